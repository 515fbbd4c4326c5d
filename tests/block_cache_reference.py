"""Plain fp64 / exact-fp32 reference of the block-scaled 8-bit KV cache and of the page tables
(CPU, no code shared with the library), and the seeded inputs of their tests.

A cache is kept as logical arrays here: codes as uint8 bytes [num_pages, page bytes], scales
fp32 [num_pages, 2, Hkv, page_size / block_tokens].
"""

from types import SimpleNamespace

import numpy as np
import torch

INT8, FP8 = 3, 4  # PA_KV_INT8_BLOCK, PA_KV_FP8_BLOCK
LIMIT = {INT8: 127.0, FP8: 448.0}
F32_MAX = np.finfo(np.float32).max


# ------------------------------------------------------------------------------ codes
def values(codes, fmt):
    """fp64 values of a uint8 code array."""
    if fmt == INT8:
        return codes.view(np.int8).astype(np.float64)
    return torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn).double().numpy()


def encode(y, fmt):
    """Codes (uint8) of fp32 values: nearest even, saturating."""
    y = np.asarray(y, dtype=np.float32)
    if fmt == INT8:
        z = np.where(np.isnan(y), 0.0, np.clip(np.rint(np.nan_to_num(y, nan=0.0)), -127, 127))
        return z.astype(np.int8).view(np.uint8)
    t = torch.from_numpy(np.ascontiguousarray(y)).clamp(-448, 448)
    return t.to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def inverse(s):
    with np.errstate(divide="ignore", over="ignore"):
        r = np.minimum(np.float32(1.0) / np.float32(s), np.float32(F32_MAX)).astype(np.float32)
    return np.where(np.asarray(s) > 0, r, np.float32(0)).astype(np.float32)


# ------------------------------------------------------------------------------ append
def rows_view(cache, c, side):
    """[num_pages, Hkv, page_size, d] view of the K (0) or V (1) codes."""
    n = c.Hkv * c.page_size
    k = n * c.d_qk
    part = cache[:, :k] if side == 0 else cache[:, k:]
    return part.reshape(cache.shape[0], c.Hkv, c.page_size, c.d_qk if side == 0 else c.d_vo)


def append(c, cache, scales):
    """The cache and scales after appending c's new rows (copies), block by block."""
    cache, scales = cache.copy(), scales.copy()
    lim = np.float32(np.float32(1.0) / np.float32(LIMIT[c.fmt]))
    for side, new in ((0, c.k_new), (1, c.v_new)):
        x_all = new.float().numpy()  # [total, Hkv, d]
        k = c.Hkv * c.page_size * c.d_qk
        for b, n in enumerate(c.n_new):
            start = c.kv_lens[b] - n
            t = start
            while t < c.kv_lens[b]:
                end = min((t // c.bt + 1) * c.bt, c.kv_lens[b])
                page = c.kv_indices[c.kv_indptr[b] + t // c.page_size]
                blk = t % c.page_size // c.bt
                first = blk * c.bt  # the block's first slot
                old = t - t // c.bt * c.bt if t == start else 0
                i0 = c.append_indptr[b] + t - start
                for h in range(c.Hkv):
                    d = new.shape[2]
                    base = (0 if side == 0 else k) + h * c.page_size * d
                    rows = cache[page, base:base + c.page_size * d].reshape(c.page_size, d)
                    x = x_all[i0:i0 + end - t, h]
                    mag = np.abs(x[np.isfinite(x)])
                    amax = np.float32(mag.max()) if mag.size else np.float32(0)
                    s_old = scales[page, side, h, blk] if old else np.float32(0)
                    s = np.float32(max(s_old, np.float32(amax * lim)))
                    r = np.float32(inverse(s))
                    if old and s > s_old:
                        ratio = np.float32(s_old * r)
                        was = values(rows[first:first + old].copy(), c.fmt).astype(np.float32)
                        rows[first:first + old] = encode(was * ratio, c.fmt)
                    with np.errstate(invalid="ignore", over="ignore"):
                        y = x * r if s > 0 else np.zeros_like(x)
                    rows[first + old:first + old + end - t] = encode(y, c.fmt)
                    scales[page, side, h, blk] = s
                t = end
    return cache, scales


# ------------------------------------------------------------------------------ attention
def attend(c, cache, scales):
    """(out, lse, out bound, lse bound) of every query row, fp64.

    The bounds count what the kernels may round, per row with scores s_j, probabilities p_j:
      e_s   the fp32 score: the sum of d_qk products may lose 2^-23 of their magnitudes' sum
            at each of d_qk additions, and its scaling 2^-22 of it;
      p_j   then relative e_s, 2^-20 for the exponential and the running rescales, and half an
            f16 step (2^-11) for the rounded probability times V scale; below f16's normal
            range that half step is 2^-25 absolute, where the sequence's largest V scale
            stands at 2^5 or more: 2^-30 of the largest code times the largest V scale per key;
      out   sum_j p_j |v_j| times twice that (numerator and denominator), the same for fp32
            sums over n keys (n 2^-23), and half a bf16 step (2^-8) of the result.
    """
    outs, lses, ob, lb = [], [], [], []
    q = c.q.double().numpy()
    g = c.Hq // c.Hkv
    for b, L in enumerate(c.kv_lens):
        n = c.qo_lens[b]
        r0 = c.qo_indptr[b]
        out = np.zeros((n, c.Hq, c.d_vo))
        lse = np.full((n, c.Hq), -np.inf)
        o_b, l_b = np.zeros((n, c.Hq, c.d_vo)), np.zeros((n, c.Hq))
        if L > 0 and n > 0:
            pages = c.kv_indices[c.kv_indptr[b]:c.kv_indptr[b + 1]]
            pos = np.arange(L - n, L)[:, None]
            j = np.arange(L)[None]
            see = (j <= pos) if c.causal else np.ones((n, L), bool)
            if c.window_left >= 0:
                see = see & (j >= pos - c.window_left)
            if c.mask is not None:
                see = see & c.mask[b]
            for h in range(c.Hkv):
                kv = []
                for side in (0, 1):
                    x = values(np.ascontiguousarray(rows_view(cache, c, side)[pages, h]), c.fmt)
                    s = np.repeat(scales[pages, side, h].astype(np.float64), c.bt, axis=1)
                    kv.append((x * s[..., None]).reshape(-1, x.shape[-1])[:L])
                k, v = kv
                qh = q[r0:r0 + n, h * g:(h + 1) * g]  # [n, g, d]
                s = np.einsum("ngd,ld->ngl", qh, k) * c.sm_scale
                mag = np.einsum("ngd,ld->ngl", np.abs(qh), np.abs(k)) * abs(c.sm_scale)
                s = np.where(see[:, None], s, -np.inf)
                m = s.max(-1, keepdims=True)
                p = np.exp(s - np.where(np.isfinite(m), m, 0.0))
                l = p.sum(-1)
                ok = l > 0
                pn = p / np.where(ok, l, 1.0)[..., None]
                out[:, h * g:(h + 1) * g] = pn @ v
                with np.errstate(divide="ignore"):
                    lse[:, h * g:(h + 1) * g] = np.where(ok, m[..., 0] + np.log(l), -np.inf)
                e_s = (np.where(see[:, None], mag, 0.0).max(-1)) * (c.d_qk * 2.0 ** -23 + 2.0 ** -22)
                rel = 2 * (e_s + 2.0 ** -20) + 2.0 ** -11 + L * 2.0 ** -22
                vmax = LIMIT[c.fmt] * float(np.nanmax(scales[pages, 1, h]))
                o_b[:, h * g:(h + 1) * g] = (rel[..., None] * (pn @ np.abs(v)) + 2.0 ** -8 * np.abs(pn @ v) +
                                             L * 2.0 ** -30 * vmax + 1e-37)
                l_b[:, h * g:(h + 1) * g] = e_s + 2.0 ** -19 + np.where(ok, np.abs(lse[:, h * g:(h + 1) * g]), 0) * 2.0 ** -21
        outs.append(out)
        lses.append(lse)
        ob.append(o_b)
        lb.append(l_b)
    return np.concatenate(outs), np.concatenate(lses), np.concatenate(ob), np.concatenate(lb)


def check(out, lse, ref, what=""):
    """Compare the library's tensors with attend()'s results under its bounds."""
    r_out, r_lse, o_b, l_b = ref
    o, l = out.float().cpu().double().numpy(), lse.cpu().double().numpy()
    assert np.isfinite(o).all(), f"{what}: non-finite output"
    bad = np.abs(o - r_out) > o_b
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outputs out of bound, worst {(np.abs(o - r_out) / o_b).max():.3g} of it"
    gone = np.isneginf(r_lse)
    assert np.array_equal(np.isneginf(l), gone), f"{what}: lse of empty rows"
    assert (o[gone] == 0).all(), f"{what}: output of empty rows"
    if (~gone).any():
        bad = np.abs(l - r_lse)[~gone] > l_b[~gone]
        assert not bad.any(), f"{what}: lse off by up to {np.abs(l - r_lse)[~gone].max():.3g}"


# ------------------------------------------------------------------------------ inputs
def make(*, kv_lens, fmt, Hkv=2, group=4, d_qk=512, d_vo=512, page_size=16, bt=16, seed=0, n_new=None, qo_lens=None,
         spread=0.5, window_left=-1, causal=True, odd_scales=False, masks=None, spare=3):
    """A cache of random codes and scales (unused slots and blocks hold NaN codes, where the
    format has them, and NaN scales), queries, and, with n_new, the new rows of an append."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    B, ps, nb = len(kv_lens), page_size, page_size // bt
    pages = [-(-L // ps) for L in kv_lens]
    num_pages = sum(pages) + spare
    perm = rng.permutation(num_pages).astype(np.int32)
    indptr = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
    c = SimpleNamespace(fmt=fmt, Hkv=Hkv, Hq=Hkv * group, d_qk=d_qk, d_vo=d_vo, page_size=ps, bt=bt, kv_lens=list(kv_lens),
                        num_pages=num_pages, kv_indptr=indptr, kv_indices=perm[:indptr[-1]].copy(),
                        last=np.array([(L - 1) % ps + 1 if L else 0 for L in kv_lens], np.int32),
                        sm_scale=d_qk ** -0.5, window_left=window_left, causal=causal, mask=masks)
    width = Hkv * ps * (d_qk + d_vo)
    if fmt == INT8:
        cache = rng.integers(-127, 128, size=(num_pages, width)).astype(np.int8).view(np.uint8)
    else:
        cache = encode(rng.normal(size=(num_pages, width)).astype(np.float32) * 60, FP8)
    # values of about unit size: int8 codes are uniform (rms 73), e4m3 codes normal (rms 60)
    scales = np.exp(spread * rng.normal(size=(num_pages, 2, Hkv, nb))).astype(np.float32) / np.float32(66)
    if odd_scales:
        pick = rng.random(scales.shape)
        scales[pick < 0.1] = 0.0
        scales[(pick >= 0.1) & (pick < 0.15)] *= np.float32(2.0 ** -40)
        pick_v = rng.random(scales[:, 1].shape)
        scales[:, 1][pick_v < 0.05] *= np.float32(2.0 ** 12)
    # what no token owns: NaN
    used = np.zeros((num_pages, ps), bool)
    for b, L in enumerate(kv_lens):
        for i, p in enumerate(c.kv_indices[indptr[b]:indptr[b + 1]]):
            used[p, :min(ps, L - i * ps)] = True
    scales[np.broadcast_to(~used.reshape(num_pages, nb, bt).any(-1)[:, None, None], scales.shape)] = np.nan
    c.cache, c.scales = cache, scales
    if fmt == FP8:
        for side in (0, 1):
            k = Hkv * ps * d_qk
            part = cache[:, :k] if side == 0 else cache[:, k:]
            view = part.reshape(num_pages, Hkv, ps, -1)
            view[np.broadcast_to(~used[:, None], view.shape[:3])] = 0x7F
            if side == 0:
                cache[:, :k] = view.reshape(num_pages, -1)
            else:
                cache[:, k:] = view.reshape(num_pages, -1)
    c.qo_lens = list(qo_lens) if qo_lens is not None else [1] * B
    c.qo_indptr = np.concatenate([[0], np.cumsum(c.qo_lens)]).astype(np.int32)
    c.q = torch.randn(int(c.qo_indptr[-1]), c.Hq, d_qk, generator=gen).bfloat16()
    if n_new is not None:
        c.n_new = list(n_new)
        c.append_indptr = np.concatenate([[0], np.cumsum(n_new)]).astype(np.int32)
        total = int(c.append_indptr[-1])
        amp = torch.exp(1.0 * torch.randn(total, Hkv, 1, generator=gen))
        c.k_new = (torch.randn(total, Hkv, d_qk, generator=gen) * amp).bfloat16()
        c.v_new = (torch.randn(total, Hkv, d_vo, generator=gen) * amp).bfloat16()
    return c


# ------------------------------------------------------------------------------ tables
def resize(table, row_ids, lens, deltas, free, count, ps):
    """What paged_attn_resize_tables does, on copies; None where it must refuse."""
    table, lens, free = table.copy(), lens.copy(), free.copy()
    width = table.shape[1]
    todo = []
    for b, d in enumerate(deltas):
        row = b if row_ids is None else int(row_ids[b])
        if row < 0:
            continue
        if row >= table.shape[0]:
            return None
        old, new = int(lens[row]), int(lens[row]) + int(d)
        if not (0 <= old <= width * ps and 0 <= new <= width * ps):
            return None
        todo.append((row, -(-old // ps), -(-new // ps), new))
    if not 0 <= count <= len(free):
        return None
    for row, po, pn, _ in todo:
        for i in range(pn, po):
            if count >= len(free):
                return None
            free[count] = table[row, i]
            count += 1
    for row, po, pn, _ in todo:
        for i in range(po, pn):
            if count == 0:
                return None
            count -= 1
            table[row, i] = free[count]
    for row, _, _, new in todo:
        lens[row] = new
    return table, lens, free, count


def build(table, row_ids, lens, counts, ps, num_pages, num_tokens):
    """The six outputs of paged_attn_build_tables for inputs without errors; kv_indices holds
    the used entries only."""
    indptr, indices, last, new_indptr, slots, positions = [0], [], [], [0], [], []
    for b, n in enumerate(counts):
        row = b if row_ids is None else int(row_ids[b])
        L, n = (int(lens[row]), max(0, int(n))) if row >= 0 else (0, 0)
        pages = [int(x) for x in table[row, :-(-L // ps)]] if row >= 0 else []
        indices += pages
        indptr.append(len(indices))
        last.append((L - 1) % ps + 1 if L else 0)
        new_indptr.append(new_indptr[-1] + n)
        for pos in range(L - n, L):
            slots.append(pages[pos // ps] * ps + pos % ps)
            positions.append(pos)
    pad = [-1] * (num_tokens - len(slots))
    return indptr, indices, last, new_indptr, slots + pad, positions + pad
