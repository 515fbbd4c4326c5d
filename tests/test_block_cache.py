"""Block-scaled 8-bit cache and page tables: what the host refuses, and pins of the reference
that the GPU tests compare with (CPU only)."""

import ctypes

import numpy as np
import pytest
import torch

import block_cache_reference as ref
import paged_gqa_attention_hd512_gb300 as pa
from paged_gqa_attention_hd512_gb300 import build as pa_build

FAKE = 0x10000  # never dereferenced: validation rejects before any CUDA call


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return pa.load()


def _attn(lib, call, **over):
    a = dict(batch=2, num_pages=4, hq=8, hkv=2, dqk=512, dvo=512, ps=16, dt=pa.PA_KV_INT8_BLOCK, scales=FAKE, bt=16,
             no_struct=False)
    a.update(over)
    sc = pa._Scales(None, None, None, a["scales"], a["bt"])
    scp = None if a["no_struct"] else ctypes.byref(sc)
    shape = (a["batch"], a["num_pages"], a["hq"], a["hkv"], a["dqk"], a["dvo"], a["ps"], 0.04, -1)
    if call == "prefill":
        return lib.paged_attn_prefill(FAKE, FAKE, 10, FAKE, FAKE, FAKE, FAKE, *shape, 1, a["dt"], scp, FAKE, None, None)
    fn = lib.paged_attn_decode if call == "decode" else lib.paged_attn_decode_noalloc
    return fn(FAKE, FAKE, FAKE, FAKE, FAKE, *shape, a["dt"], scp, FAKE, None, None)


@pytest.mark.parametrize("call", ["decode", "noalloc", "prefill"])
@pytest.mark.parametrize("dt", [pa.PA_KV_INT8_BLOCK, pa.PA_KV_FP8_BLOCK])
def test_attention_refusals(lib, call, dt):
    pa._Scales(None, None, None)  # the three-field form stays valid
    assert _attn(lib, call, dt=dt, scales=None) == pa.PA_ERR_INVALID_ARG
    assert _attn(lib, call, dt=dt, no_struct=True) == pa.PA_ERR_INVALID_ARG
    assert _attn(lib, call, dt=dt, bt=0) == pa.PA_ERR_INVALID_ARG
    assert _attn(lib, call, dt=dt, bt=32) == pa.PA_ERR_INVALID_ARG  # more than a page
    assert _attn(lib, call, dt=dt, bt=12) == pa.PA_ERR_INVALID_ARG
    assert _attn(lib, call, dt=dt, scales=FAKE + 2) == pa.PA_ERR_ALIGNMENT
    assert _attn(lib, call, dt=dt, ps=24) == pa.PA_ERR_UNSUPPORTED
    assert _attn(lib, call, dt=dt, dqk=256) == pa.PA_ERR_UNSUPPORTED
    assert _attn(lib, call, dt=5) == pa.PA_ERR_INVALID_ARG


def _append(lib, **over):
    a = dict(k=FAKE, v=FAKE, ai=FAKE, total=8, cache=FAKE, ip=FAKE, ind=FAKE, last=FAKE, batch=2, num_pages=4,
             hkv=2, dqk=512, dvo=256, ps=16, dt=pa.PA_KV_INT8_BLOCK, scales=FAKE, bt=8)
    a.update(over)
    return lib.paged_attn_append_kv_block(a["k"], a["v"], a["ai"], a["total"], a["cache"], a["ip"], a["ind"],
                                          a["last"], a["batch"], a["num_pages"], a["hkv"], a["dqk"], a["dvo"],
                                          a["ps"], a["dt"], a["scales"], a["bt"], None)


def test_append_refusals(lib):
    assert _append(lib, batch=0) == pa.PA_OK and _append(lib, total=0) == pa.PA_OK  # nothing to write
    for bad in (dict(k=None), dict(v=None), dict(ai=None), dict(cache=None), dict(ip=None), dict(ind=None),
                dict(last=None), dict(scales=None), dict(total=-1), dict(batch=-1), dict(num_pages=0), dict(hkv=0),
                dict(bt=0), dict(bt=32), dict(bt=6), dict(dt=pa.PA_KV_FP8_E4M3), dict(dt=5)):
        assert _append(lib, **bad) == pa.PA_ERR_INVALID_ARG, bad
    for bad in (dict(ps=24), dict(ps=128), dict(dqk=256, dvo=512)):
        assert _append(lib, **bad) == pa.PA_ERR_UNSUPPORTED, bad
    for bad in (dict(k=FAKE + 8), dict(v=FAKE + 2), dict(cache=FAKE + 8), dict(scales=FAKE + 1), dict(ip=FAKE + 2)):
        assert _append(lib, **bad) == pa.PA_ERR_ALIGNMENT, bad
    # the per-tensor append keeps refusing these dtypes
    assert lib.paged_attn_append_kv(FAKE, FAKE, FAKE, 8, FAKE, FAKE, FAKE, FAKE, 2, 4, 2, 512, 512, 16,
                                    pa.PA_KV_INT8_BLOCK, FAKE, FAKE, FAKE, None) == pa.PA_ERR_INVALID_ARG


def _resize(lib, **over):
    a = dict(table=FAKE, rows=4, width=8, stride=8, ids=FAKE, lens=FAKE, deltas=FAKE, batch=2, ps=16, free=FAKE,
             size=40, count=FAKE)
    a.update(over)
    return lib.paged_attn_resize_tables(a["table"], a["rows"], a["width"], a["stride"], a["ids"], a["lens"],
                                        a["deltas"], a["batch"], a["ps"], a["free"], a["size"], a["count"], None)


def _build(lib, **over):
    a = dict(table=FAKE, rows=4, width=8, stride=8, ids=FAKE, lens=FAKE, counts=FAKE, batch=2, ps=16, pages=40,
             indptr=FAKE, ind=FAKE, most=20, last=FAKE, new=FAKE, slots=FAKE, pos=FAKE, tokens=9)
    a.update(over)
    return lib.paged_attn_build_tables(a["table"], a["rows"], a["width"], a["stride"], a["ids"], a["lens"],
                                       a["counts"], a["batch"], a["ps"], a["pages"], a["indptr"], a["ind"], a["most"],
                                       a["last"], a["new"], a["slots"], a["pos"], a["tokens"], None)


@pytest.mark.parametrize("call", [_resize, _build])
def test_table_refusals(lib, call):
    for bad in (dict(table=None), dict(lens=None), dict(rows=-1), dict(width=-1), dict(stride=7), dict(batch=-1),
                dict(ids=None, batch=5)):
        assert call(lib, **bad) == pa.PA_ERR_INVALID_ARG, bad
    for bad in (dict(ps=0), dict(ps=3), dict(ps=128), dict(width=1 << 27, stride=1 << 27)):
        assert call(lib, **bad) == pa.PA_ERR_UNSUPPORTED, bad
    for bad in (dict(table=FAKE + 2), dict(ids=FAKE + 1), dict(lens=FAKE + 2)):
        assert call(lib, **bad) == pa.PA_ERR_ALIGNMENT, bad


def test_table_refusals_of_one_call(lib):
    assert _resize(lib, batch=0) == pa.PA_OK  # nothing to do
    for bad in (dict(deltas=None), dict(free=None), dict(count=None), dict(size=-1)):
        assert _resize(lib, **bad) == pa.PA_ERR_INVALID_ARG, bad
    assert _resize(lib, free=FAKE + 2) == pa.PA_ERR_ALIGNMENT
    for bad in (dict(counts=None), dict(indptr=None), dict(new=None), dict(last=None), dict(ind=None), dict(pages=0),
                dict(most=-1), dict(tokens=-1)):
        assert _build(lib, **bad) == pa.PA_ERR_INVALID_ARG, bad
    assert _build(lib, slots=FAKE + 4) == pa.PA_ERR_ALIGNMENT


def test_binding_refuses_wrong_tensors(lib):
    t = torch.zeros(4, 8, dtype=torch.int32)
    with pytest.raises(ValueError):  # CPU tensors
        pa.paged_attn_resize_tables(t, None, t[0], t[1], t[2], t[3], page_size=16)
    with pytest.raises(ValueError):
        pa.paged_attn_build_tables(t.long(), None, t[0], t[1], page_size=16, num_pages=4, max_indices=4, num_tokens=4)
    with pytest.raises(ValueError):  # no scales
        pa.paged_attn_decode(torch.zeros(1, 8, 512, dtype=torch.bfloat16), torch.zeros(10, dtype=torch.uint8),
                             t[0], t[0], t[0], num_kv_heads=1, head_dim_vo=512, page_size=16, sm_scale=1.0,
                             num_pages=1, kv_dtype=pa.PA_KV_INT8_BLOCK)


# ------------------------------------------------------------------------------ pins of the reference
def test_codes():
    assert ref.encode([0.5, 1.5, 2.5, -0.5, 126.5, 127.4, 300.0, -300.0, np.nan], ref.INT8).view(np.int8).tolist() == \
        [0, 2, 2, 0, 126, 127, 127, -127, 0]
    assert ref.values(ref.encode([448.0, 1e9, -1e9, 17.0, 19.0], ref.FP8), ref.FP8).tolist() == [448, 448, -448, 16, 20]
    every = np.arange(256, dtype=np.uint8)
    for fmt in (ref.INT8, ref.FP8):  # every code is the code of its value
        v = ref.values(every, fmt)
        ok = np.isfinite(v) & (np.abs(v) <= ref.LIMIT[fmt])
        assert np.array_equal(ref.encode(v[ok], fmt)[v[ok] != 0], every[ok][v[ok] != 0])


@pytest.mark.parametrize("fmt,half", [(ref.INT8, 0.5), (ref.FP8, 16.0)])
def test_append_error_stays_within_half_a_step(fmt, half):
    """A block written at once: |x - code s| <= half a step at the top of the range (int8: 1/2,
    e4m3: 32 / 2), plus the roundings of s, r and the product (4 units of 2^-24 of x)."""
    c = ref.make(kv_lens=[40, 7], n_new=[40, 7], fmt=fmt, Hkv=2, d_qk=256, d_vo=256, page_size=16, bt=8, seed=1)
    cache, scales = ref.append(c, c.cache, c.scales)
    for b, L in enumerate(c.kv_lens):
        pages = c.kv_indices[c.kv_indptr[b]:c.kv_indptr[b + 1]]
        for side, new in ((0, c.k_new), (1, c.v_new)):
            x = new.double().numpy()[c.append_indptr[b]:c.append_indptr[b + 1]].transpose(1, 0, 2)
            s = np.repeat(scales[pages, side].astype(np.float64), c.bt, 2)[..., None]
            got = (ref.values(np.ascontiguousarray(ref.rows_view(cache, c, side)[pages]), fmt) * s)
            got = got.transpose(1, 0, 2, 3).reshape(c.Hkv, -1, c.d_qk)[:, :L]
            s = s.transpose(1, 0, 2, 3).reshape(c.Hkv, -1, 1)[:, :L]
            assert (np.abs(got - x) <= half * s + np.abs(x) * 2.0 ** -22).all()


def test_append_in_steps_grows_scales():
    """Token by token: a block's scale is the largest so far, earlier codes follow it, and
    each growth adds at most half a step (the grown one) to their error."""
    c = ref.make(kv_lens=[16], n_new=[16], fmt=ref.INT8, Hkv=1, d_qk=256, d_vo=256, page_size=16, bt=16, seed=2)
    x = c.k_new.double().numpy()[:, 0]
    cache, scales = c.cache, c.scales
    bound = np.zeros(16)
    for t in range(16):
        step = ref.make(kv_lens=[t + 1], n_new=[1], fmt=ref.INT8, Hkv=1, d_qk=256, d_vo=256, page_size=16, bt=16, seed=2)
        step.k_new, step.v_new = c.k_new[t:t + 1], c.v_new[t:t + 1]
        step.kv_indices, old = c.kv_indices, scales[c.kv_indices[0], 0, 0, 0]
        cache, scales = ref.append(step, cache, scales)
        s = float(scales[c.kv_indices[0], 0, 0, 0])
        if t == 0 or s > old:
            bound[:t] += 0.5 * s
        bound[t] = 0.5 * s
        got = ref.values(np.ascontiguousarray(ref.rows_view(cache, c, 0)[c.kv_indices[0], 0]), ref.INT8) * s
        assert (np.abs(got[:t + 1] - x[:t + 1]).max(-1) <= bound[:t + 1] + np.abs(x[:t + 1]).max() * 2.0 ** -20).all()
    assert abs(scales[c.kv_indices[0], 0, 0, 0] - np.abs(x).max() / 127) <= np.abs(x).max() / 127 * 2.0 ** -22


def test_attention_reference_against_one_key_and_uniform_keys():
    c = ref.make(kv_lens=[1, 5], fmt=ref.INT8, Hkv=1, group=2, d_qk=256, d_vo=256, page_size=8, bt=4, seed=3)
    out, lse, _, _ = ref.attend(c, c.cache, c.scales)
    v = ref.values(np.ascontiguousarray(ref.rows_view(c.cache, c, 1)[c.kv_indices[0], 0, 0]), c.fmt) * \
        float(c.scales[c.kv_indices[0], 1, 0, 0])
    assert np.allclose(out[0], v[None], rtol=1e-12, atol=0)
    c.q[:] = 0  # every score 0: the mean, lse = ln n
    out, lse, _, _ = ref.attend(c, c.cache, c.scales)
    assert np.allclose(lse[1], np.log(5))


def test_tables_reference_conserves_pages():
    rng = np.random.default_rng(4)
    ps, rows, width, n = 4, 6, 9, 40
    table, lens = np.full((rows, width), -1, np.int32), np.zeros(rows, np.int32)
    free, count = rng.permutation(n).astype(np.int32), n
    for _ in range(200):
        ids = rng.permutation(rows)[:4]
        d = [int(rng.integers(-lens[r], width * ps - lens[r] + 1)) for r in ids]
        got = ref.resize(table, ids, lens, d, free, count, ps)
        if got is None:
            assert sum(max(0, -(-(lens[r] + x) // ps) - -(-lens[r] // ps)) for r, x in zip(ids, d)) > 0
            continue
        table, lens, free, count = got
        held = [int(p) for r in range(rows) for p in table[r, :-(-lens[r] // ps)]]
        assert sorted(held + free[:count].tolist()) == list(range(n))
