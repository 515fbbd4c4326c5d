"""Block-scaled 8-bit cache on the GPU: append codes and scales byte for byte, decode and
prefill against fp64 under the bounds of block_cache_reference.attend, and a serving loop of
the table calls, appends and attention together, eager and captured."""

import numpy as np
import pytest
import torch

import block_cache_reference as ref
import paged_gqa_attention_hd512_gb300 as pa
from block_cache_reference import FP8, INT8
from parity import ensure_built

pytestmark = pytest.mark.gpu
SHAPES = [(512, 512), (512, 256), (256, 256)]


@pytest.fixture(autouse=True)
def _built():
    ensure_built()
    yield
    torch.cuda.synchronize()
    assert pa.paged_attn_check_device_error() == 0


def gpu(x):
    return (torch.from_numpy(np.ascontiguousarray(x)) if isinstance(x, np.ndarray) else x).cuda()


def kwargs(c):
    return dict(num_kv_heads=c.Hkv, head_dim_vo=c.d_vo, page_size=c.page_size, sm_scale=c.sm_scale,
                window_left=c.window_left, kv_dtype=c.fmt, block_tokens=c.bt, num_pages=c.num_pages)


def pack_masks(masks):
    """(bits, byte offsets) of per-sequence boolean grids."""
    parts, off = [], [0]
    for m in masks:
        parts.append(np.packbits(m.reshape(-1), bitorder="little"))
        off.append(off[-1] + len(parts[-1]))
    return np.concatenate(parts + [np.zeros(1, np.uint8)]), np.array(off, np.int64)


def decode(c, call=pa.paged_attn_decode, **more):
    kw = dict(kwargs(c), block_scales=gpu(c.scales), **more)
    if call is pa.paged_attn_decode_noalloc:
        kw.update(out=torch.empty(len(c.kv_lens), c.Hq, c.d_vo, dtype=torch.bfloat16, device="cuda"),
                  lse=torch.empty(len(c.kv_lens), c.Hq, device="cuda"))
    return call(gpu(c.q), gpu(c.cache), gpu(c.kv_indptr), gpu(c.kv_indices), gpu(c.last), **kw)


def prefill(c, **more):
    kw = dict(kwargs(c), block_scales=gpu(c.scales), causal=c.causal, **more)
    if c.mask is not None:
        bits, off = pack_masks(c.mask)
        kw.update(custom_mask=gpu(bits), mask_indptr=gpu(off))
    return pa.paged_attn_prefill(gpu(c.q), gpu(c.qo_indptr), gpu(c.cache), gpu(c.kv_indptr), gpu(c.kv_indices),
                                 gpu(c.last), **kw)


# ------------------------------------------------------------------------------ append
APPENDS = [
    # kv_lens after the append, new rows, page size, block tokens
    ([1], [1], 16, 16),
    ([5, 17, 64, 33], [1, 1, 1, 1], 16, 16),          # a decode step: first row of a block, last, inside
    ([40, 7, 0, 130], [40, 3, 0, 65], 32, 8),          # across pages, an empty sequence
    ([64, 65, 66], [64, 1, 66], 64, 64),               # a scale per page
    ([19, 3], [11, 3], 8, 1),                          # a scale per token
    ([9, 10], [9, 4], 1, 1),                           # pages of one token
    ([300, 20], [290, 7], 64, 32),
]


@pytest.mark.parametrize("fmt", [INT8, FP8])
@pytest.mark.parametrize("case", range(len(APPENDS)))
@pytest.mark.parametrize("shape", SHAPES)
def test_append_bytes(shape, case, fmt):
    kv_lens, n_new, ps, bt = APPENDS[case]
    c = ref.make(kv_lens=kv_lens, n_new=n_new, fmt=fmt, Hkv=3, d_qk=shape[0], d_vo=shape[1], page_size=ps, bt=bt,
                 seed=case)
    # old blocks hold scales that some appends raise and others do not
    want = ref.append(c, c.cache, c.scales)
    cache, scales = gpu(c.cache), gpu(c.scales)
    pa.paged_attn_append_kv_block(gpu(c.k_new), gpu(c.v_new), gpu(c.append_indptr), cache, gpu(c.kv_indptr),
                                  gpu(c.kv_indices), gpu(c.last), scales, page_size=ps, block_tokens=bt, kv_dtype=fmt)
    assert np.array_equal(scales.cpu().numpy(), want[1], equal_nan=True)
    assert np.array_equal(cache.cpu().numpy(), want[0])


@pytest.mark.parametrize("fmt", [INT8, FP8])
def test_append_special_values(fmt):
    """Zeros, infinities, NaN, subnormal and huge rows; a fresh block over a poisoned scale."""
    c = ref.make(kv_lens=[48, 3], n_new=[40, 3], fmt=fmt, Hkv=2, d_qk=256, d_vo=256, page_size=16, bt=8, seed=5)
    k, v = c.k_new.float(), c.v_new.float()
    k[0:8] = 0.0                                   # a block of zeros
    v[0:8, 0] = -0.0
    k[8, 0, :4] = torch.tensor([np.inf, -np.inf, np.nan, 2.0])
    v[16:24] = torch.tensor(np.inf)                # nothing finite: scale 0
    k[24:32] *= 2.0 ** -126                        # bf16 subnormals: 1/s saturates
    v[24:32] = 2.0 ** -133
    k[32:40] *= 2.0 ** 110
    c.k_new, c.v_new = k.bfloat16(), v.bfloat16()
    want = ref.append(c, c.cache, c.scales)
    cache, scales = gpu(c.cache), gpu(c.scales)
    pa.paged_attn_append_kv_block(gpu(c.k_new), gpu(c.v_new), gpu(c.append_indptr), cache, gpu(c.kv_indptr),
                                  gpu(c.kv_indices), gpu(c.last), scales, page_size=16, block_tokens=8, kv_dtype=fmt)
    assert np.array_equal(scales.cpu().numpy(), want[1], equal_nan=True)
    got = cache.cpu().numpy()
    # NaN codes compare as NaN (their sign is not specified)
    same = (got == want[0]) | ((fmt == FP8) & (got & 0x7F == 0x7F) & (want[0] & 0x7F == 0x7F))
    assert same.all()


@pytest.mark.parametrize("fmt", [INT8, FP8])
def test_append_steps_equal_reference_steps(fmt):
    """Twelve single-token appends: scales grow, earlier codes are rounded again each time."""
    lens = [3, 14, 8]
    full = ref.make(kv_lens=[x + 12 for x in lens], n_new=[12] * 3, fmt=fmt, Hkv=2, d_qk=512, d_vo=256, page_size=32,
                    bt=16, seed=6)
    cache, scales = gpu(full.cache), gpu(full.scales)
    want = (full.cache, full.scales)
    for t in range(12):
        step = ref.make(kv_lens=[x + t + 1 for x in lens], n_new=[1] * 3, fmt=fmt, Hkv=2, d_qk=512, d_vo=256,
                        page_size=32, bt=16, seed=6)
        step.kv_indices, step.kv_indptr = full.kv_indices, full.kv_indptr  # (32 tokens: one page each)
        rows = torch.tensor([12 * b + t for b in range(3)])
        step.k_new, step.v_new = full.k_new[rows], full.v_new[rows]
        want = ref.append(step, *want)
        pa.paged_attn_append_kv_block(gpu(step.k_new), gpu(step.v_new), gpu(step.append_indptr), cache,
                                      gpu(full.kv_indptr), gpu(full.kv_indices), gpu(step.last), scales, page_size=32,
                                      block_tokens=16, kv_dtype=fmt)
    assert np.array_equal(scales.cpu().numpy(), want[1], equal_nan=True)
    assert np.array_equal(cache.cpu().numpy(), want[0])


def test_append_many_sequences_and_padded_rows():
    """1100 sequences (several rounds of the sequence search); rows behind the last sequence are ignored."""
    lens = [1 + (7 * i) % 40 for i in range(1100)]
    new = [1 + (3 * i) % 3 if lens[i] >= 3 else 1 for i in range(1100)]
    c = ref.make(kv_lens=lens, n_new=new, fmt=INT8, Hkv=1, d_qk=256, d_vo=256, page_size=8, bt=8, seed=7)
    want = ref.append(c, c.cache, c.scales)
    cache, scales = gpu(c.cache), gpu(c.scales)
    pad = torch.full((13, 1, 256), float("nan")).bfloat16()
    pa.paged_attn_append_kv_block(gpu(torch.cat([c.k_new, pad])), gpu(torch.cat([c.v_new, pad])), gpu(c.append_indptr),
                                  cache, gpu(c.kv_indptr), gpu(c.kv_indices), gpu(c.last), scales, page_size=8,
                                  block_tokens=8, kv_dtype=INT8)
    assert np.array_equal(scales.cpu().numpy(), want[1], equal_nan=True)
    assert np.array_equal(cache.cpu().numpy(), want[0])


def test_append_reports_rows_without_a_place():
    c = ref.make(kv_lens=[4, 20], n_new=[4, 5], fmt=INT8, Hkv=1, d_qk=256, d_vo=256, page_size=8, bt=8, seed=8)
    want = ref.append(c, c.cache, c.scales)
    cache, scales = gpu(c.cache), gpu(c.scales)
    ip = c.append_indptr.copy()
    rows = torch.cat([c.k_new[:4], torch.ones(6, 1, 256).bfloat16(), c.k_new[4:]])  # 4 rows for 4 tokens, then 6 more
    vrows = torch.cat([c.v_new[:4], torch.ones(6, 1, 256).bfloat16(), c.v_new[4:]])
    ip[1:] += 6
    pa.paged_attn_append_kv_block(gpu(torch.cat([rows[4:10], rows[:4], rows[10:]])),
                                  gpu(torch.cat([vrows[4:10], vrows[:4], vrows[10:]])), gpu(ip), cache, gpu(c.kv_indptr),
                                  gpu(c.kv_indices), gpu(c.last), scales, page_size=8, block_tokens=8, kv_dtype=INT8)
    assert np.array_equal(cache.cpu().numpy(), want[0])  # the ten rows' last four are the four tokens
    assert pa.paged_attn_check_device_error() == 301
    bad = c.kv_indices.copy()
    bad[0] = c.num_pages  # the first sequence's page
    cache, scales = gpu(c.cache), gpu(c.scales)
    pa.paged_attn_append_kv_block(gpu(c.k_new), gpu(c.v_new), gpu(c.append_indptr), cache, gpu(c.kv_indptr), gpu(bad),
                                  gpu(c.last), scales, page_size=8, block_tokens=8, kv_dtype=INT8)
    assert pa.paged_attn_check_device_error() == 301
    pages = c.kv_indices[1:]
    assert np.array_equal(cache.cpu().numpy()[pages], want[0][pages])


@pytest.mark.parametrize("bt", [4, 8, 64])
@pytest.mark.parametrize("fmt", [INT8, FP8])
def test_append_long(fmt, bt):
    """Several blocks per CTA of the streamed form (8 tokens a block or more), sequences that
    begin and end inside blocks, special values, and rows behind the last sequence."""
    c = ref.make(kv_lens=[700, 5, 1300, 64, 900], n_new=[650, 5, 1299, 64, 0], fmt=fmt, Hkv=3, d_qk=512, d_vo=256,
                 page_size=64, bt=bt, seed=9)
    k, v = c.k_new.float(), c.v_new.float()
    k[100:170] = 0.0
    k[300, 1, 5], v[301, 2, 7], v[800:900] = np.inf, np.nan, -np.inf
    c.k_new, c.v_new = k.bfloat16(), v.bfloat16()
    want = ref.append(c, c.cache, c.scales)
    cache, scales = gpu(c.cache), gpu(c.scales)
    pad = torch.full((70, 3, 512), float("nan")).bfloat16()
    pa.paged_attn_append_kv_block(gpu(torch.cat([c.k_new, pad])), gpu(torch.cat([c.v_new, pad[..., :256]])),
                                  gpu(c.append_indptr), cache, gpu(c.kv_indptr), gpu(c.kv_indices), gpu(c.last), scales,
                                  page_size=64, block_tokens=bt, kv_dtype=fmt)
    assert np.array_equal(scales.cpu().numpy(), want[1], equal_nan=True)
    got = cache.cpu().numpy()
    same = (got == want[0]) | ((fmt == FP8) & (got & 0x7F == 0x7F) & (want[0] & 0x7F == 0x7F))
    assert same.all()


@pytest.mark.parametrize("bt,ps", [(8, 8), (16, 32), (64, 64)])
def test_append_rounds(bt, ps):
    """Tens of blocks per CTA: the ring of the streamed form goes round many times."""
    c = ref.make(kv_lens=[9000, 12000, 77], n_new=[8990, 12000, 70], fmt=INT8, Hkv=4, d_qk=512, d_vo=256, page_size=ps,
                 bt=bt, seed=11)
    want = ref.append(c, c.cache, c.scales)
    cache, scales = gpu(c.cache), gpu(c.scales)
    for _ in range(3):
        pa.paged_attn_append_kv_block(gpu(c.k_new), gpu(c.v_new), gpu(c.append_indptr), cache, gpu(c.kv_indptr),
                                      gpu(c.kv_indices), gpu(c.last), scales, page_size=ps, block_tokens=bt)
        assert np.array_equal(scales.cpu().numpy(), want[1], equal_nan=True)
        assert np.array_equal(cache.cpu().numpy(), want[0])


def test_bad_data_does_not_end_the_waits_of_later_calls():
    """The word that a refused resize or a skipped row sets is not the one that waits look at."""
    t, n = gpu(np.zeros((1, 1), np.int32)), gpu(np.zeros(1, np.int32))
    pa.paged_attn_resize_tables(t, None, n, gpu(np.array([5], np.int32)), n, n, page_size=16)  # no free page
    c = ref.make(fmt=INT8, kv_lens=[5000, 300], qo_lens=[200, 300], n_new=[100, 300], Hkv=2, group=6, page_size=64,
                 bt=32, seed=10)
    want = ref.append(c, c.cache, c.scales)
    cache, scales = gpu(c.cache), gpu(c.scales)
    pa.paged_attn_append_kv_block(gpu(c.k_new), gpu(c.v_new), gpu(c.append_indptr), cache, gpu(c.kv_indptr),
                                  gpu(c.kv_indices), gpu(c.last), scales, page_size=64, block_tokens=32)
    assert np.array_equal(cache.cpu().numpy(), want[0])
    out, lse = prefill(c)
    ref.check(out, lse, ref.attend(c, c.cache, c.scales))
    assert pa.paged_attn_check_device_error() == 401


@pytest.mark.parametrize("bt", [8, 64])
def test_append_after_a_wait_gave_up(bt):
    """With the waits' error word set (here from the host) a streamed append gives up and
    returns, with no copy of its ring still on the way; once the word is cleared the same
    append is right."""
    c = ref.make(fmt=INT8, kv_lens=[9000, 300], n_new=[9000, 300], Hkv=2, page_size=64, bt=bt, seed=12)
    want = ref.append(c, c.cache, c.scales)
    cache, scales = gpu(c.cache), gpu(c.scales)
    args = (gpu(c.k_new), gpu(c.v_new), gpu(c.append_indptr), cache, gpu(c.kv_indptr), gpu(c.kv_indices), gpu(c.last),
            scales)
    assert pa.load().paged_attn_debug_set_error_word(0, 7) == pa.PA_OK
    pa.paged_attn_append_kv_block(*args, page_size=64, block_tokens=bt)
    assert pa.paged_attn_check_device_error() == 7
    cache.copy_(gpu(c.cache))
    scales.copy_(gpu(c.scales))
    pa.paged_attn_append_kv_block(*args, page_size=64, block_tokens=bt)
    assert np.array_equal(scales.cpu().numpy(), want[1], equal_nan=True)
    assert np.array_equal(cache.cpu().numpy(), want[0])


# ------------------------------------------------------------------------------ decode
DECODES = [
    dict(kv_lens=[37, 64], Hkv=1, group=8, page_size=16, bt=16),
    dict(kv_lens=[1, 0, 2, 63, 64, 65, 129], Hkv=2, group=6, page_size=16, bt=4),
    dict(kv_lens=[500, 33], Hkv=3, group=16, page_size=64, bt=64),
    dict(kv_lens=[300, 1, 77], Hkv=2, group=1, page_size=32, bt=8, window_left=40),
    dict(kv_lens=[300, 130], Hkv=2, group=3, page_size=64, bt=64, window_left=0),
    dict(kv_lens=[40, 11], Hkv=2, group=5, page_size=4, bt=2),
    dict(kv_lens=[23, 9], Hkv=1, group=12, page_size=1, bt=1),
    dict(kv_lens=[700, 250], Hkv=2, group=4, page_size=16, bt=1, odd_scales=True, spread=3.0),
]


@pytest.mark.parametrize("fmt", [INT8, FP8])
@pytest.mark.parametrize("case", range(len(DECODES)))
@pytest.mark.parametrize("shape", SHAPES)
def test_decode(shape, case, fmt):
    c = ref.make(fmt=fmt, d_qk=shape[0], d_vo=shape[1], seed=20 + case, **DECODES[case])
    want = ref.attend(c, c.cache, c.scales)
    name = "int8_block" if fmt == INT8 else "fp8_block"
    for direct, chunk in ((-1, 0), (0, 0), (0, 1), (0, 3)):
        pa.paged_attn_set_decode_direct(direct)
        pa.paged_attn_set_decode_chunk_pages(chunk)
        try:
            out, lse = decode(c)
            assert name in pa.paged_attn_last_variant()
        finally:
            pa.paged_attn_set_decode_direct(-1)
            pa.paged_attn_set_decode_chunk_pages(0)
        ref.check(out, lse, want, f"direct {direct} chunk {chunk}")
    out, lse = decode(c, pa.paged_attn_decode_noalloc)
    ref.check(out, lse, want, "noalloc")


@pytest.mark.parametrize("fmt", [INT8, FP8])
def test_decode_long_sequences(fmt):
    c = ref.make(fmt=fmt, kv_lens=[9000, 4097, 1], Hkv=2, group=6, page_size=64, bt=32, seed=40)
    out, lse = decode(c)
    ref.check(out, lse, ref.attend(c, c.cache, c.scales))


@pytest.mark.parametrize("batch", [511, 700, 1300])
def test_decode_many_sequences(batch):
    """Runs found by each CTA (up to 512 sequences) and by the planner (more, in one round of
    threads or two), over sequences of very different lengths, some empty, some windowed."""
    lens = [(37 * i) % 90 if i % 11 else 0 for i in range(batch)]
    lens[3], lens[-1] = 3000, 1500
    for window in (-1, 60):
        c = ref.make(fmt=INT8, kv_lens=lens, Hkv=2, group=3, d_qk=256, d_vo=256, page_size=16, bt=8, seed=42,
                     window_left=window)
        out, lse = decode(c)
        ref.check(out, lse, ref.attend(c, c.cache, c.scales), f"window {window}")


def test_decode_v_scales_over_the_whole_float_range():
    """Later blocks 2^100 above or below earlier ones, and blocks of zeros: the probabilities
    stay representable because they follow the largest V scale so far."""
    for order in (1, -1):
        c = ref.make(fmt=INT8, kv_lens=[256], Hkv=1, group=4, d_qk=256, d_vo=256, page_size=64, bt=64, seed=41, spread=0.1)
        p = c.kv_indices[::order]
        for i, e in enumerate((0, -100, -30, 60)):
            c.scales[p[i], 1] = np.float32(2.0 ** e / 66)
        c.scales[p[0], 1] = 0
        want = ref.attend(c, c.cache, c.scales)
        for chunk in (0, 1):
            pa.paged_attn_set_decode_chunk_pages(chunk)
            try:
                out, lse = decode(c)
            finally:
                pa.paged_attn_set_decode_chunk_pages(0)
            ref.check(out, lse, want, f"order {order} chunk {chunk}")


# ------------------------------------------------------------------------------ prefill
PREFILLS = [
    dict(kv_lens=[130, 70], qo_lens=[130, 70], Hkv=2, group=4, page_size=16, bt=16),
    dict(kv_lens=[1, 0, 200, 129], qo_lens=[1, 0, 7, 129], Hkv=1, group=6, page_size=32, bt=8),
    dict(kv_lens=[400, 65], qo_lens=[300, 1], Hkv=2, group=3, page_size=64, bt=64, window_left=50),
    dict(kv_lens=[150, 90], qo_lens=[40, 90], Hkv=1, group=16, page_size=8, bt=8, causal=False),
    dict(kv_lens=[150, 33], qo_lens=[40, 33], Hkv=2, group=1, page_size=4, bt=2),     # padded pages
    dict(kv_lens=[70], qo_lens=[33], Hkv=1, group=5, page_size=1, bt=1, window_left=20),
    dict(kv_lens=[600, 300], qo_lens=[200, 300], Hkv=2, group=4, page_size=16, bt=1, odd_scales=True, spread=3.0),
]


@pytest.mark.parametrize("fmt", [INT8, FP8])
@pytest.mark.parametrize("case", range(len(PREFILLS)))
@pytest.mark.parametrize("shape", SHAPES)
def test_prefill(shape, case, fmt):
    spec = PREFILLS[case]
    c = ref.make(fmt=fmt, d_qk=shape[0], d_vo=shape[1], seed=60 + case, **spec)
    want = ref.attend(c, c.cache, c.scales)
    out, lse = prefill(c)
    name = "int8_block" if fmt == INT8 else "fp8_block"
    assert name in pa.paged_attn_last_variant()
    ref.check(out, lse, want, pa.paged_attn_last_variant())
    pa.paged_attn_set_prefill_split_kv(0)
    try:
        out, lse = prefill(c)
        assert "splitkv" not in pa.paged_attn_last_variant()
        ref.check(out, lse, want, "no split")
        if c.page_size >= 8:  # converted in the kernel
            pa.paged_attn_set_prefill_dequant_limit(0)
            out, lse = prefill(c)
            assert "dequant" not in pa.paged_attn_last_variant()
            ref.check(out, lse, want, "in the kernel")
    finally:
        pa.paged_attn_set_prefill_split_kv(-1)
        pa.paged_attn_set_prefill_dequant_limit(-1)


@pytest.mark.parametrize("fmt", [INT8, FP8])
@pytest.mark.parametrize("shape", [(512, 512), (256, 256)])
@pytest.mark.parametrize("page_size", [2, 16])
def test_prefill_custom_mask(page_size, shape, fmt):
    rng = np.random.default_rng(70)
    lens, q = [150, 90], [60, 90]
    masks = [rng.random((n, L)) < 0.4 for n, L in zip(q, lens)]
    masks[0][5] = False  # a row that sees nothing
    c = ref.make(fmt=fmt, kv_lens=lens, qo_lens=q, Hkv=2, group=4, d_qk=shape[0], d_vo=shape[1], page_size=page_size,
                 bt=2, seed=71, causal=False, masks=masks)
    want = ref.attend(c, c.cache, c.scales)
    limits = (-1, 0) if page_size >= 8 else (-1,)
    for limit in limits:
        pa.paged_attn_set_prefill_dequant_limit(limit)
        try:
            out, lse = prefill(c)
        finally:
            pa.paged_attn_set_prefill_dequant_limit(-1)
        ref.check(out, lse, want, f"limit {limit}")


@pytest.mark.parametrize("fmt", [INT8, FP8])
@pytest.mark.parametrize("shape", SHAPES)
def test_prefill_extend_splits_the_prefix(shape, fmt):
    c = ref.make(fmt=fmt, kv_lens=[5000, 2500], qo_lens=[20, 33], Hkv=2, group=4, d_qk=shape[0], d_vo=shape[1],
                 page_size=32, bt=16, seed=80)
    want = ref.attend(c, c.cache, c.scales)
    for limit in (-1, 0):
        pa.paged_attn_set_prefill_dequant_limit(limit)
        try:
            out, lse = prefill(c)
        finally:
            pa.paged_attn_set_prefill_dequant_limit(-1)
        assert "splitkv" in pa.paged_attn_last_variant()
        ref.check(out, lse, want, f"limit {limit}")


@pytest.mark.parametrize("fmt", [INT8, FP8])
@pytest.mark.parametrize("shape", SHAPES)
def test_prefill_in_the_kernel_again_and_again(shape, fmt):
    """The converters' staging ring under load: the same bits every time."""
    c = ref.make(fmt=fmt, kv_lens=[5120, 2500], qo_lens=[20, 33], Hkv=2, group=4, d_qk=shape[0], d_vo=shape[1],
                 page_size=32, bt=16, seed=89)
    want = ref.attend(c, c.cache, c.scales)
    pa.paged_attn_set_prefill_dequant_limit(0)
    try:
        runs = [prefill(c) for _ in range(12)]
    finally:
        pa.paged_attn_set_prefill_dequant_limit(-1)
    ref.check(*runs[0], want)
    assert all(torch.equal(o, runs[0][0]) and torch.equal(l, runs[0][1]) for o, l in runs[1:])


@pytest.mark.parametrize("order", [1, -1])
@pytest.mark.parametrize("shape", [(512, 512), (256, 256)])
def test_prefill_v_scales_over_the_whole_float_range(shape, order):
    """As for decode; the scale steps up from tile to tile, so that O is rescaled (and, with
    head_dim_vo 512, the rescales replayed in the second pass)."""
    c = ref.make(fmt=INT8, kv_lens=[640], qo_lens=[300], Hkv=1, group=4, d_qk=shape[0], d_vo=shape[1], page_size=64, bt=64,
                 seed=81, spread=0.1)
    for i, p in enumerate(c.kv_indices[::order]):
        c.scales[p, 1] = np.float32(2.0 ** (12 * i - 70) / 66)
    c.scales[c.kv_indices[4], 1] = 0
    want = ref.attend(c, c.cache, c.scales)
    for limit in (-1, 0):
        pa.paged_attn_set_prefill_dequant_limit(limit)
        pa.paged_attn_set_prefill_split_kv(0)
        try:
            out, lse = prefill(c)
        finally:
            pa.paged_attn_set_prefill_dequant_limit(-1)
            pa.paged_attn_set_prefill_split_kv(-1)
        ref.check(out, lse, want, f"limit {limit}")


@pytest.mark.parametrize("phase", ["decode", "prefill"])
def test_scales_before_the_window_are_not_used(phase):
    """NaN scales in blocks wholly before every query's window, in pages that hold visible
    tokens and in others."""
    new = [1, 1] if phase == "decode" else [9, 40]
    c = ref.make(fmt=INT8, kv_lens=[500, 290], qo_lens=new, Hkv=2, group=4, page_size=64, bt=8, seed=83, window_left=90)
    want = ref.attend(c, c.cache, c.scales)
    for b, (L, n) in enumerate(zip(c.kv_lens, new)):
        lo = L - n - 90  # the first visible token
        for i in range(lo // 8):  # blocks before it
            c.scales[c.kv_indices[c.kv_indptr[b] + i * 8 // 64], :, :, i * 8 % 64 // 8] = np.nan
    for limit in (-1, 0):
        pa.paged_attn_set_prefill_dequant_limit(limit)
        try:
            out, lse = decode(c) if phase == "decode" else prefill(c)
        finally:
            pa.paged_attn_set_prefill_dequant_limit(-1)
        ref.check(out, lse, want, f"limit {limit}")


def test_given_outputs_and_stream():
    """out, lse and stream arguments: written in place, on that stream."""
    c = ref.make(fmt=FP8, kv_lens=[300, 41], qo_lens=[20, 41], n_new=[5, 41], Hkv=2, group=3, page_size=16, bt=8, seed=84)
    side = torch.cuda.Stream()
    cache, scales = gpu(c.cache), gpu(c.scales)
    args = [gpu(x) for x in (c.kv_indptr, c.kv_indices, c.last)]
    k, v, ai, q, qi = (gpu(x) for x in (c.k_new, c.v_new, c.append_indptr, c.q, c.qo_indptr))
    out = torch.empty(61, 6, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(61, 6, device="cuda")
    torch.cuda.synchronize()
    pa.paged_attn_append_kv_block(k, v, ai, cache, *args, scales, page_size=16, block_tokens=8, kv_dtype=FP8, stream=side)
    got = pa.paged_attn_prefill(q, qi, cache, *args, out=out, lse=lse, stream=side, block_scales=scales, **kwargs(c))
    assert got[0] is out and got[1] is lse
    side.synchronize()
    after = ref.append(c, c.cache, c.scales)
    assert np.array_equal(cache.cpu().numpy(), after[0])
    ref.check(out, lse, ref.attend(c, *after))
    out2, none = pa.paged_attn_decode(q[:2], cache, *args, return_lse=False, block_scales=scales, **kwargs(c))
    assert none is None and out2.shape == (2, 6, 512)


def test_prefill_longer_than_the_probability_scratch():
    """More than 64 KV tiles: head_dim_vo 512 recomputes the scores in its second pass."""
    c = ref.make(fmt=INT8, kv_lens=[8400], qo_lens=[6], Hkv=1, group=4, page_size=64, bt=64, seed=82)
    pa.paged_attn_set_prefill_split_kv(0)
    try:
        out, lse = prefill(c)
    finally:
        pa.paged_attn_set_prefill_split_kv(-1)
    ref.check(out, lse, ref.attend(c, c.cache, c.scales))


def test_pages_past_32_bit_offsets():
    """Pages more than 2^32 bytes into the cache: append, decode, prefill by copy (limit raised)
    and in the kernel (the default limit)."""
    c = ref.make(fmt=INT8, kv_lens=[300, 130], qo_lens=[100, 130], n_new=[60, 130], Hkv=4, group=2, page_size=64, bt=16,
                 seed=85)
    n, first = 18000, 17000  # pages of 256 KiB
    pages = first + torch.arange(c.num_pages)
    cache = torch.zeros(n, c.cache.shape[1], dtype=torch.uint8, device="cuda")
    scales = torch.zeros(n, *c.scales.shape[1:], device="cuda")
    cache[pages.cuda()], scales[pages.cuda()] = gpu(c.cache), gpu(c.scales)
    indices = gpu(c.kv_indices + np.int32(first))
    args = (gpu(c.kv_indptr), indices, gpu(c.last))
    pa.paged_attn_append_kv_block(gpu(c.k_new), gpu(c.v_new), gpu(c.append_indptr), cache, *args, scales, page_size=64,
                                  block_tokens=16)
    after = ref.append(c, c.cache, c.scales)
    assert np.array_equal(cache[pages.cuda()].cpu().numpy(), after[0])
    assert np.array_equal(scales[pages.cuda()].cpu().numpy(), after[1], equal_nan=True)
    kw = dict(kwargs(c), num_pages=n, block_scales=scales)
    want = ref.attend(c, *after)
    for limit in (-1, 32 << 30):
        pa.paged_attn_set_prefill_dequant_limit(limit)
        try:
            out, lse = pa.paged_attn_prefill(gpu(c.q), gpu(c.qo_indptr), cache, *args, **kw)
        finally:
            pa.paged_attn_set_prefill_dequant_limit(-1)
        assert ("dequant" in pa.paged_attn_last_variant()) == (limit > 0)
        ref.check(out, lse, want, f"limit {limit}")
    d = ref.SimpleNamespace(**vars(c))
    d.qo_lens, d.qo_indptr, d.q = [1, 1], np.array([0, 1, 2], np.int32), c.q[[99, 229]]
    out, lse = pa.paged_attn_decode(gpu(d.q), cache, *args, **kw)
    ref.check(out, lse, ref.attend(d, *after))
    pa.paged_attn_release_workspace()  # (the copy took gigabytes)


def test_binding_refusals():
    """What the Python calls refuse, with nothing launched."""
    c = ref.make(fmt=INT8, kv_lens=[40], n_new=[40], Hkv=2, group=2, page_size=16, bt=8, seed=86)
    q, cache, scales = gpu(c.q), gpu(c.cache), gpu(c.scales)
    ip, ix, last, ai, k, v = (gpu(x) for x in (c.kv_indptr, c.kv_indices, c.last, c.append_indptr, c.k_new, c.v_new))
    kw = kwargs(c)

    def dec(**more):
        return pa.paged_attn_decode(more.pop("q", q), cache, ip, ix, last, **{**kw, "block_scales": scales, **more})

    def app(**more):
        a = dict(k=k, v=v, ai=ai, cache=cache, ip=ip, scales=scales, ps=16, bt=8, fmt=INT8)
        a.update(more)
        pa.paged_attn_append_kv_block(a["k"], a["v"], a["ai"], a["cache"], a["ip"], ix, last, a["scales"], page_size=a["ps"],
                                      block_tokens=a["bt"], kv_dtype=a["fmt"])

    for bad in (dict(num_pages=len(c.cache) + 1), dict(block_scales=None), dict(block_scales=scales.double()),
                dict(block_scales=scales[:-1]), dict(block_scales=scales.cpu()), dict(block_tokens=0), dict(block_tokens=32), dict(block_tokens=3),
                dict(q=q[:, :, ::2]), dict(q=q[0])):
        with pytest.raises(ValueError):
            dec(**bad)
    many = torch.zeros(4096, device="cuda")
    for bad in (dict(block_tokens=3, block_scales=many), dict(sm_scale=float("inf")), dict(kv_dtype=9)):
        with pytest.raises(pa.PagedAttnError):
            dec(**bad)
    for bad in (dict(k=k.float()), dict(v=v[:-1]), dict(ai=ai.long()), dict(ip=ip[:1]), dict(scales=None),
                dict(scales=scales.half()), dict(k=k.transpose(0, 1).contiguous().transpose(0, 1)), dict(bt=17)):
        with pytest.raises(ValueError):
            app(**bad)
    with pytest.raises(pa.PagedAttnError):
        app(fmt=pa.PA_KV_FP8_E4M3)
    with pytest.raises(TypeError):
        app(ai=[0, 40])
    assert np.array_equal(cache.cpu().numpy(), c.cache)


def test_a_graph_outlives_its_workspace_growing():
    """A later call on the stream needs a larger workspace than the one whose address a graph
    has: the graph's stays allocated, and its replays are right."""
    c = ref.make(fmt=INT8, kv_lens=[3000, 41], Hkv=2, group=3, page_size=16, bt=8, seed=87)
    q, cache, scales = gpu(c.q), gpu(c.cache), gpu(c.scales)
    args = [gpu(x) for x in (c.kv_indptr, c.kv_indices, c.last)]
    kw = dict(kwargs(c), block_scales=scales)
    pa.paged_attn_release_workspace()
    want, want_lse = pa.paged_attn_decode(q, cache, *args, **kw)
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.paged_attn_decode(q, cache, *args, out=out, lse=lse, **kw)
    big = ref.make(fmt=FP8, kv_lens=[6000, 5000], qo_lens=[700, 900], Hkv=4, group=4, page_size=32, bt=32, seed=88)
    prefill(big)
    keep = [torch.full((1 << 20,), 9, dtype=torch.int32, device="cuda") for _ in range(8)]  # whatever was freed is used
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert all(bool((t == 9).all()) for t in keep)
    assert pa.paged_attn_check_device_error() == 0


# ------------------------------------------------------------------------------ together
class Server:
    """Requests on block-table rows, pages on a free list, an int8 / e4m3 cache: the state of a
    small serving loop, and its reference twin on the host."""

    def __init__(self, fmt, rows=5, width=12, ps=16, bt=8, Hkv=2, group=3, d=256, pages=40, seed=90):
        self.fmt, self.ps, self.bt, self.Hkv, self.Hq, self.d, self.pages = fmt, ps, bt, Hkv, Hkv * group, d, pages
        rng = np.random.default_rng(seed)
        self.gen = torch.Generator().manual_seed(seed)
        self.table, self.lens = np.full((rows, width), -1, np.int32), np.zeros(rows, np.int32)
        self.free, self.count = rng.permutation(pages).astype(np.int32), pages
        self.cache = np.zeros((pages, Hkv * ps * 2 * d), np.uint8)
        self.scales = np.full((pages, 2, Hkv, ps // bt), np.nan, np.float32)
        self.g = dict(table=gpu(self.table), lens=gpu(self.lens), free=gpu(self.free),
                      count=gpu(np.array([pages], np.int32)), cache=gpu(self.cache), scales=gpu(self.scales))

    def inputs(self, ids, counts, padded=0):
        n = sum(counts)
        draw = lambda *s: torch.randn(*s, generator=self.gen).bfloat16()  # noqa: E731
        return dict(ids=gpu(np.array(ids, np.int32)), counts=gpu(np.array(counts, np.int32)),
                    k=gpu(draw(n + padded, self.Hkv, self.d)), v=gpu(draw(n + padded, self.Hkv, self.d)),
                    q=gpu(draw(n + padded, self.Hq, self.d)))

    def step_gpu(self, x, one_token, num_tokens):
        g = self.g
        pa.paged_attn_resize_tables(g["table"], x["ids"], g["lens"], x["counts"], g["free"], g["count"], page_size=self.ps)
        indptr, indices, last, new_indptr, slots, pos = pa.paged_attn_build_tables(
            g["table"], x["ids"], g["lens"], x["counts"], page_size=self.ps, num_pages=self.pages,
            max_indices=self.pages, num_tokens=num_tokens)
        pa.paged_attn_append_kv_block(x["k"], x["v"], new_indptr, g["cache"], indptr, indices, last, g["scales"],
                                      page_size=self.ps, block_tokens=self.bt, kv_dtype=self.fmt)
        kw = dict(num_kv_heads=self.Hkv, head_dim_vo=self.d, page_size=self.ps, sm_scale=self.d ** -0.5,
                  kv_dtype=self.fmt, block_scales=g["scales"], block_tokens=self.bt, num_pages=self.pages)
        if one_token:
            return (*pa.paged_attn_decode(x["q"], g["cache"], indptr, indices, last, **kw), slots, pos)
        return (*pa.paged_attn_prefill(x["q"], new_indptr, g["cache"], indptr, indices, last, **kw), slots, pos)

    def step_ref(self, x, num_tokens):
        ids, counts = x["ids"].cpu().numpy(), x["counts"].cpu().numpy()
        self.table, self.lens, self.free, self.count = ref.resize(self.table, ids, self.lens, counts, self.free,
                                                                  self.count, self.ps)
        indptr, indices, last, new, slots, pos = ref.build(self.table, ids, self.lens, counts, self.ps, self.pages,
                                                           num_tokens)
        c = ref.SimpleNamespace(
            fmt=self.fmt, Hkv=self.Hkv, Hq=self.Hq, d_qk=self.d, d_vo=self.d, page_size=self.ps, bt=self.bt,
            num_pages=self.pages, kv_indptr=np.array(indptr), kv_indices=np.array(indices, np.int32),
            kv_lens=[int(self.lens[i]) if i >= 0 else 0 for i in ids], n_new=np.diff(new).tolist(),
            append_indptr=np.array(new), qo_lens=np.diff(new).tolist(), qo_indptr=np.array(new), sm_scale=self.d ** -0.5,
            window_left=-1, causal=True, mask=None, q=x["q"].cpu(), k_new=x["k"].cpu(), v_new=x["v"].cpu())
        self.cache, self.scales = ref.append(c, self.cache, self.scales)
        return ref.attend(c, self.cache, self.scales), slots, pos

    def same(self):
        g = self.g
        assert np.array_equal(g["table"].cpu().numpy(), self.table) and np.array_equal(g["lens"].cpu().numpy(), self.lens)
        assert int(g["count"]) == self.count and np.array_equal(g["free"].cpu().numpy(), self.free)
        assert np.array_equal(g["cache"].cpu().numpy(), self.cache)
        assert np.array_equal(g["scales"].cpu().numpy(), self.scales, equal_nan=True)


@pytest.mark.parametrize("fmt", [INT8, FP8])
def test_serving_loop(fmt):
    """Prompts admitted, decode steps, one request released and its row used again, a captured
    decode step replayed (with a padding sequence): tables, cache, scales, slots and outputs."""
    s = Server(fmt)

    def eager(ids, counts, one):
        x, n = s.inputs(ids, counts), sum(counts) + 2
        out, lse, slots, pos = s.step_gpu(x, one, n)
        want, w_slots, w_pos = s.step_ref(x, n)
        ref.check(out, lse, want)
        assert slots.tolist() == w_slots and pos.tolist() == w_pos

    eager([3, 0, 4], [40, 17, 1], False)
    for _ in range(3):
        eager([0, 3, 4], [1, 1, 1], True)
    gone = gpu(np.array([-int(s.lens[3])], np.int32))
    pa.paged_attn_resize_tables(s.g["table"], gpu(np.array([3], np.int32)), s.g["lens"], gone, s.g["free"], s.g["count"],
                                page_size=s.ps)
    s.table, s.lens, s.free, s.count = ref.resize(s.table, [3], s.lens, gone.tolist(), s.free, s.count, s.ps)
    eager([1, 3], [100, 5], False)
    s.same()
    # a decode step of rows 0, 3, 1 captured with a fourth, padding, sequence (its query row
    # sees nothing; its new row lies behind the last sequence)
    x = s.inputs([0, 3, 1, -1], [1, 1, 1, 0], padded=1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    saved = {k: v.clone() for k, v in s.g.items()}
    with torch.cuda.stream(side):
        s.step_gpu(x, True, 4)  # warm-up: grows the stream's workspace
        for k, v in saved.items():
            s.g[k].copy_(v)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out, lse, slots, pos = s.step_gpu(x, True, 4)
    for _ in range(20):  # crosses blocks and pages
        y = s.inputs([0, 3, 1, -1], [1, 1, 1, 0], padded=1)
        for k in ("k", "v", "q"):
            x[k].copy_(y[k])
        graph.replay()
        want, w_slots, w_pos = s.step_ref(x, 4)
        torch.cuda.synchronize()
        ref.check(out[:3], lse[:3], want)
        assert (out[3] == 0).all() and torch.isneginf(lse[3]).all()
        assert slots.tolist() == w_slots and pos.tolist() == w_pos
    s.same()


def test_two_streams():
    """Appends and decodes of two caches on two streams give what each gives alone."""
    cs = [ref.make(kv_lens=[200, 90], n_new=[30, 1], fmt=f, Hkv=2, d_qk=512, d_vo=512, page_size=16, bt=16, seed=95 + f)
          for f in (INT8, FP8)]
    want = [ref.append(c, c.cache, c.scales) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    state = [dict(k=gpu(c.k_new), v=gpu(c.v_new), ai=gpu(c.append_indptr), cache=gpu(c.cache), ip=gpu(c.kv_indptr),
                  ind=gpu(c.kv_indices), last=gpu(c.last), scales=gpu(c.scales), q=gpu(c.q)) for c in cs]
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for c, st, s in zip(cs, state, streams):
            with torch.cuda.stream(s):
                pa.paged_attn_append_kv_block(st["k"], st["v"], st["ai"], st["cache"], st["ip"], st["ind"], st["last"],
                                              st["scales"], page_size=16, block_tokens=16, kv_dtype=c.fmt)
                got.append(pa.paged_attn_decode(st["q"], st["cache"], st["ip"], st["ind"], st["last"],
                                                block_scales=st["scales"], **kwargs(c)))
    torch.cuda.synchronize()
    for i, (c, st) in enumerate(zip(cs, state)):
        assert np.array_equal(st["cache"].cpu().numpy(), want[i][0])
        full = ref.attend(c, *want[i])
        for out, lse in got[i::2]:
            ref.check(out, lse, full)
