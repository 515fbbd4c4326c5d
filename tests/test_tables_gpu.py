"""paged_attn_resize_tables and paged_attn_build_tables against their plain references."""

import numpy as np
import pytest
import torch

import block_cache_reference as ref
import paged_gqa_attention_hd512_gb300 as pa
from parity import ensure_built

pytestmark = pytest.mark.gpu
RESIZE, BUILD = 401, 402


@pytest.fixture(autouse=True)
def _built():
    ensure_built()


def gpu(x, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, dtype=dtype))).cuda()


def state(rng, rows, width, ps, pages, fill=0.7):
    """A block table with random lengths, and the free list of the other pages."""
    lens = np.minimum(rng.integers(0, width * ps + 1, size=rows), int(fill * pages * ps / rows)).astype(np.int32)
    perm = rng.permutation(pages).astype(np.int32)
    table, at = np.full((rows, width), -1, np.int32), 0
    for r in range(rows):
        n = -(-int(lens[r]) // ps)
        table[r, :n] = perm[at:at + n]
        at += n
    free = np.concatenate([perm[at:], np.full(at, -5, np.int32)])
    return table, lens, free, pages - at


def run_resize(table, ids, lens, deltas, free, count, ps):
    t, l, f, c = gpu(table), gpu(lens), gpu(free), gpu([count])
    pa.paged_attn_resize_tables(t, None if ids is None else gpu(ids), l, gpu(deltas), f, c, page_size=ps)
    return t.cpu().numpy(), l.cpu().numpy(), f.cpu().numpy(), int(c)


def same(a, b):
    return all(np.array_equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("ps", [1, 16, 64])
@pytest.mark.parametrize("batch,rows,width", [(1, 1, 1), (3, 7, 40), (300, 320, 12), (1024, 1024, 3), (2500, 2600, 5)])
def test_resize(batch, rows, width, ps):
    rng = np.random.default_rng(batch + ps)
    pages = max(4, rows * width * 3 // 4)
    st = state(rng, rows, width, ps, pages)
    for step in range(6):
        ids = rng.permutation(rows)[:batch].astype(np.int32)
        if step == 5:
            ids = np.where(rng.random(batch) < 0.3, -1, ids).astype(np.int32)  # padding
        old = st[1][np.maximum(ids, 0)].astype(np.int64)
        room = width * ps - old
        kind = step % 3
        d = np.zeros(batch, np.int64) if kind == 0 else -old  # one token more; release; any change
        if kind == 0:
            d = np.minimum(1, room)
        elif kind == 2:
            d = rng.integers(-old, np.minimum(room, old // 2 + 3) + 1)
        want = ref.resize(st[0], ids, st[1], d, st[2], st[3], ps)
        got = run_resize(st[0], ids, st[1], d, st[2], st[3], ps)
        if want is None:  # not enough pages: nothing changes
            assert same(got, st) and pa.paged_attn_check_device_error() == RESIZE
            continue
        assert same(got, want) and pa.paged_attn_check_device_error() == 0
        st = want


def test_resize_takes_pages_given_back_in_the_same_call():
    rng = np.random.default_rng(1)
    table = np.array([[0, 1, 2, 3], [9, 9, 9, 9]], np.int32)
    lens, free = np.array([16, 0], np.int32), np.full(4, -1, np.int32)
    got = run_resize(table, None, lens, [-9, 8], free, 0, 4)  # two pages back, two taken
    want = ref.resize(table, None, lens, [-9, 8], free, 0, 4)
    assert same(got, want) and got[3] == 0 and got[0][1, :2].tolist() == [3, 2]
    assert pa.paged_attn_check_device_error() == 0
    del rng


def test_resize_refuses_without_changing_anything():
    table = np.arange(12, dtype=np.int32).reshape(3, 4)
    lens, free = np.array([16, 5, 0], np.int32), np.arange(12, 20, dtype=np.int32)
    bad = [
        ([0, 3], [1, 1], 2, None),           # row id past the table
        ([1, 0], [4, 1], 8, None),           # past the row's pages
        ([1, 2], [1, -1], 8, None),          # below zero
        ([2, 1], [16, 11], 5, None),         # six pages wanted, five free
        ([0], [-16], 6, None),               # four pages back, room for two
        ([0], [1 << 30], 8, None),
        ([0], [-(1 << 31)], 8, None),
        ([0], [-1], 9, None),                # a count past the list
        ([0], [-1], -1, None),
    ]
    for ids, d, count, _ in bad:
        got = run_resize(table, ids, lens, d, free, count, 4)
        assert same(got, (table, lens, free, count)), (ids, d)
        assert pa.paged_attn_check_device_error() == RESIZE
        assert ref.resize(table, ids, lens, d, free, count, 4) is None


def test_resize_rows_of_a_wider_table():
    rng = np.random.default_rng(2)
    table, lens, free, count = state(rng, 6, 8, 16, 40)
    wide = np.full((6, 13), 77, np.int32)
    wide[:, 2:10] = table
    t, l, f, c = gpu(wide), gpu(lens), gpu(free), gpu([count])
    d = np.minimum(20, 8 * 16 - lens)
    pa.paged_attn_resize_tables(t[:, 2:10], None, l, gpu(d), f, c, page_size=16)
    want = ref.resize(table, None, lens, d, free, count, 16)
    assert want is not None and np.array_equal(t.cpu().numpy()[:, 2:10], want[0]) and int(c) == want[3]
    assert (t.cpu().numpy()[:, [0, 1, 10, 11, 12]] == 77).all()
    assert pa.paged_attn_check_device_error() == 0


def run_build(table, ids, lens, counts, ps, pages, most, tokens):
    n = len(counts)
    out = (torch.full((n + 1,), -9, dtype=torch.int32, device="cuda"), torch.full((most,), -9, dtype=torch.int32, device="cuda"),
           torch.full((n,), -9, dtype=torch.int32, device="cuda"), torch.full((n + 1,), -9, dtype=torch.int32, device="cuda"),
           torch.full((tokens,), -9, dtype=torch.int64, device="cuda"), torch.full((tokens,), -9, dtype=torch.int32, device="cuda"))
    got = pa.paged_attn_build_tables(gpu(table), None if ids is None else gpu(ids), gpu(lens), gpu(counts), page_size=ps,
                                     num_pages=pages, max_indices=most, num_tokens=tokens, out=out)
    return [x.cpu().tolist() for x in got]


@pytest.mark.parametrize("ps", [1, 16, 64])
@pytest.mark.parametrize("batch,rows,width", [(1, 1, 1), (3, 7, 400), (300, 320, 12), (1024, 1024, 3), (2500, 2600, 5)])
def test_build(batch, rows, width, ps):
    rng = np.random.default_rng(batch + 3 * ps)
    pages = max(4, rows * width * 3 // 4)
    table, lens, _, _ = state(rng, rows, width, ps, pages)
    ids = rng.permutation(rows)[:batch].astype(np.int32)
    ids[rng.random(batch) < 0.1] = -1
    for counts in (np.minimum(1, lens[np.maximum(ids, 0)]), rng.integers(-2, lens[np.maximum(ids, 0)] + 1),
                   lens[np.maximum(ids, 0)], np.zeros(batch, np.int64)):
        total = int(np.maximum(np.where(ids >= 0, counts, 0), 0).sum())
        want = ref.build(table, ids, lens, counts, ps, pages, total + 3)
        most = len(want[1]) + 5
        got = run_build(table, ids, lens, counts, ps, pages, most, total + 3)
        assert got[1][len(want[1]):] == [-9] * 5  # behind the last entry: as they were
        got[1] = got[1][:len(want[1])]
        assert got == list(want)
        assert pa.paged_attn_check_device_error() == 0


def test_build_slots_past_32_bits():
    """Slots of pages whose number times page_size does not fit 31 bits."""
    pages = 1 << 26
    table = np.array([[pages - 1, 5, pages - 2]], np.int32)
    got = run_build(table, None, np.array([170], np.int32), [170], 64, pages, 3, 170)
    assert got == list(ref.build(table, None, np.array([170], np.int32), [170], 64, pages, 170))
    assert max(got[4]) > 1 << 31 and pa.paged_attn_check_device_error() == 0


def test_build_reports_bad_entries():
    table = np.array([[0, 1, 2, 3], [4, 5, 6, 7], [8, 99, -3, 9]], np.int32)
    lens = np.array([16, 5, 12], np.int32)
    ok = ref.build(table, [1], lens, [2], 4, 10, 6)
    # a row past the table, more new tokens than tokens, a bad length: listed without tokens
    for ids, l, counts in (([1, 3], lens, [2, 1]), ([1, 0], lens, [2, 17]),
                           ([1, 0], np.array([17, 5, 0], np.int32), [2, 1]), ([1, 0], np.array([-1, 5, 0], np.int32), [2, 0])):
        got = run_build(table, ids, l, counts, 4, 10, 20, 6)
        assert got[0] == ok[0] + [ok[0][-1]] and got[2] == ok[2] + [0] and got[3] == ok[3] + [2] and got[4] == ok[4]
        assert pa.paged_attn_check_device_error() == BUILD
    # page ids outside the pool: page 0, slot -1
    got = run_build(table, [2], lens, [6], 4, 10, 20, 6)
    assert got[1][:3] == [8, 0, 0] and got[4] == [-1] * 6 and got[5] == list(range(6, 12))
    assert pa.paged_attn_check_device_error() == BUILD
    # more pages or new tokens than the outputs hold: an empty batch
    for most, tokens in ((5, 6), (6, 2)):
        got = run_build(table, [0, 1], lens, [1, 2], 4, 10, most, tokens)
        assert got == [[0, 0, 0], [-9] * most, [0, 0], [0, 0, 0], [-1] * tokens, [-1] * tokens]
        assert pa.paged_attn_check_device_error() == BUILD


def test_build_of_an_empty_batch():
    got = run_build(np.zeros((2, 3), np.int32), np.zeros(0, np.int32), np.zeros(2, np.int32), np.zeros(0, np.int32), 16, 4, 2, 3)
    assert got == [[0], [-9, -9], [], [0], [-1] * 3, [-1] * 3] and pa.paged_attn_check_device_error() == 0


def test_binding_refusals():
    t, n = gpu(np.zeros((2, 3))), gpu(np.zeros(2))
    for bad in (dict(t=t.long()), dict(t=t.t()), dict(t=t.cpu()), dict(t=t[0]), dict(lens=n[:1]), dict(lens=n.long()),
                dict(ids=n[:1]), dict(free=n.float()), dict(count=n[:0])):
        a = dict(t=t, ids=None, lens=n, free=n, count=n)
        a.update(bad)
        with pytest.raises(ValueError):
            pa.paged_attn_resize_tables(a["t"], a["ids"], a["lens"], n, a["free"], a["count"], page_size=16)
    out = pa.paged_attn_build_tables(t, None, n, n, page_size=16, num_pages=4, max_indices=2, num_tokens=3)
    assert [x.numel() for x in out] == [3, 2, 2, 3, 3, 3] and out[4].dtype == torch.int64
    for bad in (out[:5], list(out), (*out[:4], out[5], out[4]), (out[0][:1], *out[1:])):
        with pytest.raises(ValueError):
            pa.paged_attn_build_tables(t, None, n, n, page_size=16, num_pages=4, max_indices=2, num_tokens=3, out=bad)
    for bad in (dict(page_size=24), dict(num_pages=0)):
        kw = dict(page_size=16, num_pages=4, max_indices=2, num_tokens=3)
        kw.update(bad)
        with pytest.raises(pa.PagedAttnError):
            pa.paged_attn_build_tables(t, None, n, n, **kw)
    assert pa.paged_attn_check_device_error() == 0
