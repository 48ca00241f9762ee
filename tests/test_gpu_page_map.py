"""Block tables and slot maps on the GPU against the request-by-request oracle (whole numbers: equal)."""

import numpy as np
import pytest
import torch

import chunked_prefill_hybrid_sar_gb300 as sar
from chunked_prefill_hybrid_sar_gb300 import _lib
from oracle import kv8

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def batch(seed, n, page, longest, grow, spare=10):
    """Lengths, new tokens, tables, free list and count of a mixed batch."""
    g = np.random.default_rng(seed)
    lens = g.integers(0, longest + 1, n)
    new = g.choice([-1, 0, 1, 1, 1, 2], n) if grow == 1 else g.integers(-1, grow + 1, n)
    lens[g.random(n) < 0.1] = 0
    held = -(-lens // page)
    need = -(-(lens + np.maximum(new, 0)) // page)
    stride = int(need.max(initial=0)) + 2
    pool = int(held.sum() + (need - held).sum() + spare)
    pages = g.permutation(pool)
    tables = np.full((n, stride), -1)
    at = 0
    for i in range(n):
        tables[i, :held[i]] = pages[at:at + held[i]]
        at += held[i]
    free = np.full(pool, -7)
    free[:pool - at] = pages[at:]
    return lens, new, tables, free, pool - at


def run(lens, new, tables, free, count, page, max_rows, in_place=False, extra=0):
    n = len(lens)
    wide = torch.full((max(n, 1), tables.shape[1] + extra), -9, dtype=torch.int32, device="cuda")
    tab = wide[:n, :tables.shape[1]]
    tab.copy_(ints(tables))
    l, f, c = ints(lens), ints(free), ints([count])
    lo, co = (l, c) if in_place else (torch.empty_like(l), torch.empty_like(c))
    off = torch.full((n + 1,), -5, dtype=torch.int32, device="cuda")
    pos, slots = (torch.full((max_rows,), -5, dtype=torch.int32, device="cuda") for _ in range(2))
    sar.page_map(l, ints(new), tab, f, c, off, pos, slots, page_size=page, lens_out=None if in_place else lo,
                 free_count_out=None if in_place else co)
    assert extra == 0 or bool((wide[:, tables.shape[1]:] == -9).all())
    return [t.cpu().numpy() for t in (lo, tab, f, co, off, pos, slots)]


def check(lens, new, tables, free, count, page, max_rows, **kw):
    got = run(lens, new, tables, free, count, page, max_rows, **kw)
    *want, refused = kv8.page_map(lens, new, tables, free, count, page, max_rows)
    for name, x, y in zip(("lens", "tables", "free", "count", "offsets", "positions", "slots"), got, want):
        assert np.array_equal(np.atleast_1d(x).ravel(), np.atleast_1d(y).ravel()), name
    return refused


@pytest.mark.parametrize("n", [1, 2, 31, 33, 200, 513, 1500])
@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("grow", [1, 70])
def test_mixed_batches(n, page, grow):
    b = batch(n + page, n, page, 300, grow)
    rows = int(np.maximum(b[1], 0).sum())
    assert check(*b, page, rows + 3, in_place=n % 2 == 0, extra=n % 3) == []
    sar.op_sync_status()


def test_long_requests_and_many_rows():
    b = batch(5, 7, 16, 60000, 9000)
    assert check(*b, 16, int(np.maximum(b[1], 0).sum())) == []
    sar.op_sync_status()


def test_most_requests():
    b = batch(6, 8192, 16, 40, 1)
    assert check(*b, 16, 8192 * 2) == []
    sar.op_sync_status()


@pytest.mark.parametrize("spare", [0, -1, -4, -30])
def test_too_few_pages(spare):
    lens, new, tables, free, count = batch(8, 60, 16, 100, 40, spare=0)
    count += spare - 0
    new = np.maximum(new, 0)  # (none are given back)
    refused = check(lens, new, tables, free, count, 16, int(new.sum()))
    if refused:
        with pytest.raises(sar.SarError) as e:
            sar.op_sync_status()
        assert e.value.code == _lib.SAR_ERR_NO_PAGES
    assert bool(refused) == (spare < 0)
    sar.op_sync_status()


@pytest.mark.parametrize("last,refused", [(16, []), (33, [2])])
def test_pages_given_back_are_taken_in_the_same_call(last, refused):
    """One page on the list and three given back; 33 + 60 tokens take three, 1 + 16 one more, 1 + 33 two."""
    lens, new, tables, free, count = [40, 33, 1], [-1, 60, last], np.full((3, 9), -1), np.array([4, 0, 0, 0, 0, 0, 0, 0]), 1
    tables[0, :3], tables[1, :3], tables[2, :1] = (1, 2, 3), (5, 6, 7), 0
    assert check(lens, new, tables, free, count, 16, 60 + last) == refused
    if refused:
        with pytest.raises(sar.SarError):
            sar.op_sync_status()
    sar.op_sync_status()


@pytest.mark.parametrize("max_rows", [0, 1, 17, 40])
def test_rows_that_do_not_fit(max_rows):
    lens, new, tables, free, count = batch(9, 20, 16, 100, 8)
    refused = check(lens, new, tables, free, count, 16, max_rows)
    assert refused
    with pytest.raises(sar.SarError) as e:
        sar.op_sync_status()
    assert e.value.code == _lib.SAR_ERR_BOUNDS


def test_no_requests():
    got = run([], [], np.zeros((0, 3), int), np.array([3, 1, 2]), 2, 16, 4)
    assert got[3].tolist() == [2] and got[4].tolist() == [0] and got[6].tolist() == [-1] * 4 and got[5].tolist() == [0] * 4
    sar.op_sync_status()


def test_bad_requests_wait_and_are_reported():
    tables = np.full((4, 2), -1)
    tables[1, 0], tables[3] = 3, (1, 2)
    lens, tab, free, count, off, pos, slots = run([-4, 5, 10 ** 6, 32], [3, 1, -1, 4], tables, np.array([0, 4, 5, 0, 0, 0]), 3, 16, 6)
    assert lens.tolist() == [0, 6, 10 ** 6, 32] and np.array_equal(tab, tables) and count.tolist() == [3]
    assert off.tolist() == [0, 0, 1, 1, 1] and slots.tolist() == [3 * 16 + 5] + [-1] * 5
    with pytest.raises(sar.SarError) as e:
        sar.op_sync_status()
    assert e.value.code == _lib.SAR_ERR_BOUNDS


def test_a_bad_page_gets_no_slots():
    tables = np.array([[99, -1], [1, -1]])
    got = run([3, 3], [1, 1], tables, np.array([0, 2]), 1, 16, 2)
    assert got[6].tolist() == [-1, 1 * 16 + 3]
    with pytest.raises(sar.SarError):
        sar.op_sync_status()


def test_replayed_steps():
    """A captured decode step's map, replayed: lengths, tables and list move on in place."""
    lens, new, tables, free, count = batch(11, 9, 16, 30, 1, spare=40)
    new = np.ones(9, int)
    tables = np.concatenate([tables, np.full((9, 6), -1)], 1)
    l, a, tab, f, c = ints(lens), ints(new), ints(tables), ints(free), ints([count])
    off, pos, slots = (torch.zeros(k, dtype=torch.int32, device="cuda") for k in (10, 9, 9))
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        sar.page_map(l, a, tab, f, c, off, pos, slots, page_size=16)
    for _ in range(50):
        graph.replay()
        torch.cuda.synchronize()
        lens, tables, free, count, o, p, s, refused = kv8.page_map(lens, new, tables, free, count, 16, 9)
        assert refused == [] and s.tolist() == slots.tolist() and p.tolist() == pos.tolist()
    assert lens.tolist() == l.tolist() and np.array_equal(tables, tab.cpu().numpy()) and c.tolist() == [count]
    sar.op_sync_status()
