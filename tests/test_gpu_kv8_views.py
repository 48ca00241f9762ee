"""Block tables that are columns of wider ones: requests and sequences that outgrow them (whole numbers, and
rows left as they were: equal)."""

import numpy as np
import pytest
import torch

import chunked_prefill_hybrid_sar_gb300 as sar
from chunked_prefill_hybrid_sar_gb300 import _lib
from oracle import kv8

from test_gpu_kv8_attention import Batch

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def bounds():
    with pytest.raises(sar.SarError) as e:
        sar.op_sync_status()
    assert e.value.code == _lib.SAR_ERR_BOUNDS
    sar.op_sync_status()


@pytest.mark.parametrize("first,last", [(4, 8), (0, 4), (2, 6), (0, 8)])
@pytest.mark.parametrize("rows", [5, 2000])
def test_requests_that_outgrow_a_view_wait(first, last, rows):
    """Of five requests with all columns but one in use, the second and the last want two pages more."""
    n, page, cols = 5, 16, last - first
    held = cols - 1
    wide = torch.full((n, 8), -9, dtype=torch.int32, device="cuda")
    tables = np.full((n, cols), -1)
    tables[:, :held] = np.arange(n * held).reshape(n, held)
    view = wide[:, first:last]
    view.copy_(ints(tables))
    lens, new, free = [held * page] * n, [1, page + 1, 0, page, page + 1], np.arange(n * held, n * held + 9)
    free = np.concatenate([free, np.full(n * held, -7)])
    l, f, c = ints(lens), ints(free), ints([9])
    off, pos, slots = ints([0] * (n + 1)), ints([0] * rows), ints([0] * rows)
    sar.page_map(l, ints(new), view, f, c, off, pos, slots, page_size=page)
    bounds()
    # (a request that would pass its table waits as one that asks for nothing)
    want = kv8.page_map(lens, [1, 0, 0, page, 0], tables, list(free), 9, page, rows)
    for got, w in zip((l, view, f, c, off, pos, slots), want):
        assert np.array_equal(got.cpu().numpy().ravel(), np.asarray(w).ravel())
    assert bool((wide[:, :first] == -9).all()) and bool((wide[:, last:] == -9).all())


def test_a_view_is_used_to_its_last_column():
    wide = torch.full((2, 6), -9, dtype=torch.int32, device="cuda")
    view = wide[:, 3:]
    l, f, c = ints([0, 0]), ints(range(6)), ints([6])
    off, pos, slots = ints([0] * 3), ints([0] * 96), ints([0] * 96)
    sar.page_map(l, ints([48, 48]), view, f, c, off, pos, slots, page_size=16)
    assert view.tolist() == [[5, 4, 3], [2, 1, 0]] and bool((wide[:, :3] == -9).all()) and c.item() == 0
    sar.op_sync_status()


@pytest.mark.parametrize("rows", [1, 20])
def test_sequences_longer_than_a_views_columns_are_left_out(rows):
    b = Batch([(1, 50), (rows, 70), (2, 40), (rows, 64)], 4, 2, 128, 16, "f16")
    n, need = len(b.seqs), 5
    want = b.run()
    wide = torch.zeros(n, 11, dtype=torch.int32)  # (page 0 is a page of the pool)
    out = torch.full((b.rows, b.q.shape[1]), 77.0, dtype=b.q.dtype, device="cuda")
    for cols, gone in ((5, ()), (4, (1,)), (3, (0, 1, 3))):
        wide.zero_()
        wide[:, 11 - cols:] = b.tables[:, :cols]
        tables = wide.cuda()[:, 11 - cols:]
        out.fill_(77)
        sar.kv8_attention(b.q.cuda(), b.cache(), b.off.cuda(), b.lens.cuda(), tables, out)
        if gone:
            bounds()
        else:
            sar.op_sync_status()
        got = out.double().cpu().numpy().reshape(want.shape)
        for i in range(n):
            a, e = int(b.off[i]), int(b.off[i + 1])
            assert (got[a:e] == 77).all() if i in gone else np.array_equal(got[a:e], want[a:e]), (cols, i)
    assert need == max(-(-m // 16) for _, m in b.seqs)
