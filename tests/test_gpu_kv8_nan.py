"""NaN codes of values under chunks: where they go, and that they cost a call little."""

import numpy as np
import pytest
import torch

import chunked_prefill_hybrid_sar_gb300 as sar

from test_gpu_kv8_attention import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seqs,heads,kv_heads,d,page", [
    ([(40, 1500)], 4, 2, 128, 16),                        # one tile, in pieces
    ([(200, 1000)], 4, 2, 64, 32),                        # several tiles
    ([(130, 600), (3, 400), (70, 70)], 8, 1, 128, 64),
    ([(256, 300)], 1, 1, 64, 16),                         # tile A ends a block before tile B
    ([(9, 640)] * 90, 8, 2, 128, 32),                     # a CTA's pieces one behind the other
    ([(1300, 1300)], 32, 8, 64, 16),                      # a unit to a CTA
])
def test_nan_values_reach_the_rows_that_see_them(seqs, heads, kv_heads, d, page):
    """At every place of a block, in first and last blocks, several to a row, next to blocks without one."""
    b = Batch(seqs, heads, kv_heads, d, page, "bf16", seed=d)
    clean = b.run()
    g = np.random.default_rng(page)
    want = np.zeros(clean.shape, bool)
    group = heads // kv_heads
    for i, (r, m) in enumerate(seqs):
        if i % 3 == 2 and len(seqs) > 3:
            continue  # (sequences without any)
        first = m - r
        for key in {0, m - 1, first, min(127, m - 1), min(128, m - 1), *g.integers(0, m, 6).tolist()}:
            h, dim = int(g.integers(0, kv_heads)), int(g.integers(0, d))
            b.codes[1, b.tables[i, key // page], h, key % page, dim] = 0x7F if dim % 2 else 0xFF
            a, e = int(b.off[i]), int(b.off[i + 1])
            want[a + max(0, key - first):e, h * group:(h + 1) * group, dim] = True
    got = b.run()
    assert np.array_equal(np.isnan(got), want)
    assert np.array_equal(got[~want], clean[~want])
    sar.op_sync_status()


def test_windows_keep_nan_out():
    b = Batch([(60, 700), (20, 300)], 4, 2, 64, 16, "f16", seed=3)
    clean = b.run(window=100)
    keys = (0, 540, 560, 641, 660, 699)
    want = np.zeros(clean.shape, bool)
    for key in keys:
        b.codes[1, b.tables[0, key // 16], 1, key % 16, 7] = 0x7F
        for row in range(60):
            want[row, 2:, 7] |= 640 + row - 100 < key <= 640 + row
    got = b.run(window=100)
    assert np.array_equal(np.isnan(got), want) and np.array_equal(got[~want], clean[~want])


@pytest.mark.parametrize("many", [False, True])
def test_one_nan_costs_a_long_context_little(many):
    """64 rows behind 200000 tokens: with a NaN in the first page, or in every thousandth key, not five times as long
    as without (a search through all of the rows' keys took 25 times as long)."""
    heads, kv_heads, d, page, m = 8, 2, 128, 64, 200000
    pages = -(-m // page)
    codes = torch.randint(0, 120, (2, pages, kv_heads, page, d), dtype=torch.uint8, device="cuda")
    scales = torch.full((2, pages, kv_heads), 2.0 ** -6, device="cuda")
    cache = sar.KV8Cache(codes[0], codes[1], scales[0], scales[1])
    q = torch.randn(64, heads * d, device="cuda").bfloat16()
    tables = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    off, lens = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 64], [m]))
    out = torch.empty_like(q)
    space = torch.empty(sar.kv8_attention_workspace(cache, q, 1), dtype=torch.uint8, device="cuda")

    def took():
        best = 1e9
        for _ in range(4):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            sar.kv8_attention(q, cache, off, lens, tables, out, workspace=space)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    clean = took()
    assert not torch.isnan(out).any()
    for key in range(0, m, 1000) if many else (3,):
        codes[1, key // page, :, key % page, 5] = 0x7F
    dirty = took()
    assert bool(torch.isnan(out.view(64, heads, d)[:, :, 5]).all()) and int(torch.isnan(out).sum()) == 64 * heads
    print(f"clean {clean * 1e3:.0f} us, with NaN {dirty * 1e3:.0f} us")
    assert dirty < 5 * clean
    sar.op_sync_status()
