"""Pages whose value scales lie far apart: the small ones' values come out as exactly as if they stood alone.

Half the pages hold values in the first half of the dims alone, the others, of a smaller scale, in the second
half, so that a dim's result is one kind's.  Tolerance as in attention's own test, but for each dim: the
output's half step, 2^-10 of the weighted mean of that dim's |V| (weights rounded to 2^-11, scores, queries,
exponentials), and weights under fp16's normal numbers.  Those are off by 2^-25 of 2^-7 of the largest weight;
pages whose scales differ by up to 2^8 are weighed together: 2^-24 of the row's largest probability a key, times
the dim's largest |V|.  fp16 results below its normal numbers: 2^-25.
"""

import numpy as np
import pytest
import torch

import chunked_prefill_hybrid_sar_gb300 as sar
from oracle import kv8

from test_gpu_kv8_attention import TYPES, Batch

pytestmark = pytest.mark.gpu


def is_small(pattern, j, pages, page):
    """Whether page j of a sequence's is one of the small kind."""
    return {"turns": j % 2 == 1, "large first": j >= pages // 2, "small first": j < pages // 2,
            "one large": j != pages // 3, "one small": j == pages // 3}[pattern]


def spread(b, pattern, top, gap):
    """The batch's values: two kinds of pages, of scales 2^top and 2^(top - gap)."""
    half = b.d // 2
    for i, (_, m) in enumerate(b.seqs):
        pages = -(-m // b.page)
        for j in range(pages):
            p = int(b.tables[i, j])
            small = is_small(pattern, j, pages, b.page)
            live = min(b.page, m - j * b.page)
            b.scales[1, p] = 2.0 ** (top - gap if small else top)
            dims = slice(0, half) if small else slice(half, b.d)
            b.codes[1, p, :, :live, dims] = 0


def check(b, window=0, **kw):
    got = b.run(window=window, **kw)
    q = b.q.double().numpy().reshape(b.rows, -1, b.d)
    kind = b.q.dtype
    eps, least = torch.finfo(kind).eps / 2, 2.0 ** -25 if kind is torch.float16 else 0.0
    for i, (r, m) in enumerate(b.seqs):
        if r == 0 or m == 0:
            continue
        a, e = int(b.off[i]), int(b.off[i + 1])
        k, v = b.keys(i, 0), b.keys(i, 1)
        want, mean = (kv8.attention(q[a:e], k, x, r, window) for x in (v, np.abs(v)))
        far = np.repeat(np.abs(v).max(0), q.shape[1] // v.shape[1], 0) * m * 2.0 ** -24
        off = np.abs(got[a:e] - want)
        tol = eps * np.abs(want) + 2.0 ** -10 * mean + far + least
        assert (off <= tol).all(), (i, float((off / np.maximum(tol, 1e-300)).max()))
    sar.op_sync_status()


SEQS = [(1, 500), (40, 300), (1, 33), (200, 700), (3, 140), (1, 64)]


@pytest.mark.parametrize("pattern", ["turns", "large first", "small first", "one large", "one small"])
@pytest.mark.parametrize("kind,top,gap", [("bf16", 0, 7), ("bf16", 0, 9), ("bf16", 3, 14), ("f16", 5, 20), ("f16", 5, 24), ("bf16", 0, 26),
                                          ("bf16", 20, 40), ("bf16", 60, 70), ("bf16", 60, 100)])
@pytest.mark.parametrize("heads,kv_heads,d,page", [(4, 2, 128, 16), (8, 1, 64, 64)])
def test_scales_apart(pattern, kind, top, gap, heads, kv_heads, d, page):
    b = Batch(SEQS, heads, kv_heads, d, page, kind, seed=gap)
    spread(b, pattern, top, gap)
    check(b)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("window", [50, 200])
def test_scales_apart_under_a_window(kind, page, window):
    b = Batch(SEQS, 8, 2, 128, page, kind, seed=window)
    spread(b, "turns", 4, 24)
    check(b, window=window)


@pytest.mark.parametrize("rows,m", [(1, 20000), (5, 9000), (64, 5000)])
def test_scales_apart_in_pieces(rows, m):
    """A long context, which many CTAs share."""
    b = Batch([(rows, m)], 4, 2, 64, 16, "bf16", seed=m)
    spread(b, "turns", 0, 30)
    check(b)


def test_scales_that_grow_from_page_to_page():
    """Every page's scale 2^12 above the one before it, and the other way round; the dims of a page are its own."""
    for turn in (False, True):
        b = Batch([(1, 130), (60, 130)], 4, 2, 128, 16, "bf16")
        for i in range(2):
            for j in range(9):
                p, live = int(b.tables[i, j]), min(16, 130 - 16 * j)
                b.scales[1, p] = 2.0 ** (12 * (8 - j if turn else j) - 38)
                keep = b.codes[1, p, :, :live, 14 * j:14 * j + 14].clone()
                b.codes[1, p, :, :live] = 0
                b.codes[1, p, :, :live, 14 * j:14 * j + 14] = keep
        check(b)


def test_a_nan_in_a_page_of_a_small_scale():
    b = Batch([(30, 200), (1, 200)], 4, 2, 128, 16, "bf16")
    spread(b, "turns", 0, 40)
    clean = b.run()
    want = np.zeros(clean.shape, bool)
    for seq, first in ((0, 0), (1, 30)):
        b.codes[1, b.tables[seq, 11], 1, 9, 5] = 0x7F  # key 185 of the second head
    want[15:30, 2:, 5] = want[30:, 2:, 5] = True
    got = b.run()
    assert np.array_equal(np.isnan(got), want) and np.array_equal(got[~want], clean[~want])


@pytest.mark.parametrize("gap", [-30, 20])
def test_one_page_of_another_scale_costs_a_long_context_little(gap):
    """64 rows behind 200000 tokens, whose first page's scale is far from all others'; its codes are zero, so that the
    result is that of an ordinary scale, up to the order of sums (twice the output's half step and the weights')."""
    heads, kv_heads, d, page, m = 8, 2, 128, 64, 200000
    pages = -(-m // page)
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(0, 120, (2, pages, kv_heads, page, d), dtype=torch.uint8, device="cuda", generator=g)
    codes[1, 0] = 0
    scales = torch.full((2, pages, kv_heads), 2.0 ** -6, device="cuda")
    cache = sar.KV8Cache(codes[0], codes[1], scales[0], scales[1])
    q = torch.randn(64, heads * d, device="cuda", generator=g).bfloat16()
    tables = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    off, lens = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 64], [m]))
    space = torch.empty(sar.kv8_attention_workspace(cache, q, 1), dtype=torch.uint8, device="cuda")

    def run():
        best, out = 1e9, torch.empty_like(q)
        for _ in range(4):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            sar.kv8_attention(q, cache, off, lens, tables, out, workspace=space)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best, out.double()

    usual, want = run()
    scales[1, 0] = 2.0 ** (gap - 6)
    took, got = run()
    print(f"usual {usual * 1e3:.0f} us, one page apart {took * 1e3:.0f} us")
    assert bool(((got - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -9 * want.abs().max()).all())
    assert took < 4 * usual
    sar.op_sync_status()
