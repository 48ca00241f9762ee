"""Attention over the 8-bit cache against the float64 oracle.

Tolerance: the output's rounding (half a step), and of the weighted mean of |V|:
weights rounded to fp16 (2^-11); scores of D <= 128 products added up in fp32 (D
2^-23 of their magnitudes' sum, about sqrt(D) here: under 2^-12.5, in numerator and
sum alike); a query's elements off by 2^-17 of its largest (D of them of either sign
add up to about sqrt(D), times a scale of 1 / sqrt(D): under 2^-14); exponentials and factors (2^-20).  Together below 2^-10.  A weight
under fp16's smallest normal number is off by 2^-25 of the largest: times the keys,
2^-25 n of the largest |V| of the row's keys.
"""

import numpy as np
import pytest
import torch

import chunked_prefill_hybrid_sar_gb300 as sar
from chunked_prefill_hybrid_sar_gb300 import _lib
from oracle import kv8

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


class Batch:
    """Sequences (rows, length) over scattered pages; everything outside them is NaN."""

    def __init__(self, seqs, heads, kv_heads, d, page, kind, seed=0, spread=0, table_fill=-1):
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.page, self.d = seqs, page, d
        need = [-(-m // page) for _, m in seqs]
        pool = sum(need) + 5
        order = torch.randperm(pool, generator=g)
        stride = max(need + [1]) + 1
        tables = torch.full((len(seqs), stride), table_fill, dtype=torch.int32)
        codes = torch.full((2, pool, kv_heads, page, d), 0x7F, dtype=torch.uint8)
        scales = torch.full((2, pool, kv_heads), float("nan"))
        at = 0
        for i, (_, m) in enumerate(seqs):
            p = order[at:at + need[i]]
            at += need[i]
            tables[i, :need[i]] = p.int()
            x = torch.randn(2, need[i], kv_heads, page, d, generator=g)
            c = (x * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            live = torch.arange(need[i] * page).view(need[i], page) < m
            c = torch.where(live[None, :, None, :, None], c, torch.tensor(0x7F, dtype=torch.uint8))
            codes[:, p] = c
            e = torch.randint(-spread, spread + 1, (2, need[i], kv_heads), generator=g).float()
            e[0] = e[0].clamp(-2, 1)
            s = torch.exp2(e) / 60
            if not spread:
                s = torch.full_like(s, 2.0 ** -6)
            scales[:, p] = s
        self.codes, self.scales, self.tables = codes, scales, tables
        self.rows = sum(r for r, _ in seqs)
        self.q = (1.3 * torch.randn(self.rows, heads * d, generator=g)).to(TYPES[kind])
        self.off = torch.tensor([0] + list(np.cumsum([r for r, _ in seqs])), dtype=torch.int32)
        self.lens = torch.tensor([m for _, m in seqs], dtype=torch.int32)

    def keys(self, i, kind):
        m = self.seqs[i][1]
        p = self.tables[i, :-(-m // self.page)].long()
        x = kv8.E4M3[self.codes[kind, p].numpy()] * self.scales[kind, p].double().numpy()[:, :, None, None]
        return x.transpose(0, 2, 1, 3).reshape(-1, x.shape[1], self.d)[:m]

    def cache(self):
        return sar.KV8Cache(*(t.contiguous().cuda() for t in (self.codes[0], self.codes[1], self.scales[0], self.scales[1])))

    def run(self, extra=0, cache=None, **kw):
        self.out = torch.full((self.rows + extra, self.q.shape[1]), 77.0, dtype=self.q.dtype, device="cuda")
        q = torch.cat([self.q, self.q[:1].expand(extra, -1)]).cuda()
        sar.kv8_attention(q, cache or self.cache(), self.off.cuda(), self.lens.cuda(), self.tables.cuda(), self.out, **kw)
        assert bool((self.out[self.rows:] == 77).all())
        return self.out[:self.rows].double().cpu().numpy().reshape(self.rows, -1, self.d)

    def check(self, window=0, scale=None, **kw):
        got = self.run(window=window, scale=0.0 if scale is None else scale, **kw)
        q = self.q.double().numpy().reshape(self.rows, -1, self.d)
        eps = torch.finfo(self.q.dtype).eps / 2
        for i, (r, m) in enumerate(self.seqs):
            if r == 0:
                continue
            a, b = int(self.off[i]), int(self.off[i + 1])
            k, v = self.keys(i, 0), self.keys(i, 1)
            want = kv8.attention(q[a:b], k, v, r, window, scale)
            mean = kv8.attention(q[a:b], k, np.abs(v), r, window, scale)
            far = np.abs(v).max(initial=0) * m * 2.0 ** -25
            off = np.abs(got[a:b] - want)
            assert np.isfinite(got[a:b]).all(), i
            assert (off <= eps * np.abs(want) + 2.0 ** -10 * mean + far).all(), (i, off.max())
        return got


SHAPES = [(32, 8, 128), (8, 1, 128), (7, 1, 128), (4, 4, 64), (6, 2, 64), (10, 2, 128)]


@pytest.mark.parametrize("heads,kv_heads,d", SHAPES)
@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("kind", list(TYPES))
def test_single_tokens(heads, kv_heads, d, page, kind):
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 200, 513]
    Batch([(1, m) for m in lens], heads, kv_heads, d, page, kind, seed=page + d).check(max_rows=1)
    sar.op_sync_status()


@pytest.mark.parametrize("heads,kv_heads,d", SHAPES)
@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("kind", list(TYPES))
def test_rows_of_every_number(heads, kv_heads, d, page, kind):
    """Chunks from the start and deep into a prompt, beside single tokens, empty and idle sequences."""
    seqs = [(1, 40), (5, 5), (2, 70), (0, 33), (17, 17), (1, 0), (3, 130), (33, 200), (1, 1), (4, 2), (64, 64), (1, 300)]
    Batch(seqs, heads, kv_heads, d, page, kind, seed=page).check(extra=2)
    sar.op_sync_status()


@pytest.mark.parametrize("n,m", [(1, 5000), (3, 2111), (1, 20000)])
def test_long_contexts_are_shared_out(n, m):
    Batch([(1, m - 7 * i) for i in range(n)], 4, 2, 128, 16, "f16", seed=m).check(max_rows=1)


def test_very_different_lengths():
    Batch([(1, m) for m in (1, 4000, 3, 0, 900, 17, 1, 1, 2500, 64)], 8, 2, 64, 32, "bf16").check()


@pytest.mark.parametrize("window", [1, 7, 16, 33, 100, 1000])
@pytest.mark.parametrize("kind", list(TYPES))
def test_windows(window, kind):
    seqs = [(1, 1), (1, 50), (1, 257), (20, 20), (30, 300), (1, 700), (3, 8)]
    Batch(seqs, 4, 2, 128, 16, kind, seed=window).check(window=window)
    Batch(seqs, 4, 2, 64, 64, kind, seed=window).check(window=window)
    sar.op_sync_status()


def test_pages_behind_a_window_may_be_gone():
    b = Batch([(1, 300), (1, 90), (20, 400)], 4, 2, 128, 16, "f16")
    full = b.run(window=40)
    for i, first in enumerate((300 - 40, 90 - 40, 400 - 20 - 39)):
        b.tables[i, :first // 16] = -1
    assert np.array_equal(b.run(window=40), full)
    sar.op_sync_status()


@pytest.mark.parametrize("spread", [1, 4, 9])
@pytest.mark.parametrize("rows", [1, 40])
def test_scales_of_every_size_beside_each_other(spread, rows):
    """Page scales that are no powers of two, and differ from page to page."""
    Batch([(rows, 333), (1, 50)], 4, 2, 128, 16, "f16", seed=spread, spread=spread).check()
    Batch([(rows, 333), (1, 50)], 8, 1, 64, 32, "bf16", seed=spread, spread=spread).check()


@pytest.mark.parametrize("exponent", [-100, -20, 20, 100])
def test_bf16_queries_of_any_size(exponent):
    """Query rows far outside fp16's range, undone by the scale."""
    b = Batch([(1, 60), (30, 90)], 4, 2, 128, 16, "bf16")
    same = b.run()
    b.q = (b.q.float() * 2.0 ** exponent).bfloat16()
    got = b.run(scale=2.0 ** -exponent * 128 ** -0.5)
    assert np.array_equal(got, same)


def test_large_scores():
    b = Batch([(1, 200), (40, 200)], 4, 2, 128, 16, "f16")
    b.q *= 40
    # (fp32 sums of scores this large are off by 40 times as much)
    got = b.run()
    q = b.q.double().numpy().reshape(b.rows, -1, 128)
    for i, (r, m) in enumerate(b.seqs):
        a, e = int(b.off[i]), int(b.off[i + 1])
        want = kv8.attention(q[a:e], b.keys(i, 0), b.keys(i, 1), r)
        assert np.abs(got[a:e] - want).max() <= 2.0 ** -6 * np.abs(b.keys(i, 1)).max()


@pytest.mark.parametrize("scale", [0.01, 0.5])
def test_scale(scale):
    Batch([(1, 77), (12, 77)], 4, 2, 64, 16, "f16").check(scale=scale)


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("d", [64, 128])
def test_nan_reaches_the_rows_that_see_it_alone(page, d):
    """A NaN value stays in its dim of the rows that see its key; a NaN key fills them."""
    b = Batch([(40, 100), (1, 100), (1, 60)], 4, 2, d, page, "f16")
    clean = b.run()

    def poke(kind, seq, key, head, dim):
        b.codes[kind, b.tables[seq, key // page], head, key % page, dim] = 0xFF

    poke(1, 0, 90, 1, 5)   # seen by rows 30.. of the chunk
    poke(0, 0, 95, 0, 9)   # rows 35..
    poke(1, 1, 50, 0, 33)
    poke(0, 2, 10, 1, 0)
    got = b.run()
    want = np.zeros(got.shape, bool)
    want[30:40, 2:, 5] = True
    want[35:40, :2] = True
    want[40, :2, 33] = True
    want[41, 2:] = True
    assert np.array_equal(np.isnan(got), want) and np.array_equal(got[~want], clean[~want])


def test_queries_that_are_not_finite():
    b = Batch([(1, 50), (1, 50), (9, 50)], 4, 2, 128, 16, "bf16")
    clean = b.run()
    b.q[0, 3], b.q[1, 130], b.q[5, 200] = float("nan"), float("inf"), float("-inf")
    got = b.run()
    bad = np.zeros(got.shape[:2], bool)
    bad[0, 0] = bad[1, 1] = bad[5, 1] = True
    assert np.isnan(got[bad]).all() and np.array_equal(got[~bad], clean[~bad])


def test_nothing_to_see_is_zero():
    got = Batch([(1, 0), (4, 2), (3, 0), (1, 5)], 4, 2, 128, 16, "f16").run()
    assert not got[0].any() and not got[1:3].any() and got[3:5].any(-1).all() and not got[5:8].any()
    sar.op_sync_status()


@pytest.mark.parametrize("shift,extra", [(8, 8), (1, 1), (2, 0), (3, 5)])
def test_strided_and_unaligned_rows(shift, extra):
    b = Batch([(1, 50), (30, 90), (1, 400)], 4, 2, 128, 16, "f16")
    want = b.run()
    n, w = b.q.shape
    q = torch.zeros(n, shift + w + extra, dtype=b.q.dtype, device="cuda")
    out = torch.full_like(q, 5.0)
    q[:, shift:shift + w] = b.q.cuda()
    sar.kv8_attention(q[:, shift:shift + w], b.cache(), b.off.cuda(), b.lens.cuda(), b.tables.cuda(), out[:, shift:shift + w])
    assert np.array_equal(out[:, shift:shift + w].double().cpu().numpy().reshape(want.shape), want)
    assert bool((out[:, :shift] == 5).all()) and bool((out[:, shift + w:] == 5).all())


def test_bad_sequences_are_left_out_and_reported():
    b = Batch([(1, 50), (1, 60), (2, 70), (1, 80)], 4, 2, 128, 16, "f16")
    want = b.run()
    sar.op_sync_status()
    b.lens[1] = 10 ** 6  # past its block table
    got = b.run()
    assert (got[1] == 77).all() and np.array_equal(np.delete(got, 1, 0), np.delete(want, 1, 0))
    with pytest.raises(sar.SarError) as e:
        sar.op_sync_status()
    assert e.value.code == _lib.SAR_ERR_BOUNDS
    b.lens[1] = 60
    got = b.run(max_rows=1)  # the third has two
    assert (got[2:4] == 77).all() and np.array_equal(got[[0, 1, 4]], want[[0, 1, 4]])
    with pytest.raises(sar.SarError):
        sar.op_sync_status()
    b.off[2] = 0  # the second's offsets fall, the third takes its rows too
    b.off[2:] = torch.tensor([0, 9, 10])
    b.run()
    with pytest.raises(sar.SarError):
        sar.op_sync_status()


def test_bad_pages_are_reported():
    b = Batch([(1, 50), (1, 60), (20, 70)], 4, 2, 128, 16, "f16")
    want = b.run()
    for bad in (-1, 10 ** 6):
        b.tables[1, 1] = bad
        got = b.run()
        assert np.array_equal(np.delete(got, 1, 0), np.delete(want, 1, 0))
        with pytest.raises(sar.SarError) as e:
            sar.op_sync_status()
        assert e.value.code == _lib.SAR_ERR_BOUNDS
    b.tables[1, 1], b.tables[2, 2] = 0, -5
    assert np.array_equal(b.run()[:1], want[:1])
    with pytest.raises(sar.SarError):
        sar.op_sync_status()


def test_two_streams_and_a_captured_call():
    """Two calls under way at once with workspaces of their own, and a replayed one on new lengths."""
    b = [Batch([(1, 900 + 50 * i) for i in range(20)] + [(30, 200)], 4, 2, 128, 16, "f16", seed=s) for s in (1, 2)]
    want = [x.run() for x in b]
    streams = [torch.cuda.Stream() for _ in b]
    args = [(x.q.cuda(), x.cache(), x.off.cuda(), x.lens.cuda(), x.tables.cuda(), torch.empty_like(x.out)) for x in b]
    torch.cuda.synchronize()
    for _ in range(5):
        for a, s in zip(args, streams):
            sar.kv8_attention(*a, stream=s)
    torch.cuda.synchronize()
    for a, w in zip(args, want):
        assert np.array_equal(a[5].double().cpu().numpy().reshape(w.shape), w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sar.kv8_attention(*args[0])
    for cut in (0, 37, 500):
        lens = b[0].lens - cut * (b[0].lens > 600).int()
        args[0][3].copy_(lens)
        graph.replay()
        torch.cuda.synchronize()
        c = Batch([(1, 900 + 50 * i) for i in range(20)] + [(30, 200)], 4, 2, 128, 16, "f16", seed=1)
        c.lens = lens
        assert np.array_equal(args[0][5].double().cpu().numpy().reshape(want[0].shape), c.run())


def test_results_repeat():
    b = Batch([(1, 3001), (1, 17), (70, 900)], 8, 2, 128, 16, "bf16")
    first = b.run()
    for _ in range(3):
        assert np.array_equal(b.run(), first)


def test_python_refusals():
    b = Batch([(1, 20), (2, 30)], 4, 2, 128, 16, "f16")
    good = dict(q=b.q.cuda(), cache=b.cache(), row_offsets=b.off.cuda(), lens=b.lens.cuda(), block_tables=b.tables.cuda(),
                out=torch.empty_like(b.q, device="cuda"))
    for kw in (dict(q=good["q"].float()), dict(q=good["q"][:, :-1]), dict(out=good["out"][:2]), dict(out=good["out"].bfloat16()),
               dict(row_offsets=good["row_offsets"][:2]), dict(lens=good["lens"].long()), dict(block_tables=good["block_tables"][:1]),
               dict(workspace=torch.empty(4, device="cuda")), dict(lens=good["lens"].cpu())):
        with pytest.raises(ValueError):
            sar.kv8_attention(**(good | kw))
    with pytest.raises(sar.SarError):
        sar.kv8_attention(**good, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    empty = good["q"][:0]
    sar.kv8_attention(empty, good["cache"], good["row_offsets"][:1], good["lens"][:0], good["block_tables"], empty)


@pytest.mark.parametrize("seqs,heads,kv_heads,d", [
    ([(2 + i % 4, 20 + i) for i in range(270)], 4, 2, 64),                   # more sequences than a call shares out
    ([(400, 500)] + [(2 + i % 5, 100 + i) for i in range(74)], 32, 8, 64),   # four units and more to an SM
    ([(1300, 1300)], 32, 8, 64),                                             # one and more
    ([(3, 60 + i % 50) if i % 3 else (1, 200) for i in range(150)], 56, 8, 128),
])
def test_many_chunks(seqs, heads, kv_heads, d):
    Batch(seqs, heads, kv_heads, d, 16, "bf16", seed=len(seqs)).check(extra=1)
    sar.op_sync_status()


def on_device(heads, kv_heads, d, page, pages, seqs, seed, room=0):
    """Sequences over the last pages of a pool that is filled there, and on the device their float64 attention."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-m // page) for _, m in seqs]
    first = room
    order = first + torch.randperm(pages, generator=g, device="cuda")
    codes = [torch.empty(first + pages, kv_heads, page, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((first + pages, kv_heads), 2.0 ** -6, device="cuda") for _ in range(2)]
    for c in codes:
        for at in range(first, first + pages, 512):  # (a piece at a time)
            part = c[at:at + 512]
            x = torch.randn(part.shape, generator=g, device="cuda") * 60
            part.copy_(x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    tables = torch.full((len(seqs), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        tables[i, :n] = order[at:at + n].int()
        at += n
    rows = [r for r, _ in seqs]
    off = torch.tensor([0] + list(np.cumsum(rows)), dtype=torch.int32, device="cuda")
    lens = torch.tensor([m for _, m in seqs], dtype=torch.int32, device="cuda")
    # (large queries: a few keys decide, wherever they lie)
    q = (3.0 * torch.randn(sum(rows), heads * d, generator=g, device="cuda")).half()
    table = torch.tensor(kv8.E4M3, device="cuda")

    def want(i):
        a, b, m = int(off[i]), int(off[i + 1]), seqs[i][1]
        p = tables[i, :need[i]].long()
        k, v = (table[c[p].long()].mul_(2.0 ** -6).transpose(1, 2).reshape(-1, kv_heads, d)[:m] for c in codes)
        x = q[a:b].double().view(b - a, kv_heads, heads // kv_heads, d)
        s = torch.einsum("rhgd,khd->rhgk", x, k) * d ** -0.5
        pos = torch.arange(m - (b - a), m, device="cuda")
        s.masked_fill_(torch.arange(m, device="cuda")[None, None, None] > pos[:, None, None, None], float("-inf"))
        w = torch.softmax(s, -1)
        far = v.abs().max() * m * 2.0 ** -25
        out, mean = (torch.einsum("rhgk,khd->rhgd", w, u).reshape(b - a, -1) for u in (v, v.abs()))
        return slice(a, b), out, 2.0 ** -11 * out.abs() + 2.0 ** -10 * mean + far

    return q, sar.KV8Cache(*codes, *scales), off, lens, tables, want


def test_more_keys_than_one_wave_of_stretches():
    """Single tokens over so many keys that the line's end is shared out a second time."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    seqs = [(1, sms * 1100 - 1111 * i) for i in range(12)]  # over 3 * 256 * 32 keys to an SM, in two heads
    assert sum(m for _, m in seqs) * 2 // 32 > 3 * sms * 256
    q, cache, off, lens, tables, want = on_device(4, 2, 64, 64, sum(-(-m // 64) for _, m in seqs), seqs, 1)
    out = torch.empty_like(q)
    sar.kv8_attention(q, cache, off, lens, tables, out, max_rows=1)
    for i in range(len(seqs)):
        rows, w, tol = want(i)
        assert bool(((out[rows].double() - w).abs() <= tol).all()), i
    # and cut by hints, into fewer stretches, and with a window
    for kw in (dict(max_len=1000), dict(max_len=10 ** 8)):
        again = torch.empty_like(q)
        sar.kv8_attention(q, cache, off, lens, tables, again, max_rows=1, **kw)
        assert bool(((again[rows].double() - w).abs() <= tol).all())
    sar.op_sync_status()


def test_codes_beyond_four_gigabytes():
    """Pages whose codes lie more than 2^32 bytes into the cache: appended to, and read by both kernels."""
    heads, kv_heads, d, page = 8, 4, 128, 64
    room = 2 ** 32 // (kv_heads * d * page) + 5
    seqs = [(1, 1000), (70, 333), (1, 64), (2, 129)]
    q, cache, off, lens, tables, want = on_device(heads, kv_heads, d, page, 30, seqs, 2, room=room)
    out = torch.empty_like(q)
    sar.kv8_attention(q, cache, off, lens, tables, out)
    for i in range(len(seqs)):
        rows, w, tol = want(i)
        assert bool(((out[rows].double() - w).abs() <= tol).all()), i
    # a key of 2^-6 * 64 in the last page's last place: code 2^6, of a scale that stays
    k = torch.ones(1, kv_heads * d, dtype=torch.float16, device="cuda")
    slot = (room + 30) * page - 1
    sar.qk_norm_rope(None, k, None, head_dim=d, v=k, cache=cache, slots=torch.tensor([slot], dtype=torch.int32, device="cuda"))
    one = torch.tensor([64.0]).to(torch.float8_e4m3fn).view(torch.uint8).item()
    for codes, scales in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)):
        assert bool((codes[-1, :, -1] == one).all()) and bool((scales[-1] == 2.0 ** -6).all())
    sar.op_sync_status()


@pytest.mark.parametrize("seqs,window", [
    ([(64, 2000)], 0), ([(50, 1500)] * 3 + [(1, 300)], 0), ([(3, 700)] * 20, 256), ([(130, 130)], 0), ([(2, 5000)], 0),
    ([(40, 1200), (40, 400), (40, 30)], 0), ([(9, 640)] * 90, 0),
])
@pytest.mark.parametrize("kind", list(TYPES))
def test_units_alike_and_not(seqs, window, kind):
    """Chunks whose units get the same number of CTAs each, and some of very different lengths."""
    Batch(seqs, 8, 2, 128, 32, kind, seed=len(seqs)).check(window=window)
    sar.op_sync_status()
