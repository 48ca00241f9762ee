"""Head norms, rotation and the 8-bit append against the float64 oracle.

Rows that are written: off by the rounding to 16 bits (half a step) and by fp32
steps: a norm's sum, root and two products, a rotation's sine (2^-23) and three
operations, under 16 roundings of 2^-24 on values up to sqrt(2) times the head's
largest: within 2^-19 of it.  Codes: as near, and the rounding to e4m3 (half a
step: 2^-4 of the value, 2^-10 of the scale near zero).  Values, and keys without
norm and rotation, take no arithmetic but exact scaling: equal codes.
"""

import numpy as np
import pytest
import torch

import chunked_prefill_hybrid_sar_gb300 as sar
from chunked_prefill_hybrid_sar_gb300 import _lib
from oracle import kv8

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS, BASE = 1e-5, 10000.0


def runs(page, kind, seed=0):
    """Slots of rows, position by position: single tokens, chunks, odd ends, rows that are not cached."""
    g = np.random.default_rng(seed)
    pages = list(g.permutation(60))

    def chunk(first, n):
        out, p = [], pages.pop()
        for j in range(first, first + n):
            if j and j % page == 0 and out:
                p = pages.pop()
            out.append(p * page + j % page)
        return out

    if kind == "singles":
        return sum([chunk(int(g.integers(0, page)), 1) for _ in range(37)], [])
    if kind == "chunk":
        return chunk(page - 3, 2 * page + 11)
    if kind == "aligned":
        return chunk(0, 3 * page)
    # a hybrid step, with rows behind the last and refused ones in between
    return chunk(5, page + 30) + [-1, -1] + chunk(0, 1) + chunk(page - 1, 1) + chunk(page - 1, 5) + [-1] + chunk(0, 20) + [-1] * 3


def case(kind, slots, heads, kv_heads, d, page, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    rows = len(slots)
    q, k, v = (spread * torch.randn(rows, h * d, generator=g) for h in (heads, kv_heads, kv_heads))
    k *= torch.exp2(torch.randint(-6, 7, (rows, 1), generator=g).float())
    v *= torch.exp2(torch.randint(-6, 7, (rows, 1), generator=g).float())
    x = [t.to(TYPES[kind]).cuda() for t in (q, k, v)]
    codes = [torch.randint(0, 127, (60, kv_heads, page, d), generator=g, dtype=torch.uint8).cuda() for _ in range(2)]
    scales = [torch.exp2(torch.randint(-9, 4, (60, kv_heads), generator=g).float()).cuda() for _ in range(2)]
    cache = sar.KV8Cache(codes[0], codes[1], scales[0], scales[1])
    pos = torch.randint(0, 70000, (rows,), generator=g, dtype=torch.int32)
    return x, cache, pos


def heads_of(t, d):
    return t.double().cpu().numpy().reshape(t.shape[0], -1, d)


def want_rows(x, gain, pos, d):
    gain = None if gain is None else gain.double().cpu().numpy()
    return np.stack([np.stack([kv8.turned(h, gain, EPS, None if pos is None else int(pos[r]), BASE) for h in row])
                     for r, row in enumerate(heads_of(x, d))])


def near(got, want, x, gain, d):
    """Written rows against the oracle's; x: the heads before, whose largest value is the scale of the fp32 steps."""
    most = np.abs(want).max(-1, keepdims=True)
    eps = torch.finfo(got.dtype).eps / 2
    bad = np.abs(heads_of(got, d) - want) > eps * np.abs(want) + 2.0 ** -19 * most * 2 ** 0.5 + 2.0 ** -25
    assert not bad.any()


def check_cache(cache, before, y, v, slots, exact_k):
    for name, rows, exact in (("k", y, exact_k), ("v", v, True)):
        old_codes, old_scales = (t.cpu().numpy() for t in before[name])
        codes, scales = (getattr(cache, f"{name}_{w}").cpu().numpy() for w in ("codes", "scales"))
        want_codes, want_scales = kv8.write(old_codes, old_scales, rows, slots)
        assert np.array_equal(scales, want_scales.astype(np.float32)), name
        if exact:
            assert np.array_equal(kv8.E4M3[codes], kv8.E4M3[want_codes], equal_nan=True), name
            continue
        fresh = np.zeros(codes.shape[:3], bool).transpose(0, 2, 1)
        page = codes.shape[2]
        for r, s in enumerate(slots):
            if s < 0:
                continue
            p, o = divmod(s, page)
            fresh[p, o] = True
            sc = scales[p][:, None]
            off = np.abs(kv8.E4M3[codes[p, :, o]] * sc - rows[r])
            most = np.abs(rows[r]).max(-1, keepdims=True)
            assert (off <= np.maximum(np.abs(rows[r]) * 2.0 ** -4, sc * 2.0 ** -10) + 2.0 ** -19 * 2 ** 0.5 * most).all()
        # what was there: as the oracle has it, anew where the scale grew
        assert np.array_equal(kv8.E4M3[codes].transpose(0, 2, 1, 3)[~fresh], kv8.E4M3[want_codes].transpose(0, 2, 1, 3)[~fresh],
                              equal_nan=True)


def snapshot(cache):
    return {n: (getattr(cache, n + "_codes").clone(), getattr(cache, n + "_scales").clone()) for n in "kv"}


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("pattern", ["singles", "chunk", "aligned", "hybrid"])
@pytest.mark.parametrize("heads,kv_heads,d,page", [(8, 2, 128, 16), (7, 1, 128, 64), (4, 4, 64, 32), (6, 2, 64, 16), (5, 5, 128, 32)])
def test_rows_and_cache(kind, pattern, heads, kv_heads, d, page):
    slots = runs(page, pattern, heads)
    (q, k, v), cache, pos = case(kind, slots, heads, kv_heads, d, page, heads * d + page)
    norm, turn = pattern != "chunk", pattern != "aligned"
    gains = [(1 + 0.2 * torch.randn(d)).cuda() for _ in range(2)] if norm else [None, None]
    at = pos if turn else None
    out_t = torch.bfloat16 if kind == "bf16" else torch.float16
    q_out = torch.empty(q.shape, dtype=out_t, device="cuda")
    k_out = torch.empty(k.shape, dtype=out_t, device="cuda") if pattern != "singles" else None
    before = snapshot(cache)
    sar.qk_norm_rope(q, k, q_out, head_dim=d, positions=None if at is None else at.cuda(), v=v, k_out=k_out, cache=cache,
                     slots=torch.tensor(slots, dtype=torch.int32, device="cuda"), q_gain=gains[0], k_gain=gains[1], eps=EPS,
                     rope_base=BASE)
    near(q_out, want_rows(q, gains[0], at, d), q, gains[0], d)
    y = want_rows(k, gains[1], at, d)
    if k_out is not None:
        near(k_out, y, k, gains[1], d)
    check_cache(cache, before, y, heads_of(v, d), slots, exact_k=not norm and not turn)
    sar.op_sync_status()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [1, 15, 16, 17, 33, 600])
def test_without_a_cache_and_in_place(d, rows):
    (q, k, _), _, pos = case("bf16", [-1] * rows, 3, 2, d, 16, rows)
    gain = (1 + 0.2 * torch.randn(d)).cuda()
    want_q, want_k = want_rows(q, gain, pos, d), want_rows(k, None, pos, d)
    sar.qk_norm_rope(q, k, q, head_dim=d, positions=pos.cuda(), k_out=k, q_gain=gain, eps=EPS)
    near(q, want_q, q, gain, d)
    near(k, want_k, k, None, d)


def test_only_keys_and_only_queries():
    (q, k, v), cache, pos = case("f16", [3, 4], 4, 2, 128, 16, 1)
    q_out = torch.empty_like(q)
    sar.qk_norm_rope(q, None, q_out, head_dim=128, positions=pos.cuda())
    near(q_out, want_rows(q, None, pos, 128), q, None, 128)
    before = snapshot(cache)
    sar.qk_norm_rope(None, k, None, head_dim=128, v=v, cache=cache, slots=torch.tensor([3, 4], dtype=torch.int32, device="cuda"))
    check_cache(cache, before, heads_of(k, 128), heads_of(v, 128), [3, 4], exact_k=True)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("shift,extra", [(0, 0), (4, 4), (1, 3), (8, 1)])
def test_strided_and_unaligned_rows(kind, shift, extra):
    """Queries, keys and values side by side in one buffer, as a fused projection leaves them."""
    d, heads, kv_heads, slots = 128, 3, 2, runs(16, "hybrid")
    (q, k, v), cache, pos = case(kind, slots, heads, kv_heads, d, 16, 3)
    n = len(slots)
    wide = torch.full((n, shift + q.shape[1] + 2 * k.shape[1] + extra), 7.0, dtype=q.dtype, device="cuda")
    views, at = [], shift
    for t in (q, k, v):
        views.append(wide[:, at:at + t.shape[1]])
        views[-1].copy_(t)
        at += t.shape[1]
    out_t = torch.bfloat16 if kind == "bf16" else torch.float16
    out = torch.full((n, shift + q.shape[1] + extra), 7.0, dtype=out_t, device="cuda")
    q_out = out[:, shift:shift + q.shape[1]]
    before = snapshot(cache)
    sar.qk_norm_rope(*views[:2], q_out, head_dim=d, positions=pos.cuda(), v=views[2], cache=cache,
                     slots=torch.tensor(slots, dtype=torch.int32, device="cuda"), eps=EPS)
    near(q_out, want_rows(q, None, pos, d), q, None, d)
    check_cache(cache, before, want_rows(k, None, pos, d), heads_of(v, d), slots, exact_k=False)
    assert bool((out[:, :shift] == 7).all()) and bool((out[:, shift + q.shape[1]:] == 7).all())


def test_growing_page_token_by_token():
    """One page filled a token at a time, its rows ever larger: as the oracle's, codes and scales."""
    d, page = 64, 32
    cache = sar.KV8Cache.empty(3, 2, page, d)
    codes, scales = np.zeros((3, 2, page, d), np.uint8), np.zeros((3, 2))
    vc, vs = codes.copy(), scales.copy()
    for j in range(page):
        x = (torch.randn(1, 2 * d) * 2.0 ** (j / 3 - 5)).half().cuda()
        y = (torch.randn(1, 2 * d) * 2.0 ** (5 - j)).half().cuda()
        sar.qk_norm_rope(None, x, None, head_dim=d, v=y, cache=cache, slots=torch.tensor([page + j], dtype=torch.int32, device="cuda"))
        codes, scales = kv8.write(codes, scales, heads_of(x, d), [page + j])
        vc, vs = kv8.write(vc, vs, heads_of(y, d), [page + j])
    for got, want in ((cache.k_codes, codes), (cache.v_codes, vc)):
        assert np.array_equal(kv8.E4M3[got.cpu().numpy()], kv8.E4M3[want])
    assert np.array_equal(cache.k_scales.cpu().numpy(), scales) and np.array_equal(cache.v_scales.cpu().numpy(), vs)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_borders_zeros_and_what_is_not_finite(kind):
    d, n = 128, 9
    x = torch.zeros(n, d)
    x[1, 0], x[2, 0], x[3, 0], x[4, 5] = 448, 449 if kind == "f32" else 452, 1e-30, 3e38
    x[5, 3], x[6, 4], x[7, 9] = float("nan"), float("inf"), float("-inf")
    x[5:8, 100] = 3.0
    x[8, :8] = torch.tensor([448, 26, 1.0625, -0.001953125, 0.0009765625, 2 ** -11, 464, -17])
    slots = [16 * i for i in range(n)]  # a page each
    k = x.to(TYPES[kind]).cuda()
    cache = sar.KV8Cache.empty(10, 1, 16, d)
    before = snapshot(cache)
    sar.qk_norm_rope(None, k, None, head_dim=d, v=k, cache=cache, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    check_cache(cache, before, heads_of(k, d), heads_of(k, d), slots, exact_k=True)
    assert cache.k_scales[3].item() == cache.k_scales[0].item() == 2.0 ** -40


def test_far_positions():
    """The angle of position 2^31 - 1, to fp32."""
    d = 128
    pos = torch.tensor([2 ** 31 - 1, 1234567891, 0, 1], dtype=torch.int32)
    q = torch.randn(4, d, generator=torch.Generator().manual_seed(1)).half().cuda()
    out = torch.empty_like(q)
    for base in (10000.0, 500000.0, 1.0):
        sar.qk_norm_rope(q, None, out, head_dim=d, positions=pos.cuda(), rope_base=base)
        x = heads_of(q, d)
        want = np.stack([np.stack([kv8.turned(h, None, 0, int(p), np.longdouble(base)) for h in row]) for row, p in zip(x, pos)])
        # (theta's own rounding in doubles: 2^-53 of an angle of up to 2^31)
        assert np.abs(heads_of(out, d) - want).max() <= (2.0 ** -11 + 2.0 ** -18 + 2.0 ** -19) * np.abs(x).max() * 2 ** 0.5


def test_slots_out_of_range_are_reported():
    (q, k, v), cache, _ = case("f16", [5, 6, 7, 8], 2, 1, 128, 16, 2)
    before = snapshot(cache)
    slots = [17, 60 * 16, -2, 33]
    sar.qk_norm_rope(None, k, None, head_dim=128, v=v, cache=cache, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    check_cache(cache, before, heads_of(k, 128), heads_of(v, 128), slots, exact_k=True)
    with pytest.raises(sar.SarError) as e:
        sar.op_sync_status()
    assert e.value.code == _lib.SAR_ERR_BOUNDS


def test_python_refusals():
    (q, k, v), cache, pos = case("f16", [5, 6], 2, 1, 128, 16, 2)
    slots = torch.tensor([5, 6], dtype=torch.int32, device="cuda")
    for kw in (dict(v=None), dict(slots=None), dict(v=v[:1]), dict(v=v.float()), dict(slots=slots[:1]), dict(slots=slots.long()),
               dict(k_gain=torch.ones(64, device="cuda")), dict(positions=pos.cuda()[:1]), dict(k_out=torch.empty_like(q)),
               dict(slots=slots.cpu())):
        with pytest.raises(ValueError):
            sar.qk_norm_rope(None, k, None, head_dim=128, **(dict(v=v, cache=cache, slots=slots) | kw))
    with pytest.raises(sar.SarError):
        sar.qk_norm_rope(q, None, torch.empty_like(q).bfloat16(), head_dim=128)


@pytest.mark.parametrize("kind,d,page", [("bf16", 128, 64), ("f32", 64, 16), ("f16", 128, 16), ("f32", 128, 32)])
def test_many_rows_are_as_few_at_a_time(kind, d, page):
    """So many rows that a CTA takes several heads: equal to the same rows in calls of a page each."""
    heads, kv_heads, pages = 24, 8, 7000 // page
    g = torch.Generator().manual_seed(page + d)
    order = torch.randperm(pages, generator=g).tolist()
    parts, at = [], 0  # runs of slots: whole pages, their ends, single tokens, rows that are not cached
    for p in order:
        first = 0 if at % 3 else int(torch.randint(0, page, (1,), generator=g))
        last = page if at % 4 else first + 1
        parts.append([p * page + o for o in range(first, last)])
        if at % 50 == 7:
            parts.append([-1] * 3)
        at += 1
    slots = torch.tensor(sum(parts, []), dtype=torch.int32, device="cuda")
    rows = slots.numel()
    x = torch.randn(rows, (heads + 2 * kv_heads) * d, generator=g).to(TYPES[kind]).cuda()
    pos = torch.randint(0, 200000, (rows,), generator=g, dtype=torch.int32).cuda()
    gain = (torch.rand(d, generator=g) + 0.5).cuda()
    out_type = torch.bfloat16 if kind == "f32" else TYPES[kind]

    def run(cuts):
        cache = sar.KV8Cache.empty(pages, kv_heads, page, d)
        for s in (cache.k_scales, cache.v_scales):
            s.fill_(2.0 ** -8)
        q_out = torch.zeros(rows, heads * d, dtype=out_type, device="cuda")
        k_out = torch.zeros(rows, kv_heads * d, dtype=out_type, device="cuda")
        for a, b in zip(cuts, cuts[1:]):
            q, k, v = x[a:b].split([heads * d, kv_heads * d, kv_heads * d], 1)
            sar.qk_norm_rope(q, k, q_out[a:b], d, positions=pos[a:b], v=v, k_out=k_out[a:b], cache=cache, slots=slots[a:b],
                             q_gain=gain, k_gain=gain)
        return q_out, k_out, cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales

    whole = run([0, rows])
    for got, want in zip(whole, run(np.cumsum([0] + [len(p) for p in parts]).tolist())):
        assert torch.equal(got, want)
    assert bool((whole[2] != 0).any()) and bool((whole[0] != 0).any(-1).all())
    sar.op_sync_status()
