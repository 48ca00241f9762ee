"""Measured cases of the 8-bit KV cache.

Three operators, in the order in which a serving step meets them: block tables
and slot maps are built on the GPU from the requests' lengths (``map``); a
step's queries and keys are normalised for each head and rotated, and its keys
and values written into the paged cache in 8 bits with a power-of-two scale for
each page and head (``append``); rows attend to what the cache holds, single
tokens and chunks (``attend``).

Where ``own`` is false, ``run`` computes them from elementary torch operations
in 32 bits; where it is true it makes the framework's calls.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
LEAST, MOST = -40, 60  # exponents of a page's scale
EPS, BASE = 1e-5, 10000.0


# ---- cases -------------------------------------------------------------------


def listed():
    return [
        # the next token of one request: latency
        dict(name="map decode 1", op="map", n=1, longest=500, grow=1, page=16, mixed=False),
        # a full batch of decodes, some of which end, wait or come in with a chunk
        dict(name="map mixed 256", op="map", n=256, longest=8192, grow=64, page=16, mixed=True),
        # prompts admitted together, each up to 2048 tokens of a chunk
        dict(name="map prefill 64", op="map", n=64, longest=4096, grow=2048, page=64, mixed=False),
        # one decoding request's row
        dict(name="append decode 1", op="append", singles=1, chunks=0, chunk_rows=0, longest=500, hq=32, hkv=8, d=128,
             page=16, norm=True, type="bf16"),
        # a hybrid step: a 512-token chunk and five decodes
        dict(name="append hybrid 517", op="append", singles=5, chunks=1, chunk_rows=512, longest=1024, hq=32, hkv=8,
             d=128, page=16, norm=True, type="f16"),
        # two long prefills of a wide model, whose keys have no norm
        dict(name="append prefill 12288", op="append", singles=0, chunks=2, chunk_rows=8192, longest=8192, hq=56, hkv=8,
             d=128, page=64, norm=False, type="bf16"),
        # one decoding request over a short history: latency
        dict(name="attend decode 1", op="attend", singles=1, longest=500, chunks=0, chunk_rows=0, chunk_len=0, hq=32,
             hkv=8, d=128, page=16, window=0, type="bf16"),
        # a full batch of decodes of every length: the cache's bytes
        dict(name="attend decode 128", op="attend", singles=128, longest=8192, chunks=0, chunk_rows=0, chunk_len=0,
             hq=32, hkv=8, d=128, page=16, window=0, type="bf16"),
        # a few very long contexts of a wide model
        dict(name="attend long 4", op="attend", singles=4, longest=131072, chunks=0, chunk_rows=0, chunk_len=0, hq=56,
             hkv=8, d=128, page=64, window=0, type="f16"),
        # a hybrid step: one prompt's chunk deep into it, and decodes
        dict(name="attend hybrid 517", op="attend", singles=5, longest=1024, chunks=1, chunk_rows=512, chunk_len=16384,
             hq=32, hkv=8, d=128, page=16, window=0, type="f16"),
        # a whole prompt at once
        dict(name="attend prefill 8192", op="attend", singles=0, longest=0, chunks=1, chunk_rows=8192, chunk_len=8192,
             hq=32, hkv=8, d=128, page=32, window=0, type="bf16"),
        # a few guessed tokens a request to verify, under a sliding window
        dict(name="attend verify 32", op="attend", singles=7, longest=2000, chunks=25, chunk_rows=6, chunk_len=5000,
             hq=16, hkv=4, d=64, page=32, window=1024, type="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = [(32, 8, 128), (56, 8, 128), (32, 8, 128), (8, 1, 128), (16, 4, 64), (4, 4, 64), (12, 2, 64), (6, 6, 128)]


def draw(rng):
    op = rng.choice(["map", "append", "append", "attend", "attend", "attend", "attend"])
    page = rng.choice([16, 32, 64])
    if op == "map":
        n, mixed = _log(rng, 1, 1024), rng.random() < 0.6
        grow = rng.choice([1, 1, _log(rng, 1, 2048)])
        return dict(op=op, n=n, longest=_log(rng, 1, 16384), grow=min(grow, max(1, 131072 // n)), page=page, mixed=mixed)
    hq, hkv, d = rng.choice(HEADS)
    kind = rng.choice(["bf16", "f16"])
    if op == "append":
        chunks = rng.choice([0, 1, 2, 5])
        rows = _log(rng, 1, 8192 // max(1, chunks)) if chunks else 0
        return dict(op=op, singles=_log(rng, 1, 512) if chunks != 1 or rng.random() < 0.5 else 0, chunks=chunks,
                    chunk_rows=rows, longest=max(rows, _log(rng, 1, 16384)), hq=hq, hkv=hkv, d=d, page=page,
                    norm=rng.random() < 0.6, type=kind)
    singles = rng.choice([0, 1, _log(rng, 1, 256), _log(rng, 1, 256)])
    longest = _log(rng, 1, 131072)
    longest = max(1, min(longest, 128 * 8192 * 8 * 128 // max(1, singles * hkv * d)))
    chunks = rng.choice([0, 1, 3, _log(rng, 1, 32)]) if singles else rng.choice([1, 4])
    rows = _log(rng, 1, 4096) if chunks else 0
    most = int(math.sqrt(8192 * 8192 * 32 * 128 / (hq * d * max(1, chunks))))
    rows = min(rows, most)
    length = max(rows, min(_log(rng, 1, 32768), most * most // max(1, rows))) if chunks else 0
    length = max(rows, min(length, 128 * 8192 * 8 // max(1, chunks * hkv)))
    return dict(op=op, singles=singles, longest=longest if singles else 0, chunks=chunks, chunk_rows=rows,
                chunk_len=length, hq=hq, hkv=hkv, d=d, page=page, window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]),
                type=kind)


def _spread(n, longest):
    """n lengths from short to the longest."""
    return [max(1, longest * (i + 1) // n) for i in range(n)]


def _batch(case):
    """(rows, length with them) of each sequence, in the order of ``prepare`` but for its shuffling."""
    single = [(1, m) for m in _spread(case["singles"], case["longest"])] if case["singles"] else []
    if not case["chunks"]:
        return single
    rows = _spread(case["chunks"], case["chunk_rows"])
    length = case["chunk_len"] if case["op"] == "attend" else case["longest"]
    return [(r, max(r, m)) for r, m in zip(rows, reversed(_spread(case["chunks"], length)))] + single


# ---- inputs ------------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _tables(g, need, stride, page_count):
    """Block tables whose pages are scattered over the pool, and the pages left."""
    pages = torch.randperm(page_count, generator=g, device=DEV).to(torch.int32)
    first = torch.tensor([0] + need, device=DEV).cumsum(0)
    j = torch.arange(stride, device=DEV)
    at = first[:-1, None] + j
    inside = j < torch.tensor(need, device=DEV)[:, None]
    return torch.where(inside, pages[at.clamp(max=page_count - 1)], -1), pages[int(first[-1]):].contiguous()


def _scales_of(amax):
    """The smallest power of two that brings a magnitude down to 448."""
    m, e = torch.frexp(amax)  # amax = m 2^e, 0.5 <= m < 1; 448 = 0.875 2^9
    e = torch.where(amax > 0, e - 9 + (m > 0.875), LEAST).clamp(LEAST, MOST)
    return torch.ldexp(torch.ones_like(amax), e)


def _codes_of(x, s):
    """e4m3 codes of x / s, s a power of two; what is not finite becomes NaN."""
    t = (x / s).clamp(-448, 448)
    return torch.where(torch.isfinite(x), t, math.nan).to(E4M3).view(torch.uint8)


def _cache(g, pages, hkv, page, d):
    """Codes and scales of keys and values as a model makes them: heads and channels differ in size."""
    out = []
    for kind in range(2):
        codes = torch.empty(pages, hkv, page, d, dtype=torch.uint8, device=DEV)
        scales = torch.empty(pages, hkv, device=DEV)
        gain = torch.exp(0.7 * torch.randn(hkv, 1, d, generator=g, device=DEV)) if kind == 0 else 1.0
        step = max(1, (1 << 26) // (hkv * page * d))
        for p in range(0, pages, step):
            n = min(step, pages - p)
            x = torch.randn(n, hkv, page, d, generator=g, device=DEV) * gain
            x = x * torch.exp(0.5 * torch.randn(n, hkv, 1, 1, generator=g, device=DEV))
            s = _scales_of(x.abs().amax((2, 3)))
            scales[p:p + n] = s
            codes[p:p + n] = _codes_of(x, s[:, :, None, None])
        out += [codes, scales]
    return out


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    if case["op"] == "map":
        _prepare_map(st, g)
        return st
    batch = _batch(case)
    order = torch.randperm(len(batch), generator=g, device=DEV).tolist()
    batch = [batch[i] for i in order]
    page, hq, hkv, d = st["page"], st["hq"], st["hkv"], st["d"]
    need = [-(-m // page) for _, m in batch]
    pool = sum(need) + 7
    st["tables"], _ = _tables(g, need, max(need), pool)
    st["lens"] = _ints([m for _, m in batch])
    st["offsets"] = torch.cat([_ints([0]), _ints([r for r, _ in batch]).cumsum(0).to(torch.int32)])
    rows = st["rows"] = sum(r for r, _ in batch)
    st["k_codes"], st["k_scales"], st["v_codes"], st["v_scales"] = _cache(g, pool, hkv, page, d)
    dt = TYPES[st["type"]]
    st["out"] = torch.empty(rows, hq * d, dtype=dt, device=DEV)
    if case["op"] == "attend":
        st["q"] = (1.5 * torch.randn(rows, hq * d, generator=g, device=DEV)).to(dt)
        st["most_rows"] = max(r for r, _ in batch)
        st["most_len"] = max(m for _, m in batch)
        one = [i for i, (r, _) in enumerate(batch) if r == 1]
        more = [i for i, (r, _) in enumerate(batch) if r > 1]
        st["groups"] = [(torch.tensor(v, device=DEV), max(batch[i][0] for i in v), max(batch[i][1] for i in v)) if v else None
                        for v in (one, more)]
        return st
    # the projection's fused rows: queries, keys, values side by side
    st["qkv"] = torch.randn(rows, (hq + 2 * hkv) * d, generator=g, device=DEV).to(dt)
    st["gains"] = [1 + 0.2 * torch.randn(d, generator=g, device=DEV) for _ in range(2)] if st["norm"] else [None, None]
    pos = torch.cat([torch.arange(m - r, m, device=DEV) for r, m in batch])
    seq = torch.cat([torch.full((r,), i, device=DEV) for i, (r, _) in enumerate(batch)])
    st["positions"] = pos.to(torch.int32)
    st["slots"] = (st["tables"][seq, pos // page] * page + pos % page).to(torch.int32)
    return st


def _map_batch(case):
    """(cached, new) of each request; -1 new: it has ended, 0: it waits."""
    out = []
    for i, m in enumerate(_spread(case["n"], case["longest"])):
        new = _spread(case["n"], case["grow"])[case["n"] - 1 - i] if case["grow"] > 1 else 1
        if case["mixed"]:
            new = (new, 1, 1, -1, 1, 0, 1, 1)[i % 8]
            m = 0 if i % 8 == 0 else m  # it comes in
        out.append((m, new))
    return out


def _prepare_map(st, g):
    batch = _map_batch(st)
    order = torch.randperm(len(batch), generator=g, device=DEV).tolist()
    batch = [batch[i] for i in order]
    page = st["page"]
    held = [-(-m // page) for m, _ in batch]
    need = [-(-(m + max(0, a)) // page) for m, a in batch]
    st["stride"] = max(need) + 1
    st["pool"] = sum(need) + 16
    tables, left = _tables(g, held, st["stride"], st["pool"])
    st["tables"], st["n_free"] = tables.contiguous(), left.numel()
    st["free"] = torch.full((st["pool"],), -1, dtype=torch.int32, device=DEV)
    st["free"][:left.numel()] = left
    st["count"] = _ints([left.numel()])
    st["count_out"] = torch.empty_like(st["count"])
    st["lens"], st["new"] = _ints([m for m, _ in batch]), _ints([a for _, a in batch])
    st["lens_out"] = torch.empty_like(st["lens"])
    # a fixed number of rows, as a captured step has: more than this batch takes
    st["rows"] = sum(max(0, a) for _, a in batch) + 5
    st["offsets"] = torch.empty(st["n"] + 1, dtype=torch.int32, device=DEV)
    st["positions"] = torch.empty(st["rows"], dtype=torch.int32, device=DEV)
    st["slots"] = torch.empty(st["rows"], dtype=torch.int32, device=DEV)


# ---- one pass ----------------------------------------------------------------


def run(st):
    return {"map": _run_map, "append": _run_append, "attend": _run_attend}[st["op"]](st)


def _handle(st):
    """The cache's handle, made once over the state's tensors."""
    if "cache" not in st:
        import chunked_prefill_hybrid_sar_gb300 as sar

        st["cache"] = sar.KV8Cache(st["k_codes"], st["v_codes"], st["k_scales"], st["v_scales"])
    return st["cache"]


def _run_map(st):
    if own:
        import chunked_prefill_hybrid_sar_gb300 as sar

        sar.page_map(st["lens"], st["new"], st["tables"], st["free"], st["count"], st["offsets"], st["positions"],
                     st["slots"], page_size=st["page"], lens_out=st["lens_out"], free_count_out=st["count_out"])
    else:
        _plain_map(st)
    return [st[k] for k in ("lens_out", "tables", "free", "count_out", "offsets", "positions", "slots")]


def _plain_map(st):
    page, pool, n, stride, most = st["page"], st["pool"], st["n"], st["stride"], st["rows"]
    lens, new = st["lens"].long(), st["new"].long()
    zero = torch.zeros(1, dtype=torch.int64, device=DEV)
    add = new.clamp(min=0)
    held = (lens + page - 1) // page
    rows_at = torch.cat([zero, add.cumsum(0)])
    fits = (rows_at[1:] <= most) | (add == 0)
    take = torch.where(fits, (lens + add + page - 1) // page - held, 0)
    give = torch.where(new < 0, held, 0)
    f = st["count"].long()
    take_at = torch.cat([zero, take.cumsum(0)])
    give_at = torch.cat([zero, give.cumsum(0)])
    have = f + give_at[-1]
    ok = fits & ((take == 0) | (take_at[1:] <= have))
    # the list with the pages given back behind it
    j = torch.arange(stride, device=DEV)
    behind = torch.where(j < give[:, None], f + give_at[:-1, None] + j, pool)
    free = torch.cat([st["free"], st["free"][:1]])
    full = free.scatter(0, behind.clamp(max=pool).view(-1), st["tables"].view(-1))[:pool]
    # every request's new pages, from the end of the list
    at = have - 1 - (take_at[:-1, None] + j - held[:, None])
    fresh = (j >= held[:, None]) & (j < (held + take)[:, None]) & ok[:, None]
    st["tables"].copy_(torch.where(fresh, full[at.clamp(0, pool - 1)], st["tables"]))
    i = torch.arange(pool, device=DEV)
    taken = torch.where(ok & (take > 0), take_at[1:], 0).amax()
    left = have - taken
    st["free"].copy_(torch.where((i >= f) & (i < left), full, st["free"]))
    st["count_out"].copy_(left)
    st["lens_out"].copy_(torch.where(new < 0, 0, torch.where(ok, lens + add, lens)))
    st["offsets"].copy_(rows_at.clamp(max=most))
    r = torch.arange(most, device=DEV)
    seq = torch.searchsorted(rows_at[1:], r, right=True)
    live = seq < n
    seq = seq.clamp(max=n - 1)
    pos = lens[seq] + r - rows_at[seq]
    pages = st["tables"][seq, (pos // page).clamp(max=stride - 1)].long()
    st["positions"].copy_(torch.where(live, pos, 0))
    st["slots"].copy_(torch.where(live & ok[seq], pages * page + pos % page, -1))


def _run_append(st):
    hq, hkv, d = st["hq"], st["hkv"], st["d"]
    q, k, v = st["qkv"].split([hq * d, hkv * d, hkv * d], 1)
    if own:
        import chunked_prefill_hybrid_sar_gb300 as sar

        sar.qk_norm_rope(q, k, st["out"], head_dim=d, positions=st["positions"], v=v, cache=_handle(st), slots=st["slots"],
                         q_gain=st["gains"][0], k_gain=st["gains"][1], eps=EPS, rope_base=BASE)
    else:
        _plain_append(st, q, k, v)
    return [st["out"], st["k_codes"].view(E4M3), st["v_codes"].view(E4M3), st["k_scales"], st["v_scales"]]


def _turned(x, gain, cos, sin):
    """Heads normalised (where there is a gain) and rotated, in 32 bits."""
    if gain is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gain
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_append(st, q, k, v):
    rows, hq, hkv, d = st["rows"], st["hq"], st["hkv"], st["d"]
    i = torch.arange(d // 2, dtype=torch.float64, device=DEV)
    angle = st["positions"].double()[:, None] * torch.pow(BASE, -2 * i / d)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    st["out"].copy_(_turned(q.float().view(rows, hq, d), st["gains"][0], cos, sin).view(rows, -1))
    page, off = st["slots"].long() // st["page"], st["slots"].long() % st["page"]
    _plain_write(_turned(k.float().view(rows, hkv, d), st["gains"][1], cos, sin), page, off, st["k_codes"], st["k_scales"])
    _plain_write(v.float().view(rows, hkv, d), page, off, st["v_codes"], st["v_scales"])


def _plain_write(x, page, off, codes, scales):
    pages, hkv, size, d = codes.shape
    amax = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
    at = page[:, None].expand(-1, hkv)
    most = torch.zeros_like(scales).scatter_reduce_(0, at, amax, "amax")
    first = torch.full((pages,), size, device=DEV).scatter_reduce_(0, page, off, "amin")  # its first new token
    part = ((first > 0) & (first < size))[:, None]  # pages that go on
    s = torch.where(part, torch.maximum(_scales_of(most), scales), _scales_of(most))
    s = torch.where((first < size)[:, None], s, scales)
    # what touched pages hold already, under their new scale
    old = codes[page].view(E4M3).float() * (scales / s)[page][:, :, None, None]
    keep = torch.arange(size, device=DEV) < first[page][:, None]
    codes[page] = torch.where(keep[:, None, :, None], _codes_of(old, torch.ones_like(old)), codes[page])
    codes[page, :, off] = _codes_of(x, s[page][:, :, None])
    scales.copy_(s)


def _run_attend(st):
    if own:
        import chunked_prefill_hybrid_sar_gb300 as sar

        if "space" not in st:  # kept beside the plan
            st["space"] = torch.empty(sar.kv8_attention_workspace(_handle(st), st["q"], st["lens"].numel(),
                                                                  max_rows=st["most_rows"], max_len=st["most_len"]),
                                      dtype=torch.uint8, device=DEV)
        sar.kv8_attention(st["q"], _handle(st), st["offsets"], st["lens"], st["tables"], st["out"],
                          max_rows=st["most_rows"], max_len=st["most_len"], window=st["window"], workspace=st["space"])
        return st["out"]
    if st["groups"][0] is not None:
        _plain_attend(st, *st["groups"][0])
    if st["groups"][1] is not None:
        _plain_attend(st, *st["groups"][1])
    return st["out"]


def _plain_attend(st, seqs, most_rows, most_len):
    """Sequences padded to one size."""
    hq, hkv, d, page = st["hq"], st["hkv"], st["d"], st["page"]
    n, group = seqs.numel(), hq // hkv
    first = st["offsets"].long()[seqs]
    rows = st["offsets"].long()[seqs + 1] - first
    lens = st["lens"].long()[seqs]
    key = torch.arange(most_len, device=DEV)
    pages = st["tables"][seqs][:, key // page].long().clamp(min=0)
    k = st["k_codes"][pages, :, key % page].view(E4M3).float() * st["k_scales"][pages][..., None]
    v = st["v_codes"][pages, :, key % page].view(E4M3).float() * st["v_scales"][pages][..., None]
    r = torch.minimum(torch.arange(most_rows, device=DEV), rows[:, None] - 1)  # (rows behind repeat the last)
    at = first[:, None] + r
    q = st["q"][at].float().view(n, most_rows, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)
    s = torch.matmul(q, k.permute(0, 2, 3, 1)) * d ** -0.5
    pos = (lens[:, None] - rows[:, None] + r)[:, None, None, :, None]
    seen = key <= pos
    if st["window"]:
        seen = seen & (key > pos - st["window"])
    s = s.view(n, hkv, group, most_rows, most_len).masked_fill_(~seen, -math.inf)
    s = s.sub_(s.amax(-1, keepdim=True)).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(n, hkv, -1, most_len), v.permute(0, 2, 1, 3)).view(n, hkv, group, most_rows, d) / total
    st["out"][at] = o.permute(0, 3, 1, 2, 4).reshape(n, most_rows, hq * d).to(st["out"].dtype)


# ---- what a pass cannot do without -------------------------------------------


def work(case):
    if case["op"] == "map":
        b = _map_batch(case)
        page = case["page"]
        taken = sum(-(-(m + max(0, a)) // page) - -(-m // page) for m, a in b)
        given = sum(-(-m // page) for m, a in b if a < 0)
        return {"bytes": 16 * len(b) + 8 * (taken + given) + 8 * (sum(max(0, a) for _, a in b) + 5), "flops": 0}
    batch = _batch(case)
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    rows = sum(r for r, _ in batch)
    if case["op"] == "append":
        elements = rows * d
        pages = sum(-(-m // page) - (m - r) // page for r, m in batch)
        return {"bytes": elements * (2 * (hq + 2 * hkv) + 2 * hq + 2 * hkv) + 8 * rows + 16 * pages * hkv,
                "flops": elements * (hq + hkv) * (7 if case["norm"] else 3)}
    w = case["window"] or 1 << 40
    keys = sum(m - max(0, m - r + 1 - w) for r, m in batch)  # what a sequence's rows see together
    pairs = sum(sum(min(p + 1, w) for p in range(m - r, m)) for r, m in batch)
    return {"bytes": keys * hkv * d * 2 + keys // page * hkv * 8 + 4 * rows * hq * d, "flops": 4.0 * pairs * hq * d}


# ---- the definition in 64 bits -----------------------------------------------


def _values(codes):
    """What e4m3 codes stand for, from their bits."""
    c = torch.arange(256, device=DEV)
    e, m = c // 8 % 16, c % 8
    v = torch.where(e == 0, m.double() / 8 * 2.0 ** -6, (1 + m.double() / 8) * torch.exp2(e.double() - 7))
    v = torch.where(c % 128 == 127, math.nan, torch.where(c >= 128, -v, v))
    return v[codes.long()]


def _nearest(x):
    """The e4m3 value nearest to each x, ties to the even code."""
    grid = _values(torch.arange(127, device=DEV))
    a = x.abs().clamp(max=448)
    hi = torch.searchsorted(grid, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    down, up = a - grid[lo], grid[hi] - a
    return torch.where((down < up) | ((down == up) & (lo % 2 == 0)), grid[lo], grid[hi]) * torch.sign(x)


def exact(case, seed):
    if case["op"] == "map":
        return None  # whole numbers alone
    st = prepare(case, seed)
    return _append64(st) if case["op"] == "append" else _attend64(st)


def _append64(st):
    rows, hq, hkv, d, size = st["rows"], st["hq"], st["hkv"], st["d"], st["page"]
    x = st["qkv"].double().view(rows, -1, d)
    inv = torch.tensor([BASE ** (-2 * i / d) for i in range(d // 2)], dtype=torch.float64, device=DEV)
    z = torch.polar(torch.ones(rows, d // 2, dtype=torch.float64, device=DEV), st["positions"].double()[:, None] * inv)

    def turned(h, gain):
        if gain is not None:
            h = h / ((h * h).sum(-1, keepdim=True) / d + EPS).sqrt() * gain.double()
        w = torch.complex(h[..., :d // 2].contiguous(), h[..., d // 2:].contiguous()) * z[:, None]
        return torch.cat([w.real, w.imag], -1)

    q = turned(x[:, :hq], st["gains"][0]).view(rows, -1)
    out = [q]
    slots = st["slots"].tolist()
    for name, y in (("k", turned(x[:, hq:hq + hkv], st["gains"][1])), ("v", x[:, hq + hkv:])):
        value, scale = _values(st[name + "_codes"]), st[name + "_scales"].double()
        r = 0
        while r < rows:  # the rows of one page
            p, o = divmod(slots[r], size)
            n = 1
            while r + n < rows and o + n < size and slots[r + n] == slots[r] + n:
                n += 1
            amax = y[r:r + n].abs().amax((0, 2))
            e = torch.ceil(torch.log2(amax / 448)).clamp(LEAST, MOST)
            e = torch.where(amax > 448 * torch.exp2(e), e + 1, torch.where(amax <= 448 * torch.exp2(e - 1), e - 1, e))
            s = torch.exp2(e.clamp(LEAST, MOST))
            if o:
                s = torch.maximum(s, scale[p])
                value[p, :, :o] = _nearest(value[p, :, :o] * (scale[p] / s)[:, None, None])
            value[p, :, o:o + n] = _nearest(y[r:r + n].transpose(0, 1) / s[:, None, None])
            scale[p] = s
            r += n
        out += [value, scale]
    return [out[0], out[1], out[3], out[2], out[4]]


def _attend64(st):
    hq, hkv, d, page, w = st["hq"], st["hkv"], st["d"], st["page"], st["window"]
    out = torch.empty(st["rows"], hq, d, dtype=torch.float64, device=DEV)
    q = st["q"].double().view(st["rows"], hq, d)
    off, lens = st["offsets"].tolist(), st["lens"].tolist()
    for i, m in enumerate(lens):
        pages = st["tables"][i, :-(-m // page)].long()
        for h in range(hkv):
            k, v = ((_values(st[c + "_codes"][pages, h]) * st[c + "_scales"][pages, h].double()[:, None, None]).view(-1, d)[:m]
                    for c in "kv")
            heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            for r0 in range(off[i], off[i + 1], 1024):
                r1 = min(r0 + 1024, off[i + 1])
                s = torch.einsum("rgd,ld->grl", q[r0:r1, heads], k) / math.sqrt(d)
                pos = m - off[i + 1] + torch.arange(r0, r1, device=DEV)[:, None]
                key = torch.arange(m, device=DEV)
                gone = (key > pos) | (key <= pos - w) if w else key > pos
                p = torch.softmax(s.masked_fill(gone, -math.inf), -1)
                out[r0:r1, heads] = torch.einsum("grl,ld->rgd", p, v)
    return out.view(st["rows"], -1)
