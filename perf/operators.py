"""Measured cases of the 4-bit linear layer and of the logits controls.

Five operators, as a serving program meets them: 16-bit rows are quantised to
4-bit floating point with a scale per block (``quantise``) and turned back
(``dequantise``); two such matrices are multiplied (``product``); a table keeps
which tokens each request has seen (``state``); and logits are changed by
penalties, biases and a grammar's mask before the largest is picked
(``control``).

Where ``own`` is false, ``run`` computes them from elementary torch operations
in 32 bits; where it is true it makes the framework's calls.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = {"nv": 16, "mx": 32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- cases -------------------------------------------------------------------


def listed():
    return [
        # one decoding request through a 4096-wide projection: latency
        dict(name="product decode 1", op="product", m=1, n=4096, k=4096, fmt="nv", epi="store", type="bf16"),
        # the LM head of a batch of decodes, fp32 logits: the weight's bytes
        dict(name="product head 33", op="product", m=33, n=32000, k=4096, fmt="nv", epi="f32", type="bf16"),
        # gate and up of a hybrid step: a 512-token budget and five decodes
        dict(name="product gate/up 517", op="product", m=517, n=28672, k=4096, fmt="nv", epi="swiglu", type="bf16"),
        # the down projection of a wide model over a long prefill, into the residual stream
        dict(name="product down 8192", op="product", m=8192, n=7168, k=20480, fmt="mx", epi="residual", type="f16"),
        # one token's activations
        dict(name="quantise row 1", op="quantise", rows=1, cols=4096, fmt="nv", type="bf16"),
        # a whole gate/up weight at load time
        dict(name="quantise weight", op="quantise", rows=28672, cols=4096, fmt="nv", type="bf16"),
        # a chunk's FFN rows turned back for a check against the 16-bit path
        dict(name="dequantise 517", op="dequantise", rows=517, cols=14336, fmt="mx", type="f16"),
        # a stored 4-bit weight handed to the 16-bit model
        dict(name="dequantise weight", op="dequantise", rows=20480, cols=7168, fmt="nv", type="bf16"),
        # one request's pick under its penalties and grammar
        dict(name="control 1", op="control", rows=1, vocab=32000, type="f32", penalties=True, biases=12, masks=1,
             out=False, count=True),
        # a full batch whose adjusted logits go on to a sampler
        dict(name="control 256", op="control", rows=256, vocab=64000, type="f32", penalties=True, biases=48, masks=9,
             out=True, count=False),
        # a step's picks appended for a batch of 256 decodes
        dict(name="state append 256", op="state", rows=256, vocab=32000, longest=1, reset=False),
        # requests admitted (or resumed) with their whole histories
        dict(name="state admit 64", op="state", rows=64, vocab=64000, longest=8192, reset=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "product", "product", "quantise", "dequantise", "control", "control", "state"])
    if op == "product":
        epi = rng.choice(["store", "store", "f32", "residual", "swiglu"])
        m, n, k = _log(rng, 1, 8192), _log(rng, 64, 32768), 32 * _log(rng, 4, 640)
        n = max(128, n // 128 * 128) if epi == "swiglu" else rng.choice([n, n // 8 * 8, max(64, n // 64 * 64)])
        m = max(1, min(m, 8192 * 7168 * 20480 // (n * k)))
        return dict(op=op, m=m, n=n, k=k, fmt=rng.choice(["nv", "mx"]), epi=epi, type=rng.choice(["bf16", "f16"]))
    if op in ("quantise", "dequantise"):
        cols = 32 * _log(rng, 1, 640)
        rows = max(1, min(_log(rng, 1, 32768), 28672 * 4096 // cols))
        return dict(op=op, rows=rows, cols=cols, fmt=rng.choice(["nv", "mx"]), type=rng.choice(["bf16", "f16", "f32"]))
    if op == "control":
        vocab = rng.choice([_log(rng, 1000, 131072), 8 * _log(rng, 1000, 16384)])
        rows = max(1, min(_log(rng, 1, 512), 256 * 64000 // vocab))
        return dict(op=op, rows=rows, vocab=vocab, type=rng.choice(["f32", "f32", "bf16", "f16"]),
                    penalties=rng.random() < 0.75, biases=rng.choice([0, 1, 20, 300]), masks=rng.choice([0, 1, 5]),
                    out=rng.random() < 0.6, count=rng.random() < 0.5)
    vocab = _log(rng, 1000, 131072)
    reset = rng.random() < 0.6
    rows = max(1, min(_log(rng, 1, 256), 64 * 64000 // vocab)) if reset else _log(rng, 1, 256)
    return dict(op=op, rows=rows, vocab=vocab, longest=_log(rng, 1, 8192) if reset else rng.choice([1, 1, 5, 128]),
                reset=reset)


# ---- 4-bit layout ------------------------------------------------------------
# Codes: two to a byte, the even column in the low nibble.  Scales: one byte per
# block; 128 rows x 4 blocks form a tile of 512 bytes, row r and block b of the
# tile at (r % 32) * 16 + (r / 32) * 4 + b; a row block's tiles follow along
# the columns.


def _tile_scales(s):
    rows, nb = s.shape
    rb, kg = -(-rows // 128), -(-nb // 4)
    p = torch.zeros(rb * 128, kg * 4, dtype=torch.uint8, device=s.device)
    p[:rows, :nb] = s
    return p.view(rb, 4, 32, kg, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _untile_scales(t, rows, nb):
    rb, kg = -(-rows // 128), -(-nb // 4)
    return t.view(rb, kg, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rb * 128, kg * 4)[:rows, :nb]


def _powers(e, dtype=torch.float32):
    """2^e for whole -127 <= e <= 127, exactly."""
    return torch.tensor([2.0 ** i for i in range(-127, 128)], dtype=dtype, device=e.device)[e.long() + 127]


def _quantise(x, fmt, inv_g):
    """Codes and tiled scales of x * inv_g."""
    rows, cols = x.shape
    nb = cols // BLOCK[fmt]
    t = (x.float() * inv_g).view(rows, nb, BLOCK[fmt])
    amax = t.abs().amax(-1)
    bad = ~torch.isfinite(amax)
    if fmt == "nv":
        s = (amax / 6).clamp(max=448).to(torch.float8_e4m3fn)
        sb = torch.where(bad, 0x7F, s.view(torch.uint8))
        s = s.float().unsqueeze(-1)
        q = torch.where(s > 0, t / s, 0.0)
    else:
        e = (torch.frexp(amax).exponent - 3).clamp(min=-127)
        e = torch.where(amax > 0, e, -127)
        sb = torch.where(bad, 0xFF, e + 127).to(torch.uint8)
        q = t * _powers(-e).unsqueeze(-1)
    a = q.abs()
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5
    code |= torch.signbit(q).to(torch.uint8) << 3
    code = torch.where(bad.unsqueeze(-1), 0, code).view(rows, cols // 2, 2)
    return code[..., 0] | code[..., 1] << 4, _tile_scales(sb)


def _scale_values(t, rows, nb, fmt):
    s = _untile_scales(t, rows, nb).contiguous()
    if fmt == "nv":
        return s.view(torch.float8_e4m3fn).float()
    return torch.where(s == 255, math.nan, _powers(s.int().clamp(max=254) - 127))


def _dequantise(codes, scales, cols, fmt, g):
    """fp32 values of codes and tiled scales."""
    rows = codes.shape[0]
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    pair = torch.stack([codes & 15, codes >> 4], -1).view(rows, cols)
    v = lut[pair.int()].view(rows, -1, BLOCK[fmt])
    return (v * _scale_values(scales, rows, v.shape[1], fmt).unsqueeze(-1)).view(rows, cols) * g


# ---- inputs ------------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _activations(g, rows, cols, dtype):
    """Normalised activations: a few columns are much larger than the others."""
    x = torch.randn(rows, cols, generator=g, device=DEV)
    gain = torch.exp(0.5 * torch.randn(cols, generator=g, device=DEV))
    return (x * gain).to(dtype)


def _weights(g, rows, cols, dtype=torch.bfloat16):
    return (0.02 * torch.randn(rows, cols, generator=g, device=DEV)).to(dtype)


W_SCALE = 2.0 ** -12  # the weights' tensor scale (e4m3 block scales near 2^4)


def _tensor_scale(fmt):
    return W_SCALE if fmt == "nv" else 1.0


def _tokens(g, n, vocab):
    """Token ids with frequent and rare ones."""
    u = torch.rand(n, generator=g, device=DEV)
    return (u * u * u * vocab).to(torch.int32).clamp(max=vocab - 1)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = dict(case)
    if op == "product":
        m, n, k, fmt, epi = case["m"], case["n"], case["k"], case["fmt"], case["epi"]
        dt = TYPES[case["type"]]
        wg = _tensor_scale(fmt)
        st["a"], st["sa"] = _quantise(_activations(g, m, k, dt), fmt, 1.0)
        st["w"], st["sw"] = _quantise(_weights(g, n, k), fmt, 1.0 / wg)
        st["alpha"] = wg
        st["r"] = torch.randn(m, n, generator=g, device=DEV) if epi == "residual" else None
        out = (m, n // 2) if epi == "swiglu" else (m, n)
        st["c"] = torch.empty(out, device=DEV, dtype=dt if epi in ("store", "swiglu") else torch.float32)
    elif op == "quantise":
        x = _activations(g, case["rows"], case["cols"], TYPES[case["type"]])
        if case["rows"] >= 4096:
            x = _weights(g, case["rows"], case["cols"], TYPES[case["type"]])
        st["g"] = _tensor_scale(case["fmt"]) if case["rows"] >= 4096 else 1.0
        st["x"], st["y"] = x, torch.empty_like(x)
        nb = -(-case["cols"] // BLOCK[case["fmt"]])
        st["codes"] = torch.empty(case["rows"], case["cols"] // 2, dtype=torch.uint8, device=DEV)
        st["scales"] = torch.empty(-(-case["rows"] // 128) * -(-nb // 4) * 512, dtype=torch.uint8, device=DEV)
    elif op == "dequantise":
        x = _weights(g, case["rows"], case["cols"])
        st["g"] = _tensor_scale(case["fmt"])
        st["codes"], st["scales"] = _quantise(x, case["fmt"], 1.0 / st["g"])
        st["y"] = torch.empty(case["rows"], case["cols"], dtype=TYPES[case["type"]], device=DEV)
    elif op == "control":
        _prepare_control(st, g)
    else:
        _prepare_state(st, g)
    return st


def _prepare_state(st, g):
    rows, vocab, longest = st["rows"], st["vocab"], st["longest"]
    slots = rows + 3
    st["table"] = torch.zeros(slots, -(-vocab // 8) * 8, dtype=torch.int16, device=DEV)
    st["slots"] = torch.randperm(slots, generator=g, device=DEV)[:rows].to(torch.int32)
    lens = torch.randint(1, longest + 1, (rows,), generator=g, device=DEV)
    st["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), lens.cumsum(0)]).to(torch.int32)
    st["n"] = int(lens.sum())
    st["tokens"] = _tokens(g, st["n"], vocab)
    share = torch.rand(rows, generator=g, device=DEV)
    st["prompt"] = (lens * share).to(torch.int32) if st["reset"] else None


def _prepare_control(st, g):
    rows, vocab = st["rows"], st["vocab"]
    dt = TYPES[st["type"]]
    st["x"] = (3.0 * torch.randn(rows, vocab, generator=g, device=DEV)).to(dt)
    st["y"] = torch.empty_like(st["x"]) if st["out"] else None
    st["picks"] = torch.empty(rows, dtype=torch.int32, device=DEV)
    slots = rows + 2
    table = torch.zeros(slots, vocab, dtype=torch.int32, device=DEV)
    hist = _tokens(g, slots * 600, vocab).view(slots, 600).long()
    table.scatter_add_(1, hist[:, :200], torch.ones(1, 1, dtype=torch.int32, device=DEV).expand(slots, 200))
    table.scatter_(1, hist[:, 200:], table.gather(1, hist[:, 200:]) | 0x8000)
    st["table"] = torch.zeros(slots, -(-vocab // 8) * 8, dtype=torch.int16, device=DEV)
    st["table"][:, :vocab] = ((table + 0x8000) % 0x10000 - 0x8000).to(torch.int16)
    st["slots"] = torch.randperm(slots, generator=g, device=DEV)[:rows].to(torch.int32)
    on = st["penalties"]
    st["rep"] = 1.0 + 0.25 * torch.rand(rows, generator=g, device=DEV) if on else None
    st["pres"] = torch.rand(rows, generator=g, device=DEV) if on else None
    st["freq"] = 0.5 * torch.rand(rows, generator=g, device=DEV) if on else None
    st["bias"] = None
    if st["biases"]:
        lens = torch.randint(0, st["biases"] + 1, (rows,), generator=g, device=DEV)
        off = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), lens.cumsum(0)]).to(torch.int32)
        n = int(lens.sum())
        val = torch.randint(-400, 21, (n,), generator=g, device=DEV).float() / 4
        st["bias"] = (off, _tokens(g, n, vocab), val)
    st["mask"] = st["mask_rows"] = None
    if st["masks"]:
        # grammars: free text, a set of words, a handful of tokens, nothing left
        words = -(-vocab // 32)
        bits = torch.rand(st["masks"], words * 32, generator=g, device=DEV)
        share = torch.tensor([0.9, 0.2, 0.001, 0.5, 0.0], device=DEV)[torch.arange(st["masks"], device=DEV) % 5]
        on = (bits < share.unsqueeze(1)).view(st["masks"], words, 32).long()
        word = (on << torch.arange(32, device=DEV)).sum(-1)
        st["mask"] = ((word + 2 ** 31) % 2 ** 32 - 2 ** 31).to(torch.int32)
        st["mask_rows"] = torch.randint(-1, st["masks"], (rows,), generator=g, device=DEV).to(torch.int32)


# ---- one pass ----------------------------------------------------------------


def run(st):
    return _RUN[st["op"]](st)


def _run_product(st):
    if own:
        import chunked_prefill_hybrid_sar_gb300 as sar

        epi = {"store": sar.SAR_EPI_STORE, "residual": sar.SAR_EPI_RESIDUAL, "swiglu": sar.SAR_EPI_SWIGLU,
               "f32": sar.SAR_EPI_F32}[st["epi"]]
        sar.gemm_fp4(st["a"], st["sa"], st["w"], st["sw"], st["c"], residual=st["r"], alpha=st["alpha"], epilogue=epi,
                     format=sar.SAR_FP4_NV if st["fmt"] == "nv" else sar.SAR_FP4_MX)
        return st["c"]
    a = _dequantise(st["a"], st["sa"], st["k"], st["fmt"], 1.0)
    w = _dequantise(st["w"], st["sw"], st["k"], st["fmt"], 1.0)
    d = (a @ w.t()) * st["alpha"]
    if st["epi"] == "residual":
        return d + st["r"]
    if st["epi"] == "swiglu":
        d = d.view(st["m"], -1, 2, 64)
        gate, up = d[:, :, 0], d[:, :, 1]
        d = (gate / (1 + torch.exp(-gate)) * up).reshape(st["m"], -1)
    return d.to(st["c"].dtype)


def _run_quantise(st):
    if own:
        import chunked_prefill_hybrid_sar_gb300 as sar

        fmt = sar.SAR_FP4_NV if st["fmt"] == "nv" else sar.SAR_FP4_MX
        sar.fp4_quantize(st["x"], st["codes"], st["scales"], format=fmt, tensor_scale=st["g"])
        sar.fp4_dequantize(st["codes"], st["scales"], st["y"], format=fmt, tensor_scale=st["g"])
        return st["y"]
    codes, scales = _quantise(st["x"], st["fmt"], 1.0 / st["g"])
    return _dequantise(codes, scales, st["cols"], st["fmt"], st["g"]).to(st["y"].dtype)


def _run_dequantise(st):
    if own:
        import chunked_prefill_hybrid_sar_gb300 as sar

        sar.fp4_dequantize(st["codes"], st["scales"], st["y"], tensor_scale=st["g"],
                           format=sar.SAR_FP4_NV if st["fmt"] == "nv" else sar.SAR_FP4_MX)
        return st["y"]
    return _dequantise(st["codes"], st["scales"], st["cols"], st["fmt"], st["g"]).to(st["y"].dtype)


def _run_control(st):
    if own:
        import chunked_prefill_hybrid_sar_gb300 as sar

        if "controls" not in st:  # a handle over the batch's tensors, made once
            off, tok, val = st["bias"] or (None, None, None)
            st["controls"] = sar.LogitControls(
                state=st["table"], slots=st["slots"], repetition=st["rep"], presence=st["pres"],
                frequency=st["freq"], bias_offsets=off, bias_tokens=tok, bias_values=val, mask=st["mask"],
                mask_rows=st["mask_rows"], count_picks=st["count"])
        sar.logits_control(st["x"], st["controls"], out=st["y"], tokens_out=st["picks"])
    else:
        _plain_control(st)
    return [st["picks"], st["table"]] + ([st["y"]] if st["out"] else [])


def _plain_control(st):
    rows, vocab = st["rows"], st["vocab"]
    slots = st["slots"].long()
    x = st["x"].float()
    if st["penalties"]:
        s = st["table"][slots, :vocab].int() & 0xFFFF
        count = s & 0x7FFF
        r = st["rep"].unsqueeze(1)
        x = torch.where(s != 0, torch.where(x > 0, x / r, x * r), x)
        x = x - st["freq"].unsqueeze(1) * count
        x = x - st["pres"].unsqueeze(1) * (count > 0)
    if st["bias"] is not None:
        off, tok, val = st["bias"]
        row = torch.searchsorted(off[1:].long(), torch.arange(tok.numel(), device=DEV), right=True)
        b = torch.zeros_like(x).index_put_((row, tok.long()), val, accumulate=True)
        x = x + b
    if st["mask"] is not None:
        word = st["mask"][st["mask_rows"].long().clamp(min=0)]
        on = (word.unsqueeze(-1) >> torch.arange(32, device=DEV, dtype=torch.int32) & 1).view(rows, -1)[:, :vocab]
        on = (on != 0) | (st["mask_rows"] < 0).unsqueeze(1)
        x = torch.where(on, x, -math.inf)
    if st["out"]:
        st["y"].copy_(x)
    best, at = x.max(1)
    st["picks"].copy_(torch.where(best == -math.inf, -1, at))
    if st["count"]:
        at = at.unsqueeze(1)
        s = st["table"][slots].gather(1, at).int() & 0xFFFF
        up = torch.where((s & 0x7FFF) < 0x7FFF, s + 1, s)
        up = torch.where(best.unsqueeze(1) == -math.inf, s, up)
        up = torch.where(up >= 0x8000, up - 0x10000, up).to(torch.int16)
        st["table"][slots.unsqueeze(1), at] = up


def _run_state(st):
    if own:
        import chunked_prefill_hybrid_sar_gb300 as sar

        sar.token_state_add(st["table"], st["slots"], st["offsets"], st["tokens"], vocab=st["vocab"],
                            prompt_lens=st["prompt"], reset=st["reset"])
        return st["table"]
    vocab = st["vocab"]
    slots, off = st["slots"].long(), st["offsets"].long()
    old = st["table"][slots, :vocab].int() & 0xFFFF
    if st["reset"]:
        old = torch.zeros_like(old)
    i = torch.arange(st["n"], device=DEV)
    row = torch.searchsorted(off[1:], i, right=True)
    at = row * vocab + st["tokens"].long()
    made = torch.ones_like(at) if st["prompt"] is None else (i - off[row] >= st["prompt"].long()[row]).long()
    count = (old & 0x7FFF).view(-1).long().scatter_add_(0, at, made).clamp(max=0x7FFF)
    seen = (old >> 15).view(-1).long().scatter_add_(0, at, 1 - made).clamp(max=1)
    new = (count - 0x8000 * seen).to(torch.int16)
    st["table"][slots, :vocab] = new.view(-1, vocab)
    return st["table"]


_RUN = {"product": _run_product, "quantise": _run_quantise, "dequantise": _run_dequantise, "control": _run_control,
        "state": _run_state}


# ---- what a pass cannot do without -------------------------------------------


def work(case):
    op = case["op"]
    size = {"f16": 2, "bf16": 2, "f32": 4}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        four = (m + n) * k * (0.5 + 1 / BLOCK[case["fmt"]])
        out = m * n * {"store": 2, "swiglu": 1, "f32": 4, "residual": 8}[case["epi"]]
        return {"bytes": four + out, "flops": 2.0 * m * n * k}
    if op in ("quantise", "dequantise"):
        n = case["rows"] * case["cols"]
        b, four = size[case["type"]], 0.5 + 1 / BLOCK[case["fmt"]]
        # the quantised rows are written once and read back once
        return {"bytes": n * (2 * b + 2 * four if op == "quantise" else b + four), "flops": 0}
    if op == "control":
        n = case["rows"] * case["vocab"]
        b = size[case["type"]]
        mask = min(case["masks"], case["rows"]) * case["vocab"] / 8
        return {"bytes": n * (b + (2 if case["penalties"] else 0) + (b if case["out"] else 0)) + mask, "flops": 0}
    tokens = case["rows"] * (case["longest"] + 1) / 2
    return {"bytes": tokens * 4 + (2 * case["rows"] * case["vocab"] if case["reset"] else tokens * 4), "flops": 0}


# ---- the definition in 64 bits -----------------------------------------------


def _grid_e4m3():
    """The finite non-negative e4m3 values in order, index = bit pattern."""
    sub = [m * 2.0 ** -9 for m in range(8)]
    return torch.tensor(sub + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:119],
                        dtype=torch.float64, device=DEV)


def _nearest(v, grid):
    """Index of the nearest grid value, ties to the even index, saturating."""
    hi = torch.searchsorted(grid, v.contiguous()).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    dl, dh = v - grid[lo], grid[hi] - v
    return torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def _values64(codes, scales, cols, fmt, g):
    rows = codes.shape[0]
    c = torch.stack([codes % 16, codes // 16], -1).view(rows, cols).long()
    mag, sign = c % 8, 1 - 2 * (c // 8)
    # exponent and mantissa of e2m1: 0, 0.5 below the first binade
    v = torch.where(mag < 2, 0.5 * mag.double(), (2 + mag % 2).double() * _powers(mag // 2 - 2, torch.float64))
    nb = cols // BLOCK[fmt]
    r = torch.arange(rows, device=DEV).unsqueeze(1)
    b = torch.arange(nb, device=DEV).unsqueeze(0)
    s = scales[(r // 128 * (-(-nb // 4)) + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4].long()
    if fmt == "nv":
        s = torch.where(s == 127, math.nan, _grid_e4m3()[s.clamp(max=126)])
    else:
        s = torch.where(s == 255, math.nan, _powers(s.clamp(max=254) - 127, torch.float64))
    return ((sign * v).view(rows, nb, -1) * s.unsqueeze(-1)).view(rows, cols) * g


def _rounded64(x, fmt, g):
    """The values that quantising x stands for."""
    rows, cols = x.shape
    t = (x.double() / g).view(rows, -1, BLOCK[fmt])
    a = t.abs().amax(-1, keepdim=True)
    if fmt == "nv":
        grid = _grid_e4m3()
        s = grid[_nearest(a / 6, grid)]
    else:
        some = torch.isfinite(a) & (a > 0)
        s = _powers((torch.frexp(torch.where(some, a, 2.0 ** -140)).exponent - 1 - 2).clamp(-127, 127), torch.float64)
    grid = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    q = torch.where(s > 0, t.abs() / s, 0.0)
    v = grid[_nearest(q, grid)] * torch.sign(t) * s * g
    return torch.where(torch.isfinite(a), v, math.nan).view(rows, cols)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "product":
        a = _values64(st["a"], st["sa"], st["k"], st["fmt"], 1.0)
        out = []
        for j in range(0, st["n"], 8192):
            hi = min(j + 8192, st["n"])
            # (8192 is whole scale tiles of 128 rows)
            kg = -(-(st["k"] // BLOCK[st["fmt"]]) // 4) * 512
            w = _values64(st["w"][j:hi], st["sw"][j // 128 * kg:], st["k"], st["fmt"], st["alpha"])
            out.append(a @ w.t())
        d = torch.cat(out, 1)
        if st["epi"] == "residual":
            return d + st["r"].double()
        if st["epi"] == "swiglu":
            d = d.view(st["m"], st["n"] // 128, 128)
            d = (d[..., :64] * torch.sigmoid(d[..., :64]) * d[..., 64:]).reshape(st["m"], st["n"] // 2)
        return d
    if op == "quantise":
        return torch.cat([_rounded64(x, st["fmt"], st["g"]) for x in st["x"].split(4096)])
    if op == "dequantise":
        return _values64(st["codes"], st["scales"], st["cols"], st["fmt"], st["g"])
    if op == "control" and st["out"]:
        return [None, None, _control64(st)]
    return None  # token ids and counts alone


def _control64(st):
    out = []
    for r in range(st["rows"]):
        x = st["x"][r].double()
        if st["penalties"]:
            s = st["table"][int(st["slots"][r]), :st["vocab"]].long() % 65536
            rep, pres, freq = (st[k][r].double() for k in ("rep", "pres", "freq"))
            x = torch.where((s > 0) & (x > 0), x / rep, torch.where(s > 0, x * rep, x))
            made = s % 32768
            x = x - freq * made - torch.where(made > 0, pres, 0.0)
        if st["bias"] is not None:
            lo, hi = int(st["bias"][0][r]), int(st["bias"][0][r + 1])
            x = x.index_add(0, st["bias"][1][lo:hi].long(), st["bias"][2][lo:hi].double())
        if st["mask"] is not None and int(st["mask_rows"][r]) >= 0:
            v = torch.arange(st["vocab"], device=DEV)
            word = st["mask"][int(st["mask_rows"][r])].long() % 2 ** 32
            x = torch.where(word[v // 32] // 2 ** (v % 32) % 2 == 1, x, -math.inf)
        out.append(x)
    return torch.stack(out)
