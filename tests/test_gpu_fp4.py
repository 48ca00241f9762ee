"""Quantisation to 4-bit rows and back against the float64 oracle: codes,
scales and values are equal, bit for bit (every rounding has one answer)."""

import numpy as np
import pytest
import torch

import chunked_prefill_hybrid_sar_gb300 as sar
import synth
from oracle import fp4

pytestmark = pytest.mark.gpu

FMT = {"nv": sar.SAR_FP4_NV, "mx": sar.SAR_FP4_MX}
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def rows_of(kind, rows, cols, seed=0):
    """Rows with blocks of every size: ordinary, tiny, huge, zero, and whole borders."""
    g = synth.generator(seed)
    x = synth.normal(g, (rows, cols))
    x *= torch.exp2(torch.randint(-12, 12, (rows, cols // 16), generator=g).float()).repeat_interleave(16, 1)
    x[torch.rand(rows, cols, generator=g) < 0.1] *= 0
    # exact borders and their neighbours
    k = torch.randint(0, 15, (rows, cols), generator=g).float() / 4
    x = torch.where(torch.rand(rows, 1, generator=g) < 0.3, k * torch.exp2(torch.randint(-3, 3, (rows, 1), generator=g).float()), x)
    if kind != "f32":
        x = x.clamp(-30000, 30000)
    return x.to(TYPES[kind])


def quantised(x, fmt, scale=1.0):
    rows, cols = x.shape
    codes = torch.full((rows, cols // 2), 0xEE, dtype=torch.uint8, device="cuda")
    scales = torch.full((sar.fp4_scale_bytes(rows, cols, FMT[fmt]),), 0xEE, dtype=torch.uint8, device="cuda")
    sar.fp4_quantize(x, codes, scales, format=FMT[fmt], tensor_scale=scale)
    return codes, scales


def check(x, fmt, scale=1.0):
    codes, scales = quantised(x.cuda(), fmt, scale)
    code, byte = fp4.quantise(x.float().numpy(), fmt, np.float32(1) / np.float32(scale))
    assert np.array_equal(codes.cpu().numpy(), fp4.pack(code))
    assert np.array_equal(scales.cpu().numpy(), fp4.tile(byte, fill=0xEE))
    return codes, scales, code, byte


SHAPES = [(1, 32), (1, 4096), (3, 96), (33, 160), (127, 64), (128, 256), (130, 4128), (517, 480)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("fmt", list(FMT))
def test_codes_and_scales(rows, cols, kind, fmt):
    check(rows_of(kind, rows, cols, rows + cols), fmt)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("scale", [2.0 ** -12, 0.0371, 3.0])
def test_tensor_scale(kind, fmt, scale):
    x = rows_of(kind, 40, 224, 3)
    codes, scales, code, byte = check(x, fmt, scale)
    y = torch.empty(40, 224, device="cuda")
    sar.fp4_dequantize(codes, scales, y, format=FMT[fmt], tensor_scale=scale)
    # the code times its scale is exact; one fp32 rounding by the tensor scale
    want = fp4.values(code, byte, fmt).astype(np.float32) * np.float32(scale)
    assert np.array_equal(y.cpu().numpy(), want)


@pytest.mark.parametrize("fmt", list(FMT))
def test_every_16_bit_value_over_every_scale(fmt):
    """Each finite bf16 value beside a block maximum of each of 64 mantissas."""
    bits = torch.arange(0, 0x7F80, 7, dtype=torch.int32)
    v = (bits << 16).view(torch.float32)
    v = v[(v > 2.0 ** -14) & (v < 2.0 ** 14)]
    big = torch.arange(64, 128).float()
    x = torch.zeros(64, (v.numel() + 29) // 30 * 32)
    for j in range(64):
        row = x[j].view(-1, 32)
        row[:, 0] = row[:, 16] = big[j]
        flat = torch.zeros(row.shape[0] * 30)
        flat[:v.numel()] = torch.where(v < big[j], v, v / 2.0 ** 8)
        row[:, 1:16] = flat.view(-1, 30)[:, :15]
        row[:, 17:32] = -flat.view(-1, 30)[:, 15:]
    check(x, fmt)


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("kind", list(TYPES))
def test_nan_and_infinity_poison_their_block_alone(fmt, kind):
    x = rows_of(kind, 9, 192, 5)
    x[0, 0], x[2, 40], x[4, 191], x[5, 100] = float("nan"), float("inf"), float("-inf"), float("nan")
    codes, scales, code, byte = check(x, fmt)
    y = torch.empty_like(x, device="cuda")
    sar.fp4_dequantize(codes, scales, y, format=FMT[fmt])
    B = fp4.BLOCK[fmt]
    nan = torch.isnan(y.float()).cpu().view(9, -1, B)
    bad = ~torch.isfinite(x.float()).view(9, -1, B).all(-1, keepdim=True).expand_as(nan)
    assert torch.equal(nan, bad)


@pytest.mark.parametrize("fmt", list(FMT))
def test_smallest_and_largest_fp32(fmt):
    x = torch.zeros(6, 64)
    x[0, ::3], x[1, ::5], x[2, 1::2] = 2.0 ** -149, 1.2e-38, 3.4e38
    x[3, 0], x[3, 1], x[4, 7] = 2.0 ** -126, -(2.0 ** -127), 448 * 6 * 4.0
    codes, scales, code, byte = check(x, fmt)
    y = torch.empty(6, 64, device="cuda")
    sar.fp4_dequantize(codes, scales, y, format=FMT[fmt])
    assert np.array_equal(y.cpu().numpy(), fp4.values(code, byte, fmt).astype(np.float32))


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("offset,extra", [(0, 16), (1, 0), (3, 5), (8, 8)])
def test_strides_and_alignment(kind, fmt, offset, extra):
    """Rows in a wider buffer, at any element offset; columns between them untouched."""
    rows, cols = 37, 96
    ld = cols + extra
    x = rows_of(kind, rows, cols, 11)
    buf = torch.zeros(offset + rows * ld, dtype=TYPES[kind], device="cuda")
    view = buf[offset:].as_strided((rows, cols), (ld, 1))
    view.copy_(x)
    codes, scales = quantised(view, fmt)
    code, byte = fp4.quantise(x.float().numpy(), fmt)
    assert np.array_equal(codes.cpu().numpy(), fp4.pack(code))
    buf.fill_(7.0)
    sar.fp4_dequantize(codes, scales, buf[offset:].as_strided((rows, cols), (ld, 1)), format=FMT[fmt])
    want = torch.from_numpy(fp4.values(code, byte, fmt)).to(TYPES[kind])
    assert torch.equal(buf[offset:].as_strided((rows, cols), (ld, 1)).cpu(), want)
    rest = torch.ones(buf.numel(), dtype=torch.bool)
    rest[offset:].as_strided((rows, cols), (ld, 1)).fill_(False)
    assert (buf.cpu()[rest] == 7.0).all()


def test_python_refusals():
    x = torch.zeros(4, 64, device="cuda")
    c = torch.zeros(4, 32, dtype=torch.uint8, device="cuda")
    s = torch.zeros(512, dtype=torch.uint8, device="cuda")
    sar.fp4_quantize(x, c, s)
    for bad in (dict(x=x.double()), dict(x=x.t()), dict(x=x.cpu()), dict(c=c[:3]), dict(c=c.int()), dict(s=s[:511]),
                dict(s=s.int())):
        a = dict(x=x, c=c, s=s) | bad
        with pytest.raises(ValueError):
            sar.fp4_quantize(a["x"], a["c"], a["s"])
        with pytest.raises(ValueError):
            sar.fp4_dequantize(a["c"], a["s"], a["x"])
    with pytest.raises(sar.SarError):
        sar.fp4_quantize(torch.zeros(4, 48, device="cuda"), torch.zeros(4, 24, dtype=torch.uint8, device="cuda"), s)


def test_other_stream_and_graph():
    x = rows_of("bf16", 65, 320, 21).cuda()
    codes, scales = quantised(x, "nv")
    y0 = torch.empty_like(x)
    sar.fp4_dequantize(codes, scales, y0)
    y, c2, s2 = torch.empty_like(x), torch.zeros_like(codes), torch.zeros_like(scales)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        sar.fp4_quantize(x, c2, s2)
        sar.fp4_dequantize(c2, s2, y)
    for _ in range(2):
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y0) and torch.equal(c2, codes)
