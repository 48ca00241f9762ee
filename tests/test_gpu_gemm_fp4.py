"""The 4-bit product against float64.

With scales that are small powers of two every partial sum is a multiple of
2^-4 below 2^20 (products are multiples of 1/4 up to 36, scales 1/2 to 2), so
fp32 sums are exact in any order and the fp32 result has to be equal.  With
ordinary scales each MMA of 64 products may drop less than one unit of its fp32
accumulator, at most 2^-23 of the sum of magnitudes S, and the join and the
epilogue round once per K range and once for alpha: |error| <= (K / 64 + 10) *
2^-23 * S.  A 16-bit output adds half a unit of its type.
"""

import numpy as np
import pytest
import torch

import chunked_prefill_hybrid_sar_gb300 as sar
from oracle import fp4

pytestmark = pytest.mark.gpu

FMT = {"nv": sar.SAR_FP4_NV, "mx": sar.SAR_FP4_MX}
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
EPI = {"store": sar.SAR_EPI_STORE, "residual": sar.SAR_EPI_RESIDUAL, "swiglu": sar.SAR_EPI_SWIGLU, "f32": sar.SAR_EPI_F32}


@pytest.fixture(autouse=True)
def no_device_flags():
    sar.op_sync_status()
    yield
    sar.op_sync_status()


class Rows:
    """Random 4-bit rows: codes and scales on the device, their values here."""

    def __init__(self, rng, rows, cols, fmt, plain=False, garbage=0xFF):
        code = rng.integers(0, 16, (rows, cols)).astype(np.uint8)
        blocks = cols // fp4.BLOCK[fmt]
        if plain:  # 1/2, 1, 2
            one = 0x38 if fmt == "nv" else 127
            byte = one + (8 if fmt == "nv" else 1) * rng.integers(-1, 2, (rows, blocks))
        elif fmt == "nv":
            byte = rng.integers(0, 127, (rows, blocks)) * 3 // 8 + 40
        else:
            byte = rng.integers(118, 136, (rows, blocks))
        self.values = fp4.values(code, byte.astype(np.uint8), fmt)
        self.codes = torch.from_numpy(fp4.pack(code)).cuda()
        # bytes behind the last row are not used, whatever they hold (0xFF: NaN)
        self.scales = torch.from_numpy(fp4.tile(byte.astype(np.uint8), fill=garbage)).cuda()


def run(a, w, fmt, epi="f32", dtype=torch.float16, alpha=1.0, residual=None, variant=0, out=None):
    M, N = a.codes.shape[0], w.codes.shape[0]
    wide = epi in ("f32", "residual")
    shape = (M, N // 2 if epi == "swiglu" else N)
    c = torch.full(shape, 77.0, dtype=torch.float32 if wide else dtype, device="cuda") if out is None else out
    sar.gemm_fp4(a.codes, a.scales, w.codes, w.scales, c, residual=residual, alpha=alpha, epilogue=EPI[epi],
                 format=FMT[fmt], variant=variant)
    return c


def variants(M, N, K):
    v = {"auto": sar.SAR_FP4_GEMM_AUTO, "split": sar.SAR_FP4_GEMM_SPLIT, "pair": sar.SAR_FP4_GEMM_PAIR}
    for n in (1, 2, 3, 8):
        if n <= (K + 255) // 256:
            v[f"split{n}"] = sar.SAR_FP4_GEMM_SPLIT | n << 8
            v[f"split{n}x64"] = v[f"split{n}"] | sar.SAR_FP4_GEMM_TOKENS64
    if K > 256:
        v["pair2"] = sar.SAR_FP4_GEMM_PAIR | 2 << 8
    return v


SHAPES = [(1, 1, 32), (1, 128, 64), (2, 130, 96), (16, 256, 256), (17, 64, 288), (33, 200, 512), (48, 129, 800),
          (64, 512, 1024), (65, 384, 2080), (127, 127, 160), (128, 128, 2304), (129, 256, 256), (200, 1000, 544),
          (257, 300, 1088), (513, 640, 320),
          (256, 256, 1024), (512, 512, 96), (384, 700, 4384), (770, 20000, 288), (2048, 5632, 256)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("fmt", list(FMT))
def test_exact_sums(M, N, K, fmt):
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    a, w = Rows(rng, M, K, fmt, plain=True), Rows(rng, N, K, fmt, plain=True)
    want = a.values @ w.values.T
    for name, v in variants(M, N, K).items():
        got = run(a, w, fmt, variant=v).cpu().numpy()
        assert np.array_equal(got, want), (name, np.abs(got - want).max())


@pytest.mark.parametrize("M,N,K", [(1, 256, 4096), (40, 384, 2048), (130, 256, 1056), (300, 512, 3200)])
@pytest.mark.parametrize("epi", list(EPI))
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("fmt", list(FMT))
def test_epilogues(M, N, K, epi, dt, fmt):
    rng = np.random.default_rng(K + M)
    a, w = Rows(rng, M, K, fmt), Rows(rng, N, K, fmt)
    s = np.abs(a.values) @ np.abs(w.values).T
    alpha = 3.0 / s.max() * 8  # (SwiGLU's operands of ordinary size)
    alpha = float(np.float32(alpha))
    r = torch.randn(M, N, generator=torch.Generator().manual_seed(1))
    want = alpha * (a.values @ w.values.T)
    bound = (K / 64 + 10) * 2.0 ** -23 * s * alpha
    if epi == "residual":
        want = want + r.double().numpy()
        bound = bound + 2.0 ** -23 * np.abs(want)
    if epi == "swiglu":
        g, u = (x.reshape(M, N // 2) for x in np.split(want.reshape(M, N // 128, 2, 64), 2, axis=2))
        bg, bu = (x.reshape(M, N // 2) for x in np.split(bound.reshape(M, N // 128, 2, 64), 2, axis=2))
        # |silu'| <= 1.1, |silu(g)| <= |g|; the fast exponential and division: a few units, 2^-20
        want = fp4.swiglu(want)
        bound = 1.1 * bg * np.abs(u) + np.abs(g) * bu + 1.1 * bg * bu + 2.0 ** -20 * np.abs(g * u)
    for name, v in variants(M, N, K).items():
        got = run(a, w, fmt, epi, TYPES[dt], alpha, r.cuda() if epi == "residual" else None, v)
        b = bound
        if epi in ("store", "swiglu"):
            tiny = torch.finfo(TYPES[dt]).smallest_normal
            b = bound + torch.finfo(TYPES[dt]).eps / 2 * np.maximum(np.abs(want) + bound, tiny)
        off = np.abs(got.double().cpu().numpy() - want)
        assert (off <= b).all(), (name, (off - b).max(), off.max())


# The narrowest last token tile behind whole ones of 256: the fewest and the most
# tokens in it, a ragged N and K, one weight tile and more tiles than pairs of SMs,
# one and several whole token tiles.
TAILS = [(257, 128, 32), (272, 130, 96), (258, 640, 1056), (517, 20736, 320), (1029, 6400, 544), (2049, 384, 2336)]


@pytest.mark.parametrize("M,N,K", TAILS)
@pytest.mark.parametrize("epi", ["store", "f32", "residual", "in place"])
@pytest.mark.parametrize("fmt", list(FMT))
def test_a_few_tokens_behind_whole_tiles(M, N, K, epi, fmt):
    rng = np.random.default_rng(M + K)
    a, w = Rows(rng, M, K, fmt, plain=True), Rows(rng, N, K, fmt, plain=True)
    in_place, epi = epi == "in place", "residual" if epi == "in place" else epi
    dtype = torch.bfloat16 if epi == "store" else torch.float32
    want = torch.from_numpy(2.0 ** -6 * (a.values @ w.values.T) + (epi == "residual")).to(dtype)
    for offset in (0, 1):  # of C, in elements: written by tiles, and one by one
        buf = torch.full((offset + M * N + 64,), 5.0, dtype=dtype, device="cuda")
        c = buf[offset:offset + M * N].view(M, N)
        r = None if epi != "residual" else c.fill_(1.0) if in_place else torch.ones(M, N, device="cuda")
        run(a, w, fmt, epi, alpha=2.0 ** -6, residual=r, out=c, variant=sar.SAR_FP4_GEMM_PAIR)
        assert torch.equal(c.cpu(), want)
        assert (buf[:offset] == 5.0).all() and (buf[offset + M * N:] == 5.0).all()


@pytest.mark.parametrize("M,N,K", [(257, 128, 32), (264, 640, 1056), (528, 20736, 320), (1029, 6400, 544)])
@pytest.mark.parametrize("fmt", list(FMT))
def test_swiglu_of_a_few_tokens_behind_whole_tiles(M, N, K, fmt):
    test_epilogues(M, N, K, "swiglu", "bf16", fmt)


def test_residual_in_place_and_repeated():
    rng = np.random.default_rng(4)
    a, w = Rows(rng, 70, 1024, "nv", plain=True), Rows(rng, 384, 1024, "nv", plain=True)
    h = torch.arange(70 * 384, device="cuda").view(70, 384).float() % 64
    want = h.double().cpu().numpy() + 2 * (a.values @ w.values.T)
    for _ in range(2):
        run(a, w, "nv", "residual", residual=h, out=h)
    assert np.array_equal(h.cpu().numpy(), want)


@pytest.mark.parametrize("M,N", [(5, 136), (40, 131), (129, 258)])
@pytest.mark.parametrize("epi", ["store", "f32", "residual"])
@pytest.mark.parametrize("offset", [0, 1, 2])
def test_output_alignment_and_nothing_beside_it(M, N, epi, offset):
    rng = np.random.default_rng(N)
    a, w = Rows(rng, M, 320, "nv", plain=True), Rows(rng, N, 320, "nv", plain=True)
    dtype = torch.float16 if epi == "store" else torch.float32
    buf = torch.full((offset + M * N + 64,), 5.0, dtype=dtype, device="cuda")
    c = buf[offset:offset + M * N].view(M, N)
    r = torch.ones(M, N, device="cuda")
    run(a, w, "nv", epi, alpha=2.0 ** -6, residual=r if epi == "residual" else None, out=c)
    want = torch.from_numpy(2.0 ** -6 * (a.values @ w.values.T) + (epi == "residual")).to(dtype)
    assert torch.equal(c.cpu(), want)
    assert (buf[:offset] == 5.0).all() and (buf[offset + M * N:] == 5.0).all()


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("M", [3, 140])
def test_nan_scale_poisons_its_row_alone(fmt, M):
    rng = np.random.default_rng(9)
    a, w = Rows(rng, M, 512, fmt, plain=True), Rows(rng, 256, 512, fmt, plain=True)
    x = torch.randn(M, 512, device="cuda")
    x[1, 300] = float("nan")
    x[2, 511] = float("inf")
    sar.fp4_quantize(x, a.codes, a.scales, format=FMT[fmt])
    got = run(a, w, fmt)
    bad = torch.isnan(got).cpu()
    assert bad[1:3].all() and bad.sum() == 2 * 256


def test_no_tokens():
    w = Rows(np.random.default_rng(0), 64, 64, "nv")
    a = torch.empty(0, 32, dtype=torch.uint8, device="cuda")
    a = a.view(0, 32)
    n = sar.launch_count()
    sar.gemm_fp4(a, torch.empty(0, dtype=torch.uint8, device="cuda"), w.codes, w.scales,
                 torch.empty(0, 64, dtype=torch.float16, device="cuda"))
    assert sar.launch_count() == n


def test_python_refusals():
    rng = np.random.default_rng(0)
    a, w = Rows(rng, 4, 64, "nv"), Rows(rng, 128, 64, "nv")
    c = torch.empty(4, 128, dtype=torch.float16, device="cuda")
    good = dict(a=a.codes, a_scales=a.scales, w=w.codes, w_scales=w.scales, c=c)
    sar.gemm_fp4(**good)
    for bad in (dict(a=a.codes[:, :16]), dict(a=a.codes.int()), dict(a=a.codes.cpu()), dict(a_scales=a.scales[:100]),
                dict(w=w.codes.t()), dict(w_scales=w.scales.int()), dict(c=c.float()), dict(c=c[:3]), dict(c=c.t()),
                dict(residual=c.float()), dict(epilogue=sar.SAR_EPI_RESIDUAL, c=c.float()),
                dict(epilogue=sar.SAR_EPI_SWIGLU), dict(epilogue=sar.SAR_EPI_F32)):
        with pytest.raises(ValueError):
            sar.gemm_fp4(**(good | bad))


def test_captured_and_on_another_stream():
    rng = np.random.default_rng(2)
    w = Rows(rng, 512, 1024, "nv", plain=True)
    x = torch.randn(24, 1024, device="cuda", dtype=torch.bfloat16)
    codes = torch.empty(24, 512, dtype=torch.uint8, device="cuda")
    scales = torch.empty(sar.fp4_scale_bytes(24, 1024), dtype=torch.uint8, device="cuda")
    c = torch.empty(24, 512, device="cuda")

    def layer():
        sar.fp4_quantize(x, codes, scales)
        sar.gemm_fp4(codes, scales, w.codes, w.scales, c, epilogue=sar.SAR_EPI_F32)

    layer()
    first = c.clone()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        layer()
    x2 = torch.randn_like(x)
    x.copy_(x2)
    g.replay()
    torch.cuda.synchronize()
    second = c.clone()
    assert not torch.equal(first, second)
    with torch.cuda.stream(torch.cuda.Stream()):
        layer()
    torch.cuda.synchronize()
    assert torch.equal(c, second)
