"""4-bit rows without a GPU: the oracle's pins and the entry points' refusals."""

import ctypes

import numpy as np
import pytest

import chunked_prefill_hybrid_sar_gb300 as sar
from chunked_prefill_hybrid_sar_gb300 import _lib
from oracle import fp4


def test_tables():
    assert fp4.E4M3[1] == 2.0 ** -9 and fp4.E4M3[8] == 2.0 ** -6 and fp4.E4M3[126] == 448
    assert (np.diff(fp4.E4M3) > 0).all()


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_ties_go_to_the_even_code(fmt):
    row = np.tile([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], 4)[None]
    code, byte = fp4.quantise(row, fmt)  # largest 6: the scale is one in both formats
    assert fp4.scale_value(byte, fmt).tolist() == [[1.0] * (32 // fp4.BLOCK[fmt])]
    assert code[0, :8].tolist() == [0, 2, 2, 4, 4, 6, 6, 7]
    assert fp4.values(code, byte, fmt)[0, :8].tolist() == [0, 1, 1, 2, 2, 4, 4, 6]


def test_scales():
    x = np.zeros((4, 32))
    x[0, 0], x[1, 3], x[2, 5], x[3, 7] = 12.0, 7.99, 2.0 ** -20, np.inf
    assert fp4.quantise(x, "mx")[1].ravel().tolist() == [127 + 1, 127, 127 - 22, 255]
    nv = fp4.quantise(x, "nv")[1]
    assert fp4.scale_value(nv, "nv")[:3, 0].tolist() == [2.0, 1.375, 0.0] and nv[3, 0] == 127
    assert not fp4.quantise(x, "nv")[0][2].any()


def test_tile_order():
    byte = np.arange(130 * 5, dtype=np.int64).reshape(130, 5) % 251
    t = fp4.tile(byte.astype(np.uint8))
    assert t.size == 2 * 2 * 512
    for r, b in ((0, 0), (31, 3), (32, 1), (127, 4), (129, 2)):
        at = (r // 128 * 2 + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4
        assert t[at] == byte[r, b]


def test_scale_bytes():
    for rows, cols, fmt, n in ((1, 32, sar.SAR_FP4_NV, 512), (128, 64, sar.SAR_FP4_NV, 512),
                               (129, 96, sar.SAR_FP4_NV, 2 * 2 * 512), (128, 128, sar.SAR_FP4_MX, 512),
                               (1, 160, sar.SAR_FP4_MX, 1024), (0, 64, sar.SAR_FP4_NV, 0)):
        assert sar.fp4_scale_bytes(rows, cols, fmt) == n


P = 1 << 20  # an aligned address that no call gets to use


@pytest.mark.parametrize("change,code", [
    (dict(x=None), "INVALID"), (dict(codes=None), "INVALID"), (dict(scales=None), "INVALID"),
    (dict(rows=-1), "INVALID"), (dict(cols=0), "INVALID"), (dict(cols=48), "UNSUPPORTED"), (dict(ld=31), "INVALID"),
    (dict(kind=3), "INVALID"), (dict(fmt=2), "INVALID"), (dict(scale=0.0), "INVALID"), (dict(scale=-1.0), "INVALID"),
    (dict(scale=float("nan")), "INVALID"), (dict(scale=float("inf")), "INVALID"), (dict(scale=1e-40), "INVALID"),
    (dict(x=P + 1), "INVALID"), (dict(codes=P + 8), "INVALID"), (dict(scales=P + 4), "INVALID"),
    (dict(rows=2 ** 31 - 1, cols=2 ** 20, ld=2 ** 20), "UNSUPPORTED"),
])
def test_rows_are_refused(change, code):
    a = dict(x=P, ld=64, rows=3, cols=32, kind=1, fmt=0, scale=1.0, codes=P, scales=P) | change
    want = {"INVALID": _lib.SAR_ERR_INVALID_ARG, "UNSUPPORTED": _lib.SAR_ERR_UNSUPPORTED}[code]
    q = sar.lib().sar_op_fp4_quantize(a["x"], a["ld"], a["rows"], a["cols"], a["kind"], a["fmt"], a["scale"],
                                      a["codes"], a["scales"], None)
    d = sar.lib().sar_op_fp4_dequantize(a["codes"], a["scales"], a["rows"], a["cols"], a["fmt"], a["scale"], a["x"],
                                        a["ld"], a["kind"], None)
    assert (q, d) == (want, want)


def test_no_rows_is_no_work():
    lib = sar.lib()
    assert lib.sar_op_fp4_quantize(None, 32, 0, 32, 0, 0, 1.0, None, None, None) == _lib.SAR_OK
    assert lib.sar_op_fp4_dequantize(None, None, 0, 32, 0, 1.0, None, 32, 0, None) == _lib.SAR_OK
    n = ctypes.c_int64()
    assert lib.sar_op_fp4_scale_bytes(1, 33, 0, ctypes.byref(n)) == _lib.SAR_ERR_UNSUPPORTED


@pytest.mark.parametrize("change,code", [
    (dict(a=None), "INVALID"), (dict(sa=None), "INVALID"), (dict(w=None), "INVALID"), (dict(sw=None), "INVALID"),
    (dict(c=None), "INVALID"), (dict(M=-1), "INVALID"), (dict(N=0), "INVALID"), (dict(K=0), "INVALID"),
    (dict(K=48), "UNSUPPORTED"), (dict(epi=4), "INVALID"), (dict(epi=-1), "INVALID"), (dict(fmt=2), "INVALID"),
    (dict(storage=2), "INVALID"), (dict(variant=0xff), "INVALID"), (dict(variant=-1), "INVALID"),
    (dict(variant=1 << 16), "INVALID"), (dict(variant=0x100), "INVALID"), (dict(variant=0x1002), "INVALID"), (dict(variant=0x2001), "INVALID"), (dict(epi=2, N=192), "UNSUPPORTED"), (dict(epi=1), "INVALID"),
    (dict(a=P + 8), "INVALID"), (dict(w=P + 8), "INVALID"), (dict(sa=P + 1), "INVALID"), (dict(sw=P + 4), "INVALID"),
    (dict(c=P + 1), "INVALID"), (dict(epi=3, c=P + 2), "INVALID"), (dict(epi=1, r=P + 2), "INVALID"),
])
def test_product_is_refused(change, code):
    a = dict(a=P, sa=P, w=P, sw=P, c=P, r=None, M=4, N=128, K=64, alpha=1.0, epi=0, fmt=0, variant=0, storage=0) | change
    rc = sar.lib().sar_op_gemm_fp4(a["a"], a["sa"], a["w"], a["sw"], a["c"], a["r"], a["M"], a["N"], a["K"], a["alpha"],
                                   a["epi"], a["fmt"], a["variant"], a["storage"], None)
    assert rc == {"INVALID": _lib.SAR_ERR_INVALID_ARG, "UNSUPPORTED": _lib.SAR_ERR_UNSUPPORTED}[code]


def test_product_of_no_tokens_is_no_work():
    assert sar.lib().sar_op_gemm_fp4(None, None, None, None, None, None, 0, 64, 64, 1.0, 0, 0, 0, 0, None) == _lib.SAR_OK


@pytest.mark.parametrize("change", [dict(M=2 ** 31 - 1), dict(N=2 ** 31 - 1), dict(K=2 ** 31 - 32), dict(M=2 ** 30 + 1)])
def test_sides_whose_tiles_pass_32_bits_are_refused(change):
    a = dict(M=4, N=128, K=64) | change
    rc = sar.lib().sar_op_gemm_fp4(P, P, P, P, P, None, a["M"], a["N"], a["K"], 1.0, 0, 0, 0, 0, None)
    assert rc == _lib.SAR_ERR_UNSUPPORTED
