"""Float64 oracle of the microscaled 4-bit rows and of their product.

Codes are indices into the e2m1 magnitudes (bit 3 the sign); scales are e4m3
numbers (``nv``, blocks of 16) or powers of two (``mx``, blocks of 32).  Every
rounding is a search of the format's own table: nearest, ties to the even
index, saturating.
"""

from __future__ import annotations

import numpy as np

BLOCK = {"nv": 16, "mx": 32}
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# e4m3's finite non-negative numbers, index = byte: 3 mantissa bits, bias 7
E4M3 = np.array([(b & 7) * 2.0 ** -9 if b < 8 else (8 + (b & 7)) * 2.0 ** ((b >> 3) - 10) for b in range(127)])


def nearest(v: np.ndarray, table: np.ndarray) -> np.ndarray:
    """Index of the table entry nearest to each v >= 0."""
    hi = np.minimum(np.searchsorted(table, v), len(table) - 1)
    lo = np.maximum(hi - 1, 0)
    down, up = v - table[lo], table[hi] - v
    return np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)


def scale_value(byte: np.ndarray, fmt: str) -> np.ndarray:
    byte = byte.astype(np.int64)
    if fmt == "nv":
        return np.where(byte == 127, np.nan, E4M3[np.minimum(byte, 126)])
    return np.where(byte == 255, np.nan, np.ldexp(1.0, np.minimum(byte, 254).astype(np.int32) - 127))


def quantise(x: np.ndarray, fmt: str, inv_scale: float = 1.0):
    """(codes [rows, cols], scale bytes [rows, blocks]) of x times the fp32 ``inv_scale``, as float32 products."""
    with np.errstate(all="ignore"):
        t = (x.astype(np.float32) * np.float32(inv_scale)).astype(np.float64)
        t = t.reshape(x.shape[0], -1, BLOCK[fmt])
        a = np.abs(t).max(-1)
        bad = ~np.isfinite(a)
        ok = np.where(bad, 0.0, a)
        if fmt == "nv":
            byte = nearest(ok / 6, E4M3)
        else:
            byte = np.where(ok > 0, np.maximum(np.frexp(ok)[1] - 1 - 2, -127), -127) + 127
        s = scale_value(byte, fmt)[..., None]
        q = np.divide(np.abs(t), s, out=np.zeros_like(t), where=(s > 0) & ~bad[..., None])
        code = nearest(q, E2M1) + 8 * np.signbit(t)
        code = np.where(bad[..., None] | (s == 0), 0, code)
    return code.reshape(x.shape).astype(np.uint8), np.where(bad, 127 if fmt == "nv" else 255, byte).astype(np.uint8)


def values(code: np.ndarray, byte: np.ndarray, fmt: str, scale: float = 1.0) -> np.ndarray:
    v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    v = v.reshape(code.shape[0], -1, BLOCK[fmt]) * scale_value(byte, fmt)[..., None]
    return v.reshape(code.shape) * scale


def pack(code: np.ndarray) -> np.ndarray:
    """Two codes to a byte, the even column in the low half."""
    return (code[:, 0::2] | code[:, 1::2] << 4).astype(np.uint8)


def tile(byte: np.ndarray, fill: int = 0) -> np.ndarray:
    """Scale bytes in the library's order; ``fill`` in the rows behind the last."""
    rows, blocks = byte.shape
    tiles = -(-blocks // 4)
    out = np.full((-(-rows // 128), tiles, 512), fill, np.uint8)
    for r in range(rows):
        for t in range(tiles):
            at = r % 32 * 16 + r % 128 // 32 * 4
            row = np.zeros(4, np.uint8)
            row[:min(4, blocks - 4 * t)] = byte[r, 4 * t:4 * t + 4]
            out[r // 128, t, at:at + 4] = row
    return out.reshape(-1)


def swiglu(d: np.ndarray) -> np.ndarray:
    """silu(gate) * up of columns that alternate in blocks of 64."""
    m, n = d.shape
    d = d.reshape(m, n // 128, 2, 64)
    g = d[:, :, 0]
    with np.errstate(over="ignore"):
        return (g / (1 + np.exp(-g)) * d[:, :, 1]).reshape(m, n // 2)
