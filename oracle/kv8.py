"""Oracle of the 8-bit KV cache: page and slot maps, the append behind the
projection, attention over codes; NumPy, float64, one request and head at a time."""

from __future__ import annotations

import numpy as np

LEAST, MOST = -40, 60


def _table():
    c = np.arange(128)
    e, m = c // 8, c % 8
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    v[127] = np.nan
    return np.concatenate([v, -v])


E4M3 = _table()  # index = bit pattern


def codes_of(x):
    """The e4m3 code nearest to each x, ties to the even one, saturating; 0x7F for
    what is not finite."""
    x = np.asarray(x, np.float64)
    grid = E4M3[:127]
    a = np.minimum(np.abs(np.where(np.isfinite(x), x, 0)), 448)
    hi = np.clip(np.searchsorted(grid, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    down, up = a - grid[lo], grid[hi] - a
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return np.where(np.isfinite(x), code + 128 * np.signbit(x), 127).astype(np.uint8)


def scale_of(a):
    """The smallest power of two in range with a <= 448 s."""
    e = LEAST
    while e < MOST and a > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def turned(x, gain, eps, position, base):
    """One head, normalised and rotated."""
    x = np.asarray(x, np.float64)
    d = x.size
    if gain is not None:
        x = x / np.sqrt((x * x).mean() + eps) * gain
    if position is None:
        return x
    a = position * base ** (-2 * np.arange(d // 2) / d)
    u, w = x[:d // 2], x[d // 2:]
    return np.concatenate([u * np.cos(a) - w * np.sin(a), w * np.cos(a) + u * np.sin(a)])


def write(codes, scales, x, slots):
    """codes [pages, heads, size, d] and scales [pages, heads] after rows x [rows, heads, d]."""
    codes, scales = codes.copy(), scales.copy()
    pages, heads, size, d = codes.shape
    r = 0
    while r < len(slots):
        if not 0 <= slots[r] < pages * size:
            r += 1
            continue
        p, o = divmod(int(slots[r]), size)
        n = 1
        while r + n < len(slots) and o + n < size and slots[r + n] == slots[r] + n:
            n += 1
        for h in range(heads):
            y = x[r:r + n, h]
            s = scale_of(np.abs(np.where(np.isfinite(y), y, 0)).max())
            if o:
                s = max(s, float(scales[p, h]))
                if s > scales[p, h] > 0:
                    codes[p, h, :o] = codes_of(E4M3[codes[p, h, :o]] * (float(scales[p, h]) / s))
            codes[p, h, o:o + n] = codes_of(y / s)
            scales[p, h] = s
        r += n
    return codes, scales


def page_map(lens, new, tables, free, count, page, max_rows):
    """Request by request; returns lens, tables, free list, count, row offsets,
    positions, slots and the requests that got nothing of what they asked for."""
    tables, free = tables.copy(), list(free)
    lens_out, offsets, refused = [], [0], []
    stack = free[:count]
    held = [-(-int(m) // page) for m in lens]
    for i, a in enumerate(new):
        if a == -1:
            stack += [int(p) for p in tables[i, :held[i]]]
    have, wanted, dry = len(stack), 0, False
    positions, slots = np.zeros(max_rows, np.int64), np.full(max_rows, -1, np.int64)
    at = 0
    given = list(stack)
    for i, (m, a) in enumerate(zip(lens, new)):
        add = max(int(a), 0)
        rows = range(at, min(at + add, max_rows))
        ok = add == 0 or at + add <= max_rows
        take = -(-(int(m) + add) // page) - held[i] if ok else 0
        if take:
            wanted += take
            dry = dry or wanted > have
            ok = not dry
            if ok:
                for j in range(take):
                    tables[i, held[i] + j] = given.pop()
        if not ok:
            refused.append(i)
        for r in rows:
            p = int(m) + r - at
            positions[r] = p
            if ok:
                slots[r] = tables[i, p // page] * page + p % page
        lens_out.append(0 if a == -1 else int(m) + (add if ok else 0))
        at += add
        offsets.append(min(at, max_rows))
    out = np.array(free)
    out[count:len(given)] = given[count:]
    return np.array(lens_out), tables, out, len(given), np.array(offsets), positions, slots, refused


def attention(q, k, v, rows, window=0, scale=None):
    """q [rows, heads, d] of a sequence's last rows over its keys and values
    [len, kv heads, d]; zero for a row that sees nothing."""
    n, heads, d = q.shape
    group = heads // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    out = np.zeros((n, heads, d))
    for j in range(n):
        p = k.shape[0] - rows + j
        lo = max(0, p - window + 1) if window else 0
        if p < 0:
            continue
        for h in range(heads):
            with np.errstate(all="ignore"):
                s = k[lo:p + 1, h // group] @ q[j, h] * scale
                w = np.exp(s - s.max())
                out[j, h] = (w[:, None] * v[lo:p + 1, h // group]).sum(0) / w.sum()
    return out
