"""Sequences with pages out of range: their rows attend to the keys that are left (tolerance of attention's own
test), a row that has none left is NaN, and the call is reported."""

import numpy as np
import pytest

import chunked_prefill_hybrid_sar_gb300 as sar
from chunked_prefill_hybrid_sar_gb300 import _lib

from test_gpu_kv8_attention import Batch

pytestmark = pytest.mark.gpu


def left(q, k, v, rows, gone, window):
    """Attention of the last `rows` tokens over the keys that are not gone, and the same of |V|; NaN where none is."""
    n, heads, d = q.shape
    group, out = heads // k.shape[1], np.full((2, n, heads, d), np.nan)
    for j in range(n):
        p = k.shape[0] - rows + j
        seen = np.array([i for i in range(max(0, p - window + 1) if window else 0, p + 1) if not gone[i]], int)
        if seen.size == 0:
            continue
        for h in range(heads):
            s = k[seen, h // group] @ q[j, h] * d ** -0.5
            w = np.exp(s - s.max())
            for o, x in zip(out, (v, np.abs(v))):
                o[j, h] = w @ x[seen, h // group] / w.sum()
    return out


@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("heads,kv_heads,d,kind", [(8, 2, 128, "f16"), (4, 4, 64, "bf16")])
@pytest.mark.parametrize("lost", ["first", "last", "middle", "odd", "all", "all but last"])
@pytest.mark.parametrize("window", [0, 40])
def test_rows_attend_to_what_is_left(page, heads, kv_heads, d, kind, lost, window):
    seqs = [(1, 300), (20, 300), (1, 17), (3, 64), (70, 129), (1, 3000), (2, 2500), (140, 200), (1, 90)]
    b = Batch(seqs, heads, kv_heads, d, page, kind, seed=page + d)
    keys = [(b.keys(i, 0), b.keys(i, 1)) for i in range(len(seqs))]
    gone, bad = [], (-1, 10 ** 6, -2 ** 31, int(b.codes.shape[1]))
    for i, (_, m) in enumerate(seqs):
        n = -(-m // page)
        which = {"first": [0], "last": [n - 1], "middle": [n // 2], "odd": range(1, n, 2), "all": range(n),
                 "all but last": range(n - 1)}[lost]
        g = np.zeros(m, bool)
        if i != len(seqs) - 1:  # (the last sequence stays whole)
            for j in which:
                b.tables[i, j] = bad[j % 4]
                g[j * page:(j + 1) * page] = True
        gone.append(g)
    got = b.run(window=window)
    with pytest.raises(sar.SarError) as e:
        sar.op_sync_status()
    assert e.value.code == _lib.SAR_ERR_BOUNDS
    q = b.q.double().numpy().reshape(b.rows, -1, d)
    eps = 2.0 ** -11 if kind == "f16" else 2.0 ** -8
    for i, ((r, m), (k, v)) in enumerate(zip(seqs, keys)):
        a, e = int(b.off[i]), int(b.off[i + 1])
        want, mean = left(q[a:e], k, v, r, gone[i], window)
        none = np.isnan(want)
        assert np.array_equal(np.isnan(got[a:e]), none), i
        tol = eps * np.abs(want) + 2.0 ** -10 * mean + np.abs(v).max() * m * 2.0 ** -25
        assert (np.abs(got[a:e] - want) <= tol)[~none].all(), i
