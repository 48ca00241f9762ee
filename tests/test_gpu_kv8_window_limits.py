"""Windows as large as their type: they mask nothing, for rows in front of the sequence's start too."""

import numpy as np
import pytest

import chunked_prefill_hybrid_sar_gb300 as sar

from test_gpu_kv8_attention import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 30, 1 << 20])
@pytest.mark.parametrize("heads,kv_heads,d,page", [(4, 2, 128, 16), (8, 1, 64, 64)])
def test_a_window_beyond_every_key_is_none(window, heads, kv_heads, d, page):
    """Sequences with more rows than tokens, whose first rows see nothing, beside others."""
    seqs = [(5, 2), (1, 0), (300, 17), (40, 200), (9, 0), (1, 70), (64, 1), (600, 500)]
    b = Batch(seqs, heads, kv_heads, d, page, "bf16", seed=page)
    want = b.check()
    got = b.check(window=window)
    assert np.array_equal(got, want)
    for (r, m), a in zip(seqs, b.off.tolist()):
        assert not got[a:a + max(0, r - m)].any() and got[a + max(0, r - m):a + r].any(-1).all()
    sar.op_sync_status()


def test_windows_about_the_position_itself():
    """Windows one short of, equal to and one past a row's position, with rows on either side of the start."""
    seqs = [(140, 130), (3, 1), (1, 129), (20, 300)]
    for window in (1, 2, 127, 128, 129, 130, 131, 299, 300, 301):
        Batch(seqs, 4, 2, 128, 16, "f16", seed=window).check(window=window)
    sar.op_sync_status()
