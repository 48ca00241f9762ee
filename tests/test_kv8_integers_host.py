"""The 8-bit cache's entries without a GPU: numbers that the library's 32-bit fields do not hold are refused, not cut."""

import ctypes

import pytest
import torch

import chunked_prefill_hybrid_sar_gb300 as sar

from test_kv8_views_host import a_cache, calls, ints  # noqa: F401

BIG = [2 ** 31, 2 ** 32, 2 ** 32 + 16, -2 ** 31 - 1, 2 ** 63]


def attend(**kw):
    q = torch.zeros(2, 64, dtype=torch.float16)
    sar.kv8_attention(q, a_cache(), ints(4), ints(3), ints(3, 9), q.clone(), workspace=torch.zeros(16, dtype=torch.uint8), **kw)


@pytest.mark.parametrize("big", BIG)
@pytest.mark.parametrize("name", ["window", "max_rows", "max_len"])
def test_attention(calls, name, big):  # noqa: F811
    with pytest.raises(ValueError, match="32 bits"):
        attend(**{name: big})
    assert not calls
    for fits in (1, 2 ** 31 - 1):
        attend(**{name: fits})
        assert getattr(calls["sar_kv8_attention"], name) == fits


@pytest.mark.parametrize("big", BIG)
def test_workspace(big):
    q, cache = torch.zeros(2, 64, dtype=torch.float16), object.__new__(sar.KV8Cache)
    cache.head_dim, cache.ref = 64, ctypes.byref(sar._lib.sar_kv8())
    for kw in (dict(n=big), dict(n=1, max_rows=big), dict(n=1, max_len=big)):
        with pytest.raises(ValueError, match="32 bits"):
            sar.kv8_attention_workspace(cache, q, **kw)


@pytest.mark.parametrize("big", BIG)
def test_page_map(calls, big):  # noqa: F811
    with pytest.raises(ValueError, match="32 bits"):
        sar.page_map(ints(3), ints(3), ints(3, 9), ints(5), ints(1), ints(4), ints(6), ints(6), big)
    assert not calls


@pytest.mark.parametrize("head_dim", [0, -64, 2 ** 32 + 64])
def test_head_rows(calls, head_dim):  # noqa: F811
    q = torch.zeros(2, 64, dtype=torch.float16)
    for rows in ((q, None, q.clone()), (None, q, None), (q, q, q.clone())):
        with pytest.raises(ValueError, match="head_dim|32 bits"):
            sar.qk_norm_rope(*rows, head_dim=head_dim)
    assert not calls
