"""The 8-bit cache's entries without a GPU: what they hand on of tables that are views."""

import types

import pytest
import torch

import chunked_prefill_hybrid_sar_gb300 as sar

from test_kv8_host import CODE, attention, page_map


@pytest.fixture
def calls(monkeypatch):
    """The structs that reach the library, which is not called."""
    got = {}

    def keep(name):
        def call(args, *rest):
            got[name] = type(args._obj).from_buffer_copy(args._obj)
            return 0
        return call

    fake = types.SimpleNamespace(**{n: keep(n) for n in ("sar_page_map", "sar_kv8_attention", "sar_qk_norm_rope")})
    monkeypatch.setattr(sar, "lib", lambda: fake)
    monkeypatch.setattr(sar, "_launch_stream", lambda *a: None)
    return got


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def a_cache(pages=3):
    codes, scales = torch.zeros(pages, 1, 16, 64, dtype=torch.uint8), torch.zeros(pages, 1)
    return sar.KV8Cache(codes, codes.clone(), scales, scales.clone())


VIEWS = [(lambda t: t, 9, 9), (lambda t: t[:, :4], 9, 4), (lambda t: t[:, 5:], 9, 4), (lambda t: t[:, 2:3], 9, 1)]


@pytest.mark.parametrize("view,stride,columns", VIEWS)
def test_page_map_learns_a_views_columns(calls, view, stride, columns):
    sar.page_map(ints(3), ints(3), view(ints(3, 9)), ints(5), ints(1), ints(4), ints(6), ints(6), 16)
    a = calls["sar_page_map"]
    assert (a.bt_stride, a.bt_cols) == (stride, columns)


@pytest.mark.parametrize("view,stride,columns", VIEWS)
def test_attention_learns_a_views_columns(calls, view, stride, columns):
    cache = a_cache()
    q = torch.zeros(2, 64, dtype=torch.float16)
    sar.kv8_attention(q, cache, ints(4), ints(3), view(ints(3, 9)), q.clone(), workspace=torch.zeros(16, dtype=torch.uint8))
    b = calls["sar_kv8_attention"]
    assert (b.bt_stride, b.bt_cols) == (stride, columns)


@pytest.mark.parametrize("cols,code", [(-1, "INVALID"), (5, "INVALID")])
def test_columns_are_checked(cols, code):
    assert page_map(bt_stride=4, bt_cols=cols) == attention(dict(bt_stride=4, bt_cols=cols)) == CODE[code]




def test_tables_without_columns_are_refused(calls):
    with pytest.raises(ValueError, match="no columns"):
        sar.page_map(ints(3), ints(3), ints(3, 9)[:, 4:4], ints(5), ints(1), ints(4), ints(6), ints(6), 16)
    q = torch.zeros(2, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="no columns"):
        sar.kv8_attention(q, a_cache(), ints(4), ints(3), ints(3, 9)[:, 4:4], q.clone())
    assert not calls
