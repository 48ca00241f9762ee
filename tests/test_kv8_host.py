"""The 8-bit cache without a GPU: the oracle's pins and the entry points' refusals."""

import ctypes

import numpy as np
import pytest
import torch

import chunked_prefill_hybrid_sar_gb300 as sar
from chunked_prefill_hybrid_sar_gb300 import _lib
from oracle import kv8

P = 1 << 20  # an aligned address that no call gets to use
CODE = {"INVALID": _lib.SAR_ERR_INVALID_ARG, "UNSUPPORTED": _lib.SAR_ERR_UNSUPPORTED, "OK": _lib.SAR_OK}


def test_codes_are_torchs():
    c = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(c, kv8.E4M3, equal_nan=True)
    x = torch.cat([torch.linspace(-448, 448, 4001), torch.linspace(-0.05, 0.05, 4001)])
    assert np.array_equal(kv8.codes_of(x.numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert kv8.codes_of([1e9, -1e9, np.inf, np.nan]).tolist() == [126, 254, 127, 127]


def test_scale_borders():
    assert [kv8.scale_of(a) for a in (448, 448.1, 224, 224.1, 0)] == [1, 2, 0.5, 1, 2.0 ** -40]
    assert kv8.scale_of(448 * 2.0 ** 60) == kv8.scale_of(1e30) == 2.0 ** 60


def test_page_map_by_hand():
    """Three requests of pages of 2: one ends, one grows into a new page, one comes in."""
    tables = np.array([[7, 8, -1], [3, -1, -1], [-1, -1, -1]])
    lens, tab, free, count, off, pos, slots, refused = kv8.page_map([3, 2, 0], [-1, 1, 3], tables, [5, 6, 0, 0, 0], 2, 2, 6)
    # the list becomes 5 6 7 8; the second request takes 8, the third 7 and 6
    assert lens.tolist() == [0, 3, 3] and tab.tolist() == [[7, 8, -1], [3, 8, -1], [7, 6, -1]]
    assert count == 1 and off.tolist() == [0, 0, 1, 4] and refused == []
    assert pos.tolist() == [2, 0, 1, 2, 0, 0] and slots.tolist() == [16, 14, 15, 12, -1, -1]
    assert free.tolist() == [5, 6, 0, 0, 0]


def test_page_map_first_come_first_served():
    tables = np.full((4, 3), -1)
    tables[3, 0] = 9
    lens, _, _, count, _, _, slots, refused = kv8.page_map([0, 0, 0, 1], [2, 5, 1, 1], tables, [1, 2], 2, 2, 20)
    assert refused == [1, 2] and lens.tolist() == [2, 0, 0, 2] and count == 1
    assert slots[:9].tolist() == [4, 5, -1, -1, -1, -1, -1, -1, 19]


def test_attention_of_equal_keys_is_the_mean():
    v = np.random.default_rng(0).normal(size=(5, 1, 8))
    out = kv8.attention(np.ones((2, 2, 8)), np.ones((5, 1, 8)), v, 2)
    assert np.allclose(out[0, 1], v[:4, 0].mean(0)) and np.allclose(out[1, 0], v[:, 0].mean(0))
    assert np.allclose(kv8.attention(np.ones((1, 1, 8)), np.ones((5, 1, 8)), v, 1, window=2)[0, 0], v[3:, 0].mean(0))
    assert not kv8.attention(np.ones((3, 1, 8)), np.ones((2, 1, 8)), v[:2], 3)[0].any()


# ---- refusals ------------------------------------------------------------------


def cache(**change):
    a = dict(k_codes=P, v_codes=P, k_scales=P, v_scales=P, num_pages=10, n_kv_heads=2, page_size=16, head_dim=128) | change
    return _lib.sar_kv8(*a.values())


BAD_CACHES = [
    (dict(k_codes=None), "INVALID"), (dict(v_codes=None), "INVALID"), (dict(k_scales=None), "INVALID"),
    (dict(v_scales=None), "INVALID"), (dict(num_pages=0), "INVALID"), (dict(n_kv_heads=0), "INVALID"),
    (dict(page_size=8), "UNSUPPORTED"), (dict(page_size=48), "UNSUPPORTED"), (dict(head_dim=96), "UNSUPPORTED"),
    (dict(num_pages=2 ** 27), "UNSUPPORTED"), (dict(num_pages=2 ** 26, n_kv_heads=2), "UNSUPPORTED"),
    (dict(k_codes=P + 8), "INVALID"), (dict(v_codes=P + 1), "INVALID"), (dict(k_scales=P + 2), "INVALID"),
]


def page_map(**change):
    a = dict(lens=P, new_lens=P, lens_out=P, block_tables=P, free_pages=P, free_count=P, free_count_out=P, row_offsets=P,
             positions=P, slots=P, n=3, bt_stride=4, page_size=16, num_pages=10, max_rows=5) | change
    return sar.lib().sar_page_map(ctypes.byref(_lib.sar_page_map_args(*a.values())), None)


@pytest.mark.parametrize("change,code", [
    *[({name: None}, "INVALID") for name in ("lens", "new_lens", "lens_out", "block_tables", "free_pages", "free_count",
                                             "free_count_out", "row_offsets", "positions", "slots")],
    *[({name: P + 2}, "INVALID") for name in ("lens", "block_tables", "free_count", "row_offsets", "slots")],
    (dict(n=-1), "INVALID"), (dict(bt_stride=0), "INVALID"), (dict(num_pages=0), "INVALID"), (dict(max_rows=-1), "INVALID"),
    (dict(page_size=24), "UNSUPPORTED"), (dict(n=8193), "UNSUPPORTED"), (dict(n=8192, bt_stride=2 ** 17 + 1), "UNSUPPORTED"),
    (dict(max_rows=2 ** 30 + 1), "UNSUPPORTED"), (dict(num_pages=2 ** 27), "UNSUPPORTED"),
    (dict(bt_stride=2 ** 27, n=1), "UNSUPPORTED"),
])
def test_page_map_is_refused(change, code):
    assert page_map(**change) == CODE[code]


def qk(change, with_cache=True, cache_change={}):
    a = dict(q=P, k=P, v=P, q_out=2 * P, k_out=None, ldq=512, ldk=256, ldv=256, ldq_out=512, ldk_out=256, q_gain=None,
             k_gain=None, positions=P, slots=P, rows=3, n_q_heads=4, n_kv_heads=2, head_dim=128, type=1, out_type=1,
             eps=1e-5, rope_base=1e4) | change
    c = cache(**cache_change)
    return sar.lib().sar_qk_norm_rope(ctypes.byref(_lib.sar_qk_rows(*a.values())), ctypes.byref(c) if with_cache else None, None)


@pytest.mark.parametrize("change,code", [
    (dict(q=None), "INVALID"), (dict(q_out=None), "INVALID"), (dict(k=None), "INVALID"), (dict(v=None), "INVALID"),
    (dict(slots=None), "INVALID"), (dict(rows=-1), "INVALID"), (dict(n_q_heads=-1), "INVALID"), (dict(n_kv_heads=1), "INVALID"),
    (dict(type=3), "INVALID"), (dict(out_type=2), "INVALID"), (dict(out_type=0), "INVALID"), (dict(head_dim=32), "UNSUPPORTED"),
    (dict(n_q_heads=1025, ldq=2 ** 20, ldq_out=2 ** 20), "UNSUPPORTED"), (dict(rows=2 ** 30 + 1), "UNSUPPORTED"),
    (dict(q_gain=P, eps=-1.0), "INVALID"), (dict(k_gain=P, eps=float("nan")), "INVALID"), (dict(rope_base=0.0), "INVALID"),
    (dict(rope_base=float("inf")), "INVALID"), (dict(ldq=511), "INVALID"), (dict(ldk=255), "INVALID"), (dict(ldv=255), "INVALID"),
    (dict(ldq_out=511), "INVALID"), (dict(k_out=3 * P, ldk_out=255), "INVALID"), (dict(k_out=P), "INVALID"),
    (dict(q_out=P, ldq_out=520), "INVALID"), (dict(q_out=P, type=2), "INVALID"), (dict(q=P + 1), "INVALID"),
    (dict(slots=P + 2), "INVALID"), (dict(positions=P + 1), "INVALID"),
])
def test_rows_are_refused(change, code):
    assert qk(change) == CODE[code]


@pytest.mark.parametrize("change,code", BAD_CACHES)
def test_rows_into_a_bad_cache_are_refused(change, code):
    assert qk({}, cache_change=change) == CODE[code]


def attention(change, cache_change={}):
    a = dict(q=P, out=P, ldq=512, ldo=512, row_offsets=P, lens=P, block_tables=P, workspace=P, workspace_bytes=1 << 40, rows=5,
             n=2, n_q_heads=4, bt_stride=8, storage=1, max_rows=4, max_len=0, window=0, scale=0.0) | change
    b, c = _lib.sar_kv8_batch(*a.values()), cache(**cache_change)
    return sar.lib().sar_kv8_attention(ctypes.byref(b), ctypes.byref(c), None)


@pytest.mark.parametrize("change,code", [
    *[({name: None}, "INVALID") for name in ("q", "out", "row_offsets", "lens", "block_tables", "workspace")],
    (dict(rows=-1), "INVALID"), (dict(n=-1), "INVALID"), (dict(n_q_heads=0), "INVALID"), (dict(max_rows=0), "INVALID"),
    (dict(max_len=-1), "INVALID"), (dict(window=-1), "INVALID"), (dict(n_q_heads=3), "UNSUPPORTED"),
    (dict(n_q_heads=18, ldq=2304, ldo=2304), "UNSUPPORTED"), (dict(storage=2), "INVALID"), (dict(scale=-1.0), "INVALID"),
    (dict(scale=float("nan")), "INVALID"), (dict(ldq=511), "INVALID"), (dict(ldo=511), "INVALID"), (dict(bt_stride=0), "INVALID"),
    (dict(bt_stride=2 ** 27), "UNSUPPORTED"), (dict(workspace=P + 8), "INVALID"), (dict(workspace_bytes=100), "INVALID"),
    (dict(q=P + 1), "INVALID"), (dict(lens=P + 2), "INVALID"), (dict(rows=2 ** 30 + 1), "UNSUPPORTED"),
])
def test_attention_is_refused(change, code):
    assert attention(change) == CODE[code]


@pytest.mark.parametrize("change,code", BAD_CACHES)
def test_attention_over_a_bad_cache_is_refused(change, code):
    assert attention({}, change) == CODE[code]


def test_nothing_is_no_work():
    none = dict(q=None, out=None, row_offsets=None, lens=None, block_tables=None, workspace=None)
    assert attention(dict(rows=0, **none)) == attention(dict(n=0, **none)) == _lib.SAR_OK
    assert qk(dict(rows=0, q=None, k=None, v=None, q_out=None, slots=None)) == _lib.SAR_OK
    assert qk(dict(q=None, k=None, v=None, q_out=None, n_q_heads=0, n_kv_heads=0), with_cache=False) == _lib.SAR_OK


def test_null_structs():
    lib = sar.lib()
    assert lib.sar_page_map(None, None) == lib.sar_qk_norm_rope(None, None, None) == _lib.SAR_ERR_INVALID_ARG
    assert lib.sar_kv8_attention(None, None, None) == _lib.SAR_ERR_INVALID_ARG
    assert lib.sar_kv8_attention_workspace(None, None, None) == _lib.SAR_ERR_INVALID_ARG


def test_handles_check_their_tensors():
    z = torch.zeros
    with pytest.raises(ValueError, match="uint8"):
        sar.KV8Cache(z(2, 1, 16, 64), z(2, 1, 16, 64), z(2, 1), z(2, 1))
    codes = z(2, 1, 16, 64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="scales"):
        sar.KV8Cache(codes, codes, z(2, 2), z(2, 1))
    with pytest.raises(ValueError, match="keys as values"):
        sar.KV8Cache(codes, codes[:1], z(2, 1), z(2, 1))
