"""Batches without rows: nothing is read, checked for length or launched."""

import ctypes

import pytest

import chunked_prefill_hybrid_sar_gb300 as sar
from chunked_prefill_hybrid_sar_gb300 import _lib

P = 1 << 20  # an aligned address that no call gets to use


# what an empty batch's tensors (null where they hold nothing) come as
@pytest.mark.parametrize("ctl", [
    {}, dict(state=P, n_slots=4, state_ld=64), dict(state=P, n_slots=4, state_ld=64, count_picks=1),
    dict(mask=P, n_masks=2, mask_ld=2),
])
def test_controls_of_an_empty_batch(ctl):
    c = _lib.sar_logit_controls()
    for k, v in ctl.items():
        setattr(c, k, v)
    lib = sar.lib()
    for tokens in (P, None):
        assert lib.sar_logits_control(None, 64, 0, 64, 2, ctypes.byref(c), None, 0, tokens, None) == _lib.SAR_OK
    # with a row, the missing slots (or outputs) are refused as before
    if "state" in ctl:
        assert lib.sar_logits_control(P, 64, 1, 64, 2, ctypes.byref(c), None, 0, P, None) == _lib.SAR_ERR_INVALID_ARG
    assert lib.sar_logits_control(P, 64, 1, 64, 2, ctypes.byref(c), None, 0, None, None) == _lib.SAR_ERR_INVALID_ARG
