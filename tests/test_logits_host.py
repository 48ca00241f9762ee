"""Logits controls without a GPU: the oracle's pins and the entries' refusals."""

import ctypes

import numpy as np
import pytest

import chunked_prefill_hybrid_sar_gb300 as sar
from chunked_prefill_hybrid_sar_gb300 import _lib
from oracle import logits as ol

P = 1 << 20  # an aligned address that no call gets to use


def test_oracle_by_hand():
    x = np.array([2.0, -2.0, 1.0, 0.0, 5.0])
    s = np.array([0x8000, 0x8000, 3, 1, 0], np.uint16)
    y = ol.changed(x, s, 2.0, 0.5, 0.25, [(4, 1.0), (0, -1.0), (4, 2.0), (9, 7.0)], np.array([0b10111], np.uint32))
    assert y.tolist() == [0.0, -4.0, 0.5 - 0.75 - 0.5, -np.inf, 8.0]
    assert ol.pick(y) == 4 and ol.pick(np.full(3, -np.inf)) == -1 and ol.pick(np.array([np.nan, 1.0, 1.0])) == 1


def test_oracle_state():
    t = ol.state_add(np.zeros((3, 4), np.uint16), [2, 0], [[1, 1, 3], [0]], [1, 0], 4, False)
    assert t.tolist() == [[1, 0, 0, 0], [0, 0, 0, 0], [0, 0x8001, 0, 1]]
    t[0, 0] = ol.MOST
    t = ol.state_add(t, [0, 2], [[0], [3]], [0, 0], 4, False)
    assert t[0, 0] == ol.MOST and t[2, 3] == 2
    assert ol.state_add(t, [2, 2], [[1], [2]], [0, 0], 3, True)[2].tolist() == [0, 1, 0, 2]


def controls(**kw):
    c = _lib.sar_logit_controls()
    for k, v in kw.items():
        setattr(c, k, v)
    return c


GOOD = dict(logits=P, ld=64, rows=2, vocab=64, kind=2, out=P, ld_out=64, tokens=P)


@pytest.mark.parametrize("change,ctl", [
    (dict(logits=None), {}), (dict(ld=63), {}), (dict(rows=-1), {}), (dict(vocab=0), {}), (dict(kind=3), {}),
    (dict(ld_out=63), {}), (dict(out=None, tokens=None), {}), (dict(logits=P + 2), {}), (dict(out=P + 2), {}),
    (dict(tokens=P + 2), {}), (dict(kind=0, logits=P + 1), {}),
    ({}, dict(repetition=P)), ({}, dict(count_picks=1)),
    (dict(tokens=None), dict(state=P, slots=P, n_slots=1, state_ld=64, count_picks=1)),
    ({}, dict(state=P, n_slots=1, state_ld=64)), ({}, dict(state=P, slots=P, n_slots=0, state_ld=64)),
    ({}, dict(state=P, slots=P, n_slots=1, state_ld=63)), ({}, dict(state=P + 1, slots=P, n_slots=1, state_ld=64)),
    ({}, dict(state=P, slots=P + 2, n_slots=1, state_ld=64)), ({}, dict(bias_offsets=P)),
    ({}, dict(bias_offsets=P, bias_tokens=P, bias_values=P, n_biases=-1)),
    ({}, dict(mask=P, mask_ld=1, n_masks=1)), ({}, dict(mask=P, mask_ld=2, n_masks=0)), ({}, dict(mask_rows=P)),
    ({}, dict(mask=P + 1, mask_ld=2, n_masks=1)),
])
def test_controls_are_refused(change, ctl):
    a = GOOD | change
    c = controls(**ctl)
    rc = sar.lib().sar_logits_control(a["logits"], a["ld"], a["rows"], a["vocab"], a["kind"], ctypes.byref(c), a["out"],
                                      a["ld_out"], a["tokens"], None)
    assert rc == _lib.SAR_ERR_INVALID_ARG


def test_no_rows_is_no_work():
    lib = sar.lib()
    assert lib.sar_logits_control(None, 8, 0, 8, 2, ctypes.byref(controls()), None, 0, P, None) == _lib.SAR_OK
    assert lib.sar_logits_control(P, 8, 1, 8, 2, None, None, 0, P, None) == _lib.SAR_ERR_INVALID_ARG
    assert lib.sar_token_state_add(P, 8, 1, 8, P, 0, P, P, 3, None, 1, None) == _lib.SAR_OK
    assert lib.sar_token_state_add(P, 8, 1, 8, P, 4, P, P, 0, None, 0, None) == _lib.SAR_OK
    assert lib.sar_graph_set_controls(None, None) == _lib.SAR_ERR_INVALID_ARG


@pytest.mark.parametrize("change,code", [
    (dict(state=None), 1), (dict(slots=None), 1), (dict(offsets=None), 1), (dict(tokens=None), 1), (dict(ld=7), 1),
    (dict(n_slots=0), 1), (dict(vocab=0), 1), (dict(n=-1), 1), (dict(n_tokens=-1), 1), (dict(state=P + 1), 1),
    (dict(slots=P + 2), 1), (dict(offsets=P + 1), 1), (dict(tokens=P + 2), 1), (dict(prompt=P + 3), 1),
    (dict(n=65536), 7),
])
def test_state_calls_are_refused(change, code):
    a = dict(state=P, ld=8, n_slots=2, vocab=8, slots=P, n=2, offsets=P, tokens=P, n_tokens=4, prompt=None) | change
    rc = sar.lib().sar_token_state_add(a["state"], a["ld"], a["n_slots"], a["vocab"], a["slots"], a["n"], a["offsets"],
                                       a["tokens"], a["n_tokens"], a["prompt"], 0, None)
    assert rc == code


# (a thread's next step past the end of such a list, or of such rows, would not fit 32 bits)
@pytest.mark.parametrize("change,ctl", [
    (dict(rows=2 ** 31 - 1), {}), (dict(vocab=2 ** 30 + 1, ld=2 ** 30 + 1, ld_out=2 ** 30 + 1), {}),
    ({}, dict(bias_offsets=P, bias_tokens=P, bias_values=P, n_biases=2 ** 31 - 1)),
])
def test_controls_beyond_32_bits_are_refused(change, ctl):
    a = GOOD | change
    rc = sar.lib().sar_logits_control(a["logits"], a["ld"], a["rows"], a["vocab"], a["kind"], ctypes.byref(controls(**ctl)),
                                      a["out"], a["ld_out"], a["tokens"], None)
    assert rc == _lib.SAR_ERR_UNSUPPORTED


@pytest.mark.parametrize("reset", [0, 1])
@pytest.mark.parametrize("vocab,n_tokens", [(8, 2 ** 31 - 1), (2 ** 30 + 1, 4)])
def test_state_calls_beyond_32_bits_are_refused(reset, vocab, n_tokens):
    rc = sar.lib().sar_token_state_add(P, 2 ** 31, 2, vocab, P, 2, P, P, n_tokens, None, reset, None)
    assert rc == _lib.SAR_ERR_UNSUPPORTED
