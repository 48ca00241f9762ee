"""What a step graph refuses of its controls, without a GPU: no call gets to
the library or to a tensor's memory."""

import types

import pytest

import chunked_prefill_hybrid_sar_gb300 as sar
from chunked_prefill_hybrid_sar_gb300 import _lib


def graph(logit_rows=3, vocab=64, device=0):
    """A graph that was never captured: the library refuses its null handle."""
    g = object.__new__(sar.StepGraph)
    g.h = None
    g._vocab = vocab
    g._keep = (types.SimpleNamespace(logit_rows=logit_rows), None, None,
               types.SimpleNamespace(get_device=lambda: device), None)
    return g


def controls(rows=3, vocab=64, device=0):
    c = object.__new__(sar.LogitControls)
    c.rows, c.vocab, c.device, c.c = rows, vocab, device, _lib.sar_logit_controls()
    return c


@pytest.mark.parametrize("change", [dict(rows=2), dict(rows=0), dict(vocab=63), dict(vocab=1), dict(device=1)])
def test_controls_of_other_sizes_or_devices_are_refused(change):
    with pytest.raises(ValueError):
        graph().set_controls(controls(**change))


@pytest.mark.parametrize("change", [dict(), dict(rows=None), dict(rows=4, vocab=1 << 30), dict(device=None)])
def test_fitting_controls_reach_the_library(change):
    for c in (controls(**change), None):
        with pytest.raises(sar.SarError) as e:
            graph().set_controls(c)
        assert e.value.code == _lib.SAR_ERR_INVALID_ARG
