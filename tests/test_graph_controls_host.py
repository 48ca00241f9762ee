"""What a step graph refuses of its controls, without a GPU: no call gets to
the library or to a tensor's memory."""

import types
import weakref

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
    g._pending = g._controls = None
    g._earlier = []
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


def test_an_enqueued_step_keeps_its_controls(monkeypatch):
    """The step reads the arrays of the controls that it was enqueued under until
    it has been waited for, whatever the graph has been given since."""
    fake = types.SimpleNamespace(sar_graph_set_controls=lambda h, c: 0, sar_graph_wait=lambda h: 0,
                                 sar_graph_enqueue_host_tokens=lambda *a: 0, sar_graph_destroy=lambda h: 0)
    monkeypatch.setattr(sar, "lib", lambda: fake)
    g = graph()
    buf = types.SimpleNamespace(data_ptr=lambda: 0)

    def set_new():
        c = controls()
        g.set_controls(c)
        return weakref.ref(c)

    first = set_new()
    second = set_new()
    assert first() is None  # no step under way
    g.enqueue_host_tokens(buf, buf, stream=1)
    third = set_new()
    g.enqueue_host_tokens(buf, buf, stream=1)
    g.set_controls(None)
    assert second() is not None and third() is not None
    g.wait()
    assert second() is None and third() is None
