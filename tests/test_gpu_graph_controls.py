"""A step graph's controls whose tables are cut out of wider ones."""

import dataclasses

import pytest
import torch

import chunked_prefill_hybrid_sar_gb300 as sar
import synth
from chunked_prefill_hybrid_sar_gb300 import harness

pytestmark = pytest.mark.gpu


@pytest.fixture()
def step():
    case = synth.tiny_case(0, dtype=torch.bfloat16)
    dims = dataclasses.replace(case["dims"], vocab=1024)
    _, head, _ = synth.model_weights(0, dims, torch.bfloat16)
    m = harness.load_model(dims, case["layers"], head, max_tokens=64, max_decodes=8)
    kv = sar.KVCache(m, 16, 32)
    logits = torch.empty(2, dims.vocab, device="cuda")
    inp = torch.zeros(2, dtype=torch.int32, device="cuda")
    batch = sar.Batch(None, [(0, 0, [0, 1]), (1, 0, [2, 3])], in_kind=sar.SAR_IN_TOKENS)
    g = sar.StepGraph(m, kv, batch, inp, logits_out=logits)
    yield g, dims.vocab, logits
    g.close()
    m.close()


def run(g):
    host_in = torch.tensor([5, 6], dtype=torch.int32).pin_memory()
    out = torch.empty(2, dtype=torch.int32).pin_memory()
    g.launch_host_tokens(host_in, out)
    return out.tolist()


def test_narrow_views_are_refused(step):
    g, vocab, logits = step
    slots = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    table = torch.zeros(2, vocab + 16, dtype=torch.int16, device="cuda")
    words = -(-vocab // 32)
    mask = torch.full((2, words + 4), -1, dtype=torch.int32, device="cuda")
    for kw in (dict(state=table[:, 24:], slots=slots), dict(state=table[:, :vocab - 8], slots=slots),
               dict(mask=mask[:, 5:]), dict(mask=mask[:, :words - 1]), dict(state=table, slots=slots[:1])):
        with pytest.raises(ValueError):
            g.set_controls(sar.LogitControls(**kw))
    # what was refused left the graph as it was; a view of the whole width is taken
    assert run(g) == logits.argmax(1).tolist()
    table[1, 8:] = 1
    table[:, :8] = -1
    g.set_controls(sar.LogitControls(state=table[:, 8:8 + vocab], slots=slots, count_picks=True))
    picks = run(g)
    assert picks == logits.argmax(1).tolist()
    assert table[0, 8 + picks[0]] == 1 and table[1, 8 + picks[1]] == 2 and (table[:, :8] == -1).all()
