"""Batches without rows through the Python entries."""

import pytest
import torch

import chunked_prefill_hybrid_sar_gb300 as sar

pytestmark = pytest.mark.gpu


def test_an_empty_batch_changes_nothing():
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.arange(4 * 64, dtype=torch.int16, device="cuda").view(4, 64)
    before = table.clone()
    mask = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    ctl = sar.LogitControls(state=table, slots=none, repetition=torch.empty(0, device="cuda"), bias_offsets=start,
                            bias_tokens=none, bias_values=torch.empty(0, device="cuda"), mask=mask, mask_rows=none,
                            count_picks=True)
    x = torch.empty(0, 64, device="cuda")
    sar.logits_control(x, ctl, out=torch.empty_like(x), tokens_out=none)
    sar.logits_control(x, ctl, tokens_out=none)
    for reset in (True, False):
        sar.token_state_add(table, none, start, none, prompt_lens=none, reset=reset)
    q = torch.empty(0, 32, dtype=torch.uint8, device="cuda")
    s = torch.empty(0, dtype=torch.uint8, device="cuda")
    sar.fp4_quantize(x, q, s)
    sar.fp4_dequantize(q, s, x)
    w = torch.zeros(16, 32, dtype=torch.uint8, device="cuda")
    sw = torch.zeros(sar.fp4_scale_bytes(16, 64), dtype=torch.uint8, device="cuda")
    sar.gemm_fp4(q, s, w, sw, torch.empty(0, 16, device="cuda"), epilogue=sar.SAR_EPI_F32)
    sar.op_sync_status()
    assert torch.equal(table, before)
    # one row: its pick is made and counted
    pick = torch.empty(1, dtype=torch.int32, device="cuda")
    one = sar.LogitControls(state=table, slots=start, count_picks=True)
    sar.logits_control(torch.arange(64.0, device="cuda").view(1, 64), one, tokens_out=pick)
    assert pick.item() == 63 and table[0, 63] == before[0, 63] + 1
