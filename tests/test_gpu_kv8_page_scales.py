"""Rows appended to pages whose present scale is no power of two (a cache that another program filled): codes are
h / s rounded to nearest even, ties included, so equal to the oracle's."""

import numpy as np
import pytest
import torch

import chunked_prefill_hybrid_sar_gb300 as sar
from oracle import kv8

pytestmark = pytest.mark.gpu

TIES = [17, 19, 21, 23, 25, 27, 29, 31, 8.5, 9.5, 10.5, 1.0625, 1.1875, 136, 152, 2 ** -10, 3 * 2 ** -10]


@pytest.mark.parametrize("kind", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("power", [-9, 0, 5])
def test_values_between_two_codes(kind, power):
    """A page each for scales of 7 bits; every value lies just between two codes under its page's scale, so that
    the quotient (a number of few bits, exact in fp32) is a tie."""
    d, page = 64, 16
    scales = np.arange(129, 256) / 128 * 2.0 ** power
    n = len(scales)
    x = np.zeros((n, d))
    for i, s in enumerate(scales):
        t = [c * s * sign for c in TIES for sign in (1, -1)]
        t = [y for y in t if float(torch.tensor(y).to(kind)) == y]  # (those that the rows' type holds)
        x[i, :len(t)] = t
    assert (x != 0).any(1).sum() > (100 if kind == torch.float32 else 8)
    codes = torch.zeros(n, 1, page, d, dtype=torch.uint8, device="cuda")
    s = torch.tensor(scales, dtype=torch.float32, device="cuda").view(n, 1)
    cache = sar.KV8Cache(codes, codes.clone(), s, s.clone())
    rows = torch.tensor(x).to(kind).cuda()
    slots = page * np.arange(n) + 1 + np.arange(n) % (page - 1)  # each page goes on at another place
    sar.qk_norm_rope(None, rows, None, head_dim=d, v=rows, cache=cache, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    want, want_scales = kv8.write(codes.cpu().numpy() * 0, s.cpu().numpy().astype(float), x[:, None], slots)
    for name in "kv":
        assert np.array_equal(getattr(cache, f"{name}_scales").cpu().numpy(), want_scales)
        assert np.array_equal(kv8.E4M3[getattr(cache, f"{name}_codes").cpu().numpy()], kv8.E4M3[want])
    sar.op_sync_status()


def test_a_page_that_grows_out_of_such_a_scale():
    """Rows in front are rounded anew from their old scale to the power of two that takes its place."""
    d, page = 128, 32
    g = torch.Generator().manual_seed(5)
    # (e4m3 codes times a scale of 7 bits over a power of two: exact in fp32)
    codes = torch.randint(0, 127, (3, 2, page, d), generator=g, dtype=torch.uint8)
    s = torch.tensor([[129 / 128, 200 / 128], [255 / 128, 1.5], [131 / 128, 3.25]])
    cache = sar.KV8Cache(codes.cuda(), codes.clone().cuda(), s.cuda(), s.clone().cuda())
    x = torch.randn(3, 2 * d, generator=g) * 3000
    slots = [7, page + 31, 2 * page + 16]
    sar.qk_norm_rope(None, x.cuda(), None, head_dim=d, v=x.cuda(), cache=cache, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    want, want_scales = kv8.write(codes.numpy(), s.numpy().astype(float), x.double().numpy().reshape(3, 2, d), slots)
    assert np.array_equal(cache.v_scales.cpu().numpy(), want_scales) and (want_scales > s.numpy()).all()
    assert np.array_equal(kv8.E4M3[cache.v_codes.cpu().numpy()], kv8.E4M3[want])
