"""Every scale byte that a 4-bit matrix may hold, turned back at tensor scales of
every size: equal to code x scale x tensor scale rounded once to fp32 (the
float64 product is exact), and that rounded once more to a 16-bit type."""

import numpy as np
import pytest
import torch

import chunked_prefill_hybrid_sar_gb300 as sar
from oracle import fp4

pytestmark = pytest.mark.gpu

FMT = {"nv": sar.SAR_FP4_NV, "mx": sar.SAR_FP4_MX}
# both ends are the smallest and largest tensor scales that the entry takes
SCALES = [3.0e-39, 2.0 ** -126, 1.7e-30, 2.0 ** -12, 0.0371, 0.99, 1.0, 1.5, 3.0, 31.9, 2.0 ** 100, 1.3e30, 3.4e38]


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16, torch.float16])
def test_every_scale_byte(fmt, scale, kind):
    top = 128 if fmt == "nv" else 256
    B = fp4.BLOCK[fmt]
    byte = np.arange(top, dtype=np.uint8).reshape(-1, 2)
    code = np.tile(np.arange(16, dtype=np.uint8), (top // 2, 2 * B // 16))
    y = torch.empty(code.shape, dtype=kind, device="cuda")
    sar.fp4_dequantize(torch.from_numpy(fp4.pack(code)).cuda(), torch.from_numpy(fp4.tile(byte)).cuda(), y,
                       format=FMT[fmt], tensor_scale=scale)
    with np.errstate(over="ignore"):
        want = fp4.values(code, byte, fmt, np.float64(np.float32(scale))).astype(np.float32)
    want = torch.from_numpy(want).to(kind)
    got = y.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    keep = ~torch.isnan(want)
    assert torch.equal(got[keep], want[keep])
    assert torch.equal(torch.signbit(got[keep]), torch.signbit(want[keep]))
