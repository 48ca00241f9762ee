"""4-bit products with a side that only one of the tilings can launch: the
library's own choice takes them."""

import numpy as np
import pytest
import torch

import chunked_prefill_hybrid_sar_gb300 as sar
from chunked_prefill_hybrid_sar_gb300 import _lib
from oracle import fp4

pytestmark = pytest.mark.gpu

LONG = 65535 * 128 + 256  # rows: more tiles than a grid has along y or z


@pytest.fixture(autouse=True)
def no_device_flags():
    sar.op_sync_status()
    yield
    torch.cuda.empty_cache()
    sar.op_sync_status()


def short(rows, K, seed):
    """Codes and power-of-two scales (sums are exact in fp32), and their values."""
    rng = np.random.default_rng(seed)
    code = rng.integers(0, 16, (rows, K)).astype(np.uint8)
    byte = (0x38 + 8 * rng.integers(-1, 2, (rows, K // 16))).astype(np.uint8)
    return torch.from_numpy(fp4.pack(code)).cuda(), torch.from_numpy(fp4.tile(byte)).cuda(), fp4.values(code, byte, "nv")


def long(K, some, seed):
    """LONG rows of random codes under scales of one; the values of `some` rows."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (LONG, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.full((sar.fp4_scale_bytes(LONG, K),), 0x38, dtype=torch.uint8, device="cuda")
    at = codes[torch.tensor(some, device="cuda")].cpu().numpy()
    code = np.stack([at & 15, at >> 4], -1).reshape(len(some), K)
    return codes, scales, fp4.values(code, np.full((len(some), K // 16), 0x38, np.uint8), "nv")


SOME = [0, 1, 127, 128, 4_000_000, 65535 * 128 - 1, 65535 * 128, LONG - 129, LONG - 1]


@pytest.mark.parametrize("K", [64, 320])
def test_many_weight_rows(K):
    a, w = short(16, K, 1), long(K, SOME, 2)
    c = torch.full((16, LONG), 7.0, dtype=torch.float16, device="cuda")
    sar.gemm_fp4(*a[:2], *w[:2], c)
    got = c[:, torch.tensor(SOME, device="cuda")].cpu()
    assert torch.equal(got, torch.from_numpy(a[2] @ w[2].T).half())
    with pytest.raises(sar.SarError) as e:
        sar.gemm_fp4(*a[:2], *w[:2], c, variant=sar.SAR_FP4_GEMM_SPLIT)
    assert e.value.code == _lib.SAR_ERR_UNSUPPORTED


# (the long K is what makes the split tiling the faster one by its estimate)
@pytest.mark.parametrize("N,K", [(64, 64), (128, 4096)])
def test_many_token_rows(N, K):
    a, w = long(K, SOME, 3), short(N, K, 4)
    c = torch.full((LONG, N), 7.0, dtype=torch.float16, device="cuda")
    sar.gemm_fp4(*a[:2], *w[:2], c)
    got = c[torch.tensor(SOME, device="cuda")].cpu()
    assert torch.equal(got, torch.from_numpy(a[2] @ w[2].T).half())
    # (tokens in tiles of 64 pass the grid at half as many)
    half = LONG // 2
    d = torch.full((half, N), 7.0, dtype=torch.float16, device="cuda")
    with pytest.raises(sar.SarError) as e:
        sar.gemm_fp4(a[0][:half], a[1], *w[:2], d, variant=sar.SAR_FP4_GEMM_SPLIT | sar.SAR_FP4_GEMM_TOKENS64)
    assert e.value.code == _lib.SAR_ERR_UNSUPPORTED
    sar.gemm_fp4(a[0][:half], a[1], *w[:2], d, variant=sar.SAR_FP4_GEMM_SPLIT)
    near = [i for i in SOME if i < half]
    assert torch.equal(d[torch.tensor(near, device="cuda")], c[torch.tensor(near, device="cuda")])
