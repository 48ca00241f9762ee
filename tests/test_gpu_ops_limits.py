"""4-bit rows, their product and the logits controls where sizes pass 32 bits,
launches are many, or two run at once."""

import numpy as np
import pytest
import torch

import chunked_prefill_hybrid_sar_gb300 as sar
from oracle import fp4
from oracle import logits as ol

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_device_flags():
    sar.op_sync_status()
    yield
    torch.cuda.empty_cache()
    sar.op_sync_status()


def plain_rows(rng, rows, cols, fmt="nv"):
    """Codes and power-of-two scales (exact fp32 sums), and their values."""
    code = rng.integers(0, 16, (rows, cols)).astype(np.uint8)
    byte = (0x38 + 8 * rng.integers(-1, 2, (rows, cols // 16))).astype(np.uint8)
    return (torch.from_numpy(fp4.pack(code)).cuda(), torch.from_numpy(fp4.tile(byte)).cuda(), fp4.values(code, byte, fmt))


def test_more_than_2_31_elements():
    rows, cols = 530_000, 4128
    assert rows * cols > 2 ** 31
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    some = [0, 1, 260_000, 520_255, rows - 130, rows - 1]
    g = torch.Generator().manual_seed(1)
    part = torch.randn(len(some), cols, generator=g).bfloat16()
    x[torch.tensor(some, device="cuda")] = part.cuda()
    codes = torch.empty(rows, cols // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(sar.fp4_scale_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    sar.fp4_quantize(x, codes, scales)
    code, byte = fp4.quantise(part.float().numpy(), "nv")
    assert np.array_equal(codes[torch.tensor(some, device="cuda")].cpu().numpy(), fp4.pack(code))
    x.fill_(9.0)
    sar.fp4_dequantize(codes, scales, x)
    got = x[torch.tensor(some, device="cuda")].cpu()
    assert torch.equal(got, torch.from_numpy(fp4.values(code, byte, "nv")).bfloat16())
    assert int((x != 0).any(1).sum()) == len(some)


@pytest.mark.parametrize("variant", [sar.SAR_FP4_GEMM_PAIR, sar.SAR_FP4_GEMM_SPLIT, sar.SAR_FP4_GEMM_SPLIT | sar.SAR_FP4_GEMM_TOKENS64])
def test_a_product_of_more_than_2_31_results(variant):
    M, N, K = 66_003, 32_768, 64
    assert M * N > 2 ** 31
    rng = np.random.default_rng(0)
    a, w = plain_rows(rng, M, K), plain_rows(rng, N, K)
    c = torch.full((M, N), 7.0, dtype=torch.float16, device="cuda")
    sar.gemm_fp4(*a[:2], *w[:2], c, variant=variant)
    for m in (0, 127, 33_000, 65_535, 65_536, M - 3, M - 1):
        want = torch.from_numpy(a[2][m] @ w[2].T).half()
        assert torch.equal(c[m].cpu(), want), m


def test_more_rows_than_a_grid_has():
    rows, vocab = 70_001, 40
    x = torch.randn(rows, vocab, device="cuda")
    slots = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    slots[66_000] = 1
    state = torch.zeros(2, vocab, dtype=torch.int16, device="cuda")
    state[1, 3] = 2
    mask = torch.full((2, 2), -1, dtype=torch.int32, device="cuda")
    mask[1, 0] = 1 << 5
    mask_rows = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    mask_rows[rows - 1] = 1
    freq = torch.full((rows,), 50.0, device="cuda")
    y, picks = torch.empty_like(x), torch.empty(rows, dtype=torch.int32, device="cuda")
    sar.logits_control(x, sar.LogitControls(state=state, slots=slots, frequency=freq, mask=mask, mask_rows=mask_rows), out=y,
                       tokens_out=picks)
    want = x.clone()
    want[66_000, 3] -= 100.0
    want[rows - 1, :32] = float("-inf")  # (the mask's second word allows the rest)
    want[rows - 1, 5] = x[rows - 1, 5]
    assert torch.equal(y, want) and torch.equal(picks.long(), want.argmax(1))


def test_a_state_table_of_more_than_2_31_entries():
    slots, vocab = 17_000, 131_072
    table = torch.zeros(slots, vocab, dtype=torch.int16, device="cuda")
    where = torch.tensor([16_999, 0, 16_500], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 2, 3, 6], dtype=torch.int32, device="cuda")
    tok = torch.tensor([131_071, 131_071, 5, 0, 70_000, 131_071], dtype=torch.int32, device="cuda")
    for reset in (True, False):
        sar.token_state_add(table, where, off, tok, reset=reset)
    assert table[16_999, 131_071] == 4 and table[0, 5] == 2 and table[16_500, 70_000] == 2
    assert int(table.sum(dtype=torch.int64)) == 12
    picks = torch.empty(1, dtype=torch.int32, device="cuda")
    x = torch.zeros(1, vocab, device="cuda")
    x[0, 131_071], x[0, 70_000] = 3.0, 2.5
    sar.logits_control(x, sar.LogitControls(state=table, slots=where[2:], presence=torch.ones(1, device="cuda"), count_picks=True),
                       tokens_out=picks)
    assert picks.item() == 131_071 and table[16_500, 131_071] == 3


def test_two_streams_at_once():
    """Calls on two streams keep nothing that the other could overwrite."""
    rng = np.random.default_rng(5)
    work = []
    for i, (M, N, K) in enumerate([(9, 512, 4096), (300, 1024, 2048), (40, 700, 1024), (600, 512, 512)]):
        a, w = plain_rows(rng, M, K), plain_rows(rng, N, K)
        work.append((a, w, torch.empty(M, N, device="cuda")))
    x = torch.randn(64, 5000, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs = []
    for a, w, c in work:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sar.gemm_fp4(*a[:2], *w[:2], c, epilogue=sar.SAR_EPI_F32)
        graphs.append(g)
    picks = [torch.empty(64, dtype=torch.int32, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                for g in graphs[k::2]:
                    g.replay()
                sar.logits_control(x, sar.LogitControls(), tokens_out=picks[k])
                a, w, c = work[k]
                sar.gemm_fp4(*a[:2], *w[:2], c, epilogue=sar.SAR_EPI_F32)
    torch.cuda.synchronize()
    for a, w, c in work:
        assert np.array_equal(c.cpu().numpy(), a[2] @ w[2].T)
    for p in picks:
        assert torch.equal(p.long(), x.argmax(1))


def test_the_same_call_twice_gives_the_same_bits():
    rng = np.random.default_rng(6)
    x = torch.randn(70, 8192, device="cuda")
    w = torch.randn(1000, 8192, device="cuda")
    q = []
    for t in (x, w):
        codes = torch.empty(t.shape[0], 4096, dtype=torch.uint8, device="cuda")
        scales = torch.empty(sar.fp4_scale_bytes(*t.shape), dtype=torch.uint8, device="cuda")
        sar.fp4_quantize(t, codes, scales)
        q += [codes, scales]
    for v in (0, sar.SAR_FP4_GEMM_SPLIT | 7 << 8, sar.SAR_FP4_GEMM_PAIR):
        c = [torch.empty(70, 1000, device="cuda") for _ in range(2)]
        for y in c:
            sar.gemm_fp4(*q, y, epilogue=sar.SAR_EPI_F32, variant=v)
        assert torch.equal(*c)


def test_a_step_of_sampling_as_a_server_runs_it():
    """Admit, then decode rounds of control and pick with counted picks, a
    request leaving and another taking its slot: the table follows the oracle."""
    rng = np.random.default_rng(7)
    vocab, slots = 3000, 6
    table = torch.zeros(slots, vocab, dtype=torch.int16, device="cuda")
    want = np.zeros((slots, vocab), np.uint16)
    live = {0: 4, 1: 2, 2: 5}

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def admit(rows):
        nonlocal want
        lists = [rng.integers(0, vocab, 50).tolist() for _ in rows]
        off = i32([0] + np.cumsum([50] * len(rows)).tolist())
        sar.token_state_add(table, i32(rows), off, i32(sum(lists, [])), prompt_lens=i32([40] * len(rows)), reset=True)
        want = ol.state_add(want, rows, lists, [40] * len(rows), vocab, True)

    admit(list(live.values()))
    for step in range(6):
        if step == 3:
            live[1] = 2
            admit([2])  # the slot's next request
        rows = list(live.values())
        x = torch.from_numpy(rng.standard_normal((3, vocab)).astype(np.float32)).cuda()
        rep = torch.tensor([1.2, 1.0, 2.0], device="cuda")
        ctl = sar.LogitControls(state=table, slots=i32(rows), repetition=rep, frequency=torch.full((3,), 0.25, device="cuda"),
                                count_picks=True)
        picks = torch.empty(3, dtype=torch.int32, device="cuda")
        sar.logits_control(x, ctl, tokens_out=picks)
        for r in range(3):
            y = ol.changed(x[r].cpu().numpy(), want[rows[r]], rep[r].item(), None, 0.25, dtype=np.float32)
            assert picks[r].item() == ol.pick(y)
        want = ol.state_add(want, rows, [[t] for t in picks.tolist()], [0] * 3, vocab, False)
        assert np.array_equal(table.cpu().numpy().view(np.uint16), want)
