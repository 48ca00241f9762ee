"""Bias lists of every length: the search of a short list, the slices of a long
one, and the longest that a row may have."""

import numpy as np
import pytest
import torch

import chunked_prefill_hybrid_sar_gb300 as sar
from chunked_prefill_hybrid_sar_gb300 import _lib
from oracle import logits as ol
from test_gpu_logits import Case, TYPES, i32

pytestmark = pytest.mark.gpu

MOST = 1 << 21  # biases of a row


@pytest.fixture(autouse=True)
def no_device_flags():
    sar.op_sync_status()
    yield
    torch.cuda.empty_cache()
    sar.op_sync_status()


def listed(rng, n, vocab, distinct):
    """n biases over `distinct` tokens, neighbours and both ends of the vocabulary among them."""
    some = rng.integers(0, vocab, distinct)
    some[:3] = [0, vocab - 1, vocab // 2]
    some[3:40] = np.minimum(vocab // 2 + np.arange(min(37, max(0, distinct - 3))), vocab - 1)
    t = some[rng.integers(0, distinct, n)]
    return [(int(a), float(b)) for a, b in zip(t, rng.standard_normal(n).astype(np.float32))]


def check(c, y, picks):
    """Equal to the float32 oracle; and to the float64 one within six roundings of
    numbers no larger than the largest operand, plus a rounding for each of a
    token's k biases: a partial sum in list order is at most the biases'
    magnitudes' sum times (1 + 2^-24)^k, below 1.01 for k < 2^17."""
    w32, w64 = c.want(np.float32), c.want(np.float64)
    if picks is not None:
        assert picks.tolist() == [ol.pick(r) for r in w32]
    want = torch.from_numpy(w32).to(TYPES[c.kind])
    got = y.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    keep = ~torch.isnan(want)
    assert torch.equal(got[keep], want[keep])
    if c.kind != "f32":
        return
    k, size = np.zeros(w64.shape), np.zeros(w64.shape)
    for r, entries in enumerate(c.lists):
        if entries:
            tok = np.array([t for t, _ in entries])
            k[r] = np.bincount(tok, minlength=c.vocab)
            size[r] = np.bincount(tok, weights=[abs(v) for _, v in entries], minlength=c.vocab)
    fine = np.isfinite(w64)
    big = np.abs(w64) + 2 * np.abs(np.nan_to_num(c.x.numpy(), posinf=0, neginf=0)) + 32
    bound = 2.0 ** -24 * (6 * big + 1.01 * k * size)
    assert (np.abs(got.numpy()[fine] - w64[fine]) <= bound[fine]).all()


@pytest.mark.parametrize("n", [511, 512, 513, 640, 1300, 12000])
@pytest.mark.parametrize("rows,vocab,distinct", [(2, 50, 40), (3, 9001, 300), (2, 33000, 20000), (1, 131072, 700), (160, 4104, 1000)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_lists_with_repeats(n, rows, vocab, distinct, kind):
    rng = np.random.default_rng(n + vocab)
    c = Case(rows, vocab, kind, biases=5)
    c.lists[0] = listed(rng, n, vocab, distinct)
    c.lists[-1] = [(t, v) for t, v in c.lists[0][::-1]]
    x = c.x.cuda()
    y, picks = torch.full_like(x, 9.0), torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    sar.logits_control(x, c.controls(), out=y, tokens_out=picks)
    check(c, y, picks)
    only = torch.full_like(picks, -7)
    sar.logits_control(x, c.controls(), tokens_out=only)
    assert torch.equal(only, picks)
    sar.logits_control(x, c.controls(), out=x)  # in place
    check(c, x, None)


@pytest.mark.parametrize("n", [513, 3000])
def test_entries_out_of_range_in_a_long_list(n):
    rng = np.random.default_rng(n)
    c = Case(2, 5000, "f32", biases=0)
    c.lists = [listed(rng, n, 5000, 400), []]
    for at, t in ((0, -1), (7, 5000), (n - 1, 2 ** 31 - 1), (n // 2, -(2 ** 31)), (n // 3, -64)):
        c.lists[0][at] = (t, 3.0)
    x = c.x.cuda()
    y, picks = torch.empty_like(x), torch.empty(2, dtype=torch.int32, device="cuda")
    sar.logits_control(x, c.controls(), out=y, tokens_out=picks)
    with pytest.raises(sar.SarError) as e:
        sar.op_sync_status()
    assert e.value.code == _lib.SAR_ERR_BOUNDS
    c.lists[0] = [(t, v) for t, v in c.lists[0] if 0 <= t < 5000]
    check(c, y, picks)


@pytest.mark.parametrize("n,vocab", [(200_000, 40_000), (1 << 20, 1000), (MOST, 1), (MOST, 40_000), (MOST + 1, 40_000)])
def test_the_longest_lists(n, vocab):
    """Whole biases, so that their sums are exact in any order; the second row's list is short."""
    rng = np.random.default_rng(n)
    x = torch.from_numpy(rng.integers(-50, 50, (2, vocab)).astype(np.float32)).cuda()
    tok = rng.integers(0, vocab, n + 2).astype(np.int32)
    val = rng.integers(-3, 4, n + 2).astype(np.float32)
    val[n:] = 1000.0
    ctl = sar.LogitControls(bias_offsets=i32([0, n, n + 2]), bias_tokens=torch.from_numpy(tok).cuda(),
                            bias_values=torch.from_numpy(val).cuda())
    y, picks = torch.empty_like(x), torch.empty(2, dtype=torch.int32, device="cuda")
    sar.logits_control(x, ctl, out=y, tokens_out=picks)
    if n > MOST:  # passed over and reported
        with pytest.raises(sar.SarError) as e:
            sar.op_sync_status()
        assert e.value.code == _lib.SAR_ERR_BOUNDS
    want = x.cpu().numpy().astype(np.float64)
    for r, (b, e) in enumerate([(0, n if n <= MOST else 0), (n, n + 2)]):
        want[r] += np.bincount(tok[b:e], weights=val[b:e], minlength=vocab)
    assert np.array_equal(y.cpu().numpy(), want)
    assert picks.tolist() == want.argmax(1).tolist()
