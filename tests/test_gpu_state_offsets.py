"""Rows of an appending call whose offsets are out of range or fall."""

import numpy as np
import pytest
import torch

import chunked_prefill_hybrid_sar_gb300 as sar
from chunked_prefill_hybrid_sar_gb300 import _lib
from oracle import logits as ol

pytestmark = pytest.mark.gpu

TOKENS = [4, 5, 6, 7, 4, 4, 9, 5]


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.fixture(autouse=True)
def no_device_flags():
    sar.op_sync_status()
    yield
    sar.op_sync_status()


def appended(offsets, prompt=None, reset=False):
    n = len(offsets) - 1
    start = np.arange(n * 32, dtype=np.uint16).reshape(n, 32) % 5
    table = torch.from_numpy(start.view(np.int16)).cuda()
    sar.token_state_add(table, i32(list(range(n))[::-1]), i32(offsets), i32(TOKENS),
                        prompt_lens=None if prompt is None else i32(prompt), reset=reset)
    lists = [TOKENS[b:e] if 0 <= b <= e <= len(TOKENS) else None for b, e in zip(offsets, offsets[1:])]
    good = [i for i in range(n) if lists[i] is not None]
    want = ol.state_add(start, [n - 1 - i for i in good], [lists[i] for i in good],
                        [0 if prompt is None else prompt[i] for i in good], 32, reset)
    return table.cpu().numpy().view(np.uint16), want, len(good) < n


# no two good rows of these share a token
BAD = [[-3, 2, 8], [-1, 0, 8], [0, 4, 9], [0, 8, 9], [2, 5, 2 ** 31 - 1], [0, 3, 3, 2], [0, 8, 0], [8, 0, 0], [0, 4, 4, 3, 3],
       [-5, -2, 3, 8], [-(2 ** 31), 3, 8], [9, 12, 15]]


@pytest.mark.parametrize("offsets", BAD)
@pytest.mark.parametrize("prompt", [False, True])
@pytest.mark.parametrize("reset", [False, True])
def test_bad_rows_are_passed_over_and_reported(offsets, prompt, reset):
    got, want, bad = appended(offsets, [1] * (len(offsets) - 1) if prompt else None, reset)
    assert bad
    with pytest.raises(sar.SarError) as e:
        sar.op_sync_status()
    assert e.value.code == _lib.SAR_ERR_BOUNDS
    assert np.array_equal(got, want)


@pytest.mark.parametrize("offsets", [[0, 8], [0, 0, 8, 8], [3, 3, 5], [0, 2, 4, 6, 8], [8, 8, 8], [0] + [1] * 700 + [8]])
@pytest.mark.parametrize("prompt", [False, True])
def test_good_rows_are_not_reported(offsets, prompt):
    got, want, bad = appended(offsets, [1] * (len(offsets) - 1) if prompt else None)
    assert not bad and np.array_equal(got, want)


def test_more_rows_than_tokens_with_a_bad_last_one():
    """The row's report comes from a thread behind the last token's."""
    n = 1000
    offsets = [0] * n + [9]
    table = torch.zeros(1, 32, dtype=torch.int16, device="cuda")
    sar.token_state_add(table, i32([0] * n), i32(offsets), i32(TOKENS))
    with pytest.raises(sar.SarError) as e:
        sar.op_sync_status()
    assert e.value.code == _lib.SAR_ERR_BOUNDS
    assert not table.any()


@pytest.mark.parametrize("offsets", [[0, 5, 3, 8], [5, 8, 0, 8], [0, 6, 4, 5, 8], [3, 1, 8, 2, 8]])
def test_falling_offsets_count_no_token_twice(offsets):
    """Rows that overlap after a fall: each token into one row at most, into none
    that is bad, and only tokens that the row holds."""
    n = len(offsets) - 1
    table = torch.zeros(n, 32, dtype=torch.int16, device="cuda")
    sar.token_state_add(table, i32(list(range(n))), i32(offsets), i32(list(range(8))))
    with pytest.raises(sar.SarError) as e:
        sar.op_sync_status()
    assert e.value.code == _lib.SAR_ERR_BOUNDS
    assert int(table.sum(0).max()) <= 1
    for r in range(n):
        assert {int(t) for t in table[r].nonzero()} <= set(range(offsets[r], offsets[r + 1]))
