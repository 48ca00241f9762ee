"""Oracle of the logits controls and of the token state, row by row.

``changed`` works in the given NumPy float type: float64 for the definition,
float32 (every operation rounded, as the library's entry states) for equality.
"""

from __future__ import annotations

import numpy as np

PROMPT, MOST = 0x8000, 0x7FFF


def state_add(table, slots, lists, prompt_lens, vocab, reset):
    """The uint16 table after one call; ``lists``: one token list per row."""
    table = table.copy()
    done = set()
    for slot, toks, k in zip(slots, lists, prompt_lens):
        if not 0 <= slot < table.shape[0] or (reset and slot in done):
            continue
        done.add(slot)
        row = table[slot]
        if reset:
            row[:vocab] = 0
        for i, t in enumerate(toks):
            if not 0 <= t < vocab:
                continue
            if i < k:
                row[t] |= PROMPT
            elif (row[t] & MOST) < MOST:
                row[t] += 1
    return table


def changed(x, state=None, repetition=None, presence=None, frequency=None, biases=(), mask=None, dtype=np.float64):
    """One row of logits under its controls.  state: the row's uint16 entries;
    biases: (token, value) pairs; mask: uint32 words."""
    with np.errstate(all="ignore"):
        x = x.astype(dtype)
        if state is not None:
            made = (state & MOST).astype(dtype)
            seen = state != 0
            if repetition is not None:
                r = dtype(np.float32(repetition))
                x = np.where(seen, np.where(x > 0, x / r, x * r), x).astype(dtype)
            if frequency is not None:
                x = np.where(seen, x - (dtype(np.float32(frequency)) * made).astype(dtype), x).astype(dtype)
            if presence is not None:
                x = np.where(made > 0, x - dtype(np.float32(presence)), x).astype(dtype)
        total = {}
        for t, v in biases:
            if 0 <= t < x.size:
                total[t] = dtype(total[t] + dtype(v)) if t in total else dtype(v)
        for t, v in total.items():
            x[t] = dtype(x[t] + v)
        if mask is not None:
            t = np.arange(x.size)
            x = np.where(mask[t // 32] >> (t % 32).astype(np.uint32) & 1, x, -np.inf).astype(dtype)
    return x


def pick(x) -> int:
    """The lowest index of the largest value above -inf; -1 without one."""
    x = np.where(np.isnan(x), -np.inf, x)
    return int(x.argmax()) if x.size and x.max() > -np.inf else -1
