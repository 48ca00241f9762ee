"""Steps of a serving loop over the 8-bit cache: page map, head rows with the append,
attention, one behind the other on the device, against the float64 oracle.

The page map is exact.  Head rows and codes: as in the rows' own test (within 2^-19
of the head's largest before their rounding).  Attention reads what the device wrote,
with the tolerance of attention's own test.
"""

import numpy as np
import pytest
import torch

import chunked_prefill_hybrid_sar_gb300 as sar
from chunked_prefill_hybrid_sar_gb300 import _lib
from oracle import kv8

pytestmark = pytest.mark.gpu

HEADS, KV_HEADS, D, PAGE, EPS, BASE = 6, 2, 64, 16, 1e-5, 10000.0


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Loop:
    """n requests over a pool of pages, and buffers of max_rows rows."""

    def __init__(self, n, pages, max_rows, columns=20, seed=0):
        self.g = torch.Generator().manual_seed(seed)
        self.n, self.pages, self.max_rows = n, pages, max_rows
        self.cache = sar.KV8Cache.empty(pages, KV_HEADS, PAGE, D)
        self.lens, self.new, self.tables = ints([0] * n), ints([0] * n), ints([[-1] * columns] * n)
        self.free, self.count = ints(torch.randperm(pages, generator=self.g).tolist()), ints([pages])
        self.off, self.pos, self.slots = ints([0] * (n + 1)), ints([0] * max_rows), ints([0] * max_rows)
        self.gains = [torch.rand(D, generator=self.g).cuda() + 0.5 for _ in range(2)]
        self.qkv = torch.zeros(max_rows, (HEADS + 2 * KV_HEADS) * D, dtype=torch.bfloat16, device="cuda")
        self.q = torch.zeros(max_rows, HEADS * D, dtype=torch.bfloat16, device="cuda")
        self.out = torch.zeros_like(self.q)
        self.workspace = torch.empty(sar.kv8_attention_workspace(self.cache, self.q, n), dtype=torch.uint8, device="cuda")

    def state(self):
        return [t for t in (self.lens, self.tables, self.free, self.count, self.cache.k_codes, self.cache.v_codes,
                            self.cache.k_scales, self.cache.v_scales)]

    def fill(self):
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=self.g).bfloat16())
        self.out.fill_(77)

    def step(self, max_rows=None):
        q, k, v = self.qkv.split([HEADS * D, KV_HEADS * D, KV_HEADS * D], 1)
        sar.page_map(self.lens, self.new, self.tables, self.free, self.count, self.off, self.pos, self.slots, PAGE)
        sar.qk_norm_rope(q, k, self.q, D, positions=self.pos, v=v, cache=self.cache, slots=self.slots, q_gain=self.gains[0],
                         k_gain=self.gains[1], eps=EPS, rope_base=BASE)
        sar.kv8_attention(self.q, self.cache, self.off, self.lens, self.tables, self.out, max_rows=max_rows,
                          workspace=self.workspace)


def turned(x, gain, pos):
    return np.stack([np.stack([kv8.turned(h, gain, EPS, int(p), BASE) for h in row]) for row, p in zip(x, pos)])


def check_step(loop, new, refused=()):
    """One step from the loop's present state, every part of it against the oracle's."""
    lens, tables, free, count = (t.cpu().numpy() for t in (loop.lens, loop.tables, loop.free, loop.count))
    old = {name: (getattr(loop.cache, f"{name}_codes").cpu().numpy(), getattr(loop.cache, f"{name}_scales").cpu().numpy())
           for name in "kv"}
    loop.new.copy_(torch.tensor(new, dtype=torch.int32))
    loop.fill()
    loop.step()
    lens, tables, free, count, off, pos, slots, bad = kv8.page_map(lens, new, tables, list(free), int(count[0]), PAGE, loop.max_rows)
    assert tuple(bad) == tuple(refused)
    for got, want in ((loop.lens, lens), (loop.off, off), (loop.pos, pos), (loop.slots, slots), (loop.count, [count])):
        assert got.tolist() == list(want)
    assert np.array_equal(loop.tables.cpu().numpy(), tables) and loop.free.tolist()[:count] == list(free[:count])

    x = loop.qkv.double().cpu().numpy().reshape(loop.max_rows, -1, D)
    q = turned(x[:, :HEADS], loop.gains[0].double().cpu().numpy(), pos)
    k = turned(x[:, HEADS:HEADS + KV_HEADS], loop.gains[1].double().cpu().numpy(), pos)
    got_q = loop.q.double().cpu().numpy().reshape(q.shape)
    assert (np.abs(got_q - q) <= 2.0 ** -8 * np.abs(q) + 2.0 ** -18 * np.abs(q).max(-1, keepdims=True)).all()
    v_codes, v_scales = kv8.write(*old["v"], x[:, HEADS + KV_HEADS:], slots)
    codes, scales = ({name: getattr(loop.cache, f"{name}_{what}").cpu().numpy() for name in "kv"} for what in ("codes", "scales"))
    assert np.array_equal(scales["v"], v_scales) and np.array_equal(kv8.E4M3[codes["v"]], kv8.E4M3[v_codes])
    assert np.array_equal(scales["k"], kv8.write(*old["k"], k, slots)[1])
    for r in np.flatnonzero(slots >= 0):
        p, o = divmod(int(slots[r]), PAGE)
        sc = scales["k"][p][:, None]
        off_by = np.abs(kv8.E4M3[codes["k"][p, :, o]] * sc - k[r])
        assert (off_by <= np.maximum(np.abs(k[r]) * 2.0 ** -4, sc * 2.0 ** -10) + 2.0 ** -18 * np.abs(k[r]).max()).all()

    out = loop.out.double().cpu().numpy().reshape(q.shape)
    assert (out[off[-1]:] == 77).all()  # rows behind the last request
    for i in range(loop.n):
        a, b, m = int(off[i]), int(off[i + 1]), int(lens[i])
        if a == b:
            continue
        p = tables[i, :-(-m // PAGE)]
        kk, vv = ((kv8.E4M3[codes[name][p]] * scales[name][p][:, :, None, None]).transpose(0, 2, 1, 3).reshape(-1, KV_HEADS, D)[:m]
                  for name in "kv")
        want, mean = (kv8.attention(got_q[a:b], kk, w, b - a) for w in (vv, np.abs(vv)))
        far = np.abs(vv).max(initial=0) * m * 2.0 ** -25
        assert (np.abs(out[a:b] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * mean + far).all()


def test_requests_come_go_and_wait():
    loop = Loop(5, 15, 70)
    check_step(loop, [37, 0, 5, 0, 0])           # two prompts
    check_step(loop, [1, 60, 1, 0, 1])           # one more beside decoding
    sar.op_sync_status()
    check_step(loop, [12, 1, 9, 47, 1])          # chunks deep into prompts
    sar.op_sync_status()
    check_step(loop, [1, 20, 1, 30, 1], refused=(3,))  # the pool runs dry: rows without slots
    with pytest.raises(sar.SarError) as e:
        sar.op_sync_status()
    assert e.value.code == _lib.SAR_ERR_NO_PAGES
    check_step(loop, [-1, 20, 1, 30, 1])         # pages given back are enough
    check_step(loop, [25, 1, -1, 1, -1])         # the first place, with a new request
    check_step(loop, [1, 1, 0, 1, 0])
    check_step(loop, [-1, -1, 0, -1, 0])
    assert loop.count.tolist() == [15] and sorted(loop.free.tolist()) == list(range(15))
    sar.op_sync_status()


def test_captured_steps_are_the_eager_ones():
    """A decode step captured once and replayed, through page borders, beside the same steps launched."""
    loops = [Loop(4, 40, 90, seed=3) for _ in range(2)]
    for loop in loops:
        loop.new.copy_(ints([33, 15, 7, 31]))
        loop.fill()
        loop.step()
        loop.new.fill_(1)
    loop = loops[0]
    graph = torch.cuda.CUDAGraph()
    before = [t.clone() for t in loop.state()]
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        loop.step(max_rows=1)
    for t, was in zip(loop.state(), before):
        assert torch.equal(t, was)  # a capture runs nothing
    for _ in range(20):
        for x in loops:
            x.fill()
        graph.replay()
        loops[1].step(max_rows=1)
        for a, b in zip(loops[0].state() + [loops[0].q, loops[0].out], loops[1].state() + [loops[1].q, loops[1].out]):
            assert torch.equal(a, b)
    sar.op_sync_status()


def test_two_captured_loops_at_once():
    """Two loops' captured steps, each with its own workspace, replayed side by side on two streams."""
    loops = [Loop(6, 80, 200, seed=s) for s in (5, 5, 6, 6)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs = []
    for loop in loops:
        loop.new.copy_(ints([100, 1, 40, 3, 17, 30]))
        loop.fill()
        loop.step()
        loop.new.copy_(ints([1, 2, 1, 5, 0, 1]))
        loop.fill()
    torch.cuda.synchronize()
    for loop in (loops[0], loops[2]):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            loop.step()
        graphs.append(g)
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for loop in (loops[1], loops[3]):
        for _ in range(10):
            loop.step()
    for a, b in ((0, 1), (2, 3)):
        for x, y in zip(loops[a].state() + [loops[a].out], loops[b].state() + [loops[b].out]):
            assert torch.equal(x, y)
    sar.op_sync_status()


def test_a_wrong_guess_of_the_longest_changes_little():
    """max_len only shares out work: results agree whatever it says."""
    loop = Loop(3, 60, 700, columns=60)
    check_step(loop, [600, 33, 1])
    loop.new.copy_(ints([1, 1, 1]))
    loop.step()
    for max_len in (1, 64, 600, 10 ** 6):
        out = torch.full_like(loop.out, 77)
        sar.kv8_attention(loop.q, loop.cache, loop.off, loop.lens, loop.tables, out, max_len=max_len)
        assert torch.equal(out[3:], torch.full_like(out[3:], 77))
        # (equal up to the order of sums: twice the output's half step, 2^-8, and twice 2^-10 of the mean)
        assert (out[:3].double() - loop.out[:3].double()).abs().max() <= 2.0 ** -6 * loop.out[:3].double().abs().max()
    sar.op_sync_status()
