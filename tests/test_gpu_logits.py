"""Token state and logits controls against the oracle: whole numbers and picks
equal, fp32 logits equal to the float32 oracle (the entry states each rounding)
and within their roundings of the float64 one, 16-bit logits equal to the
float32 ones rounded once."""

import dataclasses

import numpy as np
import pytest
import torch

import chunked_prefill_hybrid_sar_gb300 as sar
import synth
from chunked_prefill_hybrid_sar_gb300 import _lib, harness
from oracle import logits as ol

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def no_device_flags():
    sar.op_sync_status()
    yield
    sar.op_sync_status()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def csr(lists):
    return (i32([0] + np.cumsum([len(x) for x in lists]).tolist()),
            i32([t for x in lists for t in x]) if any(lists) else torch.empty(0, dtype=torch.int32, device="cuda"))


def as_u16(t):
    return t.cpu().numpy().view(np.uint16)


def table_of(a):
    return torch.from_numpy(a.view(np.int16)).cuda()


# ---- token state -----------------------------------------------------------------


@pytest.mark.parametrize("vocab,ld,offset", [(1, 1, 0), (37, 40, 0), (1000, 1000, 0), (8192, 8192, 0), (8193, 8200, 0),
                                             (20011, 20011, 0), (8200, 8208, 1)])
@pytest.mark.parametrize("reset", [False, True])
@pytest.mark.parametrize("prompts", [False, True])
def test_state_add(vocab, ld, offset, reset, prompts):
    rng = np.random.default_rng(vocab + ld)
    n_slots, n = 7, 5
    start = rng.integers(0, 65536, (n_slots, ld)).astype(np.uint16)
    start[:, ::3] = 0
    start[:, 1::7] = ol.MOST - 1  # about to stop counting
    buf = torch.zeros(offset + n_slots * ld, dtype=torch.int16, device="cuda")
    table = buf[offset:].view(n_slots, ld)
    table.copy_(table_of(start))
    slots = rng.permutation(n_slots)[:n].tolist()
    lists = [rng.integers(0, vocab, k).tolist() for k in (0, 1, 700, 3, 5000)]
    lists[2] += [vocab - 1] * 5
    k = [min(len(x), 3) + (i == 3) * 100 for i, x in enumerate(lists)]  # row 3: more than its list
    off, tok = csr(lists)
    sar.token_state_add(table, i32(slots), off, tok, vocab=vocab, prompt_lens=i32(k) if prompts else None, reset=reset)
    want = ol.state_add(start, slots, lists, k if prompts else [0] * n, vocab, reset)
    assert np.array_equal(as_u16(table), want)


def test_state_counts_stop_at_their_limit():
    table = torch.zeros(2, 16, dtype=torch.int16, device="cuda")
    off, tok = csr([[3] * 40000 + [4], [5]])
    for reset in (True, False):
        sar.token_state_add(table, i32([1, 0]), off, tok, reset=reset)
        t = as_u16(table)
        assert t[1, 3] == ol.MOST and t[1, 4] == (1 if reset else 2) and t[0, 5] == t[1, 4]


def test_state_two_rows_of_one_slot():
    table = torch.zeros(3, 64, dtype=torch.int16, device="cuda")
    lists = [[7] * 300 + [1], [7] * 200, [2]]
    off, tok = csr(lists)
    sar.token_state_add(table, i32([1, 1, 2]), off, tok)
    assert np.array_equal(as_u16(table), ol.state_add(np.zeros((3, 64), np.uint16), [1, 1, 2], lists, [0] * 3, 64, False))
    sar.op_sync_status()
    # a resetting call takes the first and says so
    sar.token_state_add(table, i32([1, 1, 2]), off, tok, reset=True)
    assert np.array_equal(as_u16(table), ol.state_add(np.zeros((3, 64), np.uint16), [1, 1, 2], lists, [0] * 3, 64, True))
    with pytest.raises(sar.SarError) as e:
        sar.op_sync_status()
    assert e.value.code == _lib.SAR_ERR_BOUNDS


@pytest.mark.parametrize("reset", [False, True])
@pytest.mark.parametrize("bad", ["slot", "slot<0", "token", "token<0", "offset"])
def test_state_out_of_range_is_passed_over_and_reported(reset, bad):
    table = torch.zeros(3, 32, dtype=torch.int16, device="cuda")
    slots, lists = [1, 2], [[4, 5], [6, 7]]
    if bad.startswith("slot"):
        slots[0] = -1 if "<" in bad else 3
    if bad.startswith("token"):
        lists[0][1] = -3 if "<" in bad else 32
    off, tok = csr(lists)
    if bad == "offset":
        if not reset:
            pytest.skip("an appending call looks its rows up by token")
        off[2] = 9
    want = ol.state_add(np.zeros((3, 32), np.uint16), slots, lists if bad != "offset" else [lists[0], []], [0, 0], 32, reset)
    sar.token_state_add(table, i32(slots), off, tok, reset=reset)
    with pytest.raises(sar.SarError) as e:
        sar.op_sync_status()
    assert e.value.code == _lib.SAR_ERR_BOUNDS
    assert np.array_equal(as_u16(table), want)


# ---- controls ----------------------------------------------------------------------


class Case:
    def __init__(self, rows, vocab, kind, seed=0, state_ld=None, penal=True, biases=7, masks=4, ties=True):
        rng = np.random.default_rng(seed + rows * 31 + vocab)
        self.rows, self.vocab, self.kind = rows, vocab, kind
        x = torch.from_numpy(rng.standard_normal((rows, vocab)).astype(np.float32) * 3)
        if ties:  # few values: every maximum has company
            x = (x * 2).round() / 2
        x[rng.random((rows, vocab)) < 0.03] = float("-inf")
        x[rng.random((rows, vocab)) < 0.01] = float("nan")
        if vocab > 40:
            x[0, 17] = float("inf")
        self.x = x.to(TYPES[kind])
        ld = state_ld or -(-vocab // 8) * 8
        n_slots = rows + 2
        t = rng.integers(0, 4, (n_slots, ld)).astype(np.uint16) | (rng.random((n_slots, ld)) < 0.1).astype(np.uint16) << 15
        t[rng.random((n_slots, ld)) < 0.7] = 0
        t[:, :1] = 0xFFFF
        self.table = t
        self.slots = rng.permutation(n_slots)[:rows].astype(np.int64)
        if rows > 2:
            self.slots[1] = -1
        self.rep, self.pres, self.freq = (rng.uniform(0.5, 1.8, rows).astype(np.float32), rng.uniform(-1, 1, rows).astype(np.float32),
                                          rng.uniform(-0.3, 1, rows).astype(np.float32)) if penal else (None,) * 3
        self.lists = [[] for _ in range(rows)]
        if biases:
            self.lists = [[(int(t), float(v)) for t, v in zip(rng.integers(0, vocab, k), rng.standard_normal(k).astype(np.float32) * 4)]
                          for k in rng.integers(0, biases + 1, rows)]
            self.lists[-1] += self.lists[-1][:3] + [(vocab - 1, 0.1), (vocab - 1, 0.2), (vocab - 1, -0.3)]  # listed again
        self.mask = self.mask_rows = None
        if masks:
            words = -(-vocab // 32) + 1
            share = np.array([0.9, 0.5, 0.02, 0.0])[np.arange(masks) % 4]
            on = rng.random((masks, words * 32)) < share[:, None]
            self.mask = np.packbits(on.reshape(masks, words, 32), axis=-1, bitorder="little").view("<u4").reshape(masks, words)
            self.mask_rows = rng.integers(-1, masks, rows)
            self.mask_rows[-1] = min(3, masks - 1)

    def controls(self, count=False, state=None):
        f = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
        kw = {}
        if self.rep is not None or count:
            self.dev_state = table_of(self.table) if state is None else state
            kw.update(state=self.dev_state, slots=i32(self.slots.tolist()), repetition=f(self.rep), presence=f(self.pres),
                      frequency=f(self.freq), count_picks=count)
        if any(self.lists):
            off, tok = csr([[t for t, _ in x] for x in self.lists])
            kw.update(bias_offsets=off, bias_tokens=tok,
                      bias_values=torch.tensor([v for x in self.lists for _, v in x], device="cuda"))
        if self.mask is not None:
            kw.update(mask=f(self.mask.view(np.int32)), mask_rows=i32(self.mask_rows.tolist()))
        return sar.LogitControls(**kw)

    def want(self, dtype):
        out = []
        for r in range(self.rows):
            s = None
            if self.rep is not None and self.slots[r] >= 0:
                s = self.table[self.slots[r], :self.vocab]
            p = (self.rep[r], self.pres[r], self.freq[r]) if s is not None else (None,) * 3
            m = self.mask[self.mask_rows[r]] if self.mask is not None and self.mask_rows[r] >= 0 else None
            out.append(ol.changed(self.x[r].float().numpy(), s, *p, self.lists[r], m, dtype))
        return np.stack(out)

    def check(self, y, picks):
        w32 = self.want(np.float32)
        if picks is not None:
            assert picks.cpu().tolist() == [ol.pick(r) for r in w32]
        if y is None:
            return
        want = torch.from_numpy(w32).to(TYPES[self.kind])
        assert torch.equal(torch.isnan(y.cpu()), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(y.cpu(), 3e4, 6e4, -6e4), torch.nan_to_num(want, 3e4, 6e4, -6e4))
        w64 = self.want(np.float64)
        fine = np.isfinite(w64)
        if self.kind == "f32" and fine.any():
            # six roundings of numbers no larger than the largest operand
            big = np.abs(w64[fine]) + 2 * np.abs(np.nan_to_num(self.x.numpy(), posinf=0, neginf=0))[fine] + 32
            assert (np.abs(y.cpu().numpy()[fine] - w64[fine]) <= 6 * 2.0 ** -24 * big).all()


SHAPES = [(1, 1), (1, 33), (3, 96), (2, 4096), (5, 4097), (1, 32000), (7, 1111), (65, 2000), (2, 33000), (160, 4104), (1, 131072)]


@pytest.mark.parametrize("rows,vocab", SHAPES)
@pytest.mark.parametrize("kind", list(TYPES))
def test_everything_at_once(rows, vocab, kind):
    c = Case(rows, vocab, kind, biases=60)
    x = c.x.cuda()
    y, picks = torch.full_like(x, 9.0), torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    sar.logits_control(x, c.controls(), out=y, tokens_out=picks)
    c.check(y, picks)
    only = torch.full_like(picks, -7)
    sar.logits_control(x, c.controls(), tokens_out=only)
    assert torch.equal(only, picks) and torch.equal(torch.nan_to_num(x.cpu()), torch.nan_to_num(c.x))
    sar.logits_control(x, c.controls(), out=x)  # in place, without a pick
    c.check(x, None)


@pytest.mark.parametrize("part", ["none", "penalties", "biases", "masks"])
@pytest.mark.parametrize("rows,vocab", [(3, 5000), (1, 70001)])
def test_each_alone(part, rows, vocab):
    c = Case(rows, vocab, "f32", penal=part == "penalties", biases=300 if part == "biases" else 0, masks=4 if part == "masks" else 0)
    x = c.x.cuda()
    y, picks = torch.empty_like(x), torch.empty(rows, dtype=torch.int32, device="cuda")
    sar.logits_control(x, c.controls(), out=y, tokens_out=picks)
    c.check(y, picks)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("offset,extra,state_ld", [(0, 8, 5008), (1, 0, 5000), (0, 3, 5000), (3, 5, 5003), (8, 8, 5001)])
def test_strides_and_alignment(kind, offset, extra, state_ld):
    rows, vocab = 4, 5000
    c = Case(rows, vocab, kind, state_ld=state_ld)
    ld = vocab + extra
    buf = torch.zeros(offset + rows * ld, dtype=TYPES[kind], device="cuda")
    x = buf[offset:].as_strided((rows, vocab), (ld, 1))
    x.copy_(c.x)
    out = torch.full((offset + rows * ld,), 5.0, dtype=TYPES[kind], device="cuda")
    y = out[offset:].as_strided((rows, vocab), (ld, 1))
    picks = torch.empty(rows, dtype=torch.int32, device="cuda")
    sar.logits_control(x, c.controls(), out=y, tokens_out=picks)
    c.check(y.contiguous(), picks)
    rest = torch.ones(out.numel(), dtype=torch.bool)
    rest[offset:].as_strided((rows, vocab), (ld, 1)).fill_(False)
    assert (out.cpu()[rest] == 5.0).all()


@pytest.mark.parametrize("rows,vocab", [(1, 40000), (9, 3000)])
def test_picks_are_counted(rows, vocab):
    c = Case(rows, vocab, "f32", masks=4)
    ctl = c.controls(count=True)
    picks = torch.empty(rows, dtype=torch.int32, device="cuda")
    table = c.table.copy()
    for _ in range(3):  # a decode loop over the same logits: penalties grow
        sar.logits_control(c.x.cuda(), ctl, tokens_out=picks)
        c.check(None, picks)
        lists = [[] if t < 0 else [t] for t in picks.cpu().tolist()]
        c.table = table = ol.state_add(table, c.slots.tolist(), lists, [0] * rows, vocab, False)
        assert np.array_equal(as_u16(c.dev_state), table)


def test_a_mask_that_leaves_nothing():
    x = torch.randn(3, 9000, device="cuda")
    mask = torch.zeros(3, 282, dtype=torch.int32, device="cuda")
    mask[1, 281] = 1 << 7  # token 8999
    mask[2, 0] = -(1 << 31)  # token 31
    picks = torch.empty(3, dtype=torch.int32, device="cuda")
    y = torch.empty_like(x)
    state = torch.zeros(3, 9000, dtype=torch.int16, device="cuda")
    sar.logits_control(x, sar.LogitControls(mask=mask, state=state, slots=i32([0, 1, 2]), count_picks=True), out=y, tokens_out=picks)
    assert picks.cpu().tolist() == [-1, 8999, 31]
    assert torch.isneginf(y[0]).all() and torch.isfinite(y).sum() == 2
    assert state.sum() == 2 and state[1, 8999] == 1 and state[2, 31] == 1


@pytest.mark.parametrize("bad", ["slot", "mask", "offset", "bias"])
def test_out_of_range_is_passed_over_and_reported(bad):
    c = Case(4, 600, "f32")
    ctl = c.controls()
    keep = dict(zip(("state", "slots", "rep", "pres", "freq", "off", "tok", "val", "mask", "rows"), ctl._keep))
    if bad == "slot":
        keep["slots"][2] = 99
        c.slots[2] = -1
    elif bad == "mask":
        keep["rows"][2] = 99
        c.mask_rows[2] = -1
    elif bad == "offset":
        keep["off"][4] = 9999
        c.lists[3] = []
    else:
        at = int(keep["off"][3])
        keep["tok"][at] = 600
        c.lists[3] = c.lists[3][1:]
    x = c.x.cuda()
    y, picks = torch.empty_like(x), torch.empty(4, dtype=torch.int32, device="cuda")
    sar.logits_control(x, ctl, out=y, tokens_out=picks)
    with pytest.raises(sar.SarError) as e:
        sar.op_sync_status()
    assert e.value.code == _lib.SAR_ERR_BOUNDS
    c.check(y, picks)


def test_python_refusals():
    x = torch.zeros(2, 64, device="cuda")
    p = torch.empty(2, dtype=torch.int32, device="cuda")
    ok = sar.LogitControls()
    sar.logits_control(x, ok, tokens_out=p)
    assert p.tolist() == [0, 0]
    state = torch.zeros(2, 64, dtype=torch.int16, device="cuda")
    for kw in (dict(out=x.half()), dict(out=x[:1]), dict(tokens_out=p.long()), dict(tokens_out=p[:1]), dict(tokens_out=p.cpu())):
        with pytest.raises(ValueError):
            sar.logits_control(x, ok, **kw)
    for kw in (dict(slots=p[:1], state=state), dict(state=state[:, :32], slots=p), dict(mask=p.view(2, 1))):
        with pytest.raises(ValueError):
            sar.logits_control(x, sar.LogitControls(**kw), tokens_out=p)
    for kw in (dict(state=state.int()), dict(state=state, slots=p.long()), dict(bias_offsets=p), dict(mask=p),
               dict(repetition=p), dict(state=state.cpu())):
        with pytest.raises(ValueError):
            sar.LogitControls(**kw)
    with pytest.raises(sar.SarError):
        sar.logits_control(x, sar.LogitControls(repetition=torch.ones(2, device="cuda")), tokens_out=p)
    for a in ((state.int(), p, i32([0, 0, 0]), p), (state, p.long(), i32([0, 0, 0]), p), (state, p, p, p),
              (state, p, i32([0, 0, 0]), p.cpu())):
        with pytest.raises(ValueError):
            sar.token_state_add(*a)


def test_captured_and_on_another_stream():
    c = Case(6, 9001, "f32")
    ctl = c.controls()
    x = c.x.cuda()
    y, picks = torch.empty_like(x), torch.empty(6, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sar.logits_control(x, ctl, out=y, tokens_out=picks)
    torch.cuda.synchronize()
    c.check(y, picks)
    off, tok = csr([[5, 5], [9000]])
    slots = i32([0, 3])
    table = torch.zeros(8, 9001, dtype=torch.int16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sar.token_state_add(table, slots, off, tok)
        sar.logits_control(x, ctl, out=y, tokens_out=picks)
    c.x = torch.flip(c.x, [0])
    x.copy_(c.x)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    c.check(y, picks)
    assert table[0, 5] == 4 and table[3, 9000] == 2 and table.sum() == 6


# ---- the step's own path -----------------------------------------------------------


def test_graph_picks_under_controls():
    """A captured decode step whose token launches pick under controls: each
    step's picks equal the oracle's on that step's logits."""
    case = synth.tiny_case(0, dtype=torch.bfloat16)
    dims = dataclasses.replace(case["dims"], vocab=1024)
    _, head, gen = synth.model_weights(0, dims, torch.bfloat16)
    m = harness.load_model(dims, case["layers"], head, max_tokens=64, max_decodes=8)
    kv = sar.KVCache(m, 16, 32)
    n = 3
    tables = [list(range(4 * i, 4 * i + 4)) for i in range(n)]
    logits = torch.empty(n, dims.vocab, device="cuda")
    inp = torch.zeros(n, dtype=torch.int32, device="cuda")

    def batch(step):
        return sar.Batch(None, [(i, step, tables[i]) for i in range(n)], in_kind=sar.SAR_IN_TOKENS)

    g = sar.StepGraph(m, kv, batch(0), inp, logits_out=logits)
    state = torch.zeros(4, dims.vocab, dtype=torch.int16, device="cuda")
    off, tok = csr([[1, 2, 3]])
    sar.token_state_add(state, i32([2]), off, tok, prompt_lens=i32([3]), reset=True)
    words = -(-dims.vocab // 32)
    mask = torch.full((1, words), -1, dtype=torch.int32, device="cuda")
    mask[0, :20] = 0
    rep, pres = np.float32([1.3, 1.0, 1.7]), np.float32([0.5, 4.0, 0.0])
    slots, mask_rows = [0, 3, 2], [-1, -1, 0]
    boff, btok = csr([[], [7, 9], []])
    ctl = sar.LogitControls(state=state, slots=i32(slots), repetition=torch.from_numpy(rep).cuda(),
                            presence=torch.from_numpy(pres).cuda(), bias_offsets=boff, bias_tokens=btok,
                            bias_values=torch.tensor([50.0, -3.0], device="cuda"), mask=mask, mask_rows=i32(mask_rows),
                            count_picks=True)
    g.set_controls(ctl)
    host_in = torch.tensor([5, 6, 7], dtype=torch.int32).pin_memory()
    out = torch.empty(n, dtype=torch.int32).pin_memory()
    want_state = as_u16(state).copy()
    for step in range(5):
        g.update(batch(step))
        if step % 2:
            g.enqueue_host_tokens(host_in, out)
            g.wait()
        else:
            g.launch_host_tokens(host_in, out)
        raw = logits.cpu().numpy()
        picks = []
        for r in range(n):
            biases = [(7, 50.0), (9, -3.0)] if r == 1 else []
            mk = mask[0].cpu().numpy().view(np.uint32) if mask_rows[r] >= 0 else None
            picks.append(ol.pick(ol.changed(raw[r], want_state[slots[r]], rep[r], pres[r], None, biases, mk, np.float32)))
        assert out.tolist() == picks
        want_state = ol.state_add(want_state, slots, [[t] for t in picks], [0] * n, dims.vocab, False)
        assert np.array_equal(as_u16(state), want_state)
        host_in.copy_(out)
    assert out[1] != 7 or want_state[3, 7] == 5
    g.set_controls(None)
    g.update(batch(5))
    g.launch_host_tokens(host_in, out)
    assert out.tolist() == logits.argmax(1).tolist()
    g.close()
    m.close()


def test_head_in_four_bits_to_the_pick():
    """Hidden rows -> 4-bit rows -> 4-bit head -> controls -> pick, as one run,
    against the same run in float64."""
    from oracle import fp4

    rng = np.random.default_rng(3)
    n, hidden, vocab = 5, 512, 2000
    h = rng.standard_normal((n, hidden)).astype(np.float32)
    w = (rng.standard_normal((vocab, hidden)) * 0.05).astype(np.float32)
    scale = 2.0 ** -11
    dev = {}
    for name, a, g in (("h", h, 1.0), ("w", w, scale)):
        codes = torch.empty(a.shape[0], hidden // 2, dtype=torch.uint8, device="cuda")
        scales = torch.empty(sar.fp4_scale_bytes(a.shape[0], hidden), dtype=torch.uint8, device="cuda")
        sar.fp4_quantize(torch.from_numpy(a).cuda(), codes, scales, tensor_scale=g)
        dev[name] = (codes, scales)
    logits = torch.empty(n, vocab, device="cuda")
    sar.gemm_fp4(*dev["h"], *dev["w"], logits, alpha=scale, epilogue=sar.SAR_EPI_F32)
    c = Case(n, vocab, "f32", ties=False)
    picks = torch.empty(n, dtype=torch.int32, device="cuda")
    c.x = logits.cpu()
    sar.logits_control(logits, c.controls(), out=logits, tokens_out=picks)
    c.check(logits, picks)
    hq, wq = (fp4.values(*fp4.quantise(a, "nv", 1 / g), "nv", g) for a, g in ((h, 1.0), (w, scale)))
    exact = hq @ wq.T
    bound = (hidden / 64 + 10) * 2.0 ** -23 * (np.abs(hq) @ np.abs(wq).T)
    assert (np.abs(c.x.numpy() - exact) <= bound).all()


@pytest.mark.parametrize("vocab", [50, 9000, 70000])
def test_long_bias_lists_with_repeats(vocab):
    """Lists beyond what one look at them holds (512), most tokens more than once."""
    c = Case(2, vocab, "f32", biases=0)
    rng = np.random.default_rng(vocab)
    few = rng.integers(0, vocab, 400)
    c.lists = [[(int(few[i]), float(v)) for i, v in zip(rng.integers(0, 400, 1300), rng.standard_normal(1300).astype(np.float32))],
               [(int(t), float(np.float32(0.1))) for t in np.repeat(few[:40], 13)]]
    x = c.x.cuda()
    y, picks = torch.empty_like(x), torch.empty(2, dtype=torch.int32, device="cuda")
    sar.logits_control(x, c.controls(), out=y, tokens_out=picks)
    c.check(y, picks)
