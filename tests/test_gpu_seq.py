"""GPU tests of the sequence operators against the float64 oracle, with its bounds on fp32 arithmetic.

Sizes sit around the places where the kernels change what they do: a row group of 16, a piece of 64
rows, tiles of a few hundred rows, channel counts below, at and past a wave's, odd ones that force
element-wise access, one row, none.
"""
import numpy as np
import pytest
import torch

import implicit_gemm_conv_amd as igc
from implicit_gemm_conv_amd import sequence
from oracle import sequence as ref
from tests.seq_cases import DT, assert_within, f64, normal, scan_inputs, starts_of

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# dtype, B, T, C, starts, carried state
SHAPES = [
    ("bf16", 1, 1, 1, None, False), ("fp32", 2, 3, 5, "some", True), ("fp16", 3, 16, 64, None, True),
    ("bf16", 2, 17, 66, "some", True), ("fp32", 1, 64, 130, None, False), ("bf16", 2, 65, 128, "some", True),
    ("fp16", 1, 128, 256, None, True), ("fp32", 1, 129, 257, "some", False), ("bf16", 2, 300, 96, "some", True),
    ("fp32", 2, 500, 34, None, True), ("fp16", 1, 1000, 40, "some", True), ("bf16", 1, 1025, 24, None, True),
    ("bf16", 3, 33, 264, "all", True), ("fp32", 2, 31, 8, "first", True), ("fp16", 5, 48, 136, "some", False),
    ("bf16", 1, 15, 512, None, True), ("fp16", 2, 127, 7, "some", True), ("fp32", 1, 260, 192, "some", True),
]


def _conv_inputs(dtype, b, t, c, k, state, bias=True):
    d = DT[dtype]
    x, w = normal(t * 7 + c, (b, t, c), d, 1.0, DEV), normal(k + c, (c, k), d, k ** -0.5, DEV)
    return (x, w, normal(c + 1, (c,), d, 0.3, DEV) if bias else None,
            normal(t + 5, (b, k - 1, c), d, 1.0, DEV) if state else None)


def _starts_np(s):
    return None if s is None else s.cpu().numpy().astype(bool)


def _rows_of(p):
    """q as (B, T, C); the rows past T of the last group have to be zero."""
    b, g, two, c, n = p.q.shape
    rows = p.q.permute(0, 1, 2, 4, 3).reshape(b, g * two * n, c).cpu().numpy()
    t = int(np.prod(p.shape[1:-1])) if len(p.shape) > 2 else p.shape[0]
    assert not rows[:, t:].any()
    return rows[:, :t]


def _unpacked(p):
    return ref.unpack8(_rows_of(p), p.e.cpu().numpy())


def _assert_kept(p, x, what):
    q, e = ref.pack8(f64(x))
    np.testing.assert_array_equal(p.e.cpu().numpy(), e, err_msg=what)
    np.testing.assert_array_equal(_rows_of(p), q, err_msg=what)


# ---- convolution ----


@pytest.mark.parametrize("k,act", [(4, "silu"), (3, None), (1, "silu"), (2, None), (8, "silu"), (5, None)])
@pytest.mark.parametrize("dtype,b,t,c,starts,state", SHAPES)
def test_conv_forward_and_backward(dtype, b, t, c, starts, state, k, act):
    x, w, bias, st = _conv_inputs(dtype, b, t, c, k, state, bias=k != 3)
    s = starts_of(starts, b, t, DEV)
    sn, name = _starts_np(s), act or "none"
    f = igc.seq_conv(x, w, bias=bias, activation=act, state=st, starts=s, keep8=True)
    y, bound, last = ref.conv_fwd(f64(x), f64(w), f64(bias), name, f64(st), sn)
    assert_within(f.y, y, bound, "y")
    np.testing.assert_array_equal(f64(f.state), last)
    _assert_kept(f.kept, x, "x in 8 bits")
    plain = igc.seq_conv(x, w, bias=bias, activation=act, state=st, starts=s)
    assert plain.kept is None and torch.equal(plain.y, f.y)

    dy = normal(t + 11, (b, t, c), DT[dtype], 1.0, DEV)
    dlast = normal(t + 12, (b, k - 1, c), DT[dtype], 1.0, DEV) if state else None
    for kept in (False, True):
        g = igc.seq_conv_bwd(dy, f.kept if kept else x, w, bias=bias, activation=act, state=st, starts=s, dstate=dlast)
        want = ref.conv_bwd(f64(dy), _unpacked(f.kept) if kept else f64(x), f64(w), f64(bias), name, f64(st), sn,
                            f64(dlast))
        assert_within(g.dx, *want["dx"], f"dx kept={kept}")
        assert_within(g.dw, *want["dw"], f"dw kept={kept}")
        assert (g.dbias is None) == (bias is None) and (g.dstate is None) == (st is None)
        if bias is not None:
            assert_within(g.dbias, *want["dbias"], f"dbias kept={kept}")
        if st is not None:
            assert_within(g.dstate, *want["dstate"], f"dstate kept={kept}")


@pytest.mark.parametrize("dtype,b,c,k,act", [("bf16", 1, 256, 4, "silu"), ("fp32", 3, 65, 3, None), ("fp16", 17, 130, 8, "silu"),
                                             ("bf16", 300, 8, 2, None), ("fp16", 4, 1, 1, "silu")])
def test_conv_steps_follow_the_sequence(dtype, b, c, k, act):
    t = 6
    x, w, bias, st = _conv_inputs(dtype, b, t, c, k, True)
    y, bound, last = ref.conv_fwd(f64(x), f64(w), f64(bias), act or "none", f64(st))
    state = st.clone()
    other = torch.empty_like(state)
    for n in range(t):
        out, now = igc.seq_conv_step(x[:, n], w, state, bias=bias, activation=act, state_out=other if n % 2 else None)
        assert now is (other if n % 2 else state)
        assert_within(out, y[:, n], bound[:, n], f"row {n}")
        if n % 2:
            state, other = other, state
    np.testing.assert_array_equal(f64(state), last)


# ---- recurrence ----


def _check_scan(dtype, b, t, c, starts, state, wide=False, decay=8.0):
    x, gr, gi, lam, h0 = scan_inputs(t * 3 + c, b, t, c, DT[dtype], DEV, state, wide)
    s = starts_of(starts, b, t, DEV)
    sn = _starts_np(s)
    f = igc.gated_scan(x, gr, gi, lam, decay=decay, h0=h0, starts=s, train=True, keep8=True)
    h, bound, last, states = ref.scan_fwd(f64(x), f64(gr), f64(gi), f64(lam), decay, f64(h0), sn)
    assert_within(f.y, h, bound, "y")
    assert_within(f.h, *last, "h")
    for n, (v, e) in enumerate(states):
        assert_within(f.states[:, n], v, e, f"state before row {64 * n}")
    for p, v, n in zip(f.kept, (x, gr, gi), ("x", "gate_r", "gate_i")):
        _assert_kept(p, v, n + " in 8 bits")
    plain = igc.gated_scan(x, gr, gi, lam, decay=decay, h0=h0, starts=s)
    assert plain.states is None and plain.kept is None and torch.equal(plain.y, f.y) and torch.equal(plain.h, f.h)

    dy = normal(t + 21, (b, t, c), DT[dtype], 1.0, DEV)
    dh = normal(t + 22, (b, c), torch.float32, 1.0, DEV) if state else None
    for kept in (False, True):
        ins = f.kept if kept else (x, gr, gi)
        g = igc.gated_scan_bwd(dy, *ins, lam, f.states, decay=decay, starts=s, dh=dh)
        given = [_unpacked(p) for p in f.kept] if kept else [f64(v) for v in ins]
        want = ref.scan_bwd(f64(dy), *given, f64(lam), f64(f.states), decay, sn, f64(dh))
        for n in ("dx", "dgate_r", "dgate_i", "dlam", "dh0"):
            assert_within(getattr(g, n), *want[n], f"{n} kept={kept}")


@pytest.mark.parametrize("dtype,b,t,c,starts,state", SHAPES)
def test_scan_forward_and_backward(dtype, b, t, c, starts, state):
    _check_scan(dtype, b, t, c, starts, state)


@pytest.mark.parametrize("dtype,b,t,c,starts,state", [SHAPES[3], SHAPES[8], SHAPES[9], SHAPES[10]])
def test_scan_gates_wide_open_and_shut(dtype, b, t, c, starts, state):
    _check_scan(dtype, b, t, c, starts, state, wide=True, decay=3.0)


@pytest.mark.parametrize("dtype,b,c", [("bf16", 1, 256), ("fp32", 3, 65), ("fp16", 17, 130), ("bf16", 300, 8)])
def test_scan_steps_follow_the_sequence(dtype, b, c):
    t = 5
    x, gr, gi, lam, h0 = scan_inputs(c, b, t, c, DT[dtype], DEV)
    h, bound, last, _ = ref.scan_fwd(f64(x), f64(gr), f64(gi), f64(lam), 8.0, f64(h0))
    state = h0.clone()
    other = torch.empty_like(state)
    for n in range(t):
        y, now = igc.gated_scan_step(x[:, n], gr[:, n], gi[:, n], lam, state, h_out=other if n % 2 else None)
        assert_within(y, h[:, n], bound[:, n], f"row {n}")
        if n % 2:
            state, other = other, state
    assert_within(state, *last, "state")


def test_slots_pick_streams_and_skip_idle_ones():
    b, pool, c, k = 6, 9, 40, 4
    x, w, bias, _ = _conv_inputs("bf16", b, 1, c, k, False)
    state = normal(3, (pool, k - 1, c), torch.bfloat16, 1.0, DEV)
    slots = torch.tensor([4, -1, 0, 8, 9, 2], dtype=torch.int32, device=DEV)
    live = [0, 2, 3, 5]
    rows = slots[live].long()
    want_y, want_s = igc.seq_conv_step(x[live, 0], w, state[rows].contiguous(), bias=bias, activation="silu")
    before = state.clone()
    y, _ = igc.seq_conv_step(x[:, 0], w, state, bias=bias, activation="silu", slots=slots)
    assert torch.equal(y[live], want_y) and not y[[1, 4]].any()
    before[rows] = want_s
    assert torch.equal(state, before)

    xs, gr, gi, lam, _ = scan_inputs(9, b, 1, c, torch.float16, DEV)
    h = normal(4, (pool, c), torch.float32, 1.0, DEV)
    want_y, want_h = igc.gated_scan_step(xs[live, 0], gr[live, 0], gi[live, 0], lam, h[rows].contiguous())
    before = h.clone()
    y, _ = igc.gated_scan_step(xs[:, 0], gr[:, 0], gi[:, 0], lam, h, slots=slots)
    assert torch.equal(y[live], want_y) and not y[[1, 4]].any()
    before[rows] = want_h
    assert torch.equal(h, before)


# ---- 8 bits ----


@pytest.mark.parametrize("dtype,shape", [("bf16", (1, 1, 1)), ("fp32", (2, 33, 7)), ("fp16", (2, 5, 9, 65)), ("bf16", (3, 16, 128)),
                                         ("fp32", (40, 24)), ("bf16", (2, 100, 264)), ("fp16", (1, 3, 4, 5, 16)),
                                         ("bf16", (2, 47, 1001)), ("fp32", (1, 4099, 64))])
def test_eight_bits_there_and_back(dtype, shape):
    scale = torch.exp2(normal(1, shape[-1:], torch.float32, 3.0))
    x = (normal(len(shape), shape) * scale).to(DT[dtype]).to(DEV)
    p = igc.pack8(x)
    rows = f64(x).reshape(1 if len(shape) == 2 else shape[0], -1, shape[-1])
    q, e = ref.pack8(rows)
    np.testing.assert_array_equal(_rows_of(p), q)
    np.testing.assert_array_equal(p.e.cpu().numpy(), e)
    assert p.shape == x.shape and p.dtype == x.dtype
    for to in (None, torch.float32, torch.bfloat16):
        v = igc.unpack8(p, to)
        want = torch.from_numpy(ref.unpack8(q, e).reshape(shape)).to(x.dtype if to is None else to)
        assert v.dtype == want.dtype and torch.equal(v.cpu(), want)


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
def test_eight_bits_at_the_ends_of_the_type(dtype):
    d = DT[dtype]
    top, low = torch.finfo(d).max, torch.finfo(d).smallest_normal
    x = torch.zeros((1, 48, 6), dtype=torch.float64)
    x[0, 0] = torch.tensor([top, -top, low, low / 4, float("inf"), float("nan")])
    x[0, 1] = torch.tensor([top * 0.99, 1.0, -low, low / 8, 1.0, 1.0])
    x = x.to(d).to(DEV)
    p = igc.pack8(x)
    v = igc.unpack8(p)
    with np.errstate(invalid="ignore"):
        q, e = ref.pack8(f64(x))
    np.testing.assert_array_equal(p.e.cpu().numpy(), e)
    assert torch.isfinite(v[0, :, :4]).all() and torch.isnan(v[0, :16, 4:]).all() and torch.isfinite(v[0, 16:]).all()
    np.testing.assert_array_equal(f64(v[0, :, :4]), f64(torch.from_numpy(ref.unpack8(q, e)[0, :, :4]).to(d)))


# ---- strides, streams, graphs, memory ----


def test_views_give_the_same_bits():
    b, t, c, k = 3, 70, 64, 4
    for d in (torch.bfloat16, torch.float32):
        wide = normal(1, (b, t + 9, 3 * c + 1), d, 1.0, DEV)
        w, bias = normal(2, (c, k), d, 0.5, DEV), normal(3, (c,), d, 0.5, DEV)
        lam = normal(4, (c,), torch.float32, 1.0, DEV) - 4
        views = [wide[:, 4:4 + t, j * c + 1:(j + 1) * c + 1] for j in range(3)]     # one element past alignment
        views.append(wide[:1, 2:2 + t, :c].expand(b, t, c))                         # one batch for all
        views.append(wide[:, 3:4, c:2 * c].expand(b, t, c))                         # one row for all
        views.append(wide.transpose(0, 1)[4:4 + t, :, :c].transpose(0, 1))
        views.append(wide[:, 4:4 + t, :2 * c:2])                                    # channels apart: copied
        dense = [v.contiguous() for v in views]
        for v, e in zip(views, dense):
            assert torch.equal(igc.seq_conv(v, w, bias, "silu").y, igc.seq_conv(e, w, bias, "silu").y)
            assert torch.equal(igc.pack8(v).q, igc.pack8(e).q)
        for p in ((0, 1, 2), (3, 4, 5), (6, 0, 4)):
            va, ea = [views[j] for j in p], [dense[j] for j in p]
            f, g = igc.gated_scan(*va, lam, train=True, keep8=True), igc.gated_scan(*ea, lam, train=True, keep8=True)
            assert torch.equal(f.y, g.y) and all(torch.equal(m.q, n.q) for m, n in zip(f.kept, g.kept))
            for m, n in zip(igc.gated_scan_bwd(views[1], *va, lam, f.states), igc.gated_scan_bwd(dense[1], *ea, lam, f.states)):
                assert torch.equal(m, n)
            for m, n in zip(igc.seq_conv_bwd(views[2], va[0], w, bias, "silu"), igc.seq_conv_bwd(dense[2], ea[0], w, bias, "silu")):
                assert (m is None and n is None) or torch.equal(m, n)


def _train(x, gr, gi, lam, w, dy):
    f = igc.seq_conv(x, w, None, "silu", keep8=True)
    s = igc.gated_scan(f.y, gr, gi, lam, train=True, keep8=True)
    g = igc.gated_scan_bwd(dy, *s.kept, lam, s.states)
    d = igc.seq_conv_bwd(g.dx, f.kept, w, None, "silu")
    return [f.y, s.y, s.h, *g, d.dx, d.dw, igc.unpack8(igc.pack8(x))]


def _train_inputs(b=2, t=700, c=192):
    x, gr, gi, lam, _ = scan_inputs(1, b, t, c, torch.bfloat16, DEV)
    return x, gr, gi, lam, normal(5, (c, 4), torch.bfloat16, 0.5, DEV), normal(6, (b, t, c), torch.bfloat16, 1.0, DEV)


def test_the_same_call_gives_the_same_bits():
    a = _train_inputs()
    first = _train(*a)
    for _ in range(5):
        assert all(torch.equal(m, n) for m, n in zip(first, _train(*a)))


@pytest.mark.parametrize("b,t,c,calls", [(1, 65539, 1024, 400), (1, 32771, 256, 800), (4, 4096, 512, 400), (2, 1999, 321, 400)])
def test_many_calls_on_new_values_give_the_same_bits(b, t, c, calls):
    """Tiles that take over a neighbour's state before it is complete show up in few of many calls; two
    sets of values take turns, so that nothing left in memory by the call before fits.  Slow decays
    carry a state that went missing far along."""
    lam = normal(9, (c,), torch.float32, 0.5, DEV) - 5
    sets = [[normal(20 + 4 * n + k, (b, t, c), torch.bfloat16, 1.0, DEV) for k in range(4)] for n in range(2)]

    def run(x, r, i, dy):
        f = igc.gated_scan(x, r, i, lam, train=True)
        return (f.y, f.h, *igc.gated_scan_bwd(dy, x, r, i, lam, f.states))

    want = [run(*s) for s in sets]
    wrong = torch.zeros(len(want[0]), dtype=torch.int64, device=DEV)
    for n in range(calls):
        got = run(*sets[n % 2])
        wrong += torch.stack([(g != w).any() for g, w in zip(got, want[n % 2])])
    assert wrong.tolist() == [0] * len(wrong)


def test_on_another_stream():
    a = _train_inputs()
    want = _train(*a)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        inputs = [v.clone() * 1 for v in a]
        got = _train(*inputs)
    side.synchronize()
    assert all(torch.equal(m, n) for m, n in zip(want, got))


def test_in_a_graph():
    a = _train_inputs()
    for _ in range(2):
        _train(*a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _train(*a)
    for n in range(4):
        a[0].copy_(normal(50 + n, a[0].shape, torch.bfloat16, 1.0, DEV))
        graph.replay()
        torch.cuda.synchronize()
        want = _train(*a)
        assert all(torch.equal(m, v) for m, v in zip(got, want)), n
        torch.cuda.synchronize()


class _Guarded:
    """torch with empty() giving tensors between two bands of a known byte, and inputs whose
    new_empty() does."""

    BAND = 4096

    def __init__(self):
        self.whole = []

    def __getattr__(self, name):
        return getattr(torch, name)

    def empty(self, shape, dtype=torch.float32, device=None):
        shape = (shape,) if isinstance(shape, int) else tuple(shape)
        n = int(np.prod(shape)) * dtype.itemsize
        raw = torch.full((n + 2 * self.BAND,), 0xA5, dtype=torch.uint8, device=device)
        self.whole.append((raw, n))
        return raw[self.BAND:self.BAND + n].view(dtype).view(shape)

    def empty_like(self, t):
        return self.empty(t.shape, t.dtype, t.device)

    def new_empty(self, t, shape, dtype=None):
        return self.empty(shape, t.dtype if dtype is None else dtype, t.device)

    def check(self):
        for raw, n in self.whole:
            assert (raw[:self.BAND] == 0xA5).all() and (raw[self.BAND + n:] == 0xA5).all()
        count, self.whole = len(self.whole), []
        return count


@pytest.mark.parametrize("dtype,b,t,c,starts,state", [s for s in SHAPES if s[0] != "fp32" or s[3] != 31])
def test_nothing_is_written_outside_the_outputs(monkeypatch, dtype, b, t, c, starts, state):
    guard = _Guarded()
    monkeypatch.setattr(sequence, "torch", guard)
    monkeypatch.setattr(torch.Tensor, "new_empty", lambda self, shape, dtype=None: guard.new_empty(self, shape, dtype))
    x, w, bias, st = _conv_inputs(dtype, b, t, c, 4, state)
    s = starts_of(starts, b, t, DEV)
    xs, gr, gi, lam, h0 = scan_inputs(t, b, t, c, DT[dtype], DEV, state)
    f = igc.seq_conv(x, w, bias, "silu", st, s, keep8=True)
    igc.seq_conv_bwd(x, f.kept, w, bias, "silu", st, s, dstate=st)
    igc.seq_conv_bwd(x, xs, w, bias, "silu", st, s)
    g = igc.gated_scan(xs, gr, gi, lam, h0=h0, starts=s, train=True, keep8=True)
    igc.gated_scan_bwd(x, *g.kept, lam, g.states, starts=s, dh=h0)
    igc.gated_scan_bwd(x, xs, gr, gi, lam, g.states, starts=s)
    igc.unpack8(igc.pack8(x))
    torch.cuda.synchronize()
    assert guard.check() > 25


@pytest.mark.parametrize("b,t", [(0, 5), (2, 0), (0, 0)])
@pytest.mark.parametrize("k", [4, 1])
def test_empty_problems(b, t, k):
    c = 24
    x, w, bias, st = _conv_inputs("bf16", b, t, c, k, True)
    f = igc.seq_conv(x, w, bias, "silu", st, starts_of("some", b, t, DEV) if t and b else None, keep8=True)
    assert f.y.shape == (b, t, c) and f.kept.shape == (b, t, c)
    if t == 0:
        assert torch.equal(f.state, st)
    g = igc.seq_conv_bwd(x, x, w, bias, "silu", st, dstate=st)
    assert not g.dw.any() and not g.dbias.any() and g.dx.shape == x.shape
    if t == 0:
        assert torch.equal(g.dstate, st)
    xs, gr, gi, lam, h0 = scan_inputs(1, b, t, c, torch.bfloat16, DEV)
    s = igc.gated_scan(xs, gr, gi, lam, h0=h0, train=True, keep8=True)
    assert s.y.shape == (b, t, c) and s.states.shape == (b, 0 if t == 0 else 1, c)
    if t == 0:
        assert torch.equal(s.h, h0)
    d = igc.gated_scan_bwd(xs, xs, gr, gi, lam, s.states, dh=h0)
    assert not d.dlam.any() and d.dx.shape == xs.shape
    if t == 0:
        assert torch.equal(d.dh0, h0)
    assert igc.unpack8(igc.pack8(x)).shape == x.shape


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("t,at,c", [(100, 37, 40), (700, 300, 66), (300, 255, 7)])
def test_nothing_crosses_a_start(bad, t, at, c):
    """Rows of one sequence hold NaN or infinities everywhere; the sequences around it do not notice."""
    b, end = 2, at + 9
    x, w, bias, st = _conv_inputs("bf16", b, t, c, 4, True)
    xs, gr, gi, lam, h0 = scan_inputs(t, b, t, c, torch.bfloat16, DEV)
    dy = normal(2, (b, t, c), torch.bfloat16, 1.0, DEV)
    s = torch.zeros((b, t), dtype=torch.uint8, device=DEV)
    s[:, at] = s[:, end] = 1
    out = []
    for value in (1.0, bad):
        v = [z.clone() for z in (x, xs, gr, gi, dy)]
        for z in v:
            z[:, at:end] = value
        f = igc.seq_conv(v[0], w, bias, "silu", st, s, keep8=True)
        g = igc.seq_conv_bwd(v[4], v[0], w, bias, "silu", st, s, dstate=st)
        r = igc.gated_scan(*v[1:4], lam, h0=h0, starts=s, train=True)
        d = igc.gated_scan_bwd(v[4], *v[1:4], lam, r.states, starts=s, dh=h0)
        rows = [torch.cat([z[:, :at], z[:, end:]], 1) for z in (f.y, g.dx, r.y, d.dx, d.dgate_r, d.dgate_i)]
        out.append(rows + [f.state, g.dstate, r.h, d.dh0])
    for m, n in zip(*out):
        assert torch.equal(m, n) and torch.isfinite(n.float()).all()


def test_a_nan_shows_where_it_reaches():
    """Without starts a NaN row reaches the later rows of its channel, and no other channel."""
    x, gr, gi, lam, h0 = scan_inputs(8, 1, 400, 20, torch.float32, DEV)
    x[0, 150, 3] = float("nan")
    f = igc.gated_scan(x, gr, gi, lam, h0=h0)
    bad = torch.isnan(f.y[0])
    assert bad[150:, 3].all() and bad.sum() == 250 and torch.isnan(f.h[0, 3])


def test_gates_at_the_infinities():
    """gate_r = -inf holds the state (a = 1, nothing enters), to the bound on its roundings;
    gate_i = -inf lets nothing in."""
    b, t, c = 1, 90, 10
    x, gr, gi, lam, h0 = scan_inputs(3, b, t, c, torch.float32, DEV)
    gr, gi = gr.contiguous(), gi.contiguous()
    gr[:, 20:60] = -float("inf")
    gi[:, 70:80] = -float("inf")
    gr[:, 85] = float("inf")
    f = igc.gated_scan(x, gr, gi, lam, h0=h0, train=True)
    h, bound, last, states = ref.scan_fwd(f64(x), f64(gr), f64(gi), f64(lam), 8.0, f64(h0))
    assert_within(f.y, h, bound, "y")
    dy = normal(1, (b, t, c), torch.float32, 1.0, DEV)
    g = igc.gated_scan_bwd(dy, x, gr, gi, lam, f.states)
    want = ref.scan_bwd(f64(dy), f64(x), f64(gr), f64(gi), f64(lam), f64(f.states), 8.0)
    for n in ("dx", "dgate_r", "dgate_i", "dlam", "dh0"):
        assert_within(getattr(g, n), *want[n], n)


def test_pieces_carry_on_where_the_last_ended():
    b, t, c, k, cut = 2, 500, 72, 4, 203
    x, w, bias, _ = _conv_inputs("fp32", b, t, c, k, False)
    s = starts_of("some", b, t, DEV)
    f = igc.seq_conv(x, w, bias, "silu", starts=s)
    f1 = igc.seq_conv(x[:, :cut], w, bias, "silu", starts=s[:, :cut])
    f2 = igc.seq_conv(x[:, cut:], w, bias, "silu", state=f1.state, starts=s[:, cut:])
    assert torch.equal(torch.cat([f1.y, f2.y], 1), f.y) and torch.equal(f2.state, f.state)
    dy = normal(9, (b, t, c), torch.float32, 1.0, DEV)
    g = igc.seq_conv_bwd(dy, x, w, bias, "silu", starts=s)
    g2 = igc.seq_conv_bwd(dy[:, cut:], x[:, cut:], w, bias, "silu", state=f1.state, starts=s[:, cut:])
    g1 = igc.seq_conv_bwd(dy[:, :cut], x[:, :cut], w, bias, "silu", starts=s[:, :cut], dstate=g2.dstate)
    want = ref.conv_bwd(f64(dy), f64(x), f64(w), f64(bias), "silu", None, _starts_np(s))
    # the carried rows' gradient is rounded once on its way: the bound covers one addition more
    assert_within(torch.cat([g1.dx, g2.dx], 1), want["dx"][0], 2 * want["dx"][1], "dx in pieces")
    assert_within(g.dx, *want["dx"], "dx")
    assert_within(g1.dw + g2.dw, *want["dw"], "dw")


@pytest.mark.parametrize("dtype,c", [("bf16", 1088), ("fp16", 1001)])
def test_tensors_past_32_bit_offsets(dtype, c):
    """More than 2^31 values: the last rows, shut off by a start, agree with those rows alone."""
    t = (1 << 31) // c + 5003
    tail = 1000
    d = DT[dtype]
    x = torch.empty((1, t, c), dtype=d, device=DEV)
    x.normal_()
    s = torch.zeros((1, t), dtype=torch.uint8, device=DEV)
    s[0, t - tail] = 1
    w, bias = normal(1, (c, 4), d, 0.5, DEV), normal(2, (c,), d, 0.5, DEV)
    lam = normal(3, (c,), torch.float32, 1.0, DEV) - 5
    end = x[:, t - tail:]
    f = igc.seq_conv(x, w, bias, "silu", starts=s, keep8=True)
    fe = igc.seq_conv(end, w, bias, "silu")
    assert torch.equal(f.y[:, t - tail:], fe.y) and torch.equal(f.state, fe.state)
    last = (t - 1) // 16 * 16 - 160                       # whole groups near the end
    p = igc.pack8(x[:, last:])
    assert torch.equal(f.kept.q[:, last // 16:], p.q) and torch.equal(f.kept.e[:, last // 16:], p.e)
    back = igc.unpack8(f.kept)
    assert torch.equal(back[:, last:], igc.unpack8(p))
    del back
    g = igc.seq_conv_bwd(f.y, f.kept, w, bias, "silu", starts=s)
    de = igc.seq_conv_bwd(f.y[:, last + 8:], igc.unpack8(p)[:, 8:], w, bias, "silu", state=igc.unpack8(p)[:, 5:8])
    assert torch.equal(g.dx[:, last + 16:], de.dx[:, 8:])
    y = f.y
    del f, g
    r = igc.gated_scan(x, y, x, lam, starts=s, train=True)
    re = igc.gated_scan(end, y[:, t - tail:], end, lam, train=True)
    # the same rows in other tiles: the states' bounds from the oracle on a few channels
    cols = [0, 1, c // 2, c - 1]
    h, bound, hl, _ = ref.scan_fwd(*(f64(v[..., cols]) for v in (end, y[:, t - tail:], end)), f64(lam[cols]))
    assert_within(r.y[:, t - tail:, cols], h, bound, "y")
    assert_within(r.h[:, cols], *hl, "h")
    assert torch.allclose(r.h, re.h, rtol=1e-4, atol=1e-5)
    b = igc.gated_scan_bwd(x, x, y, x, lam, r.states, starts=s)
    # rows before the start take no gradient from it: the piece before it, from its own kept state
    lo = (t - tail) // 64 * 64 - 64
    hi = t - tail
    gr = ref.scan_bwd(*(f64(v[:, lo:hi][..., cols]) for v in (x, x, y, x)), f64(lam[cols]),
                      f64(r.states[:, lo // 64:(hi - 1) // 64 + 1][..., cols]))
    for n in ("dx", "dgate_r", "dgate_i"):
        assert_within(getattr(b, n)[:, lo:hi][..., cols], *gr[n], n)


@pytest.mark.parametrize("kept", [False, True])
def test_gradients_against_differences(kept):
    """The GPU's gradients against central differences of the oracle's forward pass."""
    b, t, c, k = 2, 70, 3, 4
    x, gr, gi, lam, h0 = scan_inputs(31, b, t, c, torch.float32, DEV)
    w, bias = normal(1, (c, k), torch.float32, 0.5, DEV), normal(2, (c,), torch.float32, 0.5, DEV)
    s = starts_of("some", b, t, DEV)
    sn = _starts_np(s)
    dy = normal(5, (b, t, c), torch.float32, 1.0, DEV)
    if kept:      # values that 8 bits hold, so that both passes see the same ones
        x, gr, gi = (igc.unpack8(igc.pack8(v)) for v in (x, gr, gi))
    f = igc.gated_scan(x, gr, gi, lam, decay=2.0, h0=h0, starts=s, train=True, keep8=kept)
    g = igc.gated_scan_bwd(dy, *(f.kept if kept else (x, gr, gi)), lam, f.states, decay=2.0, starts=s)
    cf = igc.seq_conv(x, w, bias, "silu", starts=s, keep8=kept)
    cg = igc.seq_conv_bwd(dy, cf.kept if kept else x, w, bias, "silu", starts=s)
    a = {n: f64(v) for n, v in (("x", x), ("gr", gr), ("gi", gi), ("lam", lam), ("h0", h0), ("w", w), ("bias", bias))}
    dyn = f64(dy)

    def scan():
        return (ref.scan_fwd(a["x"], a["gr"], a["gi"], a["lam"], 2.0, a["h0"], sn)[0] * dyn).sum()

    def conv():
        return (ref.conv_fwd(a["x"], a["w"], a["bias"], "silu", None, sn)[0] * dyn).sum()

    r = np.random.default_rng(0)
    for loss, name, got in ((scan, "x", g.dx), (scan, "gr", g.dgate_r), (scan, "gi", g.dgate_i), (scan, "lam", g.dlam),
                            (scan, "h0", g.dh0), (conv, "x", cg.dx), (conv, "w", cg.dw), (conv, "bias", cg.dbias)):
        arr, got = a[name], f64(got)
        for _ in range(6):
            at = tuple(r.integers(0, n) for n in arr.shape)
            keep, step = arr[at], 1e-5
            arr[at] = keep + step
            hi = loss()
            arr[at] = keep - step
            lo = loss()
            arr[at] = keep
            # fp32 results of sums of a few hundred terms of order 1
            assert abs((hi - lo) / (2 * step) - got[at]) < 2e-4 * max(1.0, abs(got[at])), (name, at)
