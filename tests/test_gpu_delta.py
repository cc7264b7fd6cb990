"""Gated delta rule on the GPU against its row-by-row definition in float64."""
import pytest
import torch

import implicit_gemm_conv_amd as igc
from tests.delta_cases import check, definition, inputs
from tests.seq_cases import DT, normal, starts_of

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INS = ("q", "k", "v", "log_decay", "beta")

# b, t, hk, hv, dk, dv: one of everything, around the chunk's edge, shared key heads, odd sizes, wide values
SHAPES = [(1, 1, 1, 1, 1, 1), (2, 63, 1, 2, 16, 16), (1, 64, 2, 2, 32, 32), (2, 65, 1, 1, 64, 48), (1, 130, 2, 4, 128, 128),
          (2, 100, 3, 3, 65, 100), (1, 200, 1, 4, 17, 33), (3, 5, 2, 2, 128, 256), (1, 257, 9, 9, 100, 20), (2, 2, 1, 1, 8, 3)]


def _ins(x):
    return [x[n] for n in INS]


def _both(x, scale=None, starts=None, use_h0=True, use_dh=True):
    f = igc.delta_rule(*_ins(x), scale=scale, h0=x["h0"] if use_h0 else None, starts=starts, train=True)
    g = igc.delta_rule_bwd(x["dy"], *_ins(x), f.states, scale=scale, starts=starts, dh=x["dh"] if use_dh else None)
    return {**f._asdict(), **f.states._asdict(), **g._asdict()}


def _check_all(got, ref, names=None, where=None):
    for n in names or got:
        check(got[n], ref[n], n, where)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_gradients(shape, dtype):
    b, t = shape[:2]
    for starts, use in ((None, True), ("some", True), (None, False), ("all", True)):
        x = inputs(b + 3 * t, *shape, DT[dtype], DEV)
        s = starts_of(starts, b, t, DEV)
        _check_all(_both(x, None, s, use, use), definition(x, None, s, use, use))


# enough heads and columns that a workgroup carries 32 columns: a last tile of few columns, an odd number of tiles, both
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", [(5, 130, 3, 9, 40, 100), (9, 70, 4, 8, 128, 66), (17, 3, 2, 16, 17, 5)], ids=str)
def test_many_heads(shape, dtype):
    b, t = shape[:2]
    x = inputs(b + t, *shape, DT[dtype], DEV)
    s = starts_of("some", b, t, DEV)
    _check_all(_both(x, None, s), definition(x, None, s))


@pytest.mark.parametrize("dtype", list(DT))
def test_many_heads_are_each_their_own(dtype):
    """A value that is not finite in one of many heads, and the heads one by one."""
    x = inputs(3, 9, 90, 8, 8, 64, 96, DT[dtype], DEV)
    clean = _both(x)
    x["v"][4, 50, 3, 17] = float("nan")
    got = _both(x)
    for n in ("y", "h", "dv", "dh0", "dbeta"):
        same = torch.ones(9, 8, dtype=torch.bool, device=DEV)
        same[4, 3] = False
        a, b = (t[n] if n in ("h", "dh0") else t[n].transpose(1, 2) for t in (got, clean))
        assert torch.equal(a[same], b[same]), n
    bad = ~torch.isfinite(got["y"].float())
    assert bad[4, 50:, 3, 17].all() and int(bad.sum()) == 40
    one = {n: t[4:5, 2:3] if n in ("h0", "dh") else t[4:5, :, 2:3] for n, t in x.items()}
    few = _both({n: t.contiguous() for n, t in one.items()})
    for n in ("y", "h", "dv", "dlog_decay"):
        a = got[n][4:5, 2:3] if n == "h" else got[n][4:5, :, 2:3]
        assert torch.equal(a, few[n]), n


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_long_memory_and_a_given_scale(dtype):
    x = inputs(5, 1, 700, 1, 2, 64, 64, DT[dtype], DEV, slow=True)
    _check_all(_both(x, 0.37), definition(x, 0.37))


def test_equal_keys():
    """Keys that are all the same: the chunk's linear system is as far from the identity as it gets."""
    x = inputs(6, 1, 192, 1, 1, 32, 32, torch.float32, DEV, slow=True)
    x["k"] = x["k"][:, :1].expand_as(x["k"]).contiguous()
    x["beta"] = torch.ones_like(x["beta"])
    _check_all(_both(x), definition(x))


@pytest.mark.parametrize("beta", [0.0, 1.0])
def test_gates_at_their_ends(beta):
    """beta of zero (nothing is written, gradients still flow) and one; no decay, and one that leaves nothing."""
    x = inputs(7, 2, 90, 1, 2, 32, 40, torch.float32, DEV)
    x["beta"] = torch.full_like(x["beta"], beta)
    for g in (0.0, -200.0, -float("inf")):
        x["log_decay"][:, 30:50] = g
        _check_all(_both(x), definition(x))


def test_pieces_are_the_whole():
    """A sequence in pieces that break chunks, each from the state of the one before, forward and backward."""
    x = inputs(8, 2, 200, 2, 2, 32, 32, torch.float32, DEV)
    ref = definition(x)
    edges = (0, 1, 64, 130, 200)
    h, pieces = x["h0"], []
    for lo, hi in zip(edges, edges[1:]):
        part = [v[:, lo:hi] for v in _ins(x)]
        pieces.append((part, igc.delta_rule(*part, h0=h, train=True)))
        h = pieces[-1][1].h
    check(torch.cat([f.y for _, f in pieces], 1), ref["y"], "y")
    check(h, ref["h"], "h")
    dh, grads = x["dh"], []
    for (part, f), lo, hi in zip(pieces[::-1], edges[-2::-1], edges[:0:-1]):
        grads.append(igc.delta_rule_bwd(x["dy"][:, lo:hi], *part, f.states, dh=dh))
        dh = grads[-1].dh0
    for n in ("dq", "dk", "dv", "dlog_decay", "dbeta"):
        check(torch.cat([getattr(g, n) for g in grads[::-1]], 1), ref[n], n)
    check(dh, ref["dh0"], "dh0")


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 1), (3, 2, 4, 65, 100), (2, 1, 1, 128, 64), (2, 2, 2, 64, 200), (5, 1, 3, 16, 6)], ids=str)
def test_steps_are_rows_of_the_rule(shape, dtype):
    b, hk, hv, dk, dv = shape
    x = inputs(9, b, 3, hk, hv, dk, dv, DT[dtype], DEV)
    ref = definition(x)
    h = x["h0"].clone()
    for i in range(3):
        y, h2 = igc.delta_rule_step(*[v[:, i] for v in _ins(x)], h)
        assert h2 is h
        check(y, tuple(a[:, i] for a in ref["y"]), f"y {i}")
    check(h, ref["h"], "h")


def test_step_slots():
    x = inputs(10, 4, None, 1, 2, 32, 48, torch.bfloat16, DEV)
    pool = normal(3, (7, 2, 32, 48), torch.float32, 1.0, DEV)
    slots = torch.tensor([5, -1, 0, 7], dtype=torch.int32, device=DEV)
    before = pool.clone()
    other = torch.full_like(pool, 9.0)
    y2, o = igc.delta_rule_step(*_ins(x), pool, slots=slots, h_out=other)
    assert o is other and torch.equal(pool, before)
    y, _ = igc.delta_rule_step(*_ins(x), pool, slots=slots)
    assert torch.equal(y, y2) and (y[1] == 0).all() and (y[3] == 0).all()
    for s in range(7):
        if s in (5, 0):
            i = 0 if s == 5 else 2
            one = [v[i:i + 1] for v in _ins(x)]
            yi, hi = igc.delta_rule_step(*one, before[s:s + 1].clone())
            assert torch.equal(y[i], yi[0]) and torch.equal(pool[s], hi[0]) and torch.equal(other[s], hi[0])
        else:
            assert torch.equal(pool[s], before[s]) and (other[s] == 9).all()


@pytest.mark.parametrize("first", [0, 8, 3])
def test_views(first):
    """Slices of one projection at aligned and odd offsets, swapped head and row axes, expanded heads."""
    dt = torch.bfloat16
    x = inputs(11, 2, 90, 2, 4, 32, 24, dt, DEV)
    wide = torch.zeros((2, 90, first + 64 + 64 + 96 + 5), dtype=dt, device=DEV)
    v = dict(x)
    at = first
    for n, h, d in (("q", 2, 32), ("k", 2, 32), ("v", 4, 24)):
        part = wide[..., at:at + h * d]
        part.copy_(x[n].flatten(2))
        v[n] = part.unflatten(-1, (h, d))
        at += h * d
    v["dy"] = x["dy"].transpose(1, 2).contiguous().transpose(1, 2)
    assert not v["q"].is_contiguous() and not v["dy"].is_contiguous()
    a, b = _both(x), _both(v)
    assert all(torch.equal(a[n], b[n]) for n in a)
    ex = dict(x, q=x["q"][:, :, :1].expand_as(x["q"]), v=x["v"][:1].expand_as(x["v"]))
    co = dict(ex, q=ex["q"].contiguous(), v=ex["v"].contiguous())
    a, b = _both(ex), _both(co)
    assert all(torch.equal(a[n], b[n]) for n in a)
    i = 4
    y, _ = igc.delta_rule_step(*[t[:, i] for t in _ins(v)], x["h0"].clone())
    y2, _ = igc.delta_rule_step(*[t[:, i].contiguous() for t in _ins(v)], x["h0"].clone())
    assert torch.equal(y, y2)


@pytest.mark.parametrize("shape", [(0, 5, 1, 2, 8, 8), (2, 0, 1, 2, 8, 8)], ids=str)
def test_nothing_to_do(shape):
    x = inputs(12, *shape, torch.float16, DEV)
    got = _both(x)
    assert got["y"].shape == x["v"].shape and torch.equal(got["h"], x["h0"]) and torch.equal(got["dh0"], x["dh"])
    assert got["dq"].shape == x["q"].shape and got["states"].shape == (shape[0], -(-shape[1] // 64), 2, 8, 8)
    if shape[0]:
        assert (igc.delta_rule(*_ins(x)).h == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", ["q", "k", "v", "log_decay", "beta"])
def test_a_bad_value_reaches_what_comes_after(where, bad):
    """Rows before it, other heads and the next sequence are what they are without it; with v, other columns too."""
    x = inputs(13, 1, 190, 2, 2, 32, 32, torch.float32, DEV)
    starts = torch.zeros((1, 190), dtype=torch.bool, device=DEV)
    starts[0, 150] = True   # inside the third chunk
    row = 140               # inside the third chunk too
    ref = definition(x, None, starts)
    y = dict(x)
    y[where] = x[where].clone()
    y[where][(0, row, 1) + ((5,) if x[where].dim() == 4 else ())] = bad
    f = igc.delta_rule(*_ins(y), h0=x["h0"], starts=starts, train=True)
    rows = torch.arange(190)
    free = (rows < row) | (rows >= 150)
    ok = torch.zeros((1, 190, 2, 32), dtype=torch.bool)
    ok[:, :, 0] = True
    ok[:, free, 1] = True
    if where == "q":
        ok[0, :, 1] = True
        ok[0, row, 1] = False
    if where == "v":
        ok[0, :, 1] = True
        ok[0, row:150, 1, 5] = False
    check(f.y, ref["y"], "y", ok.numpy())
    check(f.h, ref["h"], "h")
    assert not f.y.cpu()[~ok].isfinite().all()
    g = igc.delta_rule_bwd(x["dy"], *_ins(y), f.states, starts=starts, dh=x["dh"])
    # the other head, and the next sequence, whose gradients take nothing from this one
    for n in ("dq", "dk", "dv", "dlog_decay", "dbeta"):
        keep = torch.zeros((1, 190, 2) + ((1,) if getattr(g, n).dim() == 4 else ()), dtype=torch.bool)
        keep[:, :, 0] = True
        keep[:, 150:, 1] = True
        check(getattr(g, n), ref[n], n, keep.numpy())


def test_a_bad_gradient_stays_in_its_sequence():
    x = inputs(14, 1, 190, 2, 2, 32, 32, torch.float32, DEV)
    starts = torch.zeros((1, 190), dtype=torch.bool, device=DEV)
    starts[0, [20, 70, 100, 150]] = True
    ref = definition(x, None, starts)
    x = dict(x, dy=x["dy"].clone(), dh=x["dh"].clone())
    x["dy"][0, 90, 1, 3] = float("nan")
    x["dh"][0, 0, 2, 2] = float("inf")
    f = igc.delta_rule(*_ins(x), h0=x["h0"], starts=starts, train=True)
    g = igc.delta_rule_bwd(x["dy"], *_ins(x), f.states, starts=starts, dh=x["dh"])
    rows = torch.arange(190)
    for n in ("dq", "dk", "dv", "dlog_decay", "dbeta"):
        keep = torch.zeros((1, 190, 2) + ((1,) if getattr(g, n).dim() == 4 else ()), dtype=torch.bool)
        keep[:, rows < 150, 0] = True
        keep[:, (rows < 70) | (rows >= 100), 1] = True
        check(getattr(g, n), ref[n], n, keep.numpy())
        assert not getattr(g, n).cpu()[~keep.expand_as(getattr(g, n))].isfinite().all()
    check(g.dh0, ref["dh0"], "dh0")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_state_ends_at_a_start(bad):
    x = inputs(15, 1, 100, 1, 1, 32, 32, torch.float32, DEV)
    starts = torch.zeros((1, 100), dtype=torch.bool, device=DEV)
    starts[0, 10] = True
    ref = definition(x, None, starts)
    h0 = x["h0"].clone()
    h0[0, 0, 3, 4] = bad
    f = igc.delta_rule(*_ins(x), h0=h0, starts=starts)
    ok = torch.ones((1, 100, 1, 32), dtype=torch.bool)
    ok[0, :10, 0, 4] = False
    check(f.y, ref["y"], "y", ok.numpy())
    check(f.h, ref["h"], "h")
    starts[0, 0] = True
    f = igc.delta_rule(*_ins(x), h0=h0, starts=starts)
    check(f.y, definition(x, None, starts)["y"], "y")


def test_guard_bands_and_given_output():
    x = inputs(16, 2, 70, 1, 3, 20, 24, torch.float16, DEV)
    want = igc.delta_rule(*_ins(x), h0=x["h0"]).y
    n = want.numel()
    for at in (64, 3):
        room = torch.full((n + 128,), 5.0, dtype=want.dtype, device=DEV)
        out = room[at:at + n].view(want.shape)
        assert igc.delta_rule(*_ins(x), h0=x["h0"], out=out).y is out
        assert torch.equal(out, want) and (room[:at] == 5).all() and (room[at + n:] == 5).all()


def test_another_stream_and_a_graph():
    shape = (2, 150, 1, 2, 64, 64)
    x, x2 = inputs(17, *shape, torch.bfloat16, DEV), inputs(18, *shape, torch.bfloat16, DEV)
    want, want2 = _both(x), _both(x2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = _both(x)
    side.synchronize()
    assert all(torch.equal(want[n], again[n]) for n in want)
    held_in = {n: t.clone() for n, t in x.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = _both(held_in)
        ys, hs = igc.delta_rule_step(*[held_in[n][:, 0] for n in INS], held_in["h0"].clone())
    for src, ref in ((x, want), (x2, want2), (x, want)):
        for n in src:
            held_in[n].copy_(src[n])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(ref[n], held[n]) for n in ref)
        y, h = igc.delta_rule_step(*[src[n][:, 0] for n in INS], src["h0"].clone())
        assert torch.equal(y, ys) and torch.equal(h, hs)
        _both(x2, 0.5)  # eager work between the replays


def test_gradients_against_differences():
    """Central differences of a scalar of the outputs, in float32 with steps of 2^-7 along unit directions: third
    derivatives of order 2^4 at these sizes add 2^-14 / 6 * 2^4, and the two sums' roundings 2^-22 * |sum| / 2^-6."""
    x = inputs(19, 1, 70, 1, 2, 16, 12, torch.float32, DEV)

    def value(z):
        f = igc.delta_rule(*_ins(z), h0=z["h0"])
        return (f.y.double() * x["dy"].double()).sum().item() + (f.h.double() * x["dh"].double()).sum().item()

    got = _both(x)
    y, h = got["y"], got["h"]
    noise = ((y * x["dy"]).abs().sum() + (h * x["dh"]).abs().sum()).item() * 2.0 ** -22 * 2 ** 6
    for k, n in enumerate(INS + ("h0",)):
        d = normal(40 + k, x[n].shape, torch.float32, 1.0, DEV)
        d = d / d.norm()
        diff = (value(dict(x, **{n: x[n] + 2.0 ** -7 * d})) - value(dict(x, **{n: x[n] - 2.0 ** -7 * d}))) * 2 ** 6
        exact = (got["d" + n].double() * d.double()).sum().item()
        assert abs(diff - exact) <= 2.0 ** -10 / 6 * 4 + noise, (n, diff, exact)


def test_the_same_bits_every_time():
    x = inputs(20, 2, 500, 2, 4, 128, 128, torch.bfloat16, DEV)
    s = starts_of("some", 2, 500, DEV)
    first = _both(x, None, s)
    for _ in range(3):
        again = _both(x, None, s)
        assert all(torch.equal(first[n], again[n]) for n in first)


def test_offsets_past_32_bits():
    """Rows of v and y behind the first 2^31 values: the last chunk of a sequence whose state is forgotten at a start
    there equals that chunk alone."""
    t, hv, dv = 33000, 128, 512
    gen = torch.Generator(DEV).manual_seed(1)
    q = torch.randn((1, t, 1, 16), generator=gen, device=DEV).half() * 0.25
    v = torch.zeros((1, t, hv, dv), dtype=torch.float16, device=DEV)
    v[:, -40:] = torch.randn((1, 40, hv, dv), generator=gen, device=DEV).half()
    g = torch.full((1, t, hv), -0.1, device=DEV)
    beta = torch.full((1, t, hv), 0.5, device=DEV)
    starts = torch.zeros((1, t), dtype=torch.bool, device=DEV)
    starts[0, -40] = True
    f = igc.delta_rule(q, q, v, g, beta, starts=starts)
    alone = igc.delta_rule(q[:, -40:], q[:, -40:], v[:, -40:], g[:, -40:], beta[:, -40:])
    # fp32 arithmetic in another order, of values of size one: then a rounding to fp16 each
    assert (f.y[:, -40:].float() - alone.y.float()).abs().max() <= 2.0 ** -9 * alone.y.float().abs().max()
    assert (f.h - alone.h).abs().max() <= 2.0 ** -16 * alone.h.abs().max()
    assert (f.y[:, :-40] == 0).all()


@pytest.mark.parametrize("dv", [64, 37])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_kept_tensors_at_any_element(dtype, dv):
    """What the forward pass kept, and the states, may start at any fp32 element: the bits are those of aligned ones."""
    x = inputs(9, 2, 130, 1, 2, 48, dv, DT[dtype], DEV)
    f = igc.delta_rule(*_ins(x), h0=x["h0"], train=True)
    want = igc.delta_rule_bwd(x["dy"], *_ins(x), f.states, dh=x["dh"])

    def moved(t):
        to = torch.empty(t.numel() + 1, device=DEV)[1:].view(t.shape)
        return to.copy_(t)

    again = igc.delta_rule(*_ins(x), h0=moved(x["h0"]), train=True)
    assert torch.equal(again.y, f.y) and torch.equal(again.states.x, f.states.x)
    got = igc.delta_rule_bwd(x["dy"], *_ins(x), igc.DeltaStates(*map(moved, f.states)), dh=moved(x["dh"]))
    for n, t in got._asdict().items():
        assert torch.equal(t, getattr(want, n)), n


@pytest.mark.parametrize("dtype", list(DT))
def test_one_row_at_every_position(dtype):
    """Inputs whose rows are all one row in memory (a row stride of zero), in a last chunk that is not whole."""
    x = inputs(24, 2, 90, 2, 2, 32, 24, DT[dtype], DEV)
    for n in ("q", "k", "v", "dy"):
        x[n] = x[n][:, :1].expand_as(x[n])
    a, b = _both(x), _both({n: t.contiguous() for n, t in x.items()})
    assert all(torch.equal(a[n], b[n]) for n in a)
