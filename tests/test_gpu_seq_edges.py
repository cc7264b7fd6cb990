"""GPU tests of the sequence operators where a number leaves fp32's range or a buffer reaches a limit."""
import pytest
import torch

import implicit_gemm_conv_amd as igc
from tests.seq_cases import DT, normal

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF = float("inf")


def _strong(seed, b, t, c, dtype, lam):
    """x, gate_r, gate_i, lam (C): products of a over a tile lie far below fp32's smallest number."""
    x, gr, gi = (normal(seed + k, (b, t, c), dtype, 1.0, DEV) for k in range(3))
    return x, gr, gi, torch.full((c,), lam, device=DEV)


# softplus(-0.43) = 0.5: a is about e^-2 a row and a product of 64 rows about e^-128; at 20 a itself is
# e^-80 in the middle of its gate and e^-139 at two standard deviations
@pytest.mark.parametrize("lam", [-0.43, 20.0])
@pytest.mark.parametrize("dtype,b,t,c", [("fp32", 1, 900, 70), ("bf16", 2, 129, 6), ("fp16", 1, 100, 64), ("bf16", 1, 2000, 130)])
def test_an_infinity_in_the_state_stays(dtype, b, t, c, lam):
    """a = e^-u is positive, so an infinite state is infinite in all later rows of its channel, and an
    infinite gradient of the last state in all earlier ones; the other channels take no notice."""
    x, gr, gi, lam = _strong(t, b, t, c, DT[dtype], lam)
    h0 = normal(1, (b, c), torch.float32, 1.0, DEV)
    plain = igc.gated_scan(x, gr, gi, lam, h0=h0, train=True)
    up, down = slice(0, None, 3), slice(1, None, 3)
    far = h0.clone()
    far[:, up], far[:, down] = INF, -INF
    f = igc.gated_scan(x, gr, gi, lam, h0=far, train=True)
    for got, want in ((f.y, plain.y), (f.states, plain.states), (f.h, plain.h)):
        assert (got[..., up] == INF).all() and (got[..., down] == -INF).all()
        assert torch.equal(got[..., 2::3], want[..., 2::3])

    dy = normal(2, (b, t, c), DT[dtype], 1.0, DEV)
    want = igc.gated_scan_bwd(dy, x, gr, gi, lam, plain.states, dh=h0)
    got = igc.gated_scan_bwd(dy, x, gr, gi, lam, plain.states, dh=far)
    for g, w in ((got.dx, want.dx), (got.dh0, want.dh0)):
        assert (g[..., up] == INF).all() and (g[..., down] == -INF).all()
        assert torch.equal(g[..., 2::3], w[..., 2::3])


@pytest.mark.parametrize("lam", [-0.43, 20.0])
@pytest.mark.parametrize("dtype,t,at,c", [("fp32", 700, 300, 70), ("bf16", 400, 130, 6), ("fp16", 130, 3, 64)])
def test_an_infinity_that_enters_stays(dtype, t, at, c, lam):
    """An infinite x makes its row and all later ones infinite, an infinite dy its row and all earlier ones."""
    x, gr, gi, lam = _strong(t, 1, t, c, DT[dtype], lam)
    dy = normal(2, (1, t, c), DT[dtype], 1.0, DEV)
    plain = igc.gated_scan(x, gr, gi, lam, train=True)
    want = igc.gated_scan_bwd(dy, x, gr, gi, lam, plain.states)
    far = x.clone()
    far[:, at, ::2] = INF
    f = igc.gated_scan(far, gr, gi, lam)
    assert (f.y[:, at:, ::2] == INF).all() and (f.h[:, ::2] == INF).all()
    assert torch.equal(f.y[:, :at], plain.y[:, :at]) and torch.equal(f.y[..., 1::2], plain.y[..., 1::2])
    far = dy.clone()
    far[:, at, ::2] = -INF
    g = igc.gated_scan_bwd(far, x, gr, gi, lam, plain.states)
    assert (g.dx[:, :at + 1, ::2] == -INF).all() and (g.dh0[:, ::2] == -INF).all()
    assert torch.equal(g.dx[:, at + 1:], want.dx[:, at + 1:]) and torch.equal(g.dx[..., 1::2], want.dx[..., 1::2])


def test_states_that_vanish_give_the_same_bits():
    """Two of three blocks of 128 rows hold zeros, and a block's product of a underflows: what is left of
    the state must not depend on whether a later tile met the tile's step or its state.  The gates
    let it through to the outputs: a is 1 at a block's first row, where the forward pass would show
    it, and the products with the gradient stay above a half at a piece's last."""
    b, t, c = 1, 128 * 3 * 40, 1024
    x, gr, gi, lam = _strong(5, b, t, c, torch.float32, -0.43)
    block = torch.arange(t, device=DEV) // 128 % 3
    dy = normal(9, (b, t, c), torch.float32, 1.0, DEV)
    x, dy = (torch.where((block == 0)[:, None], v.sign() * (v.abs() + 1), 0.0) for v in (x, dy))
    gr[:, ::64] = -30.0
    gr[:, 63::64] = 0.0
    gi.fill_(10.0)

    def run():
        f = igc.gated_scan(x, gr, gi, lam, train=True)
        return [v.view(torch.int32) for v in (f.y, f.h, f.states, *igc.gated_scan_bwd(dy, x, gr, gi, lam, f.states))]

    want = run()
    wrong = torch.zeros(len(want), dtype=torch.int64, device=DEV)
    for _ in range(200):
        wrong += torch.stack([(g != w).any() for g, w in zip(run(), want)])
    assert wrong.tolist() == [0] * len(wrong)


@pytest.mark.parametrize("c", [(1 << 24) + 1, 1 << 24])
def test_sums_over_very_many_channels(c):
    """8 taps and a bias of 2^24 channels: 2^19 groups of 32 channels, each with nine sums of 1024 threads, are
    more threads than one dimension of a grid holds.  Small whole numbers: every sum has to be exact."""
    t, k = 2, 8
    gen = torch.Generator(DEV).manual_seed(c)

    def whole(*shape):
        return torch.randint(-3, 4, shape, generator=gen, device=DEV, dtype=torch.int8).half()

    x, dy, w, bias, state = whole(1, t, c), whole(1, t, c), whole(c, k), whole(c), whole(1, k - 1, c)
    g = igc.seq_conv_bwd(dy, x, w, bias, state=state)
    rows = torch.cat([state, x], 1)[0]
    for j in range(k):
        assert torch.equal(g.dw[:, j], sum((dy[0, n] * rows[n + j]).float() for n in range(t))), j
    assert torch.equal(g.dbias, dy[0].float().sum(0))
    assert torch.equal(g.dx[0, 1], dy[0, 1] * w[:, 7]) and torch.equal(g.dx[0, 0], dy[0, 0] * w[:, 7] + dy[0, 1] * w[:, 6])


@pytest.mark.parametrize("bad", [float("nan"), INF])
@pytest.mark.parametrize("t,at,end,c", [(100, 37, 46, 40), (700, 304, 320, 66), (300, 255, 262, 7)])
def test_from_8_bits_sequences_part_at_groups(bad, t, at, end, c):
    """Rows at .. end - 1 of one sequence hold NaN or infinities.  From 8 bits the groups of 16 rows that hold one
    are NaN whole; sequences that have no row in those groups do not notice."""
    b, lo, hi = 2, at // 16 * 16, -(-end // 16) * 16
    x, gr, gi, dy = (normal(t + k, (b, t, c), torch.bfloat16, 1.0, DEV) for k in range(4))
    w, bias = normal(1, (c, 4), torch.bfloat16, 0.5, DEV), normal(2, (c,), torch.bfloat16, 0.3, DEV)
    lam = normal(3, (c,), torch.float32, 1.0, DEV) - 5
    s = torch.zeros((b, t), dtype=torch.bool, device=DEV)
    s[:, [lo, at, end]] = True
    if hi < t:
        s[:, hi] = True
    out = []
    for value in (1.0, bad):
        v = [z.clone() for z in (x, gr, gi, dy)]
        for z in v:
            z[:, at:end] = value
        f = igc.seq_conv(v[0], w, bias, "silu", starts=s, keep8=True)
        assert torch.equal(torch.isnan(igc.unpack8(f.kept)).any(2)[0],
                           (torch.arange(t, device=DEV) // 16 * 16 >= lo) & (torch.arange(t, device=DEV) < hi) & (value != 1.0))
        g = igc.seq_conv_bwd(v[3], f.kept, w, bias, "silu", starts=s)
        r = igc.gated_scan(*v[:3], lam, starts=s, train=True, keep8=True)
        d = igc.gated_scan_bwd(v[3], *r.kept, lam, r.states, starts=s)
        out.append([torch.cat([z[:, :lo], z[:, hi:]], 1) for z in (g.dx, d.dx, d.dgate_r, d.dgate_i)] + [d.dh0])
    for m, n in zip(*out):
        assert torch.equal(m, n) and torch.isfinite(n.float()).all()


def test_slots_that_no_stream_names_are_left_alone():
    """With a second buffer, slots of idle streams keep what they hold in both."""
    b, pool, c, k = 4, 7, 24, 4
    x, w = normal(1, (b, c), torch.float16, 1.0, DEV), normal(2, (c, k), torch.float16, 0.5, DEV)
    slots = torch.tensor([5, -1, 0, 7], dtype=torch.int32, device=DEV)
    named, rest = [5, 0], [1, 2, 3, 4, 6]
    state, other = (normal(n, (pool, k - 1, c), torch.float16, 1.0, DEV) for n in (3, 4))
    was = state.clone(), other.clone()
    y, now = igc.seq_conv_step(x, w, state, slots=slots, state_out=other)
    assert now is other and torch.equal(state, was[0]) and torch.equal(other[rest], was[1][rest])
    assert torch.equal(other[named], torch.cat([was[0][named, 1:], x[[0, 2], None]], 1)) and not y[[1, 3]].any()
    h, h2 = (normal(n, (pool, c), torch.float32, 1.0, DEV) for n in (5, 6))
    was = h.clone(), h2.clone()
    y, now = igc.gated_scan_step(x, x, x, w[:, 0].float(), h, slots=slots, h_out=h2)
    assert now is h2 and torch.equal(h, was[0]) and torch.equal(h2[rest], was[1][rest])
    assert torch.equal(y[[0, 2]], h2[named].half()) and not y[[1, 3]].any()
