"""GPU tests of the sequence operators at sizes where the work of a wave, the sums over workgroups and the
carrying of states between tiles change what they do."""
import numpy as np
import pytest
import torch

import implicit_gemm_conv_amd as igc
from oracle import sequence as ref
from tests.seq_cases import DT, ROUND, assert_within, f64, normal, scan_inputs, starts_of

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E = 2.0 ** -24


def _whole(seed, shape, top, dtype):
    """Whole numbers within +-top."""
    gen = torch.Generator("cpu").manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=gen).to(dtype).to(DEV)


# dtype, B, T, C, starts: groups of 16 rows times columns of 128 channels below 8192, from there on, and
# from 16384 on (1, 2 and 4 groups a wave); T ends inside a group, a walk and a workgroup; parts of the
# sums: 7, 2200, 1030, 1821, 2050, 17, 1366
WALKS = [
    ("bf16", 7, 60, 6, None), ("fp16", 1100, 131, 6, "some"), ("fp32", 515, 130, 130, None), ("bf16", 1821, 131, 4, None),
    ("fp16", 1025, 259, 3, "some"), ("fp32", 1, 4099, 8065, "some"), ("bf16", 683, 390, 6, "some"),
]


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("dtype,b,t,c,starts", WALKS)
def test_conv_sums_of_whole_numbers(dtype, b, t, c, starts, kept):
    """Without activation and on small whole numbers, which 8 bits hold as they are, fp32 makes no
    rounding at all: every gradient has to be the exact one, in both input forms."""
    k, d = 4, DT[dtype]
    x, w, dy = _whole(1, (b, t, c), 3, d), _whole(2, (c, k), 2, d), _whole(3, (b, t, c), 2, d)
    state, dstate = _whole(4, (b, k - 1, c), 3, d), _whole(5, (b, k - 1, c), 2, d)
    bias, s = _whole(6, (c,), 2, d), starts_of(starts, b, t, DEV)
    f = igc.seq_conv(x, w, bias, state=state, starts=s, keep8=kept)
    g = igc.seq_conv_bwd(dy, f.kept if kept else x, w, bias, state=state, starts=s, dstate=dstate)

    rows = torch.cat([state, x], 1).double()
    back = torch.zeros_like(rows)
    back[:, t:] += dstate
    seg = torch.zeros((b, t + k - 1), dtype=torch.int32, device=DEV)
    if s is not None:
        seg[:, k - 1:] = torch.cumsum(s.int(), 1)
        back[:, t:] *= (seg[:, t:] == seg[:, -1:])[..., None]
    y, dw = torch.zeros((b, t, c), dtype=torch.float64, device=DEV) + bias.double(), []
    for j in range(k):
        live = (seg[:, j:j + t] == seg[:, k - 1:])[..., None]
        tap = rows[:, j:j + t] * live
        y += tap * w[:, j].double()
        dw.append((tap * dy.double()).sum((0, 1)))
        back[:, j:j + t] += dy.double() * w[:, j].double() * live
    assert torch.equal(f.y.double(), y)
    assert torch.equal(g.dw.double(), torch.stack(dw, 1)) and torch.equal(g.dbias.double(), dy.double().sum((0, 1)))
    assert torch.equal(g.dx.double(), back[:, k - 1:]) and torch.equal(g.dstate.double(), back[:, :k - 1])


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("dtype,b,t,c,starts,k", [("bf16", 1100, 131, 6, "some", 4), ("fp16", 911, 131, 130, None, 3),
                                                  ("bf16", 1821, 131, 3, "some", 8)])
def test_conv_walks_with_the_activation(dtype, b, t, c, starts, k, kept):
    d = DT[dtype]
    x, w, dy = normal(1, (b, t, c), d, 1.0, DEV), normal(2, (c, k), d, k ** -0.5, DEV), normal(3, (b, t, c), d, 1.0, DEV)
    bias, state = normal(4, (c,), d, 0.3, DEV), normal(5, (b, k - 1, c), d, 1.0, DEV)
    s = starts_of(starts, b, t, DEV)
    sn = None if s is None else s.cpu().numpy()
    p = igc.pack8(x)
    held = igc.unpack8(p, torch.float32) if kept else x
    g = igc.seq_conv_bwd(dy, p if kept else x, w, bias, "silu", state, s)
    want = ref.conv_bwd(f64(dy), f64(held), f64(w), f64(bias), "silu", f64(state), sn)
    assert_within(g.dx, *want["dx"], "dx")
    assert_within(g.dstate, *want["dstate"], "dstate")


# tiles: 79 forward and 157 backward; 8 and 16; 157 and 313
@pytest.mark.parametrize("dtype,b,t,c,starts", [("fp32", 1, 10007, 20, None), ("bf16", 2, 10007, 6, None),
                                                ("fp16", 40, 1000, 5, "rare"), ("bf16", 1, 20011, 3, "rare")])
@pytest.mark.parametrize("kept", [False, True])
def test_scan_over_many_tiles(dtype, b, t, c, starts, kept):
    """Decays slow enough that a state that went missing many tiles ago shows (from 1 - 1e-5 a row)."""
    d = DT[dtype]
    x, gr, gi, _, h0 = scan_inputs(t, b, t, c, d, DEV)
    lam = torch.linspace(-13.0, -6.0, c, device=DEV)
    s = None
    if starts == "rare":
        s = torch.zeros((b, t), dtype=torch.bool, device=DEV)
        s[:, t // 3] = s[::2, 2 * t // 3 + 5] = True
    sn = None if s is None else s.cpu().numpy()
    f = igc.gated_scan(x, gr, gi, lam, h0=h0, starts=s, train=True, keep8=kept)
    h, bound, last, states = ref.scan_fwd(f64(x), f64(gr), f64(gi), f64(lam), 8.0, f64(h0), sn)
    assert_within(f.y, h, bound, "y")
    assert_within(f.h, *last, "h")
    for n, (v, e) in enumerate(states):
        assert_within(f.states[:, n], v, e, f"state before row {64 * n}")

    dy = normal(3, (b, t, c), d, 1.0, DEV)
    dh = normal(4, (b, c), torch.float32, 1.0, DEV) * 100
    ins = f.kept if kept else (x, gr, gi)
    g = igc.gated_scan_bwd(dy, *ins, lam, f.states, starts=s, dh=dh)
    given = [f64(igc.unpack8(p, torch.float32)) for p in f.kept] if kept else [f64(v) for v in ins]
    want = ref.scan_bwd(f64(dy), *given, f64(lam), f64(f.states), 8.0, sn, f64(dh))
    for n in ("dx", "dgate_r", "dgate_i", "dh0"):
        assert_within(getattr(g, n), *want[n], n)
    # dlam against the sum of what the rows' own gradients say it is: dgate_r = e (1 - r), dlam = unit sum e.
    # Each e as the gate's gradient returns it is off by its rounding and by the rounding of 1 - r; the sum
    # adds 8 rows, 8 waves, every 32nd tile and 32 of those.
    r = ref.sigmoid(given[1])
    e = f64(g.dgate_r) / (1 - r)
    rel = ROUND[d][0] + (4 + (2 * np.abs(given[1]) + 6) * r / (1 - r)) * E
    tiles = b * -(-t // 64)
    off = (np.abs(e) * (1.1 * rel + (8 + 8 + tiles / 32 + 32) * E) + ROUND[d][1] / (1 - r)).sum((0, 1))
    lam64 = f64(lam)
    unit = ref.sigmoid(lam64) / ref.softplus(lam64)
    assert_within(g.dlam, e.sum((0, 1)) * unit, (off + 12 * E * np.abs(e.sum((0, 1)))) * unit, "dlam")


@pytest.mark.parametrize("dtype,b,t,c,calls", [("bf16", 1, 20011, 512, 200), ("fp16", 4, 4096, 256, 200), ("fp32", 2, 1999, 321, 200)])
@pytest.mark.parametrize("starts", [False, True])
def test_many_calls_that_keep_8_bits_give_the_same_bits(dtype, b, t, c, calls, starts):
    """As the plain inputs' test of the kind: with packed sequences and 8-bit inputs, two sets of values taking turns."""
    lam = normal(9, (c,), torch.float32, 0.5, DEV) - 5
    sets = [[normal(20 + 4 * n + k, (b, t, c), DT[dtype], 1.0, DEV) for k in range(4)] for n in range(2)]
    s = torch.zeros((b, t), dtype=torch.bool, device=DEV)
    s[:, 700] = s[0, t // 2] = True

    def run(x, r, i, dy):
        f = igc.gated_scan(x, r, i, lam, starts=s if starts else None, train=True, keep8=True)
        return (f.y, f.h, f.states, f.kept[0].q, *igc.gated_scan_bwd(dy, *f.kept, lam, f.states, starts=s if starts else None))

    want = [run(*v) for v in sets]
    wrong = torch.zeros(len(want[0]), dtype=torch.int64, device=DEV)
    for n in range(calls):
        wrong += torch.stack([(g != w).any() for g, w in zip(run(*sets[n % 2]), want[n % 2])])
    assert wrong.tolist() == [0] * len(wrong)
