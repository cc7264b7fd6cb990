"""Gated delta rule on the GPU: sums of 16-bit inputs' products that cancel to their last bits.

Decays are one, keys orthogonal, and every product and every partial sum here is a multiple of 2^-21 below 4 and
so exact in fp32; what is left, one or two units of 2^-21, is exact in 16 bits as well.  Arithmetic at fp32's precision has
no freedom then: the results are equal to the definition's.  1 + 2^-9 + 2^-20 has bits in three groups of 8, and an operand
held in two of them loses the last.
"""
import pytest
import torch

import implicit_gemm_conv_amd as igc
from tests.delta_cases import inputs
from tests.seq_cases import DT

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E = 2.0 ** -20
F = 1 + 2.0 ** -9


def _zeros(t, dtype):
    """One head of 8 x 4: q, k, v, dy, no decay, beta one, states of zero."""
    rows = {n: torch.zeros(1, t, 1, d, dtype=DT[dtype], device=DEV) for n, d in (("q", 8), ("k", 8), ("v", 4), ("dy", 4))}
    return dict(rows, log_decay=torch.zeros(1, t, 1, device=DEV), beta=torch.ones(1, t, 1, device=DEV),
                h0=torch.zeros(1, 1, 8, 4, device=DEV), dh=torch.zeros(1, 1, 8, 4, device=DEV))


def _row(x, name, t, *values):
    x[name][0, t, 0, :len(values)] = torch.tensor(values, device=DEV)


def _forward(x, train=False):
    return igc.delta_rule(x["q"], x["k"], x["v"], x["log_decay"], x["beta"], scale=1.0, h0=x["h0"], train=train)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_y_of_the_state_before(dtype):
    """q S = (F + 2^-20) - F."""
    x = _zeros(1, dtype)
    _row(x, "q", 0, 1, 1)
    x["h0"][0, 0, 0, :2] = F + E
    x["h0"][0, 0, 1, :2] = -F
    assert _forward(x).y[0, 0, 0].tolist() == [E, E, 0, 0]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_y_of_corrections_of_many_bits(dtype):
    """R u = u_0 + u_1, with u = beta v = (F + 2^-20) / 2 and -F / 2."""
    x = _zeros(3, dtype)
    _row(x, "k", 0, 1)
    _row(x, "k", 1, 0, 1)
    _row(x, "q", 2, 1, 1)
    _row(x, "v", 0, 1, 1)
    _row(x, "v", 1, -1, -1)
    x["beta"][0, :2, 0] = torch.tensor([(F + E) / 2, F / 2])
    assert _forward(x).y[0, 2, 0].tolist() == [E / 2, E / 2, 0, 0]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_y_of_products_of_many_bits(dtype):
    """R u = (q k_0) - (q k_1), with q k = F + 2^-20 and F."""
    x = _zeros(3, dtype)
    _row(x, "k", 0, 1, 2.0 ** -10, 1)
    _row(x, "k", 1, 0, 0, 0, 1, 1)
    _row(x, "q", 2, 1, 2.0 ** -10, 2.0 ** -9, 1, 2.0 ** -9)
    _row(x, "v", 0, 1, 1)
    _row(x, "v", 1, -1, -1)
    assert _forward(x).y[0, 2, 0].tolist() == [E, E, 0, 0]


def _dk(x):
    f = _forward(x, train=True)
    g = igc.delta_rule_bwd(x["dy"], x["q"], x["k"], x["v"], x["log_decay"], x["beta"], f.states, scale=1.0, dh=x["dh"])
    return g.dk[0, :, 0]


@pytest.mark.parametrize("bits_in", ["state", "gradient"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_dk_of_the_state_before(dtype, bits_in):
    """dk = -S dx = -((F + 2^-20) - F), the many bits in S or in dx."""
    x = _zeros(1, dtype)
    _row(x, "k", 0, 0, 1)
    many, ones = torch.tensor([F + E, F]), torch.tensor([1.0, 1.0])
    x["h0"][0, 0, 0, :2] = (many if bits_in == "state" else ones) * torch.tensor([1, -1])
    x["dh"][0, 0, 1, :2] = ones if bits_in == "state" else many
    assert _dk(x).tolist() == [[-E] + [0] * 7]


@pytest.mark.parametrize("bits_in", ["gradient", "correction"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_dk_of_the_gradient_behind(dtype, bits_in):
    """dk = dS u = (F + 2^-20) - F, the many bits in dS or in u = v - S k."""
    x = _zeros(1, dtype)
    _row(x, "k", 0, 0, 1)
    _row(x, "v", 0, 1, 1)
    if bits_in == "gradient":
        x["dh"][0, 0, 0, :2] = torch.tensor([F + E, -F])
    else:
        x["dh"][0, 0, 0, :2] = torch.tensor([1, -1])
        x["h0"][0, 0, 1, :2] = 1 - torch.tensor([F + E, F])
    assert _dk(x).tolist() == [[E] + [0] * 7]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_dk_of_the_rows_before(dtype):
    """dk_2 = -(dx_2 u_0) k_0 - (dx_2 u_1) k_1 = -((F + 2^-20) - F) in its first element."""
    x = _zeros(3, dtype)
    _row(x, "k", 0, 1, 1)
    _row(x, "k", 1, -1, 1)
    _row(x, "k", 2, 0, 0, 1)
    _row(x, "v", 0, 1)
    _row(x, "v", 1, 0, 1)
    x["dh"][0, 0, 2, :2] = torch.tensor([F + E, F])
    assert _dk(x)[2, 0].item() == -E


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_dk_of_the_rows_after(dtype):
    """dk_0 = dS u_0 - (dx_1 u_0) k_1 - (dx_2 u_0) k_2 = 2^-21 - ((F + 2^-20) - F) in its second element."""
    x = _zeros(3, dtype)
    _row(x, "k", 0, 1)
    _row(x, "k", 1, 0, 1, 1)
    _row(x, "k", 2, 0, -1, 1)
    _row(x, "v", 0, 1)
    x["dh"][0, 0, 1:3, 0] = torch.tensor([E / 2, F + E / 2])
    assert _dk(x)[0, 1].item() == -E / 2


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_dk_of_the_reads_after(dtype):
    """dk_0 = (dy_1 u_0) q_1 + (dy_2 u_0) q_2 = (F + 2^-20) - F in its second element."""
    x = _zeros(3, dtype)
    _row(x, "k", 0, 1)
    _row(x, "v", 0, 1, 1)
    x["h0"][0, 0, 0, :2] = 1 - torch.tensor([F + E, F])
    _row(x, "q", 1, 0, 1)
    _row(x, "q", 2, 0, -1)
    _row(x, "dy", 1, 1)
    _row(x, "dy", 2, 0, 1)
    assert _dk(x)[0, 1].item() == E


@pytest.mark.parametrize("power", [-90, -60, 60, 120])
def test_powers_of_two_change_no_bits(power):
    """v and the first state times 2^power: y and the last state are that much larger, bit for bit, where the smallest of an
    fp32 value's three parts is still a bf16 number and nothing overflows."""
    x = inputs(25, 1, 130, 1, 2, 32, 24, torch.float32, DEV)
    big = {n: (x[n].double() * 2.0 ** power).float() for n in ("v", "h0")}
    a, b = _forward(x), _forward({**x, **big})
    for n in ("y", "h"):
        assert torch.equal((getattr(a, n).double() * 2.0 ** power).float(), getattr(b, n)), n
