"""Gated delta rule on the GPU: log decays above zero, and gates that are not finite behind a start.

The bounds of tests/delta_cases.py are for states that no row enlarges.  With log decays above zero an error made at
row j has grown by row i by at most the product of the decays between them, and so have the decays between rows by
which a chunk's terms are scaled: every bound grows by `growth`, the product of the decays above one of a sequence.
"""
import numpy as np
import pytest
import torch

import implicit_gemm_conv_amd as igc
from tests.delta_cases import check, definition, inputs
from tests.seq_cases import DT, starts_of

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INS = ("q", "k", "v", "log_decay", "beta")


def _ins(x):
    return [x[n] for n in INS]


def _both(x, starts=None):
    f = igc.delta_rule(*_ins(x), h0=x["h0"], starts=starts, train=True)
    g = igc.delta_rule_bwd(x["dy"], *_ins(x), f.states, starts=starts, dh=x["dh"])
    return {**f._asdict(), **f.states._asdict(), **g._asdict()}


def _grown(x, starts=None):
    """The definition with its bounds grown."""
    growth = torch.exp(x["log_decay"].double().clamp(min=0).sum(1)).max().item()
    return {n: (value, bound * growth) for n, (value, bound) in definition(x, None, starts).items()}


def _check_all(got, ref):
    for n in got:
        check(got[n], ref[n], n, np.ones(1, dtype=bool))


GROWTHS = {"0.01": lambda g: torch.full_like(g, 0.01), "0.05": lambda g: torch.full_like(g, 0.05),
           "both signs": lambda g: 0.1 * torch.sigmoid(g + 2.5) - 0.06}


@pytest.mark.parametrize("growth", list(GROWTHS))
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", [(1, 64, 1, 1, 16, 16), (2, 70, 1, 2, 64, 48), (1, 100, 2, 2, 128, 20)], ids=str)
def test_log_decays_above_zero(shape, dtype, growth):
    b, t = shape[:2]
    for starts in (None, "some"):
        x = inputs(b + t, *shape, DT[dtype], DEV)
        x["log_decay"] = GROWTHS[growth](x["log_decay"])
        s = starts_of(starts, b, t, DEV)
        _check_all(_both(x, s), _grown(x, s))


@pytest.mark.parametrize("dtype", list(DT))
def test_a_prompt_and_its_steps_agree(dtype):
    """The rule over 66 rows and 66 steps, log decays on both sides of zero: both are the definition's."""
    x = inputs(5, 2, 66, 1, 2, 32, 24, DT[dtype], DEV)
    x["log_decay"] = GROWTHS["both signs"](x["log_decay"])
    ref = _grown(x)
    f = igc.delta_rule(*_ins(x), h0=x["h0"])
    h, everywhere = x["h0"].clone(), np.ones(1, dtype=bool)
    for i in range(66):
        y, _ = igc.delta_rule_step(*[v[:, i] for v in _ins(x)], h)
        check(y, tuple(a[:, i] for a in ref["y"]), f"y {i}", everywhere)
    check(h, ref["h"], "h of the steps", everywhere)
    check(f.h, ref["h"], "h of the rule", everywhere)
    check(f.y, ref["y"], "y of the rule", everywhere)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("later", [False, True])
@pytest.mark.parametrize("first", [0, 64, 70])
def test_a_bad_decay_behind_a_start(first, later, bad):
    """The sequence of the bad row begins in its 64 rows: the state that enters them shows nothing of it.  Every row of the
    sequence from there on is not finite; rows before it, other heads and other sequences are what they are without it."""
    x = inputs(13, 1, 190, 2, 2, 32, 32, torch.float32, DEV)
    starts = torch.zeros((1, 190), dtype=torch.bool, device=DEV)
    starts[0, first] = True
    row, end = first + 30, 190
    if later:
        end = first + 45
        starts[0, end] = True
    ref = definition(x, None, starts)
    y = dict(x, log_decay=x["log_decay"].clone())
    y["log_decay"][0, row, 1] = bad
    f = igc.delta_rule(*_ins(y), h0=x["h0"], starts=starts, train=True)
    rows = torch.arange(190)
    ok = torch.ones((1, 190, 2, 1), dtype=torch.bool)
    ok[:, (rows >= row) & (rows < end), 1] = False
    check(f.y, ref["y"], "y", ok.numpy())
    assert not f.y[0, row:end, 1].isfinite().any()
    if later:
        check(f.h, ref["h"], "h")
    else:
        check(f.h[:, :1], tuple(a[:, :1] for a in ref["h"]), "h")
        assert not f.h[0, 1].isfinite().any()
    g = igc.delta_rule_bwd(x["dy"], *_ins(y), f.states, starts=starts, dh=x["dh"])
    keep = torch.ones((1, 190, 2), dtype=torch.bool)
    keep[:, (rows >= first) & (rows < end), 1] = False
    for n in ("dq", "dk", "dv", "dlog_decay", "dbeta"):
        t = getattr(g, n)
        check(t, ref[n], n, (keep[..., None] if t.dim() == 4 else keep).numpy())
        assert not t[0, row:end, 1].isfinite().all(), n
    check(g.dh0, ref["dh0"], "dh0")


def test_growth_that_overflows_goes_row_by_row():
    """Decays of e^3 a row, whose products over a chunk are past fp32's range, under keys that are all one unit vector and
    beta one: every row takes away what the state held, so that y = scale q_0 v whatever it grew by.  A row's sums are of
    terms of e^3 |v|, with at most 8 roundings, and the next row takes them away as well."""
    x = inputs(21, 1, 100, 1, 1, 16, 24, torch.float32, DEV)
    x["k"] = torch.zeros_like(x["k"])
    x["k"][..., 0] = 1
    x["beta"] = torch.ones_like(x["beta"])
    x["log_decay"] = torch.full_like(x["log_decay"], 3.0)
    y = igc.delta_rule(*_ins(x)).y.double()
    want = 16 ** -0.5 * x["q"][..., :1].double() * x["v"].double()
    bound = 8 * 2.0 ** -24 * np.exp(3.0) * x["v"].abs().max().item() * 16 ** -0.5 * x["q"][..., :1].double().abs()
    assert ((y - want).abs() <= bound + 2.0 ** -24 * want.abs()).all()


@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf"), 100.0])
def test_a_decay_at_a_start_acts_on_nothing(what):
    """Whatever it is: at the first row of all, inside a chunk, at a chunk's edge, twice in a row."""
    x = inputs(22, 1, 190, 2, 2, 32, 32, torch.float32, DEV)
    starts = torch.zeros((1, 190), dtype=torch.bool, device=DEV)
    at = [0, 20, 64, 100, 101, 189]
    starts[0, at] = True
    x["log_decay"][0, at, 1] = what
    got, ref = _both(x, starts), definition(x, None, starts)
    for n in got:
        check(got[n], ref[n], n)
    assert (got["dlog_decay"][:, at] == 0).all()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("zero", [-float("inf"), -200.0, -3e38])
def test_a_decay_of_zero_is_a_start(zero, dtype):
    """A log decay whose exponential is zero in fp32: the same bits as a start at its row, whatever large values stand before
    it, and a gradient that is exactly zero."""
    x = inputs(23, 1, 190, 1, 2, 40, 32, DT[dtype], DEV)
    for n in ("v", "dy"):
        x[n][:, :100] *= 64
    at = [20, 64, 100, 101, 189]
    starts = torch.zeros((1, 190), dtype=torch.bool, device=DEV)
    starts[0, at] = True
    want = _both(x, starts)
    x["log_decay"][0, at] = zero
    got = _both(x)
    for n in got:
        assert torch.equal(got[n], want[n]), n
    assert (got["dlog_decay"][:, at] == 0).all()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", [(1, 40, 1, 1, 16, 16), (2, 150, 1, 2, 64, 48), (1, 130, 2, 2, 128, 20)], ids=str)
def test_gradients_of_strong_decays(shape, dtype):
    """Decays of e^-5 to e^-20, in every row or in one of three.  All that a log decay's gradient is made of has the decay as a
    factor, so the bound on its error has it too."""
    b, t = shape[:2]
    for every, starts in ((1, None), (3, None), (3, "some")):
        x = inputs(b + t + every, *shape, DT[dtype], DEV, slow=True)
        strong = -5 - 15 * torch.sigmoid(3 + x["log_decay"])
        x["log_decay"][:, ::every] = strong[:, ::every]
        s = starts_of(starts, b, t, DEV)
        ref = definition(x, None, s)
        value, bound = ref["dlog_decay"]
        ref["dlog_decay"] = (value, bound * torch.exp(x["log_decay"].double().cpu()))
        _check_all(_both(x, s), ref)
