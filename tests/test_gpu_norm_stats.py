"""Statistics that the group norm returns, where they are not finite or the variance is hard to take."""
import pytest
import torch

import implicit_gemm_conv_amd as igc
from tests.norm_cases import inputs
from tests.seq_cases import DT

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


# teams of less than a wave, of several waves, several pieces a lane; tiles
@pytest.mark.parametrize("n,p,c,groups", [(3, 1, 48, 4), (3, 12, 48, 4), (2, 40, 1024, 2), (2, 1, 8192, 2), (3, 2000, 48, 4)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", list(DT))
def test_statistics_of_a_bad_group(dtype, bad, n, p, c, groups):
    """A NaN or an infinity makes the mean not finite and 1 / deviation NaN, with eps of zero too, and leaves those of all
    other groups as they are."""
    x, _, w, b = inputs(6, n, p, c, DT[dtype], DEV)
    hit = torch.zeros(n, groups, dtype=torch.bool, device=DEV)
    hit[1, 1] = True
    broken = x.clone()
    broken[1, p // 2, c // groups + 5] = bad
    for eps in (1e-5, 0.0):
        clean = igc.group_norm(x, groups, weight=w, bias=b, activation="silu", eps=eps)
        got = igc.group_norm(broken, groups, weight=w, bias=b, activation="silu", eps=eps)
        assert got.rstd[hit].isnan().all() and not got.mean[hit].isfinite().any()
        assert torch.equal(got.rstd[~hit], clean.rstd[~hit]) and torch.equal(got.mean[~hit], clean.mean[~hit])


def test_runs_that_begin_with_an_outlier():
    """128 positions a thread, of which the first is 2^10 off.  A run of r values about its first one, with squares s and sum m:
    s - m^2 / r has (r + 1) half steps of s from the first term, 2 r from the second (m has r half steps of the sum of |d|, at
    most sqrt(r s)) and three more, and r times 2^20 for s; the whole variance is 2^20 / r and the spread's."""
    n, p, c, groups, r = 128, 2048, 1024, 64, 128
    gen = torch.Generator(DEV).manual_seed(3)
    x = torch.randn((n, p, c), generator=gen, device=DEV)
    x[:, ::r] += 2.0 ** 10
    f = igc.group_norm(x, groups)
    for i in (0, 77, n - 1):
        d = x[i].double().view(p, groups, c // groups)
        mean = d.mean((0, 2))
        var = ((d - mean[:, None]) ** 2).mean((0, 2))
        error = (3 * r + 4) * 2.0 ** -24 * 2.0 ** 20 / var
        rstd = torch.rsqrt(var + 1e-5)
        assert ((f.rstd[i].double() / rstd - 1).abs() <= 0.5 * error + 2.0 ** -21).all()
        # a run's mean: its first value, r half steps of the mean distance to it, and one of each
        assert ((f.mean[i].double() - mean).abs() <= (r + 3) * 2.0 ** -24 * 2.0 ** 10).all()
        y = ((d - mean[:, None]) * rstd[:, None]).view(p, c)
        assert ((f.y[i].double() - y).abs() <= (0.5 * error.max() + 2.0 ** -20) * y.abs() + (r + 3) * 2.0 ** -14 * rstd.max()).all()
