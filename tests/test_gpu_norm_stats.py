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
