"""Group norm on the GPU against its definition in float64."""
import numpy as np
import pytest
import torch

import implicit_gemm_conv_amd as igc
from tests.norm_cases import check, definition, inputs
from tests.seq_cases import DT, f64, normal

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# n, p, c, groups: rows, one value, teams of less than a wave, a wave, a workgroup; tiles whose groups are
# whole pieces of 16 bytes, share a piece, are odd, or need several workgroups' channels
SHAPES = [(1, 1, 1, 1), (2, 1, 64, 4), (3, 1, 2048, 16), (5, 1, 13, 13), (4, 1, 3000, 2), (2, 7, 65, 5), (2, 100, 24, 3),
          (3, 33, 96, 8), (1, 300, 16, 2), (2, 1030, 65, 5), (1, 2500, 128, 32), (2, 900, 256, 1), (1, 130, 4160, 2),
          (2, 515, 40, 10), (1, 150, 1025, 1), (700, 1, 96, 3), (40, 9, 32, 4)]


def _both(x, dy, g, w, b, act, eps=1e-5):
    f = igc.group_norm(x, g, weight=w, bias=b, activation=act, eps=eps)
    d = igc.group_norm_bwd(dy, x, g, f.mean, f.rstd, weight=w, bias=b, activation=act, eps=eps)
    return {**f._asdict(), **d._asdict()}


def _check_all(got, x, dy, g, w, b, act, eps=1e-5):
    ref = definition(x, dy, g, w, b, act, eps)
    for name, t in got.items():
        if t is not None:
            check(t, ref[name], name)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_gradients(shape, dtype):
    n, p, c, g = shape
    for act, params in (("silu", DT[dtype]), (None, torch.float32), ("silu", None)):
        x, dy, w, b = inputs(n + 7 * p + c, n, p, c, DT[dtype], DEV, params=params)
        got = _both(x, dy, g, w, b, act)
        assert (got["dweight"] is None) == (w is None)
        _check_all(got, x, dy, g, w, b, act)


# several pieces a lane (fewer than 4 positions) and the tiles that take over; more n than a launch's teams
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(5, 1, 8192, 1), (3, 3, 2720, 1), (3, 4, 2048, 1), (4, 2, 771, 1), (2, 1, 520, 1),
                                   (2100, 1, 2056, 1), (1500, 3, 104, 1)], ids=str)
def test_wide_groups(shape, dtype):
    n, p, c, g = shape
    x, dy, w, b = inputs(n + 7 * p + c, n, p, c, DT[dtype], DEV)
    _check_all(_both(x, dy, g, w, b, "silu"), x, dy, g, w, b, "silu")


@pytest.mark.parametrize("only", ["weight", "bias"])
def test_one_parameter_alone(only):
    x, dy, w, b = inputs(5, 2, 40, 48, torch.bfloat16, DEV)
    w, b = (w, None) if only == "weight" else (None, b)
    got = _both(x, dy, 6, w, b, "silu")
    assert (got["dbias"] is None) == (b is None) and (got["dweight"] is None) == (w is None)
    _check_all(got, x, dy, 6, w, b, "silu")


@pytest.mark.parametrize("shape", [(2, 1, 512, 4), (1, 2000, 64, 2)], ids=str)
def test_a_mean_far_from_zero(shape):
    n, p, c, g = shape
    x, dy, w, b = inputs(11, n, p, c, torch.float32, DEV, offset=3000.0)
    _check_all(_both(x, dy, g, w, b, None), x, dy, g, w, b, None)


@pytest.mark.parametrize("p", [1, 3000])
def test_groups_of_one_value_repeated(p):
    x = torch.full((2, p, 16), 7.25, device=DEV, dtype=torch.float16)
    f = igc.group_norm(x, 4, eps=1e-3)
    assert torch.equal(f.y, torch.zeros_like(x)) and torch.equal(f.mean, torch.full_like(f.mean, 7.25))
    assert f64(f.rstd) == pytest.approx(1e-3 ** -0.5, rel=2.0 ** -22)


@pytest.mark.parametrize("dims", [(2, 5, 6, 64), (2, 3, 4, 5, 64), (6, 64)])
def test_images_volumes_and_rows(dims):
    x, dy, w, b = inputs(3, dims[0], int(np.prod(dims[1:-1])), 64, torch.float16, DEV)
    got = _both(x.view(dims), dy.view(dims), 8, w, b, "silu")
    assert got["y"].shape == torch.Size(dims) and got["dx"].shape == torch.Size(dims)
    _check_all(got, x, dy, 8, w, b, "silu")


@pytest.mark.parametrize("p", [1, 9, 1500])
@pytest.mark.parametrize("first", [8, 5])
def test_views(p, first):
    """Column slices of a wider tensor, at an aligned and an odd channel; an expanded batch.  Aligned views take
    the path of a copy and give its bits; at an odd channel the sums are cut differently."""
    wide = normal(21, (3, p, 200), torch.bfloat16, 1.0, DEV)
    x, dy = wide[..., first:first + 96], wide[..., 101:197]
    _, _, w, b = inputs(4, 1, 1, 96, torch.bfloat16, DEV)
    got = _both(x, dy, 12, w, b, "silu")
    _check_all(got, x, dy, 12, w, b, "silu")
    if first == 8:
        whole = igc.group_norm(x.contiguous(), 12, weight=w, bias=b, activation="silu")
        assert torch.equal(got["y"], whole.y)
    many = x[:1].expand(3, p, 96)
    y = igc.group_norm(many, 12).y
    check(y, definition(many, dy, 12, None, None, None)["y"], "y of an expanded batch")
    assert first != 8 or torch.equal(y, igc.group_norm(many.contiguous(), 12).y)


@pytest.mark.parametrize("shape", [(0, 4, 16, 2), (3, 0, 16, 2)], ids=str)
def test_nothing_to_normalise(shape):
    n, p, c, g = shape
    x = torch.zeros((n, p, c), device=DEV)
    w = torch.ones(c, device=DEV)
    got = _both(x, x, g, w, w, "silu")
    assert got["y"].shape == x.shape and got["dx"].shape == x.shape
    assert torch.equal(got["dweight"], torch.zeros_like(w)) and torch.equal(got["dbias"], torch.zeros_like(w))
    assert torch.equal(got["mean"], torch.zeros((n, g), device=DEV))


@pytest.mark.parametrize("p", [1, 12, 2000])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_value_stays_in_its_group(p, bad):
    x, dy, w, b = inputs(6, 3, p, 48, torch.float32, DEV)
    clean = _both(x, dy, 4, w, b, "silu")
    x = x.clone()
    x[1, p // 2, 17] = bad
    got = _both(x, dy, 4, w, b, "silu")
    hit = torch.zeros(3, 4, dtype=torch.bool, device=DEV)
    hit[1, 1] = True
    where = hit.repeat_interleave(12, 1)[:, None].expand(3, p, 48)
    for name in ("y", "dx"):
        assert got[name][where].isnan().all() and torch.equal(got[name][~where], clean[name][~where])
    assert got["mean"][hit].isfinite().logical_not().all() and torch.equal(got["mean"][~hit], clean["mean"][~hit])
    cols = torch.arange(48, device=DEV) // 12 == 1
    for name in ("dweight", "dbias"):
        assert torch.equal(got[name][~cols], clean[name][~cols])


@pytest.mark.parametrize("p", [1, 9, 3000])
def test_guard_bands_and_given_output(p):
    """Nothing is written around y; a given output gets the same bits at an odd element offset."""
    x, _, w, b = inputs(8, 2, p, 72, torch.float16, DEV)
    want = igc.group_norm(x, 8, weight=w, bias=b).y
    for at in (8, 3):
        room = torch.full((x.numel() + 64,), 5.0, dtype=x.dtype, device=DEV)
        out = room[at:at + x.numel()].view(x.shape)
        f = igc.group_norm(x, 8, weight=w, bias=b, out=out)
        assert f.y is out
        assert (out.float() - want.float()).abs().max() <= 2.0 ** -8
        assert (room[:at] == 5).all() and (room[at + x.numel():] == 5).all()
        if at == 8:
            assert torch.equal(out, want)


@pytest.mark.parametrize("shape", [(4, 1, 256, 4), (2, 2100, 96, 3)], ids=str)
def test_another_stream_and_a_graph(shape):
    n, p, c, g = shape
    x, dy, w, b = inputs(9, n, p, c, torch.bfloat16, DEV)
    want = _both(x, dy, g, w, b, "silu")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = _both(x, dy, g, w, b, "silu")
    side.synchronize()
    assert all(torch.equal(want[k], again[k]) for k in want)
    x2, dy2, _, _ = inputs(10, n, p, c, torch.bfloat16, DEV)
    want2 = _both(x2, dy2, g, w, b, "silu")
    xs, ds = x.clone(), dy.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = _both(xs, ds, g, w, b, "silu")
    for src, grad, ref in ((x, dy, want), (x2, dy2, want2), (x, dy, want)):
        xs.copy_(src)
        ds.copy_(grad)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(ref[k], held[k]) for k in ref)
        _both(x2, dy2, g, w, b, None)  # eager work between the replays


def test_gradients_against_differences():
    """Central differences of a scalar of y, in float32 with steps of 2^-7: the third derivatives, of order one
    here, add 2^-14 / 6 a unit of direction and the roundings of the two sums 2^-24 * |sum| / 2^-7."""
    n, p, c, g = 2, 11, 24, 3
    x, dy, w, b = inputs(12, n, p, c, torch.float32, DEV)

    def value(x, w, b):
        y = igc.group_norm(x, g, weight=w, bias=b, activation="silu").y
        return (y.double() * dy.double()).sum().item()

    got = _both(x, dy, g, w, b, "silu")
    for k, (t, name) in enumerate(((x, "dx"), (w, "dweight"), (b, "dbias"))):
        d = normal(30 + k, t.shape, torch.float32, 1.0, DEV)
        d = d / d.norm()
        h = 2.0 ** -7
        args = lambda s: [v + s * h * d if v is t else v for v in (x, w, b)]  # noqa: E731
        diff = (value(*args(1)) - value(*args(-1))) / (2 * h)
        exact = (got[name].double() * d.double()).sum().item()
        y = igc.group_norm(x, g, weight=w, bias=b, activation="silu").y
        noise = (y.abs() * dy.abs()).sum().item() * 2.0 ** -22 / (2 * h)
        assert abs(diff - exact) <= 2.0 ** -14 * 4 * dy.abs().max().item() + noise + 2.0 ** -20 * abs(exact), (name, diff, exact)


def test_offsets_past_32_bits():
    """Positions behind the first 2^31 values: whole numbers whose statistics are known."""
    p, c = (1 << 20) + 3, 2049
    x = torch.zeros((1, p, c), dtype=torch.float16, device=DEV)
    x[0, -1] = 1
    f = igc.group_norm(x, 683, eps=0.0)  # groups of 3 channels
    mean = 1 / p
    # mean and variance of p values of which one is 1
    assert f64(f.mean) == pytest.approx(mean, rel=2.0 ** -20)
    assert f64(f.rstd) == pytest.approx((mean * (1 - mean)) ** -0.5, rel=2.0 ** -18)
    assert f64(f.y[0, -1]) == pytest.approx((1 - mean) * (mean * (1 - mean)) ** -0.5, rel=2.0 ** -11)
    assert f64(f.y[0, p - 2]) == pytest.approx(-mean * (mean * (1 - mean)) ** -0.5, rel=2.0 ** -10)


@pytest.mark.parametrize("shape", [(2, 1030, 32, 2), (1, 700, 65, 5), (3, 1, 256, 2)], ids=str)
def test_values_whose_squares_overflow(shape):
    """A mean whose square is past fp32's range over a spread that is not: 2^-64 of the values gives the same bits
    (nothing is rounded by a power of two), also where a last tile has fewer rows than a workgroup.  (The squares of
    2^14 differences of 2^54 add up to 2^122.)"""
    n, p, c, g = shape
    x = (1 + 2.0 ** -12 * normal(8, (n, p, c), torch.float32, 1.0, DEV)) * 2.0 ** 66
    big, small = igc.group_norm(x, g, eps=0.0), igc.group_norm(x * 2.0 ** -64, g, eps=0.0)
    assert torch.isfinite(big.y).all() and torch.equal(big.y, small.y)
    assert torch.equal(big.mean, small.mean * 2.0 ** 64) and torch.equal(big.rstd, small.rstd * 2.0 ** -64)
