"""The convolution, the gated delta rule and the group norm as a block puts them together
(examples/gated_delta_block.py)."""
import importlib.util
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = "cuda:0"
# fp32 throughout: sums of at most 2 * 75 rows or 64 channels, a few of them one after the other, each term
# rounded by 2^-24 of its size.  Over a whole tensor the roundings add as the root of their number (2^4), to
# terms that are up to 2^4 times the result where a recurrence, a norm and their gradients cancel: 2^-16, and
# 2^2 for the steps that follow each other.
TOL = 2.0 ** -14


def _block(**kw):
    path = os.path.join(ROOT, "examples", "gated_delta_block.py")
    spec = importlib.util.spec_from_file_location("gated_delta_block", path)
    mod = importlib.util.module_from_spec(spec)
    before = list(sys.path)
    spec.loader.exec_module(mod)
    sys.path[:] = before
    return mod, mod.GatedDeltaBlock(**{**dict(model=32, key_heads=2, heads=4, dk=16, dv=24, dtype=torch.float32), **kw})


def _reference(block, u, starts):
    """The block in float64 with autograd, its parameters and u as leaves."""
    p = {n: v.detach().cpu().double().requires_grad_() for n, v in block.params.items()}
    mat = lambda x, w: x @ w.flatten(1).t()  # noqa: E731
    x = u.detach().cpu().double().requires_grad_()
    starts = starts.cpu()
    z, gates = mat(x, p["w_in"]), mat(x, p["w_gates"])
    b, t, c = z.shape
    taps = p["w_conv"].shape[1]
    share = block.hv // block.hk
    decay = torch.exp(-torch.exp(p["rate"]) * torch.nn.functional.softplus(gates[..., :block.hv]))
    beta = torch.sigmoid(gates[..., block.hv:])
    hist, live = [torch.zeros(b, c, dtype=torch.float64)] * taps, [torch.zeros(b, 1, dtype=torch.float64)] * taps
    S = torch.zeros(b, block.hv, block.dk, block.dv, dtype=torch.float64)
    rows = []
    for n in range(t):
        go = (~starts[:, n:n + 1]).double()
        hist, live = hist[1:] + [z[:, n]], [v * go for v in live[1:]] + [torch.ones_like(go)]
        y = torch.nn.functional.silu(sum(hist[j] * live[j] * p["w_conv"][:, j] for j in range(taps)))
        q, k, v = (h.unflatten(-1, (n_, d)) for h, n_, d in zip(y.split(block.sizes, -1), (block.hk, block.hk, block.hv),
                                                                (block.dk, block.dk, block.dv)))
        q, k = (h / torch.sqrt((h * h).sum(-1, keepdim=True) + 1e-6) for h in (q, k))
        q, k = (h.repeat_interleave(share, 1) for h in (q, k))
        S = (decay[:, n] * go)[..., None, None] * S
        u_ = beta[:, n, :, None] * (v - (S * k[..., None]).sum(-2))
        S = S + k[..., None] * u_[:, :, None]
        h = block.dk ** -0.5 * (S * q[..., None]).sum(-2)
        hat = (h - h.mean(-1, keepdim=True)) / torch.sqrt(h.var(-1, unbiased=False, keepdim=True) + 1e-5)
        rows.append(mat(torch.nn.functional.silu(hat.flatten(1) * p["w_norm"] + p["b_norm"]), p["w_out"]))
    return torch.stack(rows, 1), p, x


def _inputs(t=75):
    gen = torch.Generator("cpu").manual_seed(5)
    u, dy = (torch.randn((2, t, 32), generator=gen).to(DEV) for _ in range(2))
    return u, dy, (torch.rand((2, t), generator=gen) < 0.06).to(DEV)


def _off(got, want):
    return ((got.cpu().double().view_as(want) - want).norm() / want.norm()).item()


def test_block_against_the_definition_and_its_gradients():
    _, block = _block()
    u, dy, starts = _inputs()
    y, _, kept = block.forward(u, starts=starts, train=True)
    want, p, x = _reference(block, u, starts)
    assert _off(y, want.detach()) < TOL
    want.backward(dy.cpu().double())
    du, grads = block.backward(dy, kept)
    assert _off(du, x.grad) < TOL
    assert set(grads) == set(p)
    for name, g in grads.items():
        assert _off(g, p[name].grad) < TOL, name


def test_rows_one_by_one_are_the_whole_sequence():
    ex, block = _block()
    u, _, _ = _inputs(40)
    assert _off(ex.serve(block, u, 30), block.forward(u)[0].cpu().double()) < TOL


def test_streams_share_a_pool_of_states():
    """Streams in any slots of a pool, one of them idle: each goes on as it would alone."""
    _, block = _block()
    u, _, _ = _inputs(6)
    rows, h = block.new_state(5)
    slots = torch.tensor([3, -1, 0], dtype=torch.int32, device=DEV)
    three = torch.cat([u, u[:1] * 2])
    got = torch.stack([block.step(three[:, n].contiguous(), (rows, h), slots) for n in range(6)], 1)
    alone = torch.cat([block.forward(three[i:i + 1])[0] for i in (0, 2)])
    assert _off(got[[0, 2]], alone.cpu().double()) < TOL
    assert not h[[1, 2, 4]].any() and h[0].any() and h[3].any()


def test_example_runs_in_bfloat16():
    ex, block = _block(dtype=torch.bfloat16, model=64, dk=64, dv=64)
    u = torch.randn(2, 130, 64, device=DEV).bfloat16()
    y, (rows, h), kept = block.forward(u, train=True)
    du, grads = block.backward(torch.randn_like(y), kept)
    assert y.shape == du.shape == u.shape and h.shape == (2, 4, 64, 64)
    assert all(torch.isfinite(g.float()).all() for g in (y, du, *grads.values()))


def test_block_in_a_graph():
    """Forward and backward captured once and replayed between eager calls of the same block."""
    _, block = _block()
    u, dy, starts = _inputs(70)

    def both():
        y, state, kept = block.forward(u, starts=starts, train=True)
        du, grads = block.backward(dy, kept)
        return [y, *state, du, *grads.values()]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = both()
    for scale in (1.0, -0.5, 2.0):
        u.mul_(scale)
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(captured, both()):
            assert _off(got, want.cpu().double()) < TOL if want.abs().max() > 0 else not got.any()
