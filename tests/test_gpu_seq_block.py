"""The sequence operators as a recurrent block puts them together (examples/gated_recurrent_block.py)."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = "cuda:0"


def _example():
    path = os.path.join(ROOT, "examples", "gated_recurrent_block.py")
    spec = importlib.util.spec_from_file_location("gated_recurrent_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _reference(block, u, starts):
    """The block in float64 with autograd, its parameters as leaves."""
    p = {n: v.double().clone().requires_grad_() for n, v in block.params.items()}
    mat = lambda x, w: x @ w.flatten(1).t()  # noqa: E731
    x = u.double()
    z = mat(x, p["w_in"])
    b, t, c = z.shape
    k = p["w_conv"].shape[1]
    rows, h = [], torch.zeros(b, c, dtype=torch.float64, device=u.device)
    zero = torch.zeros_like(h)
    hist, live = [zero] * k, [torch.zeros(b, 1, dtype=torch.float64, device=u.device)] * k
    for n in range(t):
        go = (~starts[:, n:n + 1]).double()
        hist, live = hist[1:] + [z[:, n]], [v * go for v in live[1:]] + [torch.ones_like(go)]
        y = sum(hist[j] * live[j] * p["w_conv"][:, j] for j in range(k)) + p["b_conv"]
        y = torch.nn.functional.silu(y)
        gr, gi = mat(y, p["w_gates"]).chunk(2, -1)
        a = torch.exp(-block.decay * torch.nn.functional.softplus(p["lam"]) * torch.sigmoid(gr))
        h = a * h * go + torch.sqrt(1 - a * a) * torch.sigmoid(gi) * y
        rows.append(mat(h, p["w_out"]))
    return torch.stack(rows, 1), p


def test_block_trains_towards_the_reference_gradients():
    ex = _example()
    block = ex.GatedRecurrentBlock(model=32, channels=64, dtype=torch.float32)
    gen = torch.Generator("cpu").manual_seed(3)
    u = torch.randn((2, 75, 32), generator=gen).to(DEV)
    dy = torch.randn((2, 75, 32), generator=gen).to(DEV)
    starts = (torch.rand((2, 75), generator=gen) < 0.06).to(DEV)
    y, _, kept = block.forward(u, starts=starts, train=True)
    want, p = _reference(block, u, starts)
    assert (y - want).abs().max() < 1e-4 * want.abs().max()
    want.backward(dy.double())
    _, grads = block.backward(dy, kept)
    for name, g in grads.items():
        w = p[name].grad
        # activations of 8 bits: a step of 2^-6 of a group's largest, uniform errors of 1/sqrt(12) of it,
        # independent from row to row, so the sums over 150 rows keep a relative error of a few percent
        off = (g.double().view_as(w) - w).norm() / w.norm()
        assert off < 0.03, (name, off.item())


def test_block_learns():
    ex = _example()
    torch.manual_seed(0)
    block = ex.GatedRecurrentBlock(model=64, channels=128)
    u = torch.randn(2, 200, 64, device=DEV).bfloat16()
    starts = torch.zeros(2, 200, dtype=torch.bool, device=DEV)
    starts[:, 90] = True
    target = torch.tanh(u.float().cumsum(1) / 16).bfloat16()
    losses = ex.train(block, u, target, starts, steps=12, rate=0.1)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_block_serves_what_it_computes_whole(dtype):
    ex = _example()
    block = ex.GatedRecurrentBlock(model=32, channels=96, dtype=dtype)
    u = torch.randn((3, 150, 32), generator=torch.Generator("cpu").manual_seed(1)).to(DEV).to(dtype)
    whole = block.forward(u)[0].float()
    rows = ex.serve(block, u, 139).float()
    # one rounding to dtype at each of the five operators
    tol = 5 * (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -20)
    assert (whole - rows).abs().max() <= tol * whole.abs().max()


def test_streams_in_slots_go_on_alone():
    ex = _example()
    block = ex.GatedRecurrentBlock(model=32, channels=64)
    u = torch.randn((5, 6, 32), generator=torch.Generator("cpu").manual_seed(2)).to(DEV).bfloat16()
    alone = block.new_state(5)
    pool = block.new_state(9)
    slots = torch.tensor([7, 2, 0, 8, 3], dtype=torch.int32, device=DEV)
    for t in range(6):
        a, b = block.step(u[:, t], alone), block.step(u[:, t], pool, slots)
        assert torch.equal(a, b)
    for whole, part in zip(pool, alone):
        assert torch.equal(whole[slots.long()], part)
