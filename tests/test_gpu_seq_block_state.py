"""The example's block on a piece of a sequence that goes on from a state (examples/gated_recurrent_block.py)."""
import pytest
import torch

from tests.test_gpu_seq_block import DEV, _example

pytestmark = pytest.mark.gpu


def _reference(block, u, state):
    """The block in float64 with autograd, from carried rows and a state that are given."""
    p = {n: v.double().clone().requires_grad_() for n, v in block.params.items()}
    rows, h = (v.double() for v in state)
    z = torch.cat([rows, u.double() @ p["w_in"].flatten(1).t()], 1)
    k = p["w_conv"].shape[1]
    out = []
    for n in range(u.shape[1]):
        y = torch.nn.functional.silu((z[:, n:n + k] * p["w_conv"].t()).sum(1) + p["b_conv"])
        gr, gi = (y @ p["w_gates"].flatten(1).t()).chunk(2, -1)
        a = torch.exp(-block.decay * torch.nn.functional.softplus(p["lam"]) * torch.sigmoid(gr))
        h = a * h + torch.sqrt(1 - a * a) * torch.sigmoid(gi) * y
        out.append(h @ p["w_out"].flatten(1).t())
    return torch.stack(out, 1), p


@pytest.mark.parametrize("t", [1, 5, 40])
def test_a_later_piece_trains_towards_the_reference_gradients(t):
    ex = _example()
    block = ex.GatedRecurrentBlock(model=32, channels=64, dtype=torch.float32)
    gen = torch.Generator("cpu").manual_seed(4)
    u0, u, dy = (torch.randn((6, n, 32), generator=gen).to(DEV) for n in (30, t, t))
    state = block.forward(u0)[1]
    y, _, kept = block.forward(u, state, train=True)
    want, p = _reference(block, u, state)
    assert (y - want).abs().max() < 1e-4 * want.abs().max()
    want.backward(dy.double())
    _, grads = block.backward(dy, kept)
    for name, g in grads.items():
        w = p[name].grad
        # activations of 8 bits: a step of 2^-6 of a group's largest, uniform errors of 1/sqrt(12) of it, of one
        # value in at most four factors of a term, 0.8% of a typical value each
        off = (g.double().view_as(w) - w).norm() / w.norm()
        assert off < 0.03, (name, off.item())
