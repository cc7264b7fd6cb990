"""A gated delta block on the library: one training step, and serving, a prompt in pieces followed
by one row at a time.

    u (B, T, C_model) --1x1 convolution--> p --causal depthwise convolution, silu--> q, k, v
    gates = 1x1 convolution of u (2 heads),  h = gated delta rule of q, k (to length one), v under them
    y = 1x1 convolution of silu(norm of h, head by head)

The 1x1 convolutions are those of gated_recurrent_block.py.

    python examples/gated_delta_block.py        # on a GPU: trains a few steps, then serves
"""
import os
import sys

import torch

sys.path[:0] = [os.path.dirname(os.path.abspath(__file__)), os.path.dirname(os.path.dirname(os.path.abspath(__file__)))]
import implicit_gemm_conv_amd as igc  # noqa: E402
from gated_recurrent_block import project, project_bwd  # noqa: E402


def unit(x):
    """x by its length, head by head, and 1 / length."""
    inv = torch.rsqrt(x.float().square().sum(-1, keepdim=True) + 1e-6)
    return (x.float() * inv).to(x.dtype), inv


def unit_bwd(dy, x, inv):
    n = x.float() * inv
    return (inv * (dy.float() - n * (n * dy.float()).sum(-1, keepdim=True))).to(x.dtype)


class GatedDeltaBlock:
    """Parameters in fp32; the projections and the convolution run in `dtype`."""

    def __init__(self, model, key_heads, heads, dk, dv, taps=4, dtype=torch.bfloat16, device="cuda:0", seed=0):
        gen = torch.Generator("cpu").manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(shape, generator=gen) * scale).to(device)

        self.dtype, self.hk, self.hv, self.dk, self.dv = dtype, key_heads, heads, dk, dv
        self.sizes = [key_heads * dk, key_heads * dk, heads * dv]
        c = sum(self.sizes)
        self.params = {
            "w_in": normal(c, 1, 1, model, scale=model ** -0.5),
            "w_conv": normal(c, taps, scale=taps ** -0.5),
            "w_gates": normal(2 * heads, 1, 1, model, scale=model ** -0.5),
            "rate": torch.linspace(-4, 0, heads, device=device),   # log of the decay's rate
            "w_norm": torch.ones(heads * dv, device=device),
            "b_norm": torch.zeros(heads * dv, device=device),
            "w_out": normal(model, 1, 1, heads * dv, scale=(heads * dv) ** -0.5),
        }

    def _weights(self):
        keep = ("rate", "w_norm", "b_norm")
        return {n: p if n in keep else p.to(self.dtype) for n, p in self.params.items()}

    def new_state(self, streams):
        """Carried rows of the convolution and states of the delta rule, one slot a stream."""
        c, k = self.params["w_conv"].shape
        device = self.params["rate"].device
        return (torch.zeros((streams, k - 1, c), dtype=self.dtype, device=device),
                torch.zeros((streams, self.hv, self.dk, self.dv), device=device))

    def _heads(self, x):
        q, k, v = x.split(self.sizes, -1)
        return q.unflatten(-1, (self.hk, self.dk)), k.unflatten(-1, (self.hk, self.dk)), v.unflatten(-1, (self.hv, self.dv))

    def _gates(self, z):
        """log_decay and beta from the projected gates."""
        a, b = z.float().chunk(2, -1)
        return -torch.exp(self.params["rate"]) * torch.nn.functional.softplus(a), torch.sigmoid(b).contiguous()

    def forward(self, u, state=None, starts=None, train=False):
        """y, the state after the last row, and with train what backward needs.  Training takes `state`
        as given: backward returns no gradient of it."""
        w = self._weights()
        rows, h0 = state if state is not None else (None, None)
        p, z = project(u, w["w_in"]), project(u, w["w_gates"])
        f = igc.seq_conv(p, w["w_conv"], activation="silu", state=rows, starts=starts)
        q, k, v = self._heads(f.y)
        (qn, qi), (kn, ki) = unit(q), unit(k)
        log_decay, beta = self._gates(z)
        s = igc.delta_rule(qn, kn, v, log_decay, beta, h0=h0, starts=starts, train=train)
        h = s.y.reshape(-1, self.hv * self.dv)
        n = igc.group_norm(h, self.hv, weight=w["w_norm"], bias=w["b_norm"], activation="silu")
        out = n.y.view(*u.shape[:2], -1)
        kept = (u, p, z, f.y, (qn, kn, qi, ki), log_decay, beta, s.states, h, n, out, rows, starts) if train else None
        return project(out, w["w_out"]), (f.state, s.h), kept

    def backward(self, dy, kept):
        """Gradients of the parameters and of u."""
        w = self._weights()
        u, p, z, x, (qn, kn, qi, ki), log_decay, beta, states, h, n, out, rows, starts = kept
        q, k, v = self._heads(x)
        g = {}
        dout, g["w_out"] = project_bwd(dy, out, w["w_out"])
        norm = igc.group_norm_bwd(dout.reshape(h.shape), h, self.hv, n.mean, n.rstd, weight=w["w_norm"], bias=w["b_norm"],
                                  activation="silu")
        g["w_norm"], g["b_norm"] = norm.dweight, norm.dbias
        s = igc.delta_rule_bwd(norm.dx.view(v.shape), qn, kn, v, log_decay, beta, states, starts=starts)
        a, _ = z.float().chunk(2, -1)
        da = s.dlog_decay * -torch.exp(w["rate"]) * torch.sigmoid(a)
        g["rate"] = (s.dlog_decay * log_decay).sum((0, 1))
        dz = torch.cat([da, s.dbeta * beta * (1 - beta)], -1).to(self.dtype)
        dx = torch.cat([t.flatten(-2) for t in (unit_bwd(s.dq, q, qi), unit_bwd(s.dk, k, ki), s.dv)], -1)
        c = igc.seq_conv_bwd(dx, p, w["w_conv"], activation="silu", state=rows, starts=starts)
        g["w_conv"] = c.dw
        du, g["w_in"] = project_bwd(c.dx, u, w["w_in"])
        du_gates, g["w_gates"] = project_bwd(dz, u, w["w_gates"])
        return du + du_gates, g

    def step(self, u, state, slots=None):
        """One row of each of many streams: u (B, C_model), states updated in place."""
        w = self._weights()
        rows, h = state
        p, z = (project(u[:, None], w[name])[:, 0] for name in ("w_in", "w_gates"))
        x, _ = igc.seq_conv_step(p, w["w_conv"], rows, activation="silu", slots=slots)
        q, k, v = self._heads(x)
        y, _ = igc.delta_rule_step(unit(q)[0], unit(k)[0], v, *self._gates(z), h, slots=slots)
        n = igc.group_norm(y.flatten(1), self.hv, weight=w["w_norm"], bias=w["b_norm"], activation="silu")
        return project(n.y[:, None], w["w_out"])[:, 0]


def serve(block, u, prompt):
    """The first `prompt` rows in two pieces, the others one by one; all outputs."""
    cut = prompt // 2
    y1, state, _ = block.forward(u[:, :cut])
    y2, state, _ = block.forward(u[:, cut:prompt], state)
    rows = [block.step(u[:, t].contiguous(), state) for t in range(prompt, u.shape[1])]
    return torch.cat([y1, y2, torch.stack(rows, 1)], 1)


def main():
    torch.manual_seed(0)
    block = GatedDeltaBlock(model=256, key_heads=2, heads=4, dk=64, dv=64)
    u = torch.randn(4, 1024, 256, device="cuda:0").bfloat16()
    starts = torch.rand(4, 1024, device="cuda:0") < 0.005
    target = torch.tanh(u.float().cumsum(1) / 32)
    for i in range(20):
        y, _, kept = block.forward(u, starts=starts, train=True)
        error = y.float() - target
        _, grads = block.backward((2 / error.numel() * error * 1024).bfloat16(), kept)   # scaled: dy is 16-bit
        for name, g in grads.items():
            block.params[name] -= 0.3 / 1024 * g.view_as(block.params[name])
        if i in (0, 19):
            print(f"step {i}: mean squared error {error.square().mean().item():.4f}")
    whole = block.forward(u[:, :96])[0]
    rows = serve(block, u[:, :96], 64)
    print(f"row by row against the whole sequence: largest difference {(whole - rows).abs().max().item():.4f}")


if __name__ == "__main__":
    main()
