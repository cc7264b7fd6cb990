"""A gated recurrent block on the library: one training step with its activations kept in 8 bits,
and serving, a prompt in pieces followed by one row at a time.

    u (B, T, C_model) --1x1 convolution--> p --causal depthwise convolution, silu--> x
    gates = 1x1 convolution of x (2 C channels),  h = gated recurrence of x under the gates
    y = 1x1 convolution of h

The 1x1 convolutions are conv_fwd / conv_bwd_data of the library on (B, 1, T, C) tensors; their
weights' gradients are one matrix product each.

    python examples/gated_recurrent_block.py        # on a GPU: trains a few steps, then serves
"""
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import implicit_gemm_conv_amd as igc  # noqa: E402


def project(x, w):
    """(B, T, C_in) by w (C_out, 1, 1, C_in)."""
    return igc.conv_fwd(x[:, None], w)[:, 0]


def project_bwd(dy, x, w):
    """Gradients of project with respect to x and w (fp32)."""
    dy = dy.contiguous()
    dx = igc.conv_bwd_data(dy[:, None], w, (x.shape[0], 1, *x.shape[1:]))[:, 0]
    dw = dy.flatten(0, 1).t().float() @ x.flatten(0, 1).float()
    return dx, dw.view(w.shape)


class GatedRecurrentBlock:
    """Parameters in fp32; the projections and the convolution run in `dtype`."""

    def __init__(self, model, channels, taps=4, dtype=torch.bfloat16, device="cuda:0", seed=0):
        gen = torch.Generator("cpu").manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(shape, generator=gen) * scale).to(device)

        self.dtype, self.decay = dtype, 8.0
        self.params = {
            "w_in": normal(channels, 1, 1, model, scale=model ** -0.5),
            "w_conv": normal(channels, taps, scale=taps ** -0.5),
            "b_conv": torch.zeros(channels, device=device),
            "w_gates": normal(2 * channels, 1, 1, channels, scale=channels ** -0.5),
            # decays of 0.9 to 0.999 a row where the gate is open
            "lam": torch.log(torch.expm1(-torch.log(torch.linspace(0.9, 0.999, channels)) / 8.0)).to(device),
            "w_out": normal(model, 1, 1, channels, scale=channels ** -0.5),
        }

    def _weights(self):
        return {n: p if n == "lam" else p.to(self.dtype) for n, p in self.params.items()}

    def new_state(self, streams):
        """Carried rows of the convolution and state of the recurrence, one slot a stream."""
        c, k = self.params["w_conv"].shape
        device = self.params["lam"].device
        return (torch.zeros((streams, k - 1, c), dtype=self.dtype, device=device),
                torch.zeros((streams, c), device=device))

    def forward(self, u, state=None, starts=None, train=False):
        """y, the state after the last row, and with train what backward needs (the carried rows of
        `state` among it, not a copy of them).  Training takes `state` as given: backward returns
        no gradient of it, so none goes back into the piece before."""
        w = self._weights()
        rows, h0 = state if state is not None else (None, None)
        p = project(u, w["w_in"])
        f = igc.seq_conv(p, w["w_conv"], bias=w["b_conv"], activation="silu", state=rows, starts=starts, keep8=train)
        gate_r, gate_i = project(f.y, w["w_gates"]).chunk(2, dim=-1)
        s = igc.gated_scan(f.y, gate_r, gate_i, w["lam"], decay=self.decay, h0=h0, starts=starts, train=train,
                           keep8=train)
        kept = (igc.pack8(u), f.kept, s.kept, s.states, igc.pack8(s.y), rows, starts) if train else None
        return project(s.y, w["w_out"]), (f.state, s.h), kept

    def backward(self, dy, kept):
        """Gradients of the parameters and of u, from activations that were kept in 8 bits."""
        w = self._weights()
        u8, p8, scan8, states, h8, rows, starts = kept
        g = {}
        dh, g["w_out"] = project_bwd(dy, igc.unpack8(h8), w["w_out"])
        s = igc.gated_scan_bwd(dh, *scan8, w["lam"], states, decay=self.decay, starts=starts)
        g["lam"] = s.dlam
        x = igc.unpack8(scan8[0])
        dgates = torch.cat([s.dgate_r, s.dgate_i], dim=-1)
        dx, g["w_gates"] = project_bwd(dgates, x, w["w_gates"])
        c = igc.seq_conv_bwd(s.dx + dx, p8, w["w_conv"], bias=w["b_conv"], activation="silu", state=rows,
                             starts=starts)
        g["w_conv"], g["b_conv"] = c.dw, c.dbias
        du, g["w_in"] = project_bwd(c.dx, igc.unpack8(u8), w["w_in"])
        return du, g

    def step(self, u, state, slots=None):
        """One row of each of many streams: u (B, C_model), states updated in place."""
        w = self._weights()
        rows, h = state
        x, _ = igc.seq_conv_step(project(u[:, None], w["w_in"])[:, 0], w["w_conv"], rows, bias=w["b_conv"],
                                 activation="silu", slots=slots)
        gate_r, gate_i = project(x[:, None], w["w_gates"])[:, 0].chunk(2, dim=-1)
        y, _ = igc.gated_scan_step(x, gate_r, gate_i, w["lam"], h, decay=self.decay, slots=slots)
        return project(y[:, None], w["w_out"])[:, 0]


def train(block, u, target, starts, steps, rate):
    """Plain gradient descent on the mean squared error; the losses."""
    losses = []
    for _ in range(steps):
        y, _, kept = block.forward(u, starts=starts, train=True)
        error = y.float() - target.float()
        losses.append(error.square().mean())
        _, grads = block.backward((2 / error.numel() * error * 1024).to(block.dtype), kept)   # scaled: dy is 16-bit
        for name, g in grads.items():
            block.params[name] -= rate / 1024 * g.view_as(block.params[name])
    return torch.stack(losses).tolist()


def serve(block, u, prompt):
    """The first `prompt` rows in two pieces, the others one by one; all outputs."""
    cut = prompt // 2
    y1, state, _ = block.forward(u[:, :cut])
    y2, state, _ = block.forward(u[:, cut:prompt], state)
    rows = [block.step(u[:, t], state) for t in range(prompt, u.shape[1])]
    return torch.cat([y1, y2, torch.stack(rows, 1)], 1)


def main():
    torch.manual_seed(0)
    block = GatedRecurrentBlock(model=256, channels=512)
    u = torch.randn(4, 1024, 256, device="cuda:0").bfloat16()
    starts = torch.rand(4, 1024, device="cuda:0") < 0.005
    target = torch.tanh(u.float().cumsum(1) / 32).bfloat16()
    losses = train(block, u, target, starts, steps=40, rate=0.3)
    print(f"mean squared error {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")
    whole = block.forward(u[:, :96])[0]
    rows = serve(block, u[:, :96], 64)
    print(f"row by row against the whole sequence: largest difference {(whole - rows).abs().max().item():.4f}")


if __name__ == "__main__":
    main()
