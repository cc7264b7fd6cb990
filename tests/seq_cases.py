"""Inputs and comparisons shared by the sequence operators' tests."""
import numpy as np
import torch

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
# largest relative error of rounding to the type (2^-p for p significand bits; fp32's is in the
# oracle's bound) and the type's smallest step
ROUND = {torch.float32: (0.0, 2.0 ** -149), torch.float16: (2.0 ** -11, 2.0 ** -24),
         torch.bfloat16: (2.0 ** -8, 2.0 ** -133)}


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def normal(seed, shape, dtype=torch.float32, scale=1.0, device="cpu"):
    gen = torch.Generator("cpu").manual_seed(seed)
    return (torch.randn(shape, generator=gen) * scale).to(dtype).to(device)


def starts_of(kind, b, t, device="cpu"):
    """None, or (B, T) bool: "some" (a few, one of them at row 0 of one batch), "all", "first"."""
    if kind is None:
        return None
    s = torch.zeros((b, t), dtype=torch.bool)
    if kind == "all":
        s[:] = True
    elif t > 0:
        s[:, 0] = True
        if kind == "some":
            s = torch.rand((b, t), generator=torch.Generator().manual_seed(b * 1009 + t)) < 0.15
            s[0, 0] = True
            s[-1, t - 1] = True
    return s.to(device)


def assert_within(got, ref, bound, what):
    """|got - ref| within the oracle's bound on fp32 arithmetic plus the rounding to got's type."""
    rel, tiny = ROUND[got.dtype]
    g = f64(got)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    # what is rounded may itself be off by the bound
    allowed = bound + rel * (np.abs(ref) + bound) + tiny
    bad = ~(np.abs(g - ref) <= allowed)
    if bad.any():
        k = np.unravel_index(np.argmax(np.where(bad, np.abs(g - ref) / allowed, 0)), g.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside; at {k}: got {g[k]!r}, expected {ref[k]!r} "
                             f"+- {allowed[k]:.3g}")


def scan_inputs(seed, b, t, c, dtype, device="cpu", h0=True, wide_gates=False):
    """x, gate_r, gate_i (column slices of one projection), lam, h0; wide_gates reaches both ends of the gates."""
    x = normal(seed, (b, t, c), dtype, 1.0, device)
    both = normal(seed + 1, (b, t, 2 * c), dtype, 6.0 if wide_gates else 1.5, device)
    lam = normal(seed + 2, (c,), torch.float32, 2.0 if wide_gates else 1.0, device) - (2.0 if wide_gates else 5.0)
    h = normal(seed + 3, (b, c), torch.float32, 1.0, device) if h0 else None
    return x, both[..., :c], both[..., c:], lam, h
