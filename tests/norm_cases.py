"""Inputs, the float64 definition and the error bounds of the group norm's tests."""
import numpy as np
import torch

from tests.seq_cases import ROUND, f64, normal

U = 2.0 ** -24  # half a step of fp32, relative
# Roundings that one sum of the kernels adds at most at the tests' sizes: a thread adds up to 32 values, the
# workgroup's rows and lanes join in up to 8 steps of 3 roundings, a group's channels in as many; fp64 beyond.
SUM = 96


def inputs(seed, n, p, c, dtype, device="cpu", offset=0.25, params=torch.float32):
    """x with channels of different scale and offset, dy, weight, bias."""
    x = normal(seed, (n, p, c)) * torch.exp2(normal(seed + 1, (c,)) * 0.7) + normal(seed + 2, (c,)) * 0.5 + offset
    w, b = None, None
    if params is not None:
        w, b = (1 + normal(seed + 3, (c,)) * 0.3).to(params).to(device), normal(seed + 4, (c,), params, 0.3, device)
    return x.to(dtype).to(device), normal(seed + 5, (n, p, c), dtype, 1.0, device), w, b


def definition(x, dy, groups, w, b, act, eps=1e-5):
    """{name: (value, bound on fp32 arithmetic)} of every output, in float64 from the formula."""
    x, dy = f64(x), f64(dy)
    n, p, c = x.shape
    cg = c // groups
    w = np.ones(c) if w is None else f64(w)
    b = np.zeros(c) if b is None else f64(b)

    def mean(a):
        return a.reshape(n, p, groups, cg).mean((1, 3)) if p else np.zeros((n, groups))

    def wide(a):
        return np.repeat(a, cg, 1)[:, None]

    mu = mean(x)
    top = np.abs(x).reshape(n, p, groups, cg).max((1, 3)) if p else np.zeros((n, groups))
    far = np.abs(x - wide(mu))
    var = mean((x - wide(mu)) ** 2)
    rstd = 1 / np.sqrt(var + eps)
    e_mu = U * (2 * top + SUM * mean(far))
    # squares about a mean that is off: twice the distance times the mean's error, and the sum's roundings
    e_var = SUM * U * var + 2 * np.sqrt(var) * e_mu + e_mu ** 2
    e_rstd = rstd * (0.5 * e_var / (var + eps) + 4 * U)
    hat = (x - wide(mu)) * wide(rstd)
    e_hat = far * wide(e_rstd) + wide(rstd * e_mu) + 3 * U * np.abs(hat) + U * wide(rstd * top)
    z = hat * w + b
    e_z = e_hat * np.abs(w) + 2 * U * (np.abs(hat * w) + np.abs(b))
    out = {"mean": (mu, e_mu), "rstd": (rstd, e_rstd)}
    if act == "silu":
        s = 1 / (1 + np.exp(-z))
        d = s * (1 + z * (1 - s))
        # the exponential's argument is rounded: an error of |z| half steps, and four more roundings
        y, e_y = z * s, 1.1 * e_z + U * np.abs(z * s) * (np.abs(z) * (1 - s) * 2 + 6)
        e_d = 0.5 * e_z + U * (np.abs(z) * s * (1 - s) * 2 * (1 + np.abs(z)) + 8 * (s + np.abs(z) * s))
    else:
        y, e_y, d, e_d = z, e_z, np.ones_like(z), np.zeros_like(z)
    out["y"] = (y, e_y)
    dz = dy * d
    e_dz = np.abs(dy) * e_d + U * np.abs(dz)
    dh, e_dh = dz * w, e_dz * np.abs(w) + U * np.abs(dz * w)
    m1, m2 = mean(dh), mean(dh * hat)
    e1 = mean(e_dh) + SUM * U * mean(np.abs(dh))
    e2 = mean(e_dh * np.abs(hat) + np.abs(dh) * e_hat) + SUM * U * mean(np.abs(dh * hat))
    inner = dh - wide(m1) - hat * wide(m2)
    e_in = e_dh + wide(e1) + np.abs(hat) * wide(e2) + e_hat * wide(np.abs(m2)) \
        + 4 * U * (np.abs(dh) + wide(np.abs(m1)) + np.abs(hat) * wide(np.abs(m2)))
    out["dx"] = (wide(rstd) * inner, wide(rstd) * e_in + np.abs(inner) * wide(e_rstd))
    out["dweight"] = ((dz * hat).sum((0, 1)), (e_dz * np.abs(hat) + np.abs(dz) * e_hat + SUM * U * np.abs(dz * hat)).sum((0, 1)))
    out["dbias"] = (dz.sum((0, 1)), (e_dz + SUM * U * np.abs(dz)).sum((0, 1)))
    return out


def check(got, ref, name):
    """got against (value, bound): the bound, one rounding to got's type, and its smallest step."""
    value, bound = ref
    rel, tiny = ROUND[got.dtype]
    rel = max(rel, U)
    g = f64(got).reshape(value.shape)
    allowed = bound + rel * (np.abs(value) + bound) + tiny
    bad = ~(np.abs(g - value) <= allowed)
    if bad.any():
        k = np.unravel_index(np.argmax(np.where(bad, np.abs(g - value) / allowed, 0)), g.shape)
        raise AssertionError(f"{name}: {bad.sum()} of {bad.size} outside; at {k}: got {g[k]!r}, expected {value[k]!r} +- {allowed[k]:.3g}")
