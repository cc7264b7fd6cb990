"""Inputs, the row-by-row float64 definition and the error bounds of the gated delta rule's tests."""
import numpy as np
import torch

from tests.seq_cases import ROUND, f64, normal

U = 2.0 ** -24  # half a step of fp32, relative
# A chunk of 64 rows goes through at most four sums one after the other (k S, H r, R u or k^T u, and H's own
# substitution), each of at most 128 products and 64 rows and so of that many roundings of its terms' size.  With
# keys of length one and beta in [0, 1] a row never enlarges a state or its gradient, so errors of chunks add.
CHUNK_SUMS = 4 * (128 + 64)
# That is the worst case for one element.  Over a whole tensor roundings add as the root of their number, to terms
# that are up to 8 times the result: the bound on the 2-norm of the difference.
NORM = U * CHUNK_SUMS ** 0.5 * 8


def inputs(seed, b, t, hk, hv, dk, dv, dtype, device="cpu", slow=False):
    """q, k of length one, v, log_decay, beta in (0, 1), dy, h0, dh; step inputs have t None."""
    rows = (b,) if t is None else (b, t)

    def unit(s):
        x = normal(s, (*rows, hk, dk))
        return (x / x.norm(dim=-1, keepdim=True).clamp(min=1e-3)).to(dtype).to(device)

    g = -torch.exp(normal(seed + 3, (*rows, hv)) * (1.0 if slow else 2.0) - (5.0 if slow else 2.5)).to(device)
    beta = torch.sigmoid(normal(seed + 4, (*rows, hv))).to(device)
    state = (b, hv, dk, dv)
    return dict(q=unit(seed), k=unit(seed + 1), v=normal(seed + 2, (*rows, hv, dv), dtype, 1.0, device), log_decay=g, beta=beta,
                dy=normal(seed + 5, (*rows, hv, dv), dtype, 1.0, device), h0=normal(seed + 6, state, torch.float32, 0.3, device),
                dh=normal(seed + 7, state, torch.float32, 0.3, device))


def _norm(x):
    """2-norm of the last dimension (vectors) per (B, T, H)."""
    return x.norm(dim=-1)


def definition(x, scale=None, starts=None, use_h0=True, use_dh=True):
    """{name: (value, bound)} of every output, row by row in float64."""
    d = {n: None if t is None else t.detach().cpu().double() for n, t in x.items()}
    b, t, hv, dv = d["v"].shape
    hk, dk = d["k"].shape[2:]
    share = hv // hk
    scale = dk ** -0.5 if scale is None else scale
    q, k = (d[n].repeat_interleave(share, 2) for n in ("q", "k"))
    v, beta, decay = d["v"], d["beta"], torch.exp(d["log_decay"])
    S = d["h0"] if use_h0 else torch.zeros((b, hv, dk, dv), dtype=torch.float64)
    live = torch.ones((b, t), dtype=torch.float64) if starts is None else (~starts.cpu().bool()).double()

    def frob(s):
        return s.flatten(-2).norm(dim=-1)

    size, back = frob(S), torch.zeros((b, hv), dtype=torch.float64)
    olds, errs, us, news, y = [], [], [], [], torch.zeros_like(v)
    kept = []
    for i in range(t):
        if i % 64 == 0:
            kept.append(S)
        old = torch.where(live[:, i, None, None, None] > 0, decay[:, i, :, None, None] * S, 0.0)
        err = v[:, i] - torch.einsum("bhkv,bhk->bhv", old, k[:, i])
        u = beta[:, i, :, None] * err
        S = old + torch.einsum("bhk,bhv->bhkv", k[:, i], u)
        y[:, i] = scale * torch.einsum("bhkv,bhk->bhv", S, q[:, i])
        size = torch.maximum(size, frob(S) + _norm(err) + _norm(v[:, i]))
        olds.append(old), errs.append(err), us.append(u), news.append(S)
    last = S
    out = {"y": y, "h": last, "x": torch.stack(errs, 1) if errs else torch.zeros_like(v),
           "states": torch.stack(kept, 1) if kept else torch.zeros((b, 0, hv, dk, dv), dtype=torch.float64)}
    dy = d["dy"]
    dS = d["dh"] if use_dh else torch.zeros_like(S)
    back = torch.maximum(back, frob(dS))
    dq, dkk, dvv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, db = torch.zeros_like(beta), torch.zeros_like(beta)
    for i in range(t - 1, -1, -1):
        old, err, u, new = olds[i], errs[i], us[i], news[i]
        dS = dS + scale * torch.einsum("bhk,bhv->bhkv", q[:, i], dy[:, i])
        dq[:, i] = scale * torch.einsum("bhkv,bhv->bhk", new, dy[:, i])
        du = torch.einsum("bhkv,bhk->bhv", dS, k[:, i])
        back = torch.maximum(back, frob(dS) + _norm(du) + scale * _norm(dy[:, i]))
        dx = beta[:, i, :, None] * du
        db[:, i], dvv[:, i] = (du * err).sum(-1), dx
        dkk[:, i] = torch.einsum("bhkv,bhv->bhk", dS, u) - torch.einsum("bhkv,bhv->bhk", old, dx)
        dS = dS - torch.einsum("bhk,bhv->bhkv", k[:, i], dx)
        dg[:, i] = (dS * old).sum((-1, -2))
        dS = torch.where(live[:, i, None, None, None] > 0, decay[:, i, :, None, None] * dS, 0.0)
    fold = lambda a: a.view(b, t, hk, share, dk).sum(3)  # noqa: E731
    tol = U * CHUNK_SUMS * max(1, -(-t // 64) + 1)
    both = size * back
    rows = lambda a: a[:, None, :, None]  # noqa: E731
    bound = {"y": tol * rows(size) * scale * _norm(q)[..., None], "h": tol * size[..., None, None], "x": tol * rows(size) * torch.ones_like(v),
             "states": tol * size[:, None, :, None, None], "dv": tol * rows(back) * torch.ones_like(v),
             "dq": fold(tol * rows(size) * scale * _norm(dy)[..., None].expand_as(q)),
             "dk": fold((4 * tol * rows(both)).expand_as(k)),
             # rows' shares of a gradient of a gate differ in sign at random: 64 errors grow as their root
             "dlog_decay": 8 * tol * both[:, None].expand_as(dg), "dbeta": 2 * tol * both[:, None].expand_as(db),
             "dh0": tol * back[..., None, None]}
    out.update(dq=fold(dq), dk=fold(dkk), dv=dvv, dlog_decay=dg, dbeta=db, dh0=dS)
    return {n: (out[n], bound[n]) for n in out}


def check(got, ref, name, where=None):
    """got against (value, bound): the bound and one rounding to got's type; where: the elements that count."""
    value, bound = (a.numpy() for a in ref)
    rel, tiny = ROUND[got.dtype]
    rel = max(rel, U)
    g = f64(got)
    assert g.shape == value.shape, (name, g.shape, value.shape)
    allowed = bound + rel * (np.abs(value) + bound) + tiny
    bad = ~(np.abs(g - value) <= allowed)
    if where is not None:
        bad &= np.broadcast_to(where, bad.shape)
    if bad.any():
        k = np.unravel_index(np.argmax(np.where(bad, np.abs(g - value) / allowed, 0)), g.shape)
        raise AssertionError(f"{name}: {bad.sum()} of {bad.size} outside; at {k}: got {g[k]!r}, expected {value[k]!r} +- "
                             f"{np.broadcast_to(allowed, g.shape)[k]:.3g}")
    if where is None:
        # gradients of log decays are sums of 64 rows' shares that cancel: 8 times more
        chunks = value.shape[1] // 64 + 2 if value.ndim > 1 else 1
        far, whole = np.linalg.norm(g - value), np.linalg.norm(value)
        assert far <= (chunks * NORM * (8 if name == "dlog_decay" else 1) + rel) * whole + tiny * g.size ** 0.5, (name, far / whole)
