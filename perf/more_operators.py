"""The gated delta rule and the channels-last group norm of this library as measured cases.

``own`` False computes each operator in its plain form, elementary torch operations in float32
(sums of log decays in float64, because their differences are what is exponentiated); ``own`` True
makes the calls a user makes of ``implicit_gemm_conv_amd``.  Formulas:

delta rule    per batch row b and value head h (its key head is h // (heads of v / heads of k)),
              with a state S of (Dk, Dv), and a_t = exp(log_decay_t):
              S' = a_t S_{t-1}   (S_{t-1} absent at a row that ``starts`` marks)
              S_t = S' + k_t (beta_t (v_t - S'^T k_t))^T,   y_t = scale * S_t^T q_t
group norm    x (N, ..., C), groups of C / G neighbouring channels; mean and variance (biased) over
              the positions and channels of each (n, group):
              z = (x - mean) / sqrt(var + eps) * weight + bias,   y = z or z * sigmoid(z)

The plain delta rule takes 64 rows at a time.  With G the sums of log decays inside a chunk,
D_ij = exp(G_i - G_j) for j <= i in the same sequence and L = D * (k k^T) below the diagonal, the
rows' corrections u solve (I + beta L) u = beta (v - exp(G) k S), so that
y = scale * (exp(G) q S + (D * q k^T) u) and S moves on to exp(G_end) S + (exp(G_end - G) k)^T u.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
CHUNK = 64


def listed():
    return [
        # Serving, one token of one small stream through the delta rule: the smallest call.
        dict(name="delta_step_b1", op="delta_step", b=1, hk=4, hv=4, dk=64, dv=64, dtype="fp16"),
        # Serving, a full batch of streams, two value heads a key head: the states' bytes count.
        dict(name="delta_step_b128", op="delta_step", b=128, hk=8, hv=16, dk=128, dv=128, dtype="bf16"),
        # A long prompt, one sequence of an odd number of rows, continued from an earlier piece.
        dict(name="delta_prefill_long", op="delta_prefill", b=1, t=16387, hk=8, hv=16, dk=128, dv=128, state=True,
             starts=False, dtype="bf16"),
        # A training step's share of one layer, sequences packed end to end: the largest.
        dict(name="delta_train", op="delta_train", b=4, t=4096, hk=16, hv=16, dk=128, dv=128, state=False, starts=True,
             dtype="bf16"),
        # Float32 training with odd head sizes and an odd length, shared key heads, a carried state.
        dict(name="delta_train_odd_f32", op="delta_train", b=2, t=777, hk=3, hv=6, dk=65, dv=100, state=True,
             starts=True, dtype="fp32"),
        # Many short sequences.
        dict(name="delta_train_short", op="delta_train", b=64, t=100, hk=4, hv=4, dk=64, dv=64, state=False,
             starts=False, dtype="fp16"),
        # Serving, the heads of a few tokens normalised each: latency.
        dict(name="norm_tokens", op="norm", n=8, p=1, c=2048, groups=16, act="silu", params="same", dtype="bf16"),
        # Inference, the volume of the 3x3x3 layers, groups of 4 channels.
        dict(name="norm_volume", op="norm", n=4, p=32 ** 3, c=128, groups=32, act="silu", params="same", dtype="fp16"),
        # Training, the images of the 3x3 layer of 256 channels.
        dict(name="norm_train_image", op="norm_train", n=32, p=56 * 56, c=256, groups=32, act="silu", params="same",
             dtype="bf16"),
        # Training, the heads of a batch of sequences, each row a group for each head.
        dict(name="norm_train_heads", op="norm_train", n=4 * 4096, p=1, c=2048, groups=16, act="silu", params="fp32",
             dtype="bf16"),
        # Training of the 65-channel volume in float32: groups of 13 channels, no whole 16 bytes.
        dict(name="norm_train_c65_f32", op="norm_train", n=4, p=32 ** 3, c=65, groups=5, act="none", params="same",
             dtype="fp32"),
        # One large volume as one group: every value in one mean, batch 1.
        dict(name="norm_train_one_group", op="norm_train", n=1, p=64 ** 3, c=64, groups=1, act="none", params="fp32",
             dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    op = rng.choice(["delta_step", "delta_prefill", "delta_train", "delta_train", "norm", "norm_train", "norm_train"])
    if op.startswith("delta"):
        hk = rng.choice([1, 2, 3, 4, 8, 16])
        hv = hk * rng.choice([1, 1, 2, 4])
        dk, dv = (rng.choice([16, 32, 64, 64, 96, 128, 128, _log(rng, 1, 128)]) for _ in range(2))
        dv = dv * rng.choice([1, 1, 1, 2])
        case = dict(op=op, hk=hk, hv=hv, dk=dk, dv=dv, dtype=dtype)
        while True:
            case["b"] = _log(rng, 1, 256 if op == "delta_step" else 64)
            if op == "delta_step":
                if case["b"] * hv * dk * dv <= 1 << 25:
                    return case
                continue
            case["t"] = _log(rng, 1, 16384)
            # whole problems of at most the listed training case
            if case["b"] * case["t"] * hv * max(dk, 32) * max(dv, 32) <= 1 << 31:
                break
        case.update(state=rng.random() < 0.5, starts=rng.random() < 0.4)
        return case
    while True:
        cg, groups = _log(rng, 1, 256), rng.choice([1, 2, 4, 5, 8, 16, 32, 32])
        case = dict(op=op, n=_log(rng, 1, 64), p=_log(rng, 1, 65536), c=cg * groups, groups=groups)
        if rng.random() < 0.25:
            case.update(n=_log(rng, 1, 16384), p=1)
        if case["c"] <= 4096 and case["c"] > 1 and case["p"] * cg > 1 and case["n"] * case["p"] * case["c"] <= 1 << 24:
            break
    case.update(act=rng.choice(["none", "silu"]), params=rng.choice(["same", "fp32", "none"]), dtype=dtype)
    return case


# ---- inputs -------------------------------------------------------------------------------------


def _delta_inputs(case, seed, device):
    gen = torch.Generator(device).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    b, hk, hv, dk, dv = (case[n] for n in ("b", "hk", "hv", "dk", "dv"))
    rows = (b,) if case["op"] == "delta_step" else (b, case["t"])

    def normal(*shape, to=dt):
        return torch.randn(shape, generator=gen, device=device).to(to)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=device)

    s = {"scale": dk ** -0.5}
    # q, k and v are column slices of one projection; a model brings q and k to length one
    all_ = normal(*rows, 2 * hk * dk + hv * dv, to=torch.float32)
    qk = all_[..., :2 * hk * dk].view(*rows, 2 * hk, dk)
    qk /= qk.square().sum(-1, keepdim=True).sqrt() + 1e-6
    all_ = all_.to(dt)
    s["q"] = all_[..., :hk * dk].view(*rows, hk, dk)
    s["k"] = all_[..., hk * dk:2 * hk * dk].view(*rows, hk, dk)
    s["v"] = all_[..., 2 * hk * dk:].view(*rows, hv, dv)
    # each head has its own memory, from a row or two to a thousand
    s["log_decay"] = -torch.exp(uniform(hv) * 6.5 - 7.0) * (0.2 + 1.6 * uniform(*rows, hv))
    s["beta"] = torch.sigmoid(normal(*rows, hv, to=torch.float32))
    s["state"] = normal(b, hv, dk, dv, to=torch.float32) * 0.3 if case.get("state", True) else None
    if case["op"] != "delta_step":
        s["starts"] = None
        if case["starts"]:
            # sequences of about a fifth of the length, packed end to end
            s["starts"] = uniform(b, case["t"]) < 5.0 / case["t"]
            s["starts"][:, 0] |= uniform(b) < 0.5
    if case["op"] == "delta_train":
        s["dy"] = normal(*rows, hv, dv)
        s["dlast"] = normal(b, hv, dk, dv, to=torch.float32) * 0.3 if case["state"] else None
    return s


def _norm_inputs(case, seed, device):
    gen = torch.Generator(device).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    n, p, c = case["n"], case["p"], case["c"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=device)

    # channels of a layer differ in scale and are not centred
    x = normal(n, p, c) * torch.exp2(normal(c) * 0.7) + normal(c) * 0.5 + 0.25
    s = {"x": x.to(dt), "groups": case["groups"], "eps": 1e-5, "weight": None, "bias": None}
    if case["params"] != "none":
        par = torch.float32 if case["params"] == "fp32" else dt
        s["weight"], s["bias"] = (1 + normal(c) * 0.3).to(par), (normal(c) * 0.3).to(par)
    if case["op"] == "norm_train":
        s["dy"] = normal(n, p, c).to(dt)
    return s


def _inputs(case, seed, device):
    s = (_delta_inputs if case["op"].startswith("delta") else _norm_inputs)(case, seed, device)
    s["case"] = case
    return s


def prepare(case, seed):
    s = _inputs(case, seed, "cuda")
    if case["op"] == "delta_step":
        # a server keeps two buffers for the streams' states and swaps them
        s["next"] = torch.empty_like(s["state"])
    return s


# ---- plain forms, float32 ---------------------------------------------------------------------


def _unit_inverse(a):
    """(I + a)^-1 for strictly lower triangular a (..., 64, 64): diagonal blocks of 1, 2, 4, ... rows."""
    n, s = a.shape[-1], 1
    x = torch.eye(n, dtype=a.dtype, device=a.device).expand(a.shape).clone()
    while s < n:
        first = torch.arange(0, n, 2 * s, device=a.device)[:, None] + torch.arange(s, device=a.device)
        up, low = first, first + s
        x[..., low[:, :, None], up[:, None]] = -(x[..., low[:, :, None], low[:, None]]
                                                 @ a[..., low[:, :, None], up[:, None]]
                                                 @ x[..., up[:, :, None], up[:, None]])
        s *= 2
    return x


def _chunks(x, heads):
    """(B, T, H, ...) as float32 (B, heads, chunks, 64, ...), rows past T zero."""
    b, t, h = x.shape[:3]
    n = -(-t // CHUNK)
    x = torch.nn.functional.pad(x.float(), (0, 0) * (x.dim() - 2) + (0, n * CHUNK - t))
    x = x.reshape(b, n, CHUNK, *x.shape[2:]).movedim(3, 1)
    return x if h == heads else x.repeat_interleave(heads // h, 1)


def _rows(x, t):
    """(B, H, chunks, 64, ...) as (B, T, H, ...)."""
    x = x.movedim(1, 3)
    return x.reshape(x.shape[0], -1, *x.shape[3:])[:, :t]


def _delta_parts(q, k, v, log_decay, beta, starts):
    """What the chunks of the delta rule hold that no state enters."""
    hv = v.shape[2]
    q, k, v = (_chunks(x, hv) for x in (q, k, v))
    beta = _chunks(beta, hv)[..., None]
    g = torch.cumsum(_chunks(log_decay, hv).double(), -1)
    after = torch.arange(CHUNK, device=q.device)
    same = after[:, None] >= after
    from_state, to_state = torch.ones_like(g, dtype=torch.bool), torch.ones_like(g, dtype=torch.bool)
    if starts is not None:
        seq = torch.cumsum(_chunks(starts[:, :, None], 1), -1)          # (B, 1, chunks, 64)
        same = same & (seq[..., :, None] == seq[..., None, :])
        from_state, to_state = (seq == 0).expand_as(g), (seq == seq[..., -1:]).expand_as(g)
    decay = torch.exp(torch.where(same, g[..., :, None] - g[..., None, :], -math.inf)).float()
    p = {"q": q, "k": k, "v": v, "beta": beta, "decay": decay}
    p["enter"] = torch.where(from_state, torch.exp(g), 0.0).float()[..., None]
    p["leave"] = torch.where(to_state, torch.exp(g[..., -1:] - g), 0.0).float()[..., None]
    p["lower"] = torch.tril(decay * (k @ k.transpose(-1, -2)), -1)
    p["read"] = decay * (q @ k.transpose(-1, -2))
    p["solve"] = _unit_inverse(beta * p["lower"])
    return p


def _plain_delta(s):
    v, starts, t = s["v"], s.get("starts"), s["v"].shape[1]
    p = _delta_parts(s["q"], s["k"], v, s["log_decay"], s["beta"], starts)
    b, hv, n = p["k"].shape[:3]
    state = s["state"]
    if state is None:
        state = torch.zeros((b, hv, p["k"].shape[-1], v.shape[-1]), device=v.device)
    u0 = p["solve"] @ (p["beta"] * p["v"])
    w = p["solve"] @ (p["beta"] * p["enter"] * p["k"])
    out_k = (p["leave"] * p["k"]).transpose(-1, -2)
    us, states = [], []
    for c in range(n):
        states.append(state)
        u = u0[:, :, c] - w[:, :, c] @ state
        us.append(u)
        state = p["enter"][:, :, c, -1:] * state + out_k[:, :, c] @ u
    if n:
        p["u"], p["states"] = torch.stack(us, 2), torch.stack(states, 2)
        y = _rows(s["scale"] * (p["enter"] * (p["q"] @ p["states"]) + p["read"] @ p["u"]), t)
    else:
        y = torch.zeros(v.shape, device=v.device)
    return y, state, p


def _fold(x, like):
    """Gradients of the value heads (B, T, Hv, D), added over the heads that share one of like's."""
    b, t, h, d = like.shape
    return x.reshape(b, t, h, -1, d).sum(3)


def _plain_delta_bwd(s, p, last):
    scale, t, hv = s["scale"], s["v"].shape[1], s["v"].shape[2]
    q, k, beta, enter, leave, u, states = (p[n] for n in ("q", "k", "beta", "enter", "leave", "u", "states"))
    dy = scale * _chunks(s["dy"], hv)
    ds = torch.zeros_like(last) if s["dlast"] is None else s["dlast"]
    du0 = p["read"].transpose(-1, -2) @ dy
    solve_t, k_out, q_in = p["solve"].transpose(-1, -2), leave * k, (enter * q).transpose(-1, -2)
    k_in = (enter * k).transpose(-1, -2)
    dxs, dss = [], []
    for c in range(u.shape[2] - 1, -1, -1):
        dss.append(ds)
        du = solve_t[:, :, c] @ (du0[:, :, c] + k_out[:, :, c] @ ds)
        dxs.append(du)
        ds = enter[:, :, c, -1:] * ds + q_in[:, :, c] @ dy[:, :, c] - k_in[:, :, c] @ (beta[:, :, c] * du)
    du, dss = torch.stack(dxs[::-1], 2), torch.stack(dss[::-1], 2)
    dx = beta * du
    x = p["v"] - enter * (k @ states) - p["lower"] @ u
    dbeta = (du * x).sum(-1)
    d_read = (dy @ u.transpose(-1, -2)) * p["decay"]
    d_low = -torch.tril((dx @ u.transpose(-1, -2)) * p["decay"], -1)
    dq = enter * (dy @ states.transpose(-1, -2)) + d_read @ k
    dk_row = -enter * (dx @ states.transpose(-1, -2)) + d_low @ k
    dk_col = leave * (u @ dss.transpose(-1, -2)) + d_read.transpose(-1, -2) @ q + d_low.transpose(-1, -2) @ k
    dg = (dq * q + dk_row * k - dk_col * k).sum(-1).double()
    after = torch.cat([states[:, :, 1:], last[:, :, None]], 2)
    dg[..., -1] += (after * dss).sum((-1, -2))
    dg = torch.flip(torch.cumsum(torch.flip(dg, [-1]), -1), [-1])
    if s["starts"] is not None:
        # the decay of a row at a start acts on nothing
        dg = torch.where(_chunks(s["starts"][:, :, None], 1) != 0, 0.0, dg)
    return (_fold(_rows(dq, t), s["q"]), _fold(_rows(dk_row + dk_col, t), s["k"]), _rows(dx, t),
            _rows(dg, t).float(), _rows(dbeta, t), ds)


def _plain_norm(s):
    x, groups = s["x"], s["groups"]
    n, p, c = x.shape
    v = x.float().view(n, p, groups, c // groups)
    mean = v.mean((1, 3), keepdim=True)
    v = v - mean
    rstd = torch.rsqrt(v.square().mean((1, 3), keepdim=True) + s["eps"])
    hat = (v * rstd).view(n, p, c)
    z = hat if s["weight"] is None else hat * s["weight"].float() + s["bias"].float()
    y = z * torch.sigmoid(z) if s["case"]["act"] == "silu" else z
    return y, mean.view(n, groups), rstd.view(n, groups), hat, z


def _plain_norm_bwd(s, rstd, hat, z):
    n, p, c = hat.shape
    groups = s["groups"]
    dz = s["dy"].float()
    if s["case"]["act"] == "silu":
        sig = torch.sigmoid(z)
        dz = dz * sig * (1 + z * (1 - sig))
    dhat = dz if s["weight"] is None else dz * s["weight"].float()
    split = (n, p, groups, c // groups)
    a, h = dhat.view(split), hat.view(split)
    dx = rstd.view(n, 1, groups, 1) * (a - a.mean((1, 3), keepdim=True) - h * (a * h).mean((1, 3), keepdim=True))
    if s["weight"] is None:
        return dx.view(n, p, c), None, None
    return dx.view(n, p, c), (dz * hat).sum((0, 1)), dz.sum((0, 1))


def _some(*outputs):
    return [o for o in outputs if o is not None]


def _run_plain(s):
    op = s["case"]["op"]
    if op.startswith("norm"):
        dt = s["x"].dtype
        y, mean, rstd, hat, z = _plain_norm(s)
        out = [y.to(dt), mean, rstd]
        if op == "norm_train":
            dx, dw, db = _plain_norm_bwd(s, rstd, hat, z)
            out += _some(dx.to(dt), dw, db)
        return out
    dt = s["v"].dtype
    if op == "delta_step":
        share = s["v"].shape[1] // s["k"].shape[1]
        q, k = (x.float().repeat_interleave(share, 1)[..., None] for x in (s["q"], s["k"]))
        old = torch.exp(s["log_decay"])[..., None, None] * s["state"]
        u = s["beta"][..., None] * (s["v"].float() - (old * k).sum(-2))
        new = old + k * u[..., None, :]
        return [(s["scale"] * (new * q).sum(-2)).to(dt), new]
    y, last, p = _plain_delta(s)
    out = [y.to(dt), last]
    if op == "delta_train":
        dq, dk, dv, dg, dbeta, dh0 = _plain_delta_bwd(s, p, last)
        out += _some(dq.to(dt), dk.to(dt), dv.to(dt), dg, dbeta, dh0 if s["state"] is not None else None)
    return out


# ---- the library's calls ------------------------------------------------------------------------


def _run_own(s):
    import implicit_gemm_conv_amd as igc

    case = s["case"]
    op = case["op"]
    if op.startswith("norm"):
        f = igc.group_norm(s["x"], s["groups"], weight=s["weight"], bias=s["bias"], activation=case["act"], eps=s["eps"])
        out = [f.y, f.mean, f.rstd]
        if op == "norm_train":
            g = igc.group_norm_bwd(s["dy"], s["x"], s["groups"], f.mean, f.rstd, weight=s["weight"], bias=s["bias"],
                                   activation=case["act"])
            out += _some(g.dx, g.dweight, g.dbias)
        return out
    ins = (s["q"], s["k"], s["v"], s["log_decay"], s["beta"])
    if op == "delta_step":
        y, h = igc.delta_rule_step(*ins, s["state"], scale=s["scale"], h_out=s["next"])
        return [y, h]
    train = op == "delta_train"
    f = igc.delta_rule(*ins, scale=s["scale"], h0=s["state"], starts=s["starts"], train=train)
    out = [f.y, f.h]
    if train:
        g = igc.delta_rule_bwd(s["dy"], *ins, f.states, scale=s["scale"], starts=s["starts"], dh=s["dlast"])
        out += _some(g.dq, g.dk, g.dv, g.dlog_decay, g.dbeta, g.dh0 if s["state"] is not None else None)
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without --------------------------------------------------------------


def work(case):
    e = DTYPES[case["dtype"]].itemsize
    op = case["op"]
    if op.startswith("norm"):
        n, c, groups = case["n"] * case["p"] * case["c"], case["c"], case["groups"]
        par = {"none": 0, "same": 2 * c * e, "fp32": 8 * c}[case["params"]]
        silu = 6 if case["act"] == "silu" else 0
        bytes_, flops = 2 * n * e + par + 8 * case["n"] * groups, n * (7 + silu)
        if op == "norm_train":
            # the forward pass's input is read again, and its statistics
            bytes_ += 3 * n * e + par + 8 * case["n"] * groups + (8 * c if par else 0)
            flops += n * (16 + 2 * silu)
        return {"bytes": bytes_, "flops": flops}
    b, t, hk, hv, dk, dv = case["b"], case.get("t", 1), case["hk"], case["hv"], case["dk"], case["dv"]
    rows, state = b * t, b * hv * dk * dv * 4
    qk, vy, gates = rows * hk * dk * e, rows * hv * dv * e, rows * hv * 4
    bytes_ = 2 * qk + 2 * vy + 2 * gates + state
    # row by row: S^T k, the update, S^T q
    flops = rows * hv * (7 * dk * dv + 4 * dv)
    if op == "delta_step" or case["state"]:
        bytes_ += state
    if op != "delta_step" and case["starts"]:
        bytes_ += rows
    if op == "delta_train":
        # dy, q, k, v and both gates read again; dq, dk, dv and the gates' gradients written
        bytes_ += 4 * qk + 3 * vy + 4 * gates + (2 * state if case["state"] else 0) + (rows if case["starts"] else 0)
        # the state's gradient and the six products with it and with the state
        flops += rows * hv * 16 * dk * dv
    return {"bytes": bytes_, "flops": flops}


# ---- the definition in 64 bits ------------------------------------------------------------------


def _exact_row(S, q, k, v, g, beta):
    """One row: S is the state before it; returns the decayed state, the correction's parts, the new state."""
    old = torch.exp(g)[..., None, None] * S
    err = v - torch.einsum("bhkv,bhk->bhv", old, k)
    u = beta[..., None] * err
    return old, err, u, old + torch.einsum("bhk,bhv->bhkv", k, u)


def _exact_delta(s):
    case, scale = s["case"], s["scale"]
    share = case["hv"] // case["hk"]
    step = case["op"] == "delta_step"
    q, k, v, g, beta = (s[n][:, None] if step else s[n] for n in ("q", "k", "v", "log_decay", "beta"))
    q, k = (x.double().repeat_interleave(share, 2) for x in (q, k))
    v, g, beta = v.double(), g.double(), beta.double()
    starts = s.get("starts")
    S = s["state"].double() if s["state"] is not None else v.new_zeros((v.shape[0], case["hv"], case["dk"], case["dv"]))
    t = v.shape[1]

    def before(S, i):
        return S if starts is None else S * (~starts[:, i]).double()[:, None, None, None]

    y, kept = torch.zeros_like(v), {}
    for i in range(t):
        if i % 32 == 0:
            kept[i] = S
        S = _exact_row(before(S, i), q[:, i], k[:, i], v[:, i], g[:, i], beta[:, i])[3]
        y[:, i] = scale * torch.einsum("bhkv,bhk->bhv", S, q[:, i])
    if case["op"] != "delta_train":
        return [y[:, 0] if step else y, S]
    dy = s["dy"].double()
    dq, dk, dv, dg, db = (torch.zeros_like(x) for x in (q, k, v, g, beta))
    dS = torch.zeros_like(S) if s["dlast"] is None else s["dlast"].double()
    last = S
    for lo in sorted(kept, reverse=True):
        run_, S = [], kept[lo]
        for i in range(lo, min(lo + 32, t)):
            first = before(S, i)
            run_.append((first, *_exact_row(first, q[:, i], k[:, i], v[:, i], g[:, i], beta[:, i])))
            S = run_[-1][4]
        for i in range(min(lo + 32, t) - 1, lo - 1, -1):
            first, old, err, u, new = run_.pop()
            dS = dS + scale * torch.einsum("bhk,bhv->bhkv", q[:, i], dy[:, i])
            dq[:, i] = scale * torch.einsum("bhkv,bhv->bhk", new, dy[:, i])
            du = torch.einsum("bhkv,bhk->bhv", dS, k[:, i])
            derr = beta[:, i, :, None] * du
            db[:, i], dv[:, i] = (du * err).sum(-1), derr
            dk[:, i] = torch.einsum("bhkv,bhv->bhk", dS, u) - torch.einsum("bhkv,bhv->bhk", old, derr)
            dS = dS - torch.einsum("bhk,bhv->bhkv", k[:, i], derr)
            dg[:, i] = (dS * old).sum((-1, -2))
            dS = before(dS * torch.exp(g[:, i])[..., None, None], i)
    b, hk = case["b"], case["hk"]
    dq, dk = (x.view(b, t, hk, share, case["dk"]).sum(3) for x in (dq, dk))
    return [y, last, dq, dk, dv, dg, db] + ([dS] if s["state"] is not None else [])


def _exact_norm(s):
    case = s["case"]
    n, p, c, groups = case["n"], case["p"], case["c"], case["groups"]
    per = p * (c // groups)

    def spread(a):
        return a.repeat_interleave(c // groups, 1)[:, None]

    def gather(a):
        return a.sum(1).view(n, groups, c // groups).sum(2)

    x = s["x"].double()
    mean = gather(x) / per
    rstd = 1 / torch.sqrt(gather((x - spread(mean)) ** 2) / per + s["eps"])
    hat = (x - spread(mean)) * spread(rstd)
    w = torch.ones(c, dtype=torch.float64, device=x.device) if s["weight"] is None else s["weight"].double()
    z = hat * w + (0 if s["bias"] is None else s["bias"].double())
    sig = 1 / (1 + torch.exp(-z))
    silu = case["act"] == "silu"
    out = [z * sig if silu else z, mean, rstd]
    if case["op"] == "norm_train":
        dz = s["dy"].double()
        if silu:
            dz = dz * (sig + z * sig * (1 - sig))
        dhat = dz * w
        mean_d, mean_h = gather(dhat) / per, gather(dhat * hat) / per
        out.append((dhat - spread(mean_d) - hat * spread(mean_h)) * spread(rstd))
        if s["weight"] is not None:
            out += [(dz * hat).sum((0, 1)), dz.sum((0, 1))]
    return out


def exact(case, seed):
    s = _inputs(case, seed, "cuda")
    if case["op"].startswith("norm"):
        return _exact_norm(s)
    if case["op"] != "delta_step":
        # a row's products pass over every state: some 20 microseconds each and their bytes
        state = case["b"] * case["hv"] * case["dk"] * case["dv"] * 8
        each = 40 * (2e-5 + state / 1e12) if case["op"] == "delta_train" else 10 * (2e-5 + state / 1e12)
        if case["t"] * each > 18:
            return None
    return _exact_delta(s)
