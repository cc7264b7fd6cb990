"""The sequence operators of this library as measured cases: the causal depthwise convolution along
a sequence, the gated linear recurrence, and activations kept in 8 bits between the two passes of
training.

``own`` False computes each operator in its plain form, elementary torch operations in float32;
``own`` True makes the calls a user makes of ``implicit_gemm_conv_amd``.  Formulas, with rows
(b, t), channels c, and ``starts[b, t]`` marking a row that begins a new sequence:

convolution   z_t = bias + sum_k w[c, k] * X(t - (K-1) + k),   y = z or z * sigmoid(z)
              X(s) is x_s, the row of ``state`` for s < 0, and nothing across a start
recurrence    r = sigmoid(gate_r), i = sigmoid(gate_i), a = exp(-decay * softplus(lam) * r)
              h_t = a * h_{t-1} + sqrt(1 - a^2) * i * x_t   (h_{t-1} absent at a start)
8 bits        16 consecutive rows of a channel share a power of two 2^s, s = floor(log2(max |x|)) - 6
              (at least -126), and hold q = round(x / 2^s) to nearest even, within +-127
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EVERY = 64    # rows between the states of the recurrence that the backward pass starts from
GROUP = 16    # rows of a channel that share a power of two in 8 bits


def listed():
    return [
        # Serving, one token of each of eight streams through the convolution: latency.
        dict(name="conv_step_b8", op="conv_step", b=8, c=1024, k=4, act="silu", bias=True, dtype="bf16"),
        # Serving, one token of a single small stream through the recurrence: the smallest call.
        dict(name="scan_step_b1", op="scan_step", b=1, c=256, dtype="fp16"),
        # Serving, a full batch of streams.
        dict(name="scan_step_b256", op="scan_step", b=256, c=2048, dtype="bf16"),
        # A long prompt, continued from an earlier piece: one sequence, an odd number of rows.
        dict(name="conv_prefill_long", op="conv_prefill", b=1, t=32771, c=1024, k=4, act="silu", bias=True,
             state=True, dtype="fp16"),
        dict(name="scan_prefill_long", op="scan_prefill", b=1, t=65539, c=1024, state=True, dtype="bf16"),
        # A training step's share of one layer: batch 4 of 4096 rows, kept in 8 bits, the
        # recurrence over sequences packed end to end.
        dict(name="conv_train_8bit", op="conv_train", b=4, t=4096, c=2048, k=4, act="silu", bias=True,
             state=False, starts=False, keep8=True, dtype="bf16"),
        dict(name="scan_train_8bit", op="scan_train", b=4, t=4096, c=2048, state=False, starts=True,
             keep8=True, dtype="bf16"),
        # Float32 training of an odd channel count on odd lengths, nothing rounded in between.
        dict(name="conv_train_odd_f32", op="conv_train", b=3, t=1023, c=321, k=3, act="none", bias=False,
             state=True, starts=True, keep8=False, dtype="fp32"),
        dict(name="scan_train_odd_f32", op="scan_train", b=3, t=1999, c=321, state=True, starts=False,
             keep8=False, dtype="fp32"),
        # Many short sequences.
        dict(name="scan_train_short", op="scan_train", b=64, t=100, c=512, state=False, starts=False,
             keep8=False, dtype="fp16"),
        # Activations of a large layer kept for the backward pass and brought back: the largest.
        dict(name="keep8_large", op="keep8", b=8, t=8192, c=2048, dtype="bf16"),
        # Channels-last image activations of the 65-channel layer, 55 x 57 positions.
        dict(name="keep8_image_c65", op="keep8", b=32, t=55 * 57, c=65, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _channels(rng, hi):
    c = _log(rng, 16, hi)
    return c if rng.random() < 0.4 or c < 64 else c // 64 * 64


def _fits(case):
    # whole problems of at most 32 Mi values, as the listed training cases
    return case["b"] * case["t"] * case["c"] <= 1 << 25


def draw(rng):
    op = rng.choice(["conv_step", "scan_step", "conv_prefill", "scan_prefill", "conv_train", "conv_train",
                     "scan_train", "scan_train", "keep8"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op.endswith("step"):
        case = dict(op=op, b=_log(rng, 1, 512), c=_channels(rng, 4096), dtype=dtype)
        if op == "conv_step":
            case.update(k=rng.choice([2, 3, 4, 4, 5, 8]), act=rng.choice(["none", "silu"]), bias=rng.random() < 0.5)
        return case
    while True:
        case = dict(op=op, b=_log(rng, 1, 64), t=_log(rng, 1, 65536), c=_channels(rng, 4096), dtype=dtype)
        if _fits(case):
            break
    if op.startswith("conv"):
        case.update(k=rng.choice([2, 3, 4, 4, 5, 8]), act=rng.choice(["none", "silu"]), bias=rng.random() < 0.5)
    if op != "keep8":
        case["state"] = rng.random() < 0.5
    if op.endswith("train"):
        case.update(starts=rng.random() < 0.5, keep8=rng.random() < 0.5)
    return case


# ---- inputs -------------------------------------------------------------------------------------


def _inputs(case, seed, device):
    gen = torch.Generator(device).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    b, c, t = case["b"], case["c"], case.get("t", 1)
    step = case["op"].endswith("step")
    rows = (b, c) if step else (b, t, c)

    def normal(shape, scale=1.0, to=dt):
        return (torch.randn(shape, generator=gen, device=device) * scale).to(to)

    s = {"x": normal(rows)}
    if case["op"] == "keep8":
        # channels of a layer differ in scale by orders of magnitude
        s["x"] = (s["x"].float() * torch.exp2(normal((c,), 2.0, torch.float32))).to(dt)
        return s
    if case["op"].startswith("conv"):
        k = case["k"]
        s["w"] = normal((c, k), 1 / math.sqrt(k))
        s["bias"] = normal((c,), 0.2) if case["bias"] else None
        s["state"] = normal((b, k - 1, c)) if step or case["state"] else None
    else:
        # the two gates come from one projection, so they are column slices of its result
        both = normal(rows[:-1] + (2 * c,), 1.5)
        s["gate_r"], s["gate_i"] = both[..., :c], both[..., c:]
        # decays between 0.9 and 0.999 a row where the gate is fully open
        slow = torch.rand((c,), generator=gen, device=device, dtype=torch.float64) * 0.099 + 0.9
        s["decay"] = 8.0
        s["lam"] = torch.log(torch.expm1(-torch.log(slow) / s["decay"])).float()
        s["state"] = normal((b, c), 0.5, torch.float32) if step or case["state"] else None
    if case["op"].endswith("train"):
        s["dy"] = normal(rows)
        s["starts"] = None
        if case["starts"]:
            # sequences of about a fifth of the length, packed end to end
            s["starts"] = torch.rand((b, t), generator=gen, device=device) < 5.0 / t
            s["starts"][:, 0] |= torch.rand((b,), generator=gen, device=device) < 0.5
        if case["op"] == "conv_train":
            s["dlast"] = normal((b, case["k"] - 1, c)) if case["state"] else None
        else:
            s["dlast"] = normal((b, c), 0.5, torch.float32) if case["state"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed, "cuda")
    s["case"] = case
    if case["op"].endswith("step"):
        # a server keeps two buffers for the streams' states and swaps them
        s["next"] = torch.empty_like(s["state"])
    return s


# ---- plain forms, float32 ---------------------------------------------------------------------


def _scan(a, b):
    """Running composition of h -> a*h + b along dim 1: the products of a and the h from zero.
    Doubling: after the step of width d each row covers the last 2d rows."""
    d = 1
    while d < a.shape[1]:
        b = torch.cat([b[:, :d], torch.addcmul(b[:, d:], a[:, d:], b[:, :-d])], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return a, b


def _gates(x, gate_r, gate_i, lam, decay):
    x = x.float()
    r, i = torch.sigmoid(gate_r.float()), torch.sigmoid(gate_i.float())
    u = decay * torch.nn.functional.softplus(lam, threshold=80.0) * r
    return x, r, i, u, torch.exp(-u), torch.sqrt(-torch.expm1(-2 * u))


def _plain_scan(x, gate_r, gate_i, lam, decay, h0, starts):
    x, r, i, u, a, m = _gates(x, gate_r, gate_i, lam, decay)
    if starts is not None:
        a = torch.where(starts[..., None], 0.0, a)
    prod, h = _scan(a, m * i * x)
    if h0 is None:
        h0 = torch.zeros_like(h[:, 0])
    h = h + prod * h0[:, None]
    return h, torch.cat([h0[:, None], h[:, EVERY - 1:-1:EVERY]], 1)


def _plain_scan_bwd(dy, x, gate_r, gate_i, lam, decay, states, starts, dlast):
    b, t, c = dy.shape
    x, r, i, u, a, m = _gates(x, gate_r, gate_i, lam, decay)
    carry = a if starts is None else torch.where(starts[..., None], 0.0, a)
    # states again, piece by piece from the kept ones
    n = states.shape[1]
    fill = (0, 0, 0, n * EVERY - t)
    pa = torch.nn.functional.pad(carry, fill).view(b * n, EVERY, c)
    pb = torch.nn.functional.pad(m * i * x, fill).view(b * n, EVERY, c)
    prod, h = _scan(pa, pb)
    s = states.reshape(b * n, 1, c)
    before = torch.cat([s, (h + prod * s)[:, :-1]], 1).view(b, n * EVERY, c)[:, :t]
    # g_t = dy_t + a_{t+1} g_{t+1}
    last = torch.zeros_like(lam).expand(b, 1, c) if dlast is None else dlast[:, None]
    g = dy.float()
    g = torch.cat([g[:, :-1], g[:, -1:] + last], 1)
    ahead = torch.cat([carry[:, 1:], torch.zeros_like(carry[:, :1])], 1)
    g = _scan(ahead.flip(1), g.flip(1))[1].flip(1)
    de = g * u * (i * x * a * a / m - carry * before)
    dv = g * m
    unit = torch.sigmoid(lam) / torch.nn.functional.softplus(lam, threshold=80.0)
    return dv * i, de * (1 - r), dv * x * i * (1 - i), de.sum((0, 1)) * unit, carry[:, 0] * g[:, 0]


def _window(x, state, starts, k):
    """X(t-(K-1)+j) for each row and j < K, and which of them belong to the row's sequence."""
    b, t, c = x.shape
    if state is None:
        state = x.new_zeros((b, k - 1, c))
    ext = torch.cat([state, x], 1).float()
    if starts is None:
        return [ext[:, j:j + t] for j in range(k)], None, ext
    seg = torch.cat([starts.new_zeros((b, k - 1), dtype=torch.int32), torch.cumsum(starts.int(), 1)], 1)
    keep = [(seg[:, j:j + t] == seg[:, k - 1:])[..., None] for j in range(k)]
    return [torch.where(keep[j], ext[:, j:j + t], 0.0) for j in range(k)], (seg, keep), ext


def _plain_conv(x, w, bias, act, state, starts):
    k = w.shape[1]
    taps, marks, ext = _window(x, state, starts, k)
    w = w.float()
    z = sum(taps[j] * w[:, j] for j in range(k))
    z = z if bias is None else z + bias.float()
    last = ext[:, x.shape[1]:]
    if marks is not None:
        seg = marks[0]
        last = torch.where((seg[:, x.shape[1]:] == seg[:, -1:])[..., None], last, 0.0)
    return z, z * torch.sigmoid(z) if act == "silu" else z, last


def _plain_conv_bwd(dy, x, w, bias, act, state, starts, dlast):
    b, t, c = dy.shape
    k = w.shape[1]
    taps, marks, _ = _window(x, state, starts, k)
    z = _plain_conv(x, w, bias, act, state, starts)[0]
    dz = dy.float()
    if act == "silu":
        s = torch.sigmoid(z)
        dz = dz * s * (1 + z * (1 - s))
    w = w.float()
    dw = torch.stack([(dz * taps[j]).sum((0, 1)) for j in range(k)], 1)
    dext = dz.new_zeros((b, t + k - 1, c))
    for j in range(k):
        part = dz * w[:, j]
        dext[:, j:j + t] += part if marks is None else torch.where(marks[1][j], part, 0.0)
    if dlast is not None:
        part = dlast.float()
        if marks is not None:
            part = torch.where((marks[0][:, t:] == marks[0][:, -1:])[..., None], part, 0.0)
        dext[:, t:] += part
    return dext[:, k - 1:], dw, dz.sum((0, 1)) if bias is not None else None, dext[:, :k - 1]


def _power(s):
    """2^s in float32 for whole numbers s of -126 to 127, by its bits."""
    return ((s + 127).int() << 23).view(torch.float32)


def _plain_keep8(x):
    """What 8 bits hold of x, as float32 values."""
    b, t, c = x.shape
    n = -(-t // GROUP)
    v = torch.nn.functional.pad(x.float(), (0, 0, 0, n * GROUP - t)).view(b, n, GROUP, c)
    s = (torch.frexp(v.abs().amax(2, keepdim=True))[1] - 7).clamp(min=-126)
    q = torch.round(v * _power(-s)).clamp(-127, 127)
    return (q * _power(s)).view(b, n * GROUP, c)[:, :t]


def _some(*outputs):
    return [o for o in outputs if o is not None]


def _run_plain(s):
    case, dt = s["case"], s["x"].dtype
    op, x = case["op"], s["x"]
    if op == "keep8":
        return [_plain_keep8(x).to(dt)]
    if op == "conv_step":
        _, y, last = _plain_conv(x[:, None], s["w"], s["bias"], case["act"], s["state"], None)
        return [y[:, 0].to(dt), last.to(dt)]
    if op == "scan_step":
        h, _ = _plain_scan(x[:, None], s["gate_r"][:, None], s["gate_i"][:, None], s["lam"], s["decay"],
                           s["state"], None)
        return [h[:, 0].to(dt), h[:, 0]]
    starts = s.get("starts")
    if op.startswith("conv"):
        _, y, last = _plain_conv(x, s["w"], s["bias"], case["act"], s["state"], starts)
        out = [y.to(dt), last.to(dt)]
        if op == "conv_train":
            kept = _plain_keep8(x) if case["keep8"] else x
            dx, dw, db, dstate = _plain_conv_bwd(s["dy"], kept, s["w"], s["bias"], case["act"], s["state"], starts,
                                                 s["dlast"])
            out += _some(dx.to(dt), dw, db, dstate.to(dt) if case["state"] else None)
        return out
    h, states = _plain_scan(x, s["gate_r"], s["gate_i"], s["lam"], s["decay"], s["state"], starts)
    out = [h.to(dt), h[:, -1]]
    if op == "scan_train":
        kept = [_plain_keep8(v) if case["keep8"] else v for v in (x, s["gate_r"], s["gate_i"])]
        dx, dr, di, dlam, dh0 = _plain_scan_bwd(s["dy"], *kept, s["lam"], s["decay"], states, starts, s["dlast"])
        out += _some(dx.to(dt), dr.to(dt), di.to(dt), dlam, dh0 if case["state"] else None)
    return out


# ---- the library's calls ------------------------------------------------------------------------


def _run_own(s):
    import implicit_gemm_conv_amd as igc

    case, x = s["case"], s["x"]
    op = case["op"]
    if op == "keep8":
        return [igc.unpack8(igc.pack8(x))]
    if op == "conv_step":
        y, last = igc.seq_conv_step(x, s["w"], s["state"], bias=s["bias"], activation=case["act"],
                                    state_out=s["next"])
        return [y, last]
    if op == "scan_step":
        y, h = igc.gated_scan_step(x, s["gate_r"], s["gate_i"], s["lam"], s["state"], decay=s["decay"],
                                   h_out=s["next"])
        return [y, h]
    starts, train = s.get("starts"), op.endswith("train")
    if op.startswith("conv"):
        f = igc.seq_conv(x, s["w"], bias=s["bias"], activation=case["act"], state=s["state"], starts=starts,
                         keep8=train and case["keep8"])
        out = [f.y, f.state]
        if train:
            g = igc.seq_conv_bwd(s["dy"], f.kept if case["keep8"] else x, s["w"], bias=s["bias"],
                                 activation=case["act"], state=s["state"], starts=starts, dstate=s["dlast"])
            out += _some(g.dx, g.dw, g.dbias, g.dstate)
        return out
    f = igc.gated_scan(x, s["gate_r"], s["gate_i"], s["lam"], decay=s["decay"], h0=s["state"], starts=starts,
                       train=train, keep8=train and case["keep8"])
    out = [f.y, f.h]
    if train:
        kept = f.kept if case["keep8"] else (x, s["gate_r"], s["gate_i"])
        g = igc.gated_scan_bwd(s["dy"], *kept, s["lam"], f.states, decay=s["decay"], starts=starts,
                               dh=s["dlast"])
        out += _some(g.dx, g.dgate_r, g.dgate_i, g.dlam, g.dh0 if case["state"] else None)
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without --------------------------------------------------------------


def work(case):
    e = DTYPES[case["dtype"]].itemsize
    b, c, t = case["b"], case["c"], case.get("t", 1)
    n = b * t * c
    op = case["op"]
    kept = n + b * -(-t // GROUP) * c        # one array in 8 bits with its powers of two
    if op == "keep8":
        return {"bytes": 2 * n * e + 2 * kept, "flops": 6 * n}
    if op.startswith("conv"):
        k = case["k"]
        par, rows = c * (k + case["bias"]) * e, b * (k - 1) * c * e
        silu = 6 if case["act"] == "silu" else 0
        bytes_, flops = 2 * n * e + par + rows, n * (2 * k + silu)
        if op == "conv_step" or case["state"]:
            bytes_ += rows
        if op == "conv_train":
            bytes_ += 2 * n * e + par + c * (k + case["bias"]) * 4 + (2 * kept if case["keep8"] else n * e)
            bytes_ += 3 * rows if case["state"] else 0
            bytes_ += 2 * b * t if case["starts"] else 0
            flops += n * (6 * k + 2 * silu)
        return {"bytes": bytes_, "flops": flops}
    rows = b * c * 4
    bytes_, flops = 4 * n * e + rows + 4 * c, 20 * n
    if op == "scan_step" or case["state"]:
        bytes_ += rows
    if op == "scan_train":
        bytes_ += 4 * n * e + 8 * c + 2 * b * -(-t // EVERY) * c * 4
        bytes_ += 6 * kept if case["keep8"] else 3 * n * e
        bytes_ += 2 * rows if case["state"] else 0
        bytes_ += 2 * b * t if case["starts"] else 0
        flops += 45 * n
    return {"bytes": bytes_, "flops": flops}


# ---- the definition in 64 bits, row by row ------------------------------------------------------


def _exact_keep8(x):
    x = x.double()
    out = torch.empty_like(x)
    for t0 in range(0, x.shape[1], GROUP):
        g = x[:, t0:t0 + GROUP]
        top = g.abs().amax(1, keepdim=True)
        s = torch.floor(torch.log2(top.clamp(min=2.0 ** -120))) - 6
        step = torch.exp2(s)
        out[:, t0:t0 + GROUP] = torch.clamp(torch.round(g / step), -127, 127) * step
    return out


def _exact_scan_values(x, gate_r, gate_i, lam, decay):
    x, lam = x.double(), lam.double()
    r, i = 1 / (1 + torch.exp(-gate_r.double())), 1 / (1 + torch.exp(-gate_i.double()))
    u = decay * torch.log1p(torch.exp(lam)) * r
    return x, r, i, u, torch.exp(-u), torch.sqrt(-torch.expm1(-2 * u))


def _exact_scan(s, x, gate_r, gate_i):
    x, r, i, u, a, m = _exact_scan_values(x, gate_r, gate_i, s["lam"], s["decay"])
    h = torch.zeros_like(x[:, 0]) if s["state"] is None else s["state"].double()
    starts = s.get("starts")
    hs, states = torch.empty_like(x), []
    for t in range(x.shape[1]):
        if t % EVERY == 0:
            states.append(h)
        h = a[:, t] * (h if starts is None else h * ~starts[:, t, None]) + m[:, t] * i[:, t] * x[:, t]
        hs[:, t] = h
    return hs, states


def _exact_scan_bwd(s, x, gate_r, gate_i, states):
    lam, decay, starts = s["lam"], s["decay"], s["starts"]
    x, r, i, u, a, m = _exact_scan_values(x, gate_r, gate_i, lam, decay)
    before = torch.empty_like(x)
    for t in range(x.shape[1]):
        h = states[t // EVERY] if t % EVERY == 0 else h
        if starts is not None:
            h = h * ~starts[:, t, None]
        before[:, t] = h
        h = a[:, t] * h + m[:, t] * i[:, t] * x[:, t]
    g = torch.zeros_like(x[:, 0]) if s["dlast"] is None else s["dlast"].double()
    gs, dy = torch.empty_like(x), s["dy"].double()
    for t in range(x.shape[1] - 1, -1, -1):
        gs[:, t] = g + dy[:, t]
        g = gs[:, t] * a[:, t]
        if starts is not None:
            g = g * ~starts[:, t, None]
    du = gs * (i * x * a * a / m - a * before)
    open_ = decay * r * du
    dx, di = gs * m * i, gs * m * x * i * (1 - i)
    dr = open_ * torch.log1p(torch.exp(lam.double())) * (1 - r)
    dlam = open_.sum((0, 1)) / (1 + torch.exp(-lam.double()))
    return dx, dr, di, dlam, g


def _exact_conv(s, x, dy=None):
    """Row by row: z, y and the last rows, and with dy the gradients as well."""
    case, w = s["case"], s["w"].double()
    k = w.shape[1]
    b, t, c = x.shape
    x, starts = x.double(), s.get("starts")
    rows = torch.zeros((b, k - 1, c), dtype=torch.float64, device=x.device) if s["state"] is None else s["state"].double()
    hist = [rows[:, j] for j in range(k - 1)]
    live = [torch.ones((b, 1), dtype=torch.float64, device=x.device)] * (k - 1)
    one = torch.ones((b, 1), dtype=torch.float64, device=x.device)
    y = torch.empty_like(x)
    dext = torch.zeros((b, t + k - 1, c), dtype=torch.float64, device=x.device)
    dw, db = torch.zeros_like(w), torch.zeros(c, dtype=torch.float64, device=x.device)
    for n in range(t):
        if starts is not None:
            go = (~starts[:, n, None]).double()
            live = [v * go for v in live]
        hist, live = hist[-(k - 1):] + [x[:, n]] if k > 1 else [x[:, n]], live[-(k - 1):] + [one] if k > 1 else [one]
        z = sum(w[:, j] * hist[j] * live[j] for j in range(k))
        if s["bias"] is not None:
            z = z + s["bias"].double()
        sig = 1 / (1 + torch.exp(-z))
        y[:, n] = z * sig if case["act"] == "silu" else z
        if dy is not None:
            dz = dy[:, n].double()
            if case["act"] == "silu":
                dz = dz * (sig + z * sig * (1 - sig))
            db += dz.sum(0)
            for j in range(k):
                dw[:, j] += (dz * hist[j] * live[j]).sum(0)
                dext[:, n + j] += dz * w[:, j] * live[j]
    ends = range(len(hist) - (k - 1), len(hist))
    last = torch.stack([hist[j] * live[j] for j in ends], 1)
    if dy is not None and s["dlast"] is not None:
        dext[:, t:] += s["dlast"].double() * torch.stack([live[j] for j in ends], 1)
    return y, last, dext[:, k - 1:], dw, db, dext[:, :k - 1]


def exact(case, seed):
    s = _inputs(case, seed, "cuda")
    s["case"] = case
    op, x = case["op"], s["x"]
    if op == "keep8":
        return [_exact_keep8(x)]
    if op == "conv_step":
        y, last = _exact_conv(s, x[:, None])[:2]
        return [y[:, 0], last]
    if op == "scan_step":
        h = _exact_scan(s, x[:, None], s["gate_r"][:, None], s["gate_i"][:, None])[0][:, 0]
        return [h, h]
    if op.startswith("conv"):
        if case["t"] * case["k"] > 70000 and op == "conv_train" or case["t"] * case["k"] > 300000:
            return None
        y, last = _exact_conv(s, x)[:2]
        if op == "conv_prefill":
            return [y, last]
        kept = _exact_keep8(x) if case["keep8"] else x
        _, _, dx, dw, db, dstate = _exact_conv(s, kept, s["dy"])
        return _some(y, last, dx, dw, db if case["bias"] else None, dstate if case["state"] else None)
    if case["t"] > 40000 and op == "scan_train":
        return None
    hs, states = _exact_scan(s, x, s["gate_r"], s["gate_i"])
    if op == "scan_prefill":
        return [hs, hs[:, -1]]
    kept = [_exact_keep8(v) if case["keep8"] else v for v in (x, s["gate_r"], s["gate_i"])]
    dx, dr, di, dlam, dh0 = _exact_scan_bwd(s, *kept, states)
    return _some(hs, hs[:, -1], dx, dr, di, dlam, dh0 if case["state"] else None)
