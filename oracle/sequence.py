"""Float64 oracle of the sequence operators -- TEST INFRASTRUCTURE, as the rest of this package.

Row-by-row numpy loops written from the formulas of include/convseq.h, sharing no code with the
library.  Beside each result they carry a bound on what correct fp32 arithmetic may add to it:
every step of the recurrence passes on its predecessor's error times a, plus the roundings of its
own terms.  E is 2^-24; the gates' relative errors come from their exponentials, whose argument's
rounding grows with the argument (|x| E log2(e) ln(2), twice that with the product's), the 1-ulp
exp2, reciprocal and square root of the hardware (2 E each) and the few products around them.
"""
import numpy as np

E = 2.0 ** -24
STATE_ROWS = 64
GROUP_ROWS = 16


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-x))


def softplus(x):
    return np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))


# ---- 8 bits ----


def pack8(x):
    """(q, e) of x (B, T, C)."""
    b, t, c = x.shape
    n = -(-t // GROUP_ROWS)
    q = np.zeros((b, t, c), np.int8)
    e = np.zeros((b, n, c), np.uint8)
    for g in range(n):
        rows = x[:, g * GROUP_ROWS:(g + 1) * GROUP_ROWS]
        top = np.abs(rows).max(1)
        bad = ~np.isfinite(top)
        s = np.maximum(np.frexp(np.where(bad | (top == 0), 1.0, top))[1] - 7, -126)
        s = np.where(top == 0, -126, s)
        e[:, g] = np.where(bad, 255, s + 127)
        with np.errstate(invalid="ignore"):
            v = np.where(bad[:, None], 0, rows) * 2.0 ** -s[:, None].astype(np.float64)
        q[:, g * GROUP_ROWS:(g + 1) * GROUP_ROWS] = np.clip(np.rint(v), -127, 127)
    return q, e


def unpack8(q, e):
    s = np.repeat(e, GROUP_ROWS, axis=1)[:, :q.shape[1]].astype(np.float64)
    return np.where(s == 255, np.nan, q * 2.0 ** (s - 127))


# ---- causal depthwise convolution ----


def _window(x, state, k):
    if state is None:
        state = np.zeros((x.shape[0], k - 1, x.shape[2]))
    return np.concatenate([state, x], 1)


def _reach(starts, b, t, k):
    """How many rows before row t belong to its sequence, up to K-1 (carried rows count)."""
    out = np.full(b, k - 1)
    for j in range(k - 1, 0, -1):
        if t - j + 1 >= 0 and starts is not None:
            out = np.where(starts[:, t - j + 1], j - 1, out)
    return out


def conv_z(x, w, bias, state, starts):
    """z before the activation, and the sum of the magnitudes of its terms."""
    b, t, c = x.shape
    k = w.shape[1]
    ext = _window(x, state, k)
    z = np.zeros((b, t, c)) + (0 if bias is None else bias)
    mag = np.abs(z)
    for n in range(t):
        reach = _reach(starts, b, n, k)
        for j in range(k):
            live = (reach >= j)[:, None]
            term = np.where(live, ext[:, n + k - 1 - j], 0) * w[:, k - 1 - j]
            z[:, n] += term
            mag[:, n] += np.abs(term)
    return z, mag


def conv_fwd(x, w, bias=None, act="none", state=None, starts=None):
    """(y, bound, carried rows)."""
    b, t, c = x.shape
    k = w.shape[1]
    z, mag = conv_z(x, w, bias, state, starts)
    err = (k + 1) * E * mag
    if act == "silu":
        s = sigmoid(z)
        y, bound = z * s, 1.1 * err + (2 * np.abs(z) + 6) * E * np.abs(z * s)
    else:
        y, bound = z, err
    ext = _window(x, state, k)
    last = ext[:, t:].copy()
    if starts is not None and t > 0:
        reach = _reach(starts, b, t - 1, k)
        for j in range(k - 1):          # carried row j is j' = K-2-j rows before row t-1
            last[:, j] = np.where((reach >= k - 2 - j)[:, None], last[:, j], 0)
    return y, bound, last


def conv_bwd(dy, x, w, bias=None, act="none", state=None, starts=None, dlast=None):
    """{name: (gradient, bound)}."""
    b, t, c = dy.shape
    k = w.shape[1]
    ext = _window(x, state, k)
    z, mag = conv_z(x, w, bias, state, starts)
    dz, dz_err = dy.copy(), np.zeros_like(dy)
    if act == "silu":
        s = sigmoid(z)
        f = s * (1 + z * (1 - s))
        dz = dy * f
        # |f''| < 1/2; f is a sum of terms of at most s (1 + |z|)
        dz_err = np.abs(dy) * (0.5 * (k + 1) * E * mag + (2 * np.abs(z) + 10) * E * s * (1 + np.abs(z)))
    dext, dext_err, dext_mag = (np.zeros((b, t + k - 1, c)) for _ in range(3))
    dw, dw_err = np.zeros((c, k)), np.zeros((c, k))
    for n in range(t):
        reach = _reach(starts, b, n, k)
        for j in range(k):
            live = (reach >= j)[:, None]
            g, row, err = (np.where(live, v, 0) for v in (dz[:, n], ext[:, n + k - 1 - j], dz_err[:, n]))
            dext[:, n + k - 1 - j] += g * w[:, k - 1 - j]
            dext_mag[:, n + k - 1 - j] += np.abs(g * w[:, k - 1 - j])
            dext_err[:, n + k - 1 - j] += err * np.abs(w[:, k - 1 - j])
            dw[:, k - 1 - j] += (g * row).sum(0)
            # a sum of b*t products, each rounded on its way at most once a row
            dw_err[:, k - 1 - j] += (err * np.abs(row) + (b * t + 1) * E * np.abs(g * row)).sum(0)
    if dlast is not None:
        reach = _reach(starts, b, t - 1, k) if t > 0 else np.full(b, k)
        for j in range(k - 1):
            g = np.where((reach >= k - 2 - j)[:, None], dlast[:, j], 0)
            dext[:, t + j] += g
            dext_mag[:, t + j] += np.abs(g)
    bound = dext_err + (k + 1) * E * dext_mag
    return {"dx": (dext[:, k - 1:], bound[:, k - 1:]), "dstate": (dext[:, :k - 1], bound[:, :k - 1]),
            "dw": (dw, dw_err),
            "dbias": (dz.sum((0, 1)), (dz_err + b * t * E * np.abs(dz)).sum((0, 1)))}


# ---- gated linear recurrence ----


class Gates:
    """r, i, u, a, m = sqrt(1 - a^2), v = i x and the relative errors fp32 may put on them."""

    def __init__(self, x, gate_r, gate_i, lam, decay):
        self.x = x
        self.r, self.i = sigmoid(gate_r), sigmoid(gate_i)
        self.u = decay * softplus(lam) * self.r
        self.a = np.exp(-self.u)
        self.m = np.sqrt(-np.expm1(-2 * self.u))
        self.v = self.i * x
        fin = lambda g: np.where(np.isfinite(g), np.abs(g), 0)  # noqa: E731
        self.er = (2 * fin(gate_r) + 6) * E
        self.ei = (2 * fin(gate_i) + 6) * E
        self.eu = self.er + 10 * E
        self.ea = self.u * (self.eu + 2 * E) + 3 * E
        self.em = 0.5 * self.eu + 16 * E


def _first(starts, t):
    return None if starts is None else starts[:, t].astype(bool)[:, None]


def scan_fwd(x, gate_r, gate_i, lam, decay=8.0, h0=None, starts=None):
    """(h, bound, h_last, states): bound also holds for the last state and the kept ones."""
    b, t, c = x.shape
    k = Gates(x, gate_r, gate_i, lam, decay)
    h = np.zeros((b, c)) if h0 is None else h0.astype(np.float64)
    err, mag = np.zeros((b, c)), np.abs(h)
    hs, bound, states = np.zeros((b, t, c)), np.zeros((b, t, c)), []
    for n in range(t):
        if n % STATE_ROWS == 0:
            states.append((h, err))
        first = _first(starts, n)
        if first is not None:
            h, err, mag = (np.where(first, 0, v) for v in (h, err, mag))
        term = k.m[:, n] * k.v[:, n]
        # work split over the rows adds roundings of products of a: one a row
        err = k.a[:, n] * (err + (k.ea[:, n] + 2 * E) * mag) + (k.em[:, n] + k.ei[:, n] + 4 * E) * np.abs(term)
        h = k.a[:, n] * h + term
        mag = k.a[:, n] * mag + np.abs(term)
        err = err + 2 * E * mag
        hs[:, n], bound[:, n] = h, err
    return hs, bound, (h, err), states


def scan_bwd(dy, x, gate_r, gate_i, lam, states, decay=8.0, starts=None, dh=None):
    """{name: (gradient, bound)}; states (B, ceil(T/64), C) are the kept ones."""
    b, t, c = dy.shape
    k = Gates(x, gate_r, gate_i, lam, decay)
    before, before_err, before_mag = (np.zeros((b, t, c)) for _ in range(3))
    for n in range(t):
        if n % STATE_ROWS == 0:
            h = states[:, n // STATE_ROWS].astype(np.float64)
            err, mag = np.zeros_like(h), np.abs(h)
        first = _first(starts, n)
        if first is not None:
            h, err, mag = (np.where(first, 0, v) for v in (h, err, mag))
        before[:, n], before_err[:, n], before_mag[:, n] = h, err, mag
        term = k.m[:, n] * k.v[:, n]
        err = k.a[:, n] * (err + (k.ea[:, n] + 2 * E) * mag) + (k.em[:, n] + k.ei[:, n] + 4 * E) * np.abs(term)
        h, mag = k.a[:, n] * h + term, k.a[:, n] * mag + np.abs(term)
        err = err + 2 * E * mag
    g = np.zeros((b, c)) if dh is None else dh.astype(np.float64)
    gerr, gmag = np.zeros((b, c)), np.abs(g)
    out = {n: (np.zeros((b, t, c)), np.zeros((b, t, c))) for n in ("dx", "dgate_r", "dgate_i")}
    sum_e, sum_err = np.zeros(c), np.zeros(c)
    for n in range(t - 1, -1, -1):
        a, u, m, v, r, i, xx = (z[:, n] for z in (k.a, k.u, k.m, k.v, k.r, k.i, x))
        g, gmag = g + dy[:, n], gmag + np.abs(dy[:, n])
        gerr = gerr + 2 * E * gmag
        um = np.where(m > 0, u / np.where(m > 0, m, 1), 0)    # u / m, which goes to zero with u
        p1, p2 = um * a * a * v, u * a * before[:, n]
        e = g * (p1 - p2)
        size = np.abs(p1) + u * a * before_mag[:, n]
        rel = k.eu[:, n] + k.em[:, n] + 2 * k.ea[:, n] + k.ei[:, n] + 10 * E
        e_err = gerr * size + (np.abs(g) + gerr) * (rel * size + u * a * before_err[:, n])
        dv, dv_rel = g * m, k.em[:, n] + k.ei[:, n] + 6 * E
        dv_err = gerr * m
        out["dx"][0][:, n], out["dx"][1][:, n] = dv * i, (dv_err + dv_rel * (np.abs(dv) + dv_err)) * i
        # 1 - i is i of the negated gate, and loses what i's rounding takes from 1
        s = xx * i * (1 - i)
        lost = np.abs(xx) * i * (k.ei[:, n] * i + E)
        out["dgate_i"][0][:, n] = dv * s
        out["dgate_i"][1][:, n] = (dv_err + dv_rel * (np.abs(dv) + dv_err)) * np.abs(s) + (np.abs(dv) + dv_err) * lost
        out["dgate_r"][0][:, n] = e * (1 - r)
        out["dgate_r"][1][:, n] = (e_err + 4 * E * np.abs(e)) * (1 - r) + (np.abs(e) + e_err) * (k.er[:, n] * r + E)
        sum_e += e.sum(0)
        sum_err += (e_err + (b * t + 4) * E * np.abs(e)).sum(0)
        gerr = a * (gerr + (k.ea[:, n] + 2 * E) * gmag)
        g, gmag = g * a, gmag * a
        first = _first(starts, n)
        if first is not None:
            g, gerr, gmag = (np.where(first, 0, z) for z in (g, gerr, gmag))
    unit = sigmoid(lam) / softplus(lam)
    out["dlam"] = (sum_e * unit, (sum_err + 12 * E * np.abs(sum_e)) * unit)
    out["dh0"] = (g, gerr + 2 * E * gmag)
    return out
