"""The sequence oracle against differences, against itself in pieces, and against hand values (CPU)."""
import numpy as np
import pytest

from oracle import sequence as ref

rng = np.random.default_rng


def _difference(f, x, step=1e-5):
    """Central differences of the scalar f with respect to the array x."""
    out = np.zeros_like(x)
    for k in np.ndindex(*x.shape):
        keep = x[k]
        x[k] = keep + step
        hi = f()
        x[k] = keep - step
        out[k] = (hi - f()) / (2 * step)
        x[k] = keep
    return out


def _some_starts(r, b, t):
    s = r.random((b, t)) < 0.25
    s[0, 0] = True
    return s


@pytest.mark.parametrize("k,act,b,t,starts", [(4, "silu", 2, 7, True), (3, "none", 1, 6, False),
                                              (4, "silu", 2, 2, False), (1, "silu", 2, 5, True), (8, "none", 2, 9, True)])
def test_conv_gradients_against_differences(k, act, b, t, starts):
    r, c = rng(k * 100 + t), 3
    x, w, bias, state = r.normal(size=(b, t, c)), r.normal(size=(c, k)), r.normal(size=c), r.normal(size=(b, k - 1, c))
    s = _some_starts(r, b, t) if starts else None
    dy, dlast = r.normal(size=(b, t, c)), r.normal(size=(b, k - 1, c))

    def loss():
        y, _, last = ref.conv_fwd(x, w, bias, act, state, s)
        return (y * dy).sum() + (last * dlast).sum()

    got = ref.conv_bwd(dy, x, w, bias, act, state, s, dlast)
    for name, arr in (("dx", x), ("dw", w), ("dbias", bias), ("dstate", state)):
        # second-order remainder of the quotient: step^2 / 6 of a third derivative of order 10
        np.testing.assert_allclose(got[name][0], _difference(loss, arr), rtol=0, atol=1e-7, err_msg=name)


@pytest.mark.parametrize("b,t,starts", [(2, 9, True), (1, 70, False), (1, 67, True)])
def test_scan_gradients_against_differences(b, t, starts):
    r, c = rng(t), 2
    x, gr, gi = (r.normal(size=(b, t, c)) for _ in range(3))
    lam, h0 = r.normal(size=c) - 1, r.normal(size=(b, c))
    s = _some_starts(r, b, t) if starts else None
    dy, dh = r.normal(size=(b, t, c)), r.normal(size=(b, c))

    def forward():
        return ref.scan_fwd(x, gr, gi, lam, 2.0, h0, s)

    def loss():
        h, _, last, _ = forward()
        return (h * dy).sum() + (last[0] * dh).sum()

    states = np.stack([v[0] for v in forward()[3]], 1)
    got = ref.scan_bwd(dy, x, gr, gi, lam, states, 2.0, s, dh)
    for name, arr in (("dx", x), ("dgate_r", gr), ("dgate_i", gi), ("dlam", lam), ("dh0", h0)):
        np.testing.assert_allclose(got[name][0], _difference(loss, arr), rtol=0, atol=2e-7, err_msg=name)


def test_pieces_carry_on():
    r = rng(5)
    b, t, c, k, cut = 2, 30, 4, 4, 13
    x, gr, gi = (r.normal(size=(b, t, c)) for _ in range(3))
    w, lam, s = r.normal(size=(c, k)), r.normal(size=c), _some_starts(r, b, t)
    y, _, last = ref.conv_fwd(x, w, None, "silu", None, s)
    y1, _, mid = ref.conv_fwd(x[:, :cut], w, None, "silu", None, s[:, :cut])
    y2, _, end = ref.conv_fwd(x[:, cut:], w, None, "silu", mid, s[:, cut:])
    np.testing.assert_allclose(np.concatenate([y1, y2], 1), y, rtol=1e-14, atol=1e-14)
    np.testing.assert_array_equal(end, last)
    h, _, hl, _ = ref.scan_fwd(x, gr, gi, lam, 8.0, None, s)
    h1, _, m, _ = ref.scan_fwd(x[:, :cut], gr[:, :cut], gi[:, :cut], lam, 8.0, None, s[:, :cut])
    h2, _, e, _ = ref.scan_fwd(x[:, cut:], gr[:, cut:], gi[:, cut:], lam, 8.0, m[0], s[:, cut:])
    np.testing.assert_allclose(np.concatenate([h1, h2], 1), h, rtol=1e-14, atol=1e-14)
    np.testing.assert_allclose(e[0], hl[0], rtol=1e-14, atol=1e-14)


def test_conv_by_hand():
    x = np.array([1.0, 2.0, 3.0]).reshape(1, 3, 1)
    w = np.array([[10.0, 1.0]])
    y, _, last = ref.conv_fwd(x, w, np.array([0.5]), "none", np.array([[[7.0]]]))
    np.testing.assert_array_equal(y.ravel(), [71.5, 12.5, 23.5])
    np.testing.assert_array_equal(last.ravel(), [3.0])
    y, _, last = ref.conv_fwd(x, w, None, "none", np.array([[[7.0]]]), np.array([[True, False, True]]))
    np.testing.assert_array_equal(y.ravel(), [1.0, 12.0, 3.0])


def test_eight_bits_by_hand():
    x = np.zeros((1, 33, 3))
    x[0, :3, 0] = [1.0, -0.5, 1 / 128]          # top 1 = 2^0: steps of 2^-6, 1/128 is half a step: to even
    x[0, 0, 1] = 127.75 / 64                    # 127.75 steps: held as 127
    x[0, 16, 1] = np.inf
    x[0, 32, 2] = 2.0 ** -149
    q, e = ref.pack8(x)
    assert e[0, 0].tolist() == [121, 121, 1] and e[0, 1].tolist() == [1, 255, 1] and e[0, 2, 2] == 1
    assert q[0, :3, 0].tolist() == [64, -32, 0] and q[0, 0, 1] == 127 and q[0, 32, 2] == 0
    v = ref.unpack8(q, e)
    assert np.isnan(v[0, 16:32, 1]).all() and np.isfinite(v[0, :16]).all()


def test_eight_bits_within_half_a_step():
    x = rng(2).normal(size=(2, 77, 5)) * np.exp2(rng(3).integers(-40, 40, size=(2, 77, 5)))
    q, e = ref.pack8(x)
    step = np.repeat(2.0 ** (e.astype(float) - 127), ref.GROUP_ROWS, 1)[:, :77]
    err = np.abs(ref.unpack8(q, e) - x)
    assert (err <= np.where(np.abs(x) > 127.5 * step, 1.0, 0.5) * step).all()
    assert (np.abs(q.astype(int)) <= 127).all()
