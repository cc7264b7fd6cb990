"""Gated delta rule on the GPU where offsets grow large: very many key heads, gradients behind 2^31 elements."""
import pytest
import torch

import implicit_gemm_conv_amd as igc

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _random(gen, *shape, scale=1.0):
    return torch.randn(shape, generator=gen, device=DEV).mul_(scale)


# rows of q and k of 2^23.9 and 2^25 elements: 64 of them lie 2^31.9 and 2^33 bytes apart in (B, T, Hk, Dk)
@pytest.mark.parametrize("t,heads,dk", [(64, 1 << 17, 120), (40, 1 << 18, 128)])
def test_very_many_key_heads(t, heads, dk):
    """Every head is its own: some of them give the bits that they give alone."""
    gen = torch.Generator(DEV).manual_seed(t)
    q, k = (_random(gen, 1, t, heads, dk, scale=dk ** -0.5) for _ in range(2))
    v, dy = (_random(gen, 1, t, heads, 1) for _ in range(2))
    g = torch.full((1, t, heads), -0.1, device=DEV)
    beta = torch.sigmoid(_random(gen, 1, t, heads))
    f = igc.delta_rule(q, k, v, g, beta, train=True)
    b = igc.delta_rule_bwd(dy, q, k, v, g, beta, f.states)
    for h in (0, 1, 65535, heads // 2 + 3, heads - 1):
        one = [x[:, :, h:h + 1].contiguous() for x in (q, k, v, g, beta)]
        f1 = igc.delta_rule(*one, train=True)
        b1 = igc.delta_rule_bwd(dy[:, :, h:h + 1], *one, f1.states)
        assert f1.y.abs().max() > 0 and torch.equal(f.y[:, :, h:h + 1], f1.y), h
        assert torch.equal(f.h[:, h:h + 1], f1.h), h
        for n in ("dq", "dk", "dv", "dlog_decay", "dbeta"):
            assert torch.equal(getattr(b, n)[:, :, h:h + 1], getattr(b1, n)), (n, h)


def test_gradients_behind_32_bits():
    """Rows of v, dy, x and z behind the first 2^31 values: a sequence that begins with the last chunk has the gradients that
    it has alone (the same rows of a chunk, and nothing crosses the start); no gradient reaches the rows before."""
    t, hv, dv, last = 33000, 128, 512, 40
    assert (t - last) % 64 == 0
    gen = torch.Generator(DEV).manual_seed(1)
    q, k = (_random(gen, 1, t, 1, 16, scale=0.25).half() for _ in range(2))
    v, dy = (torch.zeros((1, t, hv, dv), dtype=torch.float16, device=DEV) for _ in range(2))
    for x in (v, dy):
        x[:, -last:] = _random(gen, 1, last, hv, dv).half()
    g = torch.full((1, t, hv), -0.1, device=DEV)
    beta = torch.full((1, t, hv), 0.5, device=DEV)
    starts = torch.zeros((1, t), dtype=torch.bool, device=DEV)
    starts[0, -last] = True
    f = igc.delta_rule(q, k, v, g, beta, starts=starts, train=True)
    b = igc.delta_rule_bwd(dy, q, k, v, g, beta, f.states, starts=starts)
    one = [x[:, -last:].contiguous() for x in (q, k, v, g, beta)]
    f1 = igc.delta_rule(*one, train=True)
    b1 = igc.delta_rule_bwd(dy[:, -last:], *one, f1.states)
    assert torch.equal(f.y[:, -last:], f1.y) and torch.equal(f.h, f1.h)
    for n in ("dq", "dk", "dv", "dlog_decay", "dbeta"):
        got, want = getattr(b, n), getattr(b1, n)
        assert want.abs().max() > 0 and torch.equal(got[:, -last:], want), n
        assert (got[:, :-last] == 0).all(), n
