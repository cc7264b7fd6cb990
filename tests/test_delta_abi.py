"""Host-side tests of the gated delta rule's C ABI and of the binding's argument checks (no GPU needed).

Every call here returns before the library touches the GPU.
"""
import os
import re

import pytest
import torch

import implicit_gemm_conv_amd as igc
from implicit_gemm_conv_amd import delta as dl

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "convdelta.h")
OK, NULL, BAD, UNSUPPORTED, LARGE, ALIAS, MISALIGNED = 0, -1, -2, -3, -4, -5, -7
MB = 1 << 20


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*(?:int|int64_t)\s+(convdelta_\w+)\s*\(", text, flags=re.M)))
    assert names == sorted(n for n, _, _ in dl.EXPORTS)
    for n in names:
        assert hasattr(dl._delta(), n), n


def test_constants_match_the_header():
    assert f"CONVDELTA_STATE_ROWS = {dl.STATE_ROWS}" in open(HEADER).read()


def _desc(**kw):
    return dl.DeltaDesc(**{**dict(b=2, t=100, hk=2, hv=4, dk=32, dv=32, dtype=2, scale=0.5), **kw})


def _heads(at, h=2, d=32, **kw):
    return dl.Heads(at, kw.get("batch", 100 * h * d), kw.get("row", h * d), kw.get("head", d))


def _fwd(d, **kw):
    p = dict(q=_heads(1 * MB), k=_heads(2 * MB), v=_heads(3 * MB, 4), g=4 * MB, beta=5 * MB, h0=None, starts=None, y=6 * MB,
             h=7 * MB, states=None, x=None, work=64 * MB)
    p.update(kw)
    return dl._delta().convdelta_fwd(d, *p.values(), None)


def _bwd(d, **kw):
    p = dict(dy=_heads(1 * MB, 4), q=_heads(2 * MB), k=_heads(3 * MB), v=_heads(4 * MB, 4), g=5 * MB, beta=6 * MB, states=7 * MB, x=14 * MB,
             starts=None, dh=None, dq=8 * MB, dk=9 * MB, dv=10 * MB, dg=11 * MB, db=12 * MB, dh0=13 * MB, work=64 * MB)
    p.update(kw)
    return dl._delta().convdelta_bwd(d, *p.values(), None)


def _step(d, **kw):
    p = dict(q=_heads(1 * MB), k=_heads(2 * MB), v=_heads(3 * MB, 4), g=4 * MB, beta=5 * MB, state=6 * MB, out=6 * MB, slots=None,
             n=2, y=7 * MB)
    p.update(kw)
    return dl._delta().convdelta_step(d, *p.values(), None)


@pytest.mark.parametrize("field,value,code", [
    ("b", -1, BAD), ("t", -1, BAD), ("hk", 0, BAD), ("hv", 0, BAD), ("hv", 3, BAD), ("dk", 0, BAD), ("dv", 0, BAD),
    ("dk", 129, UNSUPPORTED), ("dtype", 3, UNSUPPORTED), ("dtype", -1, UNSUPPORTED), ("scale", float("nan"), BAD),
    ("scale", float("inf"), BAD), ("t", 1 << 30, LARGE), ("b", 1 << 24, LARGE), ("dv", 1 << 30, LARGE)])
def test_descriptor(field, value, code):
    d = _desc(**{field: value})
    assert _fwd(d) == code and _bwd(d) == code
    assert dl._delta().convdelta_fwd_workspace(d) == code and dl._delta().convdelta_bwd_workspace(d) == code
    if field != "t":
        assert _step(d) == code


def test_missing_and_misplaced_buffers():
    d = _desc()
    assert _fwd(None) == NULL and _bwd(None) == NULL and _step(None) == NULL
    for n in ("q", "k", "v", "g", "beta", "y", "h", "work"):
        assert _fwd(d, **{n: None}) == NULL, n
    for n in ("dy", "q", "k", "v", "g", "beta", "states", "x", "dq", "dk", "dv", "dg", "db", "dh0", "work"):
        assert _bwd(d, **{n: None}) == NULL, n
    for n in ("q", "k", "v", "g", "beta", "state", "out", "y"):
        assert _step(d, **{n: None}) == NULL, n
    assert _fwd(d, q=_heads(None)) == NULL
    for n in ("batch", "row", "head"):
        assert _fwd(d, q=_heads(MB, **{n: -1})) == BAD and _fwd(d, k=_heads(MB, **{n: 1 << 60})) == LARGE
    assert _fwd(d, q=_heads(MB + 1)) == MISALIGNED and _fwd(d, g=4 * MB + 2) == MISALIGNED and _fwd(d, work=64 * MB + 8) == MISALIGNED
    n = 2 * 100 * 4 * 32 * 2
    for y in (MB, 3 * MB + n - 2, 4 * MB, 7 * MB, 64 * MB):
        assert _fwd(d, y=y) == ALIAS, y
    assert _fwd(d, h0=7 * MB) == ALIAS and _fwd(d, states=7 * MB + 4, x=20 * MB) == ALIAS and _fwd(d, states=20 * MB, x=6 * MB) == ALIAS
    assert _fwd(d, states=20 * MB) == NULL and _fwd(d, x=20 * MB) == NULL
    for k in ("dq", "dk", "dv", "dg", "db", "dh0"):
        assert _bwd(d, **{k: 7 * MB}) == ALIAS
    assert _bwd(d, dk=8 * MB) == ALIAS and _bwd(d, dv=9 * MB) == ALIAS
    assert _step(d, n=1) == BAD and _step(d, n=-1) == BAD and _step(d, out=6 * MB + 256) == ALIAS and _step(d, y=6 * MB) == ALIAS


def test_an_empty_batch_launches_nothing():
    none = dl.Heads(None, 0, 0, 0)
    d = _desc(b=0)
    assert _fwd(d, q=none, k=none, v=none, g=None, beta=None, y=None, h=None, work=None) == OK
    assert _bwd(d, dy=none, q=none, k=none, v=none, g=None, beta=None, states=None, x=None, dq=None, dk=None, dv=None, dg=None, db=None,
                dh0=None, work=None) == OK
    assert _step(d, q=none, k=none, v=none, g=None, beta=None, state=None, out=None, n=0, y=None) == OK


def test_the_workspace_grows_with_the_problem():
    size = dl._delta().convdelta_bwd_workspace
    assert size(_desc(t=0)) == 0 and 0 < size(_desc(t=1)) < size(_desc(t=64)) < size(_desc(t=65))
    assert dl._delta().convdelta_fwd_workspace(_desc()) < size(_desc())


def test_the_binding_needs_device_tensors():
    q, g, h = torch.zeros(1, 4, 2, 8), torch.zeros(1, 4, 2), torch.zeros(1, 2, 8, 8)
    for call in (lambda: igc.delta_rule(q, q, q, g, g), lambda: igc.delta_rule_bwd(q, q, q, q, g, g, igc.DeltaStates(h[:, None], q)),
                 lambda: igc.delta_rule_step(q[:, 0], q[:, 0], q[:, 0], g[:, 0], g[:, 0], h)):
        with pytest.raises(ValueError, match="GPU only"):
            call()


@pytest.mark.gpu
def test_the_binding_refuses_what_does_not_fit():
    dev = "cuda:0"
    q, v = torch.zeros(2, 20, 2, 8, device=dev), torch.zeros(2, 20, 4, 6, device=dev)
    g, h = torch.zeros(2, 20, 4, device=dev), torch.zeros(2, 4, 8, 6, device=dev)
    st = igc.DeltaStates(h[:, None].contiguous(), v)
    one = (q[:, 0], q[:, 0], v[:, 0], g[:, 0], g[:, 0])
    for error, call in (
            (ValueError, lambda: igc.delta_rule(q[0], q, v, g, g)), (TypeError, lambda: igc.delta_rule(q.double(), q, v, g, g)),
            (ValueError, lambda: igc.delta_rule(q.half(), q, v, g, g)), (ValueError, lambda: igc.delta_rule(q, q[:, :19], v, g, g)),
            (ValueError, lambda: igc.delta_rule(q, q, v[:, :, :3], g[:, :, :3], g[:, :, :3])),
            (ValueError, lambda: igc.delta_rule(q, q, v, g[:, :, :2], g)), (ValueError, lambda: igc.delta_rule(q, q, v, g, g.half())),
            (ValueError, lambda: igc.delta_rule(q, q, v, g, None)), (ValueError, lambda: igc.delta_rule(q, q, v, g, g, h0=h[:, :2])),
            (TypeError, lambda: igc.delta_rule(q, q, v, g, g, starts=torch.zeros(2, 20, device=dev))),
            (igc.ConvError, lambda: igc.delta_rule(q, q, v, g, g, scale=float("nan"))),
            (ValueError, lambda: igc.delta_rule(q, q, v, g, g, out=torch.zeros(2, 20, 4, 7, device=dev))),
            (igc.ConvError, lambda: igc.delta_rule(q, q, v, g, g, out=v)),
            (igc.ConvError, lambda: igc.delta_rule(*[torch.zeros(2, 20, 2, 129, device=dev)] * 2, v, g, g)),
            (ValueError, lambda: igc.delta_rule_bwd(v[:, :19], q, q, v, g, g, st)),
            (ValueError, lambda: igc.delta_rule_bwd(v.half(), q, q, v, g, g, st)),
            (ValueError, lambda: igc.delta_rule_bwd(v, q, q, v, g, g, None)),
            (ValueError, lambda: igc.delta_rule_bwd(v, q, q, v, g, g, st.states)),
            (ValueError, lambda: igc.delta_rule_bwd(v, q, q, v, g, g, st._replace(states=torch.zeros(2, 2, 4, 8, 6, device=dev)))),
            (ValueError, lambda: igc.delta_rule_bwd(v, q, q, v, g, g, st._replace(x=v[:, :19]))),
            (ValueError, lambda: igc.delta_rule_bwd(v, q, q, v, g, g, st, dh=h.half())),
            (ValueError, lambda: igc.delta_rule_step(*one, h[:, :2])),
            (ValueError, lambda: igc.delta_rule_step(*one, torch.zeros(3, 4, 8, 6, device=dev))),
            (TypeError, lambda: igc.delta_rule_step(*one, h, slots=torch.zeros(2, dtype=torch.int64, device=dev))),
            (ValueError, lambda: igc.delta_rule_step(*one, h, slots=torch.zeros(3, dtype=torch.int32, device=dev)))):
        with pytest.raises(error):
            call()


def test_rows_that_are_too_far_apart():
    """Offsets of 64 rows have to fit 32 bits: v, dy and y are refused where they would not."""
    far = _heads(1 << 40, 4, row=1 << 23, batch=0)
    near = _heads(1 << 40, 4, row=(1 << 23) - 1, batch=0)
    assert _fwd(_desc(), v=far) == LARGE
    assert _bwd(_desc(), v=far) == LARGE and _bwd(_desc(), dy=far) == LARGE
    assert _fwd(_desc(), v=near, beta=None) == NULL and _fwd(_desc(dv=1 << 22)) == LARGE
    lib = dl._delta()
    assert lib.convdelta_fwd_workspace(_desc(b=1, t=1, hk=1, hv=8, dv=1 << 20)) == LARGE
    assert lib.convdelta_fwd_workspace(_desc(b=1, t=1, hk=1, hv=8, dv=(1 << 20) - 1)) > 0


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [None, 1.0])
@pytest.mark.parametrize("dk,dv", [(0, 8), (8, 0), (0, 0)])
def test_heads_without_elements_are_refused(dk, dv, scale):
    dev = "cuda:0"
    q, v, g = torch.zeros(1, 4, 1, dk, device=dev), torch.zeros(1, 4, 1, dv, device=dev), torch.zeros(1, 4, 1, device=dev)
    h = torch.zeros(1, 1, dk, dv, device=dev)
    for call in (lambda: igc.delta_rule(q, q, v, g, g, scale=scale),
                 lambda: igc.delta_rule_bwd(v, q, q, v, g, g, igc.DeltaStates(h[:, None], v), scale=scale),
                 lambda: igc.delta_rule_step(q[:, 0], q[:, 0], v[:, 0], g[:, 0], g[:, 0], h, scale=scale)):
        with pytest.raises(ValueError, match="at least one element"):
            call()
