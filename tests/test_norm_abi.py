"""Host-side tests of the group norm's C ABI and of the binding's argument checks (no GPU needed).

Every call here returns before the library touches the GPU.
"""
import os
import re

import pytest
import torch

import implicit_gemm_conv_amd as igc
from implicit_gemm_conv_amd import norm as nm
from implicit_gemm_conv_amd.sequence import Rows

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, BAD, UNSUPPORTED, LARGE, ALIAS, MISALIGNED = 0, -1, -2, -3, -4, -5, -7
MB = 1 << 20


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "convnorm.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*(?:int|int64_t)\s+(convnorm_\w+)\s*\(", text, flags=re.M)))
    assert names == sorted(n for n, _, _ in nm.EXPORTS)
    for n in names:
        assert hasattr(nm._norm(), n), n


def _desc(**kw):
    return nm.NormDesc(**{**dict(n=2, p=100, c=64, groups=4, act=1, dtype=2, param_dtype=0, eps=1e-5), **kw})


def _fwd(d, x=None, w=MB, b=2 * MB, y=4 * MB, mean=8 * MB, rstd=9 * MB, work=16 * MB):
    return nm._norm().convnorm_group_fwd(d, Rows(16, 6400, 64) if x is None else x, w, b, y, mean, rstd, work, None)


@pytest.mark.parametrize("field,value,code", [
    ("n", -1, BAD), ("p", -1, BAD), ("c", 0, BAD), ("groups", 0, BAD), ("groups", 3, BAD), ("groups", 128, BAD), ("act", 2, BAD),
    ("act", -1, BAD), ("dtype", 3, UNSUPPORTED), ("param_dtype", 1, UNSUPPORTED), ("eps", -1e-5, BAD),
    ("eps", float("nan"), BAD), ("eps", float("inf"), BAD), ("c", 1 << 26, LARGE), ("p", 1 << 30, LARGE), ("n", 1 << 30, LARGE)])
def test_descriptor(field, value, code):
    d = _desc(**{field: value})
    assert _fwd(d) == code
    assert nm._norm().convnorm_group_fwd_workspace(d) == code and nm._norm().convnorm_group_bwd_workspace(d) == code
    r = Rows(16, 6400, 64)
    assert nm._norm().convnorm_group_bwd(d, r, r, MB, None, 2 * MB, 3 * MB, 4 * MB, None, None, 16 * MB, None) == code


def test_missing_and_misplaced_buffers():
    big = _desc(p=3000)
    assert _fwd(None) == NULL
    assert nm._norm().convnorm_group_fwd(_desc(), None, MB, None, 4 * MB, 8 * MB, 9 * MB, 16 * MB, None) == NULL
    assert _fwd(_desc(), x=Rows(None, 0, 0)) == NULL
    assert _fwd(_desc(), y=None) == NULL and _fwd(_desc(), mean=None) == NULL and _fwd(_desc(), rstd=None) == NULL
    assert _fwd(big, work=None) == NULL and _fwd(big, work=16 * MB + 8) == MISALIGNED
    assert _fwd(_desc(), x=Rows(17, 6400, 64)) == MISALIGNED and _fwd(_desc(), w=MB + 2) == MISALIGNED
    assert _fwd(_desc(), x=Rows(16, -1, 64)) == BAD and _fwd(_desc(), x=Rows(16, 1 << 61, 64)) == LARGE
    for y in (16, 16 + 2 * 100 * 64 * 2 - 2, MB + 4, 8 * MB, 9 * MB + 4):
        assert _fwd(_desc(), y=y) == ALIAS
    assert _fwd(_desc(), rstd=8 * MB + 4) == ALIAS
    bwd, r = nm._norm().convnorm_group_bwd, Rows(16, 6400, 64)
    for missing in range(2):
        stats = [2 * MB, 3 * MB]
        stats[missing] = None
        assert bwd(_desc(), r, r, MB, None, *stats, 4 * MB, None, None, 16 * MB, None) == NULL
    assert bwd(_desc(), r, r, MB, None, 2 * MB, 3 * MB, None, None, None, 16 * MB, None) == NULL
    assert bwd(_desc(), r, r, MB, None, 2 * MB, 3 * MB, 4 * MB, 5 * MB, 5 * MB, 16 * MB, None) == ALIAS
    assert bwd(_desc(), r, None, MB, None, 2 * MB, 3 * MB, 4 * MB, 5 * MB, None, 16 * MB, None) == NULL


def test_an_empty_batch_launches_nothing():
    none = Rows(None, 0, 0)
    assert _fwd(_desc(n=0), x=none, w=None, b=None, y=None, mean=None, rstd=None, work=None) == OK
    assert nm._norm().convnorm_group_bwd(_desc(n=0), none, none, None, None, None, None, None, None, None, None, None) == OK


def test_the_binding_needs_device_tensors():
    x, s = torch.zeros(2, 4, 8), torch.zeros(2, 2)
    for call in (lambda: igc.group_norm(x, 2), lambda: igc.group_norm_bwd(x, x, 2, s, s)):
        with pytest.raises(ValueError, match="GPU only"):
            call()


@pytest.mark.gpu
def test_the_binding_refuses_what_does_not_fit():
    dev = "cuda:0"
    x, w = torch.zeros(2, 20, 8, device=dev), torch.zeros(8, device=dev)
    s = torch.zeros(2, 2, device=dev)
    for error, call in (
            (ValueError, lambda: igc.group_norm(w, 2)), (TypeError, lambda: igc.group_norm(x.double(), 2)),
            (ValueError, lambda: igc.group_norm(x, 3)), (ValueError, lambda: igc.group_norm(x, 0)),
            (ValueError, lambda: igc.group_norm(x, 2, activation="gelu")), (ValueError, lambda: igc.group_norm(x, 2, weight=w[:7])),
            (ValueError, lambda: igc.group_norm(x, 2, weight=w.half())),
            (ValueError, lambda: igc.group_norm(x.half(), 2, weight=w, bias=w.half())),
            (ValueError, lambda: igc.group_norm(x, 2, weight=w.cpu())), (igc.ConvError, lambda: igc.group_norm(x, 2, eps=-1.0)),
            (ValueError, lambda: igc.group_norm(x, 2, out=torch.zeros(2, 20, 9, device=dev))),
            (igc.ConvError, lambda: igc.group_norm(x, 2, out=x)),
            (ValueError, lambda: igc.group_norm_bwd(x, x[:, :19], 2, s, s)), (ValueError, lambda: igc.group_norm_bwd(x, x.half(), 2, s, s)),
            (ValueError, lambda: igc.group_norm_bwd(x, x, 2, s[:, :1], s)), (ValueError, lambda: igc.group_norm_bwd(x, x, 2, None, s)),
            (ValueError, lambda: igc.group_norm_bwd(x, x, 4, s, s))):
        with pytest.raises(error):
            call()
