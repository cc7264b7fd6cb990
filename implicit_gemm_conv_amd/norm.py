"""Group norm of libconvfwd.so (include/convnorm.h): channels last, with an activation.

    import implicit_gemm_conv_amd as igc
    f = igc.group_norm(x, 32, weight=w, bias=b, activation="silu")       # x (N,[D,]H,W,C) or (N,C)
    g = igc.group_norm_bwd(dy, x, 32, f.mean, f.rstd, weight=w, bias=b, activation="silu")

Argument marshalling only, as in the rest of the binding: the arithmetic runs in the HIP
kernels, on the current stream of the tensors' device, without synchronising; there is no CPU
fallback.  Inputs may be views with channel stride 1; others are made contiguous first.
"""
import ctypes
from typing import NamedTuple, Optional

import torch

from . import _DTYPES, lib
from .sequence import ACTIVATIONS, Rows, _call, _dense, _out, _ptr, _rows, _sequence, _workspace


class NormDesc(ctypes.Structure):
    """Mirror of convnorm_desc."""
    _fields_ = [(n, ctypes.c_int32) for n in ("n", "p", "c", "groups", "act", "dtype", "param_dtype")] \
        + [("eps", ctypes.c_float)]


_P, _I64 = ctypes.c_void_p, ctypes.c_int64
_RP, _ND = ctypes.POINTER(Rows), ctypes.POINTER(NormDesc)

# Every entry point include/convnorm.h declares: (name, restype, argtypes).
EXPORTS = [
    ("convnorm_group_fwd_workspace", _I64, [_ND]),
    ("convnorm_group_fwd", ctypes.c_int, [_ND, _RP, _P, _P, _P, _P, _P, _P, _P]),
    ("convnorm_group_bwd_workspace", _I64, [_ND]),
    ("convnorm_group_bwd", ctypes.c_int, [_ND, _RP, _RP, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
]

_lib = None


def _norm():
    """The loaded library with the norm's signatures set."""
    global _lib
    if _lib is None:
        handle = lib()
        for name, res, args in EXPORTS:
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


class GroupNorm(NamedTuple):
    y: torch.Tensor
    mean: torch.Tensor               # (N, groups) fp32
    rstd: torch.Tensor               # (N, groups) fp32: 1 / sqrt(var + eps)


class GroupNormGrad(NamedTuple):
    dx: torch.Tensor
    dweight: Optional[torch.Tensor]  # (C) fp32, where there is a weight
    dbias: Optional[torch.Tensor]    # (C) fp32, where there is a bias


def _positions(x, what, like=None):
    """x (N, ..., C) as (N, P, C): the dimensions between are positions, a 2-D x has one a row."""
    if x.dim() < 2:
        raise ValueError(f"{what} must have at least 2 dimensions, got shape {tuple(x.shape)}")
    if like is not None and x.shape != like.shape:
        raise ValueError(f"{what} must have shape {tuple(like.shape)}, got {tuple(x.shape)}")
    return _sequence(x if x.dim() == 3 else x[:, None] if x.dim() == 2 else x.flatten(1, -2), what)


def _describe(x, groups, weight, bias, activation, eps):
    """The descriptor, and weight and bias checked."""
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of 'none', 'silu', got {activation!r}")
    n, p, c = x.shape
    groups = int(groups)
    if groups < 1 or c < 1 or c % groups:
        raise ValueError(f"groups must divide the {c} channels, got {groups}")
    given = [t for t in (weight, bias) if t is not None]
    kind = given[0].dtype if given else x.dtype
    if kind not in (x.dtype, torch.float32):
        raise ValueError(f"weight and bias must be {x.dtype} or torch.float32, got {kind}")
    weight, bias = (_dense(t, (c,), kind, x.device, what) for t, what in ((weight, "weight"), (bias, "bias")))
    return NormDesc(n, p, c, groups, act, _DTYPES[x.dtype], _DTYPES[kind], eps), weight, bias


def group_norm(x, groups, weight=None, bias=None, activation=None, eps=1e-5, out=None) -> GroupNorm:
    """Group norm over channels-last positions, with an activation (None or "silu").

    x (N, ..., C): the mean and the biased variance of each n and each of `groups` runs of C / groups
    neighbouring channels are taken over all positions between (a 2-D x is normalised row by row);
    weight and bias (C) of x's dtype or fp32, both of one type, 1 and 0 where None.  Returns y in
    x's dtype and shape, and the fp32 statistics that group_norm_bwd needs."""
    rows = _positions(x, "x")
    d, weight, bias = _describe(rows, groups, weight, bias, activation, eps)
    y = rows.new_empty(x.shape) if out is None else _out(out, x.shape, x.dtype, x.device, "out")
    mean, rstd = rows.new_empty((2, d.n, d.groups), dtype=torch.float32).unbind()
    work = _workspace(_norm().convnorm_group_fwd_workspace(d), rows)
    _call(rows, _norm().convnorm_group_fwd, d, _rows(rows), _ptr(weight), _ptr(bias), y.data_ptr(), mean.data_ptr(),
          rstd.data_ptr(), _ptr(work))
    return GroupNorm(y, mean, rstd)


def group_norm_bwd(dy, x, groups, mean, rstd, weight=None, bias=None, activation=None, eps=1e-5) -> GroupNormGrad:
    """Gradients of group_norm: dy that of y; x, mean and rstd, and the other arguments, are the
    forward pass's (eps is not used: rstd holds it)."""
    d_rows, rows = _positions(dy, "dy"), _positions(x, "x", dy)
    if rows.dtype is not d_rows.dtype or rows.device != d_rows.device:
        raise ValueError(f"x must be {dy.dtype} on {dy.device}, got {x.dtype} on {x.device}")
    d, weight, bias = _describe(rows, groups, weight, bias, activation, eps)
    stats = (d.n, d.groups)
    mean = _dense(mean, stats, torch.float32, rows.device, "mean")
    rstd = _dense(rstd, stats, torch.float32, rows.device, "rstd")
    if mean is None or rstd is None:
        raise ValueError("mean and rstd are needed: they are what group_norm returned")
    dx = rows.new_empty(x.shape)
    dw, db = (None if t is None else rows.new_empty((d.c,), dtype=torch.float32) for t in (weight, bias))
    work = _workspace(_norm().convnorm_group_bwd_workspace(d), rows)
    _call(rows, _norm().convnorm_group_bwd, d, _rows(d_rows), _rows(rows), _ptr(weight), _ptr(bias), mean.data_ptr(),
          rstd.data_ptr(), dx.data_ptr(), _ptr(dw), _ptr(db), _ptr(work))
    return GroupNormGrad(dx, dw, db)
