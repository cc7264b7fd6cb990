"""Gated delta rule of libconvfwd.so (include/convdelta.h): a recurrence whose state is a matrix,
written by key and read by query.

    import implicit_gemm_conv_amd as igc
    f = igc.delta_rule(q, k, v, log_decay, beta, train=True)      # q, k (B,T,Hk,Dk), v (B,T,Hv,Dv)
    g = igc.delta_rule_bwd(dy, q, k, v, log_decay, beta, f.states)
    y, state = igc.delta_rule_step(q_t, k_t, v_t, g_t, b_t, state)      # one row a stream

Argument marshalling only, as in the rest of the binding: the arithmetic runs in the HIP
kernels, on the current stream of the tensors' device, without synchronising; there is no CPU
fallback.  q, k, v and dy may be views with element stride 1 within a head (slices of one
projection); others are made contiguous first.  Formulas and rules: include/convdelta.h.
"""
import ctypes
from typing import NamedTuple, Optional

import torch

from . import _DTYPES, lib
from .sequence import _call, _dense, _out, _ptr, _slots, _starts, _workspace

STATE_ROWS = 64   # rows between the kept states of delta_rule


class Heads(ctypes.Structure):
    """Mirror of convdelta_heads."""
    _fields_ = [("data", ctypes.c_void_p)] + [(n, ctypes.c_int64) for n in ("batch_stride", "row_stride", "head_stride")]


class DeltaDesc(ctypes.Structure):
    """Mirror of convdelta_desc."""
    _fields_ = [(n, ctypes.c_int32) for n in ("b", "t", "hk", "hv", "dk", "dv", "dtype")] + [("scale", ctypes.c_float)]


_P, _I32, _I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
_HP, _DD = ctypes.POINTER(Heads), ctypes.POINTER(DeltaDesc)

# Every entry point include/convdelta.h declares: (name, restype, argtypes).
EXPORTS = [
    ("convdelta_fwd_workspace", _I64, [_DD]),
    ("convdelta_fwd", ctypes.c_int, [_DD, _HP, _HP, _HP] + [_P] * 10),
    ("convdelta_bwd_workspace", _I64, [_DD]),
    ("convdelta_bwd", ctypes.c_int, [_DD, _HP, _HP, _HP, _HP] + [_P] * 14),
    ("convdelta_step", ctypes.c_int, [_DD, _HP, _HP, _HP, _P, _P, _P, _P, _P, _I32, _P, _P]),
]

_lib = None


def _delta():
    """The loaded library with the delta rule's signatures set."""
    global _lib
    if _lib is None:
        handle = lib()
        for name, res, args in EXPORTS:
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


class DeltaStates(NamedTuple):
    """What the forward pass keeps for the backward pass."""
    states: torch.Tensor             # (B, ceil(T/64), Hv, Dk, Dv) fp32: the state before rows 0, 64, 128, ...
    x: torch.Tensor                  # (B, T, Hv, Dv) fp32: v less what the state held for k


class DeltaRule(NamedTuple):
    y: torch.Tensor
    h: torch.Tensor                  # (B, Hv, Dk, Dv) fp32: the state after the last row
    states: Optional[DeltaStates]    # for the backward pass


class DeltaRuleGrad(NamedTuple):
    dq: torch.Tensor
    dk: torch.Tensor
    dv: torch.Tensor
    dlog_decay: torch.Tensor         # (B, T, Hv) fp32
    dbeta: torch.Tensor              # (B, T, Hv) fp32
    dh0: torch.Tensor                # (B, Hv, Dk, Dv) fp32


def _heads(x, what, dims):
    """x as a (B, T, H, D) input ((B, H, D) for a step): a device tensor with element stride 1."""
    if not x.is_cuda:
        raise ValueError(f"{what} must be a device tensor: the delta rule runs on the GPU only")
    if x.dim() != dims:
        raise ValueError(f"{what} must have {dims} dimensions, got shape {tuple(x.shape)}")
    if x.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {x.dtype}")
    return x if x.stride(-1) == 1 or x.shape[-1] == 1 and x.is_contiguous() else x.contiguous()


def _inputs(q, k, v, log_decay, beta, scale, dims):
    """The row inputs, checked, and the descriptor's extents."""
    q, k, v = _heads(q, "q", dims), _heads(k, "k", dims), _heads(v, "v", dims)
    rows, (hk, dk), (hv, dv) = v.shape[:-2], k.shape[-2:], v.shape[-2:]
    device, dtype = v.device, v.dtype
    for t, what in ((q, "q"), (k, "k")):
        if t.shape != (*rows, hk, dk) or t.dtype is not dtype or t.device != device:
            raise ValueError(f"{what} must be {dtype} of shape {(*rows, hk, dk)} on {device}, "
                             f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    if dk < 1 or dv < 1:
        raise ValueError(f"heads must have at least one element, got {dk} of q and k and {dv} of v")
    if hk < 1 or hv < 1 or hv % hk:
        raise ValueError(f"the heads of v must be a multiple of those of q and k, got {hv} and {hk}")
    gates = (*rows, hv)
    log_decay = _dense(log_decay, gates, torch.float32, device, "log_decay")
    beta = _dense(beta, gates, torch.float32, device, "beta")
    if log_decay is None or beta is None:
        raise ValueError("log_decay and beta are needed")
    return q, k, v, log_decay, beta, dk ** -0.5 if scale is None else scale


def _view(x):
    """The C struct of a (B, T, H, D) or (B, H, D) view."""
    if x.dim() == 4:
        return Heads(x.data_ptr(), x.stride(0), x.stride(1), x.stride(2))
    return Heads(x.data_ptr(), x.stride(0), 0, x.stride(1))


def _describe(k, v, t, scale):
    return DeltaDesc(v.shape[0], t, k.shape[-2], v.shape[-2], k.shape[-1], v.shape[-1], _DTYPES[v.dtype], scale)


def delta_rule(q, k, v, log_decay, beta, scale=None, h0=None, starts=None, train=False, out=None) -> DeltaRule:
    """The gated delta rule over a sequence.

    q, k (B, T, Hk, Dk), Dk <= 128, and v (B, T, Hv, Dv) of one dtype, Hv a multiple of Hk (value head h reads
    key head h // (Hv / Hk)); log_decay and beta (B, T, Hv) fp32.  With a = exp(log_decay):
    S' = a S, S = S' + k (beta (v - S'^T k))^T, y = scale S^T q; scale is Dk^-0.5 if None.  q and k are
    taken as they are: a layer brings them to length one itself.  Log decays above zero cost precision, and a
    decay of zero begins a sequence.  h0 (B, Hv, Dk, Dv) fp32 is the state before the first row (zeros if
    None); starts (B, T), bool or uint8, marks rows that begin a new
    sequence.  train returns what delta_rule_bwd needs in `states`."""
    q, k, v, log_decay, beta, scale = _inputs(q, k, v, log_decay, beta, scale, 4)
    b, t, hv, dv = v.shape
    dk, device = k.shape[-1], v.device
    h0 = _dense(h0, (b, hv, dk, dv), torch.float32, device, "h0")
    starts = _starts(starts, b, t, device)
    y = v.new_empty((b, t, hv, dv)) if out is None else _out(out, (b, t, hv, dv), v.dtype, device, "out")
    h = v.new_empty((b, hv, dk, dv), dtype=torch.float32)
    states = DeltaStates(v.new_empty((b, -(-t // STATE_ROWS), hv, dk, dv), dtype=torch.float32),
                         v.new_empty((b, t, hv, dv), dtype=torch.float32)) if train else None
    kept = states if train else (None, None)
    d = _describe(k, v, t, scale)
    work = _workspace(_delta().convdelta_fwd_workspace(d), v)
    _call(v, _delta().convdelta_fwd, d, _view(q), _view(k), _view(v), log_decay.data_ptr(), beta.data_ptr(), _ptr(h0),
          _ptr(starts), y.data_ptr(), h.data_ptr(), *map(_ptr, kept), _ptr(work))
    return DeltaRule(y, h, states)


def delta_rule_bwd(dy, q, k, v, log_decay, beta, states, scale=None, starts=None, dh=None) -> DeltaRuleGrad:
    """Gradients of delta_rule: dy (B, T, Hv, Dv) that of y, dh (B, Hv, Dk, Dv) fp32 that of the last
    state; states are the ones delta_rule returned, the other arguments are the forward pass's."""
    q, k, v, log_decay, beta, scale = _inputs(q, k, v, log_decay, beta, scale, 4)
    b, t, hv, dv = v.shape
    hk, dk, device = k.shape[-2], k.shape[-1], v.device
    dy = _heads(dy, "dy", 4)
    if dy.shape != v.shape or dy.dtype is not v.dtype or dy.device != device:
        raise ValueError(f"dy must be {v.dtype} of shape {tuple(v.shape)} on {device}, got {dy.dtype} {tuple(dy.shape)} on {dy.device}")
    if not isinstance(states, DeltaStates):
        raise ValueError("states is needed, as delta_rule returned it: call it with train=True")
    x = _dense(states.x, (b, t, hv, dv), torch.float32, device, "states.x")
    states = _dense(states.states, (b, -(-t // STATE_ROWS), hv, dk, dv), torch.float32, device, "states.states")
    dh = _dense(dh, (b, hv, dk, dv), torch.float32, device, "dh")
    starts = _starts(starts, b, t, device)
    dq, dk_ = (v.new_empty((b, t, hk, dk)) for _ in range(2))
    dv_ = v.new_empty((b, t, hv, dv))
    dg, db = (v.new_empty((b, t, hv), dtype=torch.float32) for _ in range(2))
    dh0 = v.new_empty((b, hv, dk, dv), dtype=torch.float32)
    d = _describe(k, v, t, scale)
    work = _workspace(_delta().convdelta_bwd_workspace(d), v)
    _call(v, _delta().convdelta_bwd, d, _view(dy), _view(q), _view(k), _view(v), log_decay.data_ptr(), beta.data_ptr(),
          states.data_ptr(), x.data_ptr(), _ptr(starts), _ptr(dh), dq.data_ptr(), dk_.data_ptr(), dv_.data_ptr(), dg.data_ptr(),
          db.data_ptr(), dh0.data_ptr(), _ptr(work))
    return DeltaRuleGrad(dq, dk_, dv_, dg, db, dh0)


def delta_rule_step(q, k, v, log_decay, beta, h, scale=None, slots=None, h_out=None, out=None):
    """One row of each of B streams: y (B, Hv, Dv) from q, k (B, Hk, Dk), v (B, Hv, Dv), log_decay and
    beta (B, Hv) fp32 and the states h (S, Hv, Dk, Dv) fp32, updated in place or into h_out; slots as for
    seq_conv_step.  Returns (y, h)."""
    q, k, v, log_decay, beta, scale = _inputs(q, k, v, log_decay, beta, scale, 3)
    b, hv, dv = v.shape
    device = v.device
    streams = h.shape[0] if h.dim() else -1
    pool = (streams, hv, k.shape[-1], dv)
    _out(h, pool, torch.float32, device, "h")
    if h_out is None:
        h_out = h
    else:
        _out(h_out, pool, torch.float32, device, "h_out")
    slots = _slots(slots, b, streams, device)
    y = v.new_empty((b, hv, dv)) if out is None else _out(out, (b, hv, dv), v.dtype, device, "out")
    _call(v, _delta().convdelta_step, _describe(k, v, 1, scale), _view(q), _view(k), _view(v), log_decay.data_ptr(),
          beta.data_ptr(), h.data_ptr(), h_out.data_ptr(), _ptr(slots), streams, y.data_ptr())
    return y, h_out
