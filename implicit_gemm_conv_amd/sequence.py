"""Sequence operators of libconvfwd.so (include/convseq.h): what a recurrent block puts around
its projections.

    import implicit_gemm_conv_amd as igc
    f = igc.seq_conv(x, w, bias=b, activation="silu", keep8=True)       # x (B,T,C), w (C,K)
    s = igc.gated_scan(f.y, gate_r, gate_i, lam, train=True, keep8=True)
    g = igc.gated_scan_bwd(dy, *s.kept, lam, s.states)
    d = igc.seq_conv_bwd(g.dx, f.kept, w, bias=b, activation="silu")
    y, state = igc.seq_conv_step(x_t, w, state, bias=b, activation="silu")   # one row a stream
    y, h = igc.gated_scan_step(y, r_t, i_t, lam, h)
    p = igc.pack8(x); x8 = igc.unpack8(p)

Argument marshalling only, as in the rest of the binding: the arithmetic runs in the HIP
kernels, on the current stream of the tensors' device, without synchronising; there is no
CPU fallback.  Inputs (B, T, C) may be views with channel stride 1 (a column slice of a wider
projection); others are made contiguous first.  Formulas and rules: include/convseq.h.
"""
import ctypes
import math
from typing import NamedTuple, Optional, Tuple

import torch

from . import _DTYPES, _check, lib

STATE_ROWS = 64   # rows between the kept states of gated_scan
GROUP_ROWS = 16   # rows of a channel that share a power of two in 8 bits
ACTIVATIONS = {"none": 0, None: 0, "silu": 1}


class Rows(ctypes.Structure):
    """Mirror of convseq_rows."""
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64)]


class KeptPtr(ctypes.Structure):
    """Mirror of convseq_kept."""
    _fields_ = [("q", ctypes.c_void_p), ("e", ctypes.c_void_p)]


_Kept3 = KeptPtr * 3


class ConvDesc(ctypes.Structure):
    """Mirror of convseq_conv_desc."""
    _fields_ = [(n, ctypes.c_int32) for n in ("b", "t", "c", "k", "act", "dtype")]


class ScanDesc(ctypes.Structure):
    """Mirror of convseq_scan_desc."""
    _fields_ = [(n, ctypes.c_int32) for n in ("b", "t", "c", "dtype")] + [("decay", ctypes.c_float)]


_P, _I32, _I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
_RP, _KP = ctypes.POINTER(Rows), ctypes.POINTER(KeptPtr)
_CD, _SD = ctypes.POINTER(ConvDesc), ctypes.POINTER(ScanDesc)

# Every entry point include/convseq.h declares: (name, restype, argtypes).
EXPORTS = [
    ("convseq_conv_fwd", ctypes.c_int, [_CD, _RP, _P, _P, _P, _P, _P, _P, _KP, _P]),
    ("convseq_conv_bwd_workspace", _I64, [_CD]),
    ("convseq_conv_bwd", ctypes.c_int, [_CD, _RP, _RP, _KP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    ("convseq_conv_step", ctypes.c_int, [_CD, _P, _I64, _P, _P, _P, _P, _P, _I32, _P, _P]),
    ("convseq_scan_fwd_workspace", _I64, [_SD]),
    ("convseq_scan_fwd", ctypes.c_int, [_SD, _RP, _RP, _RP, _P, _P, _P, _P, _P, _P, _KP, _P, _P]),
    ("convseq_scan_bwd_workspace", _I64, [_SD]),
    ("convseq_scan_bwd", ctypes.c_int, [_SD, _RP, _RP, _RP, _RP, _KP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    ("convseq_scan_step", ctypes.c_int, [_SD, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _P, _I32, _P, _P]),
    ("convseq_pack8", ctypes.c_int, [_I32, _I32, _I32, _I32, _RP, _KP, _P]),
    ("convseq_unpack8", ctypes.c_int, [_I32, _I32, _I32, _I32, _KP, _P, _P]),
]

_lib = None


def _seq():
    """The loaded library with the sequence entry points' signatures set."""
    global _lib
    if _lib is None:
        handle = lib()
        for name, res, args in EXPORTS:
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


class Packed8(NamedTuple):
    """A tensor in 8 bits: q (B, groups of 16 rows, 2, C, 8) int8 and e (B, groups, C) uint8; the
    value held at row t is q[b, t // 16, t % 16 // 8, c, t % 8] * 2^(e - 127), NaN where e is 255.
    shape and dtype are the original's."""
    q: torch.Tensor
    e: torch.Tensor
    shape: torch.Size
    dtype: torch.dtype


class SeqConv(NamedTuple):
    y: torch.Tensor
    state: torch.Tensor              # (B, K-1, C): the carried rows of the next piece
    kept: Optional[Packed8]          # x in 8 bits


class SeqConvGrad(NamedTuple):
    dx: torch.Tensor
    dw: torch.Tensor                 # (C, K) fp32
    dbias: Optional[torch.Tensor]    # (C) fp32, where there is a bias
    dstate: Optional[torch.Tensor]   # (B, K-1, C), where there are carried rows


class GatedScan(NamedTuple):
    y: torch.Tensor
    h: torch.Tensor                  # (B, C) fp32: the state after the last row
    states: Optional[torch.Tensor]   # (B, ceil(T/64), C) fp32, for the backward pass
    kept: Optional[Tuple[Packed8, Packed8, Packed8]]   # x, gate_r, gate_i in 8 bits


class GatedScanGrad(NamedTuple):
    dx: torch.Tensor
    dgate_r: torch.Tensor
    dgate_i: torch.Tensor
    dlam: torch.Tensor               # (C) fp32
    dh0: torch.Tensor                # (B, C) fp32


# ---- argument checks ----------------------------------------------------------------------------


def _sequence(x, what, like=None, dims=3):
    """x as a (B, T, C) input ((B, C) for a step): a device tensor with channel stride 1."""
    if not x.is_cuda:
        raise ValueError(f"{what} must be a device tensor: the sequence operators run on the GPU only")
    if x.dim() != dims:
        raise ValueError(f"{what} must have {dims} dimensions, got shape {tuple(x.shape)}")
    if like is None:
        if x.dtype not in _DTYPES:
            raise TypeError(f"unsupported dtype {x.dtype}")
    elif x.shape != like.shape or x.dtype is not like.dtype or x.device != like.device:
        raise ValueError(f"{what} must be {like.dtype} of shape {tuple(like.shape)} on {like.device}, "
                         f"got {x.dtype} {tuple(x.shape)} on {x.device}")
    return x if x.stride(-1) == 1 or x.shape[-1] == 1 and x.is_contiguous() else x.contiguous()


def _dense(t, shape, dtype, device, what):
    """A dense operand of one exact shape and type (None stays None)."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.device != device:
        raise ValueError(f"{what} must be a {dtype} tensor of shape {tuple(shape)} on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t if t.is_contiguous() else t.contiguous()


def _out(t, shape, dtype, device, what):
    """An output the caller gave: as _dense, but it has to be contiguous as it is."""
    if t.shape != shape or t.dtype is not dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t


def _starts(starts, b, t, device):
    if starts is None:
        return None
    if starts.dtype not in (torch.bool, torch.uint8):
        raise TypeError("starts must be a bool or uint8 tensor")
    return _dense(starts, (b, t), starts.dtype, device, "starts")


def _kept_input(p, shape, device, what):
    """An input given in 8 bits, standing for a (B, T, C) tensor: its C struct."""
    b, t, c = shape
    groups = -(-t // GROUP_ROWS)
    q, e, held = p.q, p.e, p.shape
    held = held[1] if len(held) == 3 else held[0] if len(held) == 2 else math.prod(held[1:-1])
    if held != t or q.shape != (b, groups, 2, c, GROUP_ROWS // 2) or e.shape != (b, groups, c) \
            or q.dtype is not torch.int8 or e.dtype is not torch.uint8 or q.device != device or e.device != device \
            or not q.is_contiguous() or not e.is_contiguous():
        raise ValueError(f"{what} in 8 bits must stand for a tensor of shape {tuple(shape)} on {device}")
    return p


def _filter(w, bias, x, activation):
    """w (C, K) and bias (C), checked, and the activation's number."""
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of 'none', 'silu', got {activation!r}")
    shape, c = w.shape, x.shape[-1]
    if len(shape) != 2 or shape[0] != c or shape[1] < 1:
        raise ValueError(f"w must be (C, K) with C = {c}, got {tuple(shape)}")
    device, dtype = x.device, x.dtype
    return (_dense(w, shape, dtype, device, "w"), None if bias is None else _dense(bias, (c,), dtype, device, "bias"),
            shape[1], act)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _rows(x):
    batch, row, _ = x.stride()
    return Rows(x.data_ptr(), batch, row)


def _new_kept(x, shape):
    """Room for x (B, T, C) in 8 bits, as the tensor of the given shape."""
    b, t, c = x.shape
    groups = -(-t // GROUP_ROWS)
    return Packed8(x.new_empty((b, groups, 2, c, GROUP_ROWS // 2), dtype=torch.int8),
                   x.new_empty((b, groups, c), dtype=torch.uint8), shape, x.dtype)


def _kept_ptr(p):
    """One convseq_kept, NULL for none."""
    return None if p is None else KeptPtr(p.q.data_ptr(), p.e.data_ptr())


def _kept_ptrs(kept):
    """A C array of three convseq_kept, NULL for none."""
    return None if kept is None else _Kept3(*[(p.q.data_ptr(), p.e.data_ptr()) for p in kept])


def _call(x, fn, *args):
    """fn(*args, stream) on the current stream of x's device, which is made current if it is not."""
    index = x.get_device()
    if index == torch.cuda.current_device():
        return _check(fn(*args, _raw_stream(index)))
    with torch.cuda.device(index):
        return _check(fn(*args, _raw_stream(index)))


def _raw_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


# the handle alone, without a Stream object around it (2 us), where this torch offers it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


def _workspace(n_bytes, x):
    return x.new_empty(_check(n_bytes), dtype=torch.uint8) if n_bytes else None


# ---- causal depthwise convolution ---------------------------------------------------------------


def seq_conv(x, w, bias=None, activation=None, state=None, starts=None, keep8=False, out=None) -> SeqConv:
    """Causal depthwise convolution along a sequence.

    x (B, T, C); w (C, K), K <= 8, and bias (C) of x's dtype; activation None or "silu"; state
    (B, K-1, C), the rows before x (zeros if None); starts (B, T), bool or uint8, marks rows that
    begin a new sequence.  keep8 also writes x in 8 bits for the backward pass, in groups of 16 rows
    that starts do not divide: one NaN or infinity is NaN in all rows of its group there.
    """
    x = _sequence(x, "x")
    b, t, c = x.shape
    w, bias, k, act = _filter(w, bias, x, activation)
    state = _dense(state, (b, k - 1, c), x.dtype, x.device, "state")
    starts = _starts(starts, b, t, x.device)
    y = x.new_empty((b, t, c)) if out is None \
        else _out(out, (b, t, c), x.dtype, x.device, "out")
    last = x.new_empty((b, k - 1, c))
    kept = _new_kept(x, x.shape) if keep8 else None
    d = ConvDesc(b, t, c, k, act, _DTYPES[x.dtype])
    _call(x, _seq().convseq_conv_fwd, d, _rows(x), w.data_ptr(), _ptr(bias), _ptr(state), _ptr(starts), y.data_ptr(),
          last.data_ptr(), _kept_ptr(kept))
    return SeqConv(y, last, kept)


def seq_conv_bwd(dy, x, w, bias=None, activation=None, state=None, starts=None, dstate=None) -> SeqConvGrad:
    """Gradients of seq_conv: dy (B, T, C) that of y, dstate (B, K-1, C) that of the carried rows
    it returned.  x is the forward input, or what it kept of it in 8 bits (Packed8); the other
    arguments are the forward pass's."""
    dy = _sequence(dy, "dy")
    b, t, c = dy.shape
    w, bias, k, act = _filter(w, bias, dy, activation)
    packed = isinstance(x, Packed8)
    x = _kept_input(x, dy.shape, dy.device, "x") if packed else _sequence(x, "x", dy)
    state = _dense(state, (b, k - 1, c), dy.dtype, dy.device, "state")
    dlast = _dense(dstate, (b, k - 1, c), dy.dtype, dy.device, "dstate")
    starts = _starts(starts, b, t, dy.device)
    dx = dy.new_empty((b, t, c))
    dw = dy.new_empty((c, k), dtype=torch.float32)
    db = None if bias is None else dy.new_empty((c,), dtype=torch.float32)
    dfirst = None if state is None else torch.empty_like(state)
    d = ConvDesc(b, t, c, k, act, _DTYPES[dy.dtype])
    work = _workspace(_seq().convseq_conv_bwd_workspace(d), dy)
    _call(dy, _seq().convseq_conv_bwd, d, _rows(dy), None if packed else _rows(x), _kept_ptr(x if packed else None),
          w.data_ptr(), _ptr(bias), _ptr(state), _ptr(starts), _ptr(dlast), dx.data_ptr(), dw.data_ptr(), _ptr(db),
          _ptr(dfirst), _ptr(work))
    return SeqConvGrad(dx, dw, db, dfirst)


def _slots(slots, b, pool, device):
    """The streams' slots in a pool of states, checked; None where stream b has slot b."""
    if slots is None:
        if pool != b:
            raise ValueError(f"state holds {pool} streams, x has {b}: give slots")
        return None
    if slots.dtype != torch.int32:
        raise TypeError("slots must be an int32 tensor")
    return _dense(slots, (b,), torch.int32, device, "slots")


def seq_conv_step(x, w, state, bias=None, activation=None, slots=None, state_out=None, out=None):
    """One row of each of B streams: y (B, C) from x (B, C) and the carried rows state
    (S, K-1, C), which move on by one, in place or into state_out.  Stream b's rows are slot b,
    or slots[b] (int32); a stream whose slot lies outside the pool is idle: its y is zero and no
    state is touched.  Slots that no stream names are not copied to state_out: where streams may be
    idle, update in place rather than swap two buffers.  Two streams must not share a slot.
    Returns (y, state)."""
    x = _sequence(x, "x", dims=2)
    b, c = x.shape
    w, bias, k, act = _filter(w, bias, x, activation)
    device, dtype = x.device, x.dtype
    streams = state.shape[0] if state.dim() else -1
    pool = (streams, k - 1, c)
    _out(state, pool, dtype, device, "state")
    if state_out is None:
        state_out = state
    else:
        _out(state_out, pool, dtype, device, "state_out")
    slots = _slots(slots, b, streams, device)
    y = x.new_empty((b, c)) if out is None else _out(out, (b, c), dtype, device, "out")
    _call(x, _seq().convseq_conv_step, ConvDesc(b, 1, c, k, act, _DTYPES[dtype]), x.data_ptr(), x.stride(0), w.data_ptr(),
          None if bias is None else bias.data_ptr(), state.data_ptr(), state_out.data_ptr(), _ptr(slots), streams,
          y.data_ptr())
    return y, state_out


# ---- gated linear recurrence --------------------------------------------------------------------


def gated_scan(x, gate_r, gate_i, lam, decay=8.0, h0=None, starts=None, train=False, keep8=False,
               out=None) -> GatedScan:
    """The gated linear recurrence h_t = a h_{t-1} + sqrt(1 - a^2) sigmoid(gate_i) x_t with
    a = exp(-decay softplus(lam) sigmoid(gate_r)), over x, gate_r, gate_i (B, T, C) of one dtype;
    lam (C) and h0 (B, C) fp32.  starts as for seq_conv; a row at a start is scaled by
    sqrt(1 - a^2) like any other.  train returns the states that
    gated_scan_bwd needs, keep8 also x, gate_r and gate_i in 8 bits (groups as for seq_conv)."""
    x = _sequence(x, "x")
    gate_r, gate_i = _sequence(gate_r, "gate_r", x), _sequence(gate_i, "gate_i", x)
    b, t, c = x.shape
    lam = _dense(lam, (c,), torch.float32, x.device, "lam")
    h0 = _dense(h0, (b, c), torch.float32, x.device, "h0")
    starts = _starts(starts, b, t, x.device)
    y = x.new_empty((b, t, c)) if out is None \
        else _out(out, (b, t, c), x.dtype, x.device, "out")
    h = x.new_empty((b, c), dtype=torch.float32)
    states = x.new_empty((b, -(-t // STATE_ROWS), c), dtype=torch.float32) if train else None
    kept = tuple(_new_kept(x, x.shape) for _ in range(3)) if keep8 else None
    d = ScanDesc(b, t, c, _DTYPES[x.dtype], decay)
    work = _workspace(_seq().convseq_scan_fwd_workspace(d), x)
    _call(x, _seq().convseq_scan_fwd, d, _rows(x), _rows(gate_r), _rows(gate_i), lam.data_ptr(), _ptr(h0), _ptr(starts),
          y.data_ptr(), h.data_ptr(), _ptr(states), _kept_ptrs(kept), _ptr(work))
    return GatedScan(y, h, states, kept)


def gated_scan_bwd(dy, x, gate_r, gate_i, lam, states, decay=8.0, starts=None, dh=None) -> GatedScanGrad:
    """Gradients of gated_scan: dy (B, T, C) that of y, dh (B, C) fp32 that of the last state.
    x, gate_r and gate_i are the forward inputs, or what it kept of them in 8 bits (Packed8, all
    three); states are the ones it returned."""
    dy = _sequence(dy, "dy")
    b, t, c = dy.shape
    ins = (x, gate_r, gate_i)
    packed = isinstance(x, Packed8)
    if any(isinstance(v, Packed8) != packed for v in ins):
        raise ValueError("x, gate_r and gate_i must all be tensors or all be in 8 bits")
    names = ("x", "gate_r", "gate_i")
    ins = tuple(_kept_input(v, dy.shape, dy.device, n) if packed else _sequence(v, n, dy) for v, n in zip(ins, names))
    lam = _dense(lam, (c,), torch.float32, dy.device, "lam")
    states = _dense(states, (b, -(-t // STATE_ROWS), c), torch.float32, dy.device, "states")
    if states is None:
        raise ValueError("states is needed: call gated_scan with train=True")
    dh = _dense(dh, (b, c), torch.float32, dy.device, "dh")
    starts = _starts(starts, b, t, dy.device)
    dx, dr, di = (dy.new_empty((b, t, c)) for _ in range(3))
    dlam = dy.new_empty((c,), dtype=torch.float32)
    dh0 = dy.new_empty((b, c), dtype=torch.float32)
    d = ScanDesc(b, t, c, _DTYPES[dy.dtype], decay)
    rows = (None,) * 3 if packed else tuple(_rows(v) for v in ins)
    work = _workspace(_seq().convseq_scan_bwd_workspace(d), dy)
    _call(dy, _seq().convseq_scan_bwd, d, _rows(dy), *rows, _kept_ptrs(ins if packed else None), lam.data_ptr(),
          states.data_ptr(), _ptr(starts), _ptr(dh), dx.data_ptr(), dr.data_ptr(), di.data_ptr(), dlam.data_ptr(),
          dh0.data_ptr(), _ptr(work))
    return GatedScanGrad(dx, dr, di, dlam, dh0)


def gated_scan_step(x, gate_r, gate_i, lam, h, decay=8.0, slots=None, h_out=None, out=None):
    """One row of each of B streams through the recurrence: y (B, C) from x, gate_r, gate_i
    (B, C) and the states h (S, C) fp32, updated in place or into h_out; slots as for
    seq_conv_step.  Returns (y, h)."""
    x = _sequence(x, "x", dims=2)
    gate_r, gate_i = _sequence(gate_r, "gate_r", x, 2), _sequence(gate_i, "gate_i", x, 2)
    b, c = x.shape
    device, dtype = x.device, x.dtype
    lam = _dense(lam, (c,), torch.float32, device, "lam")
    streams = h.shape[0] if h.dim() else -1
    _out(h, (streams, c), torch.float32, device, "h")
    if h_out is None:
        h_out = h
    else:
        _out(h_out, (streams, c), torch.float32, device, "h_out")
    slots = _slots(slots, b, streams, device)
    y = x.new_empty((b, c)) if out is None else _out(out, (b, c), dtype, device, "out")
    _call(x, _seq().convseq_scan_step, ScanDesc(b, 1, c, _DTYPES[dtype], decay), x.data_ptr(), x.stride(0),
          gate_r.data_ptr(), gate_r.stride(0), gate_i.data_ptr(), gate_i.stride(0), lam.data_ptr(), h.data_ptr(),
          h_out.data_ptr(), _ptr(slots), streams, y.data_ptr())
    return y, h_out


# ---- activations in 8 bits ----------------------------------------------------------------------


def pack8(x) -> Packed8:
    """x (B, ..., C) in 8 bits.  The dimensions between the first and the last are taken as one
    row axis (a channels-last image's positions); groups of 16 consecutive rows of a channel
    share a power of two, and are read back as NaN if one of them is NaN or infinite.  A 2-D x is
    one sequence of rows."""
    if x.dim() < 2:
        raise ValueError(f"x must have at least 2 dimensions, got shape {tuple(x.shape)}")
    shape = x.shape
    rows = _sequence(x if x.dim() == 3 else x[None] if x.dim() == 2 else x.flatten(1, -2), "x")
    b, t, c = rows.shape
    kept = _new_kept(rows, shape)
    _call(rows, _seq().convseq_pack8, b, t, c, _DTYPES[rows.dtype], _rows(rows), _kept_ptr(kept))
    return kept


def unpack8(p: Packed8, dtype=None, out=None) -> torch.Tensor:
    """The values a Packed8 holds, in its original's dtype or the one given."""
    dtype = p.dtype if dtype is None else dtype
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}")
    if not p.q.is_cuda:
        raise ValueError("q and e must be device tensors: the sequence operators run on the GPU only")
    shape, c = p.shape, p.shape[-1]
    b, t = (1, shape[0]) if len(shape) == 2 else (shape[0], math.prod(shape[1:-1]))
    _kept_input(p, (b, t, c), p.q.device, "p")
    y = p.q.new_empty(shape, dtype=dtype) if out is None else _out(out, shape, dtype, p.q.device, "out")
    _call(p.q, _seq().convseq_unpack8, b, t, c, _DTYPES[dtype], _kept_ptr(p), y.data_ptr())
    return y
