"""Host-side tests of the sequence operators' C ABI and of the binding's argument checks (no GPU needed).

Every call here returns before the library touches the GPU.
"""
import ctypes
import os
import re

import pytest
import torch

import implicit_gemm_conv_amd as igc
from implicit_gemm_conv_amd import sequence as sq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "convseq.h")
OK, NULL, BAD, UNSUPPORTED, LARGE, ALIAS, MISALIGNED = 0, -1, -2, -3, -4, -5, -7
MB = 1 << 20


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*(?:int|int64_t)\s+(convseq_\w+)\s*\(", text, flags=re.M)))
    assert names == sorted(n for n, _, _ in sq.EXPORTS)
    for n in names:
        assert hasattr(sq._seq(), n), n


def test_constants_match_the_header():
    text = open(HEADER).read()
    assert f"CONVSEQ_STATE_ROWS = {sq.STATE_ROWS}" in text and f"CONVSEQ_GROUP_ROWS = {sq.GROUP_ROWS}" in text


def _conv(**kw):
    return sq.ConvDesc(**{**dict(b=2, t=100, c=64, k=4, act=1, dtype=2), **kw})


def _scan(**kw):
    return sq.ScanDesc(**{**dict(b=2, t=100, c=64, dtype=2, decay=8.0), **kw})


def _rows(at, **kw):
    return sq.Rows(at, kw.get("batch", 6400), kw.get("row", 64))


def _conv_fwd(d, x=None, w=MB, bias=None, state=None, starts=None, y=4 * MB, last=None, kept=None):
    return sq._seq().convseq_conv_fwd(d, _rows(16) if x is None else x, w, bias, state, starts, y, last, kept, None)


@pytest.mark.parametrize("field,value,code", [("b", -1, BAD), ("t", -1, BAD), ("c", 0, BAD), ("k", 0, BAD), ("k", 9, UNSUPPORTED),
                                              ("act", 2, BAD), ("act", -1, BAD), ("dtype", 3, UNSUPPORTED),
                                              ("c", 1 << 26, LARGE), ("b", 1 << 22, LARGE), ("t", 1 << 30, LARGE)])
def test_conv_descriptor(field, value, code):
    d = _conv(**{field: value})
    assert _conv_fwd(d) == code
    assert sq._seq().convseq_conv_bwd_workspace(d) == code
    if field != "t":
        assert sq._seq().convseq_conv_step(d, 16, 64, MB, None, 2 * MB, 2 * MB, None, 2, 4 * MB, None) == code


@pytest.mark.parametrize("field,value,code", [("b", -1, BAD), ("t", -1, BAD), ("c", 0, BAD), ("dtype", -1, UNSUPPORTED),
                                              ("decay", 0.0, BAD), ("decay", -1.0, BAD), ("decay", float("nan"), BAD),
                                              ("decay", float("inf"), BAD), ("t", 1 << 30, LARGE)])
def test_scan_descriptor(field, value, code):
    d, r = _scan(**{field: value}), _rows(16)
    lib = sq._seq()
    assert lib.convseq_scan_fwd(d, r, r, r, MB, None, None, 4 * MB, None, None, None, 8 * MB, None) == code
    assert lib.convseq_scan_fwd_workspace(d) == code and lib.convseq_scan_bwd_workspace(d) == code
    if field != "t":
        assert lib.convseq_scan_step(d, 16, 64, 16, 64, 16, 64, MB, 2 * MB, 2 * MB, None, 2, 4 * MB, None) == code


def test_missing_and_misplaced_buffers():
    lib = sq._seq()
    assert _conv_fwd(None) == NULL
    assert lib.convseq_conv_fwd(_conv(), None, MB, None, None, None, 4 * MB, None, None, None) == NULL
    assert _conv_fwd(_conv(), x=_rows(None)) == NULL
    assert _conv_fwd(_conv(), w=None) == NULL and _conv_fwd(_conv(), y=None) == NULL
    assert _conv_fwd(_conv(), kept=sq.KeptPtr(8 * MB, None)) == NULL
    assert _conv_fwd(_conv(), x=_rows(17)) == MISALIGNED and _conv_fwd(_conv(dtype=0), bias=MB + 2) == MISALIGNED
    assert _conv_fwd(_conv(), x=_rows(16, row=-64)) == BAD and _conv_fwd(_conv(), x=_rows(16, batch=1 << 61)) == LARGE
    n = 2 * 100 * 64 * 2
    for y in (16, 16 + n - 2, MB, 4 * MB):
        assert _conv_fwd(_conv(), y=y, kept=sq.KeptPtr(4 * MB, 8 * MB)) == ALIAS
    assert _conv_fwd(_conv(), last=4 * MB + n - 2) == ALIAS and _conv_fwd(_conv(), last=MB + 8) == ALIAS
    r, k3 = _rows(16), (sq.KeptPtr * 3)(*[sq.KeptPtr(8 * MB + j * MB, 12 * MB + j * MB) for j in range(3)])
    bwd = lib.convseq_scan_bwd
    rest = (MB, 2 * MB, None, None, 4 * MB, 5 * MB, 6 * MB, 7 * MB, None, 32 * MB, None)
    assert bwd(_scan(), r, r, r, r, k3, *rest) == BAD            # as they were and in 8 bits at once
    assert bwd(_scan(), r, r, r, None, None, *rest) == NULL
    assert bwd(_scan(), r, None, None, None, None, *rest) == NULL
    assert bwd(_scan(), None, r, r, r, None, *rest) == NULL
    assert bwd(_scan(), r, r, r, r, None, *rest[:5], 4 * MB, *rest[6:]) == ALIAS
    assert bwd(_scan(), r, r, r, r, None, *rest[:1], None, *rest[2:]) == NULL          # states
    assert bwd(_scan(), r, r, r, r, None, *rest[:9], None, None) == NULL               # workspace
    assert bwd(_scan(), r, r, r, r, None, *rest[:9], 32 * MB + 8, None) == MISALIGNED
    cb = lib.convseq_conv_bwd
    assert cb(_conv(), r, r, sq.KeptPtr(MB, 2 * MB), *[4 * MB] * 11) == BAD
    assert cb(_conv(), r, None, None, *[4 * MB] * 11) == NULL


def test_step_pools():
    step = sq._seq().convseq_conv_step
    assert step(_conv(), 16, 64, MB, None, 2 * MB, 2 * MB, None, 1, 4 * MB, None) == BAD      # fewer slots than streams
    assert step(_conv(), 16, 64, MB, None, 2 * MB, 2 * MB, None, -1, 4 * MB, None) == BAD
    assert step(_conv(), 16, 64, MB, None, 2 * MB, 2 * MB + 128, None, 2, 4 * MB, None) == ALIAS   # neither apart nor the same
    assert step(_conv(b=0), None, 64, MB, None, None, None, None, 0, None, None) == OK


def test_empty_batches_launch_nothing():
    lib = sq._seq()
    r = _rows(None)
    assert lib.convseq_conv_fwd(_conv(b=0), r, MB, None, None, None, None, None, None, None) == OK
    assert lib.convseq_scan_fwd(_scan(b=0), r, r, r, MB, None, None, None, None, None, None, None, None) == OK
    assert lib.convseq_pack8(0, 5, 6, 1, r, sq.KeptPtr(None, None), None) == OK
    assert lib.convseq_unpack8(5, 0, 6, 1, sq.KeptPtr(None, None), None, None) == OK
    assert lib.convseq_pack8(1, 5, 0, 1, r, sq.KeptPtr(None, None), None) == BAD
    assert lib.convseq_pack8(1, 5, 6, 1, r, sq.KeptPtr(MB, MB), None) == NULL
    assert lib.convseq_unpack8(1, 5, 6, 1, None, MB, None) == NULL
    assert lib.convseq_unpack8(1, 5, 6, 0, sq.KeptPtr(MB, 2 * MB), 3 * MB + 2, None) == MISALIGNED


def test_the_binding_needs_device_tensors():
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    for call in (lambda: igc.seq_conv(x, w), lambda: igc.seq_conv_bwd(x, x, w), lambda: igc.pack8(x),
                 lambda: igc.seq_conv_step(x[0], w, x), lambda: igc.gated_scan(x, x, x, w[:, 0]),
                 lambda: igc.gated_scan_bwd(x, x, x, x, w[:, 0], x), lambda: igc.gated_scan_step(x[0], x[0], x[0], w[:, 0], x[0]),
                 lambda: igc.unpack8(igc.Packed8(x.to(torch.int8), x.to(torch.uint8), x.shape, x.dtype))):
        with pytest.raises(ValueError, match="GPU only"):
            call()


@pytest.mark.gpu
def test_the_binding_refuses_what_does_not_fit():
    dev = "cuda:0"
    x, w = torch.zeros(2, 20, 8, device=dev), torch.zeros(8, 4, device=dev)
    lam, kept = torch.zeros(8, device=dev), igc.pack8(torch.zeros(2, 20, 8, device=dev))
    states = torch.zeros(2, 1, 8, device=dev)
    half = x.half()
    for error, call in (
            (ValueError, lambda: igc.seq_conv(x[0], w)), (TypeError, lambda: igc.seq_conv(x.double(), w.double())),
            (ValueError, lambda: igc.seq_conv(x, w.half())), (ValueError, lambda: igc.seq_conv(x, w[:7])),
            (ValueError, lambda: igc.seq_conv(x, w, activation="gelu")), (ValueError, lambda: igc.seq_conv(x, w, bias=lam[:4])),
            (igc.ConvError, lambda: igc.seq_conv(x, torch.zeros(8, 9, device=dev))),
            (ValueError, lambda: igc.seq_conv(x, w, state=torch.zeros(2, 4, 8, device=dev))),
            (TypeError, lambda: igc.seq_conv(x, w, starts=torch.zeros(2, 20, device=dev))),
            (ValueError, lambda: igc.seq_conv(x, w, starts=torch.zeros(2, 19, dtype=torch.bool, device=dev))),
            (ValueError, lambda: igc.seq_conv(x, w, out=torch.zeros(2, 20, 9, device=dev))),
            (igc.ConvError, lambda: igc.seq_conv(x, w, out=x)),
            (ValueError, lambda: igc.seq_conv_bwd(x, half, w)), (ValueError, lambda: igc.seq_conv_bwd(x[:, :19], kept, w)),
            (ValueError, lambda: igc.gated_scan(x, x, x[:, :19], lam)), (ValueError, lambda: igc.gated_scan(x, half, x, lam)),
            (ValueError, lambda: igc.gated_scan(x, x, x, lam.half())), (igc.ConvError, lambda: igc.gated_scan(x, x, x, lam, decay=0.0)),
            (ValueError, lambda: igc.gated_scan(x, x, x, lam, h0=torch.zeros(2, 7, device=dev))),
            (ValueError, lambda: igc.gated_scan_bwd(x, kept, x, x, lam, states)),
            (ValueError, lambda: igc.gated_scan_bwd(x, x, x, x, lam, None)),
            (ValueError, lambda: igc.gated_scan_bwd(x, x, x, x, lam, torch.zeros(2, 2, 8, device=dev))),
            (ValueError, lambda: igc.gated_scan_step(x[0], x[0], x[0], lam, torch.zeros(19, 8, device=dev))),
            (TypeError, lambda: igc.gated_scan_step(x[0], x[0], x[0], lam, torch.zeros(30, 8, device=dev),
                                                    slots=torch.zeros(20, dtype=torch.int64, device=dev))),
            (ValueError, lambda: igc.seq_conv_step(x[0], w, torch.zeros(20, 2, 8, device=dev))),
            (ValueError, lambda: igc.pack8(lam)), (ValueError, lambda: igc.unpack8(igc.Packed8(kept.q, kept.e[:, :1], kept.shape, kept.dtype))),
            (TypeError, lambda: igc.unpack8(kept, torch.float64))):
        with pytest.raises(error):
            call()
