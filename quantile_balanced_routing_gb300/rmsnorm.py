"""The norm in front of a layer: residual addition, RMS norm, 8-bit rows, gradient.

Argument checks and allocation around ``moe_add_rmsnorm`` and
``moe_add_rmsnorm_backward`` (see include/qbmoe.h for formats and formulas); every
step runs in libqbmoe's CUDA kernels.
"""
from __future__ import annotations

import math
from typing import NamedTuple, Optional

from . import MAX_NORM, MAX_ROWS, QBMOE_BF16, QBMOE_F32, QbmoeError, _here, _p, _refuse, load_library

BLOCK = 32


class Mxfp8:
    """An MXFP8 tensor [..., K]: ``codes`` float8_e4m3fn (or its bytes as uint8)
    [..., K], and ``scales`` uint8 [..., K / 32], one E8M0 byte per 32 elements.
    Checked when it is made, so that the calls that take it need not.  Codes start
    on a 16-byte boundary; scales that do not are copied by the calls."""
    __slots__ = ("codes", "scales", "shape")

    def __init__(self, codes, scales):
        import torch
        if (codes.dtype is not torch.float8_e4m3fn and codes.dtype is not torch.uint8) or \
                scales.dtype is not torch.uint8 or not codes.is_contiguous() or not scales.is_contiguous():
            _refuse("Mxfp8", "codes are contiguous float8_e4m3fn or uint8, scales contiguous uint8")
        if codes.dim() < 1 or scales.dim() < 1:
            _refuse("Mxfp8", "codes [..., K] and scales [..., K/32]")
        (*lead, K), (*lead_s, blocks) = codes.shape, scales.shape
        if K == 0 or blocks * BLOCK != K or lead != lead_s:
            _refuse("Mxfp8", f"codes [..., K] and scales [..., K/32], K a multiple of {BLOCK}")
        self.codes, self.scales, self.shape = codes, scales, tuple(codes.shape)

    def __iter__(self):
        return iter((self.codes, self.scales))


class AddRmsNorm(NamedTuple):
    y: Optional["torch.Tensor"]       # [..., H] the normed rows (with mxfp8: the codes' values, bf16)
    q: Optional[Mxfp8]                # the normed rows in MXFP8
    total: "torch.Tensor"             # [..., H] x + residual (x without a residual)


def _rows(what, name, t, H):
    """(rows, elements between them) of t [..., H]: contiguous, or a matrix with contiguous rows."""
    if t.dim() == 2:
        ld, one = t.stride()
        rows = t.shape[0]
        if rows <= 1:
            ld = H
        if rows and ((one != 1 and H != 1) or ld < H):
            _refuse(what, f"{name} has contiguous rows")
        return rows, ld
    if not t.is_contiguous():
        _refuse(what, f"{name} is contiguous, or a matrix with contiguous rows")
    return t.numel() // H, H


def _type(what, name, t):
    import torch
    if t.dtype is torch.bfloat16:
        return QBMOE_BF16
    if t.dtype is not torch.float32:
        _refuse(what, f"{name} is fp32 or bf16")
    return QBMOE_F32


def _width(what, t, gamma, eps):
    import torch
    H = t.shape[-1] if t.dim() else 0
    if H < 1 or H > MAX_NORM:
        _refuse(what, f"rows of 1 to {MAX_NORM} elements")
    if gamma.dtype is not torch.float32 or gamma.shape != (H,) or not gamma.is_contiguous():
        _refuse(what, "gamma is contiguous fp32 [H]")
    if not 0.0 <= eps < math.inf:
        _refuse(what, "eps is finite and not negative")
    return H


def add_rmsnorm(x, gamma, residual=None, eps=1e-6, mxfp8=False, values=True, total=None, stream=None) -> AddRmsNorm:
    """RMS norm of x + residual over the last axis, times gamma [H] fp32.

    x and residual [..., H], each fp32 or bf16 (matrices may have strided rows).
    ``total`` of the result is the sum, rounded to the residual's type; the norm is that
    of the rounded sum.  The argument total takes it (the residual itself: the residual
    stream is updated in place).  Without a residual, total is x.
    ``y`` has x's type.  With mxfp8 (H a multiple of 32) ``q`` holds the normed rows as
    an :class:`Mxfp8`, which :func:`mxfp4_matvec` and :func:`mxfp4_experts` take, and y, unless
    values is False, what its codes stand for, in bf16."""
    import torch
    if stream is not None:   # outputs are allocated on the stream that writes them
        with torch.cuda.stream(stream):
            return add_rmsnorm(x, gamma, residual, eps, mxfp8, values, total)
    what = "add_rmsnorm"
    xt = _type(what, "x", x)
    H = _width(what, x, gamma, eps)
    T, ldx = _rows(what, "x", x, H)
    if T > MAX_ROWS:
        _refuse(what, f"at most {MAX_ROWS} rows")
    if mxfp8 and H % BLOCK:
        _refuse(what, f"8-bit rows have a multiple of {BLOCK} elements")
    empty, dev = torch.empty, x.device
    rt = ldr = ldt = 0
    if residual is not None:
        rt = _type(what, "residual", residual)
        if residual.shape != x.shape:
            _refuse(what, "residual is of x's shape")
        _, ldr = _rows(what, "residual", residual, H)
        if total is not None:
            if total.dtype is not residual.dtype or total.shape != x.shape:
                _refuse(what, "total is of the residual's shape and type")
            _, ldt = _rows(what, "total", total, H)
    elif total is not None:
        _refuse(what, "total goes with a residual")
    cur = _here(what, x, gamma, residual, total)
    if residual is not None and total is None:
        total, ldt = empty(x.shape, dtype=residual.dtype, device=dev), H
    y = codes = scales = None
    if mxfp8:
        codes = empty(x.shape, dtype=torch.float8_e4m3fn, device=dev)
        scales = empty((*x.shape[:-1], H // BLOCK), dtype=torch.uint8, device=dev)
    if values or not mxfp8:
        y = empty(x.shape, dtype=torch.bfloat16 if mxfp8 else x.dtype, device=dev)
    rc = load_library().moe_add_rmsnorm(T, H, xt, x.data_ptr(), ldx, rt, _p(residual), ldr, gamma.data_ptr(), eps,
                                        _p(total), ldt, _p(y), H, _p(codes), _p(scales), cur)
    if rc:
        raise QbmoeError(rc, "moe_add_rmsnorm")
    q = None
    if mxfp8:
        q = object.__new__(Mxfp8)
        q.codes, q.scales, q.shape = codes, scales, tuple(x.shape)
    return AddRmsNorm(y, q, x if residual is None else total)


def add_rmsnorm_backward(dy, total, gamma, dtotal=None, eps=1e-6, need_dgamma=True, stream=None):
    """Gradients (dx [..., H] of total's type, dgamma [H] fp32) of :func:`add_rmsnorm`.

    dy [..., H] (fp32 or bf16): gradient of the normed rows, passed straight through their
    rounding; total as add_rmsnorm returned it; dtotal, of total's type, the gradient that
    reaches the sum itself, or None.  dx is the gradient of x and of the residual alike.
    need_dgamma False: None in its place."""
    import torch
    if stream is not None:
        with torch.cuda.stream(stream):
            return add_rmsnorm_backward(dy, total, gamma, dtotal, eps, need_dgamma)
    what = "add_rmsnorm_backward"
    dt, tt = _type(what, "dy", dy), _type(what, "total", total)
    H = _width(what, total, gamma, eps)
    if dy.shape != total.shape:
        _refuse(what, "dy is of total's shape")
    T, ldt = _rows(what, "total", total, H)
    if T > MAX_ROWS:
        _refuse(what, f"at most {MAX_ROWS} rows")
    _, ldd = _rows(what, "dy", dy, H)
    ldo = 0
    if dtotal is not None:
        if dtotal.dtype is not total.dtype or dtotal.shape != total.shape:
            _refuse(what, "dtotal is of total's shape and type")
        _, ldo = _rows(what, "dtotal", dtotal, H)
    cur = _here(what, dy, total, gamma, dtotal)
    lib, dev = load_library(), total.device
    dx = torch.empty(total.shape, dtype=total.dtype, device=dev)
    dgamma, ws, nbytes = None, None, 0
    if need_dgamma:
        dgamma = torch.empty(H, dtype=torch.float32, device=dev)
        nbytes = lib.qbmoe_add_rmsnorm_workspace_bytes(T, H)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    rc = lib.moe_add_rmsnorm_backward(T, H, dt, dy.data_ptr(), ldd, tt, total.data_ptr(), ldt, gamma.data_ptr(), eps,
                                      _p(dtotal), ldo, dx.data_ptr(), H, _p(dgamma), _p(ws), nbytes, cur)
    if rc:
        raise QbmoeError(rc, "moe_add_rmsnorm_backward")
    return dx, dgamma
