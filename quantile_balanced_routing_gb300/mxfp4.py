"""MXFP4 tensors: quantisation, product and its gradients.

Argument checks and allocation around ``moe_mxfp4_*`` (see include/qbmoe.h for
formats and formulas); every step runs in libqbmoe's CUDA kernels.  The codes
and scales are the layout :class:`LatentMoE` takes for MXFP4 experts.
"""
from __future__ import annotations

from typing import NamedTuple

from . import (MAX_EXPERTS, QBMOE_BF16, QBMOE_EINVAL, QBMOE_F32, QBMOE_MXFP4, QbmoeError, _allocating_on, _check_device, _p,
               _stream_ptr, load_library)

BLOCK = 32


class Mxfp4(NamedTuple):
    """An MXFP4 tensor [..., K]: two E2M1 codes a byte (element 2i in the low
    nibble) and one E8M0 scale byte per 32 elements."""
    codes: "torch.Tensor"    # uint8 [..., K / 2]
    scales: "torch.Tensor"   # uint8 [..., K / 32]

    @property
    def shape(self):
        return tuple(self.codes.shape[:-1]) + (2 * self.codes.shape[-1],)


def _need(what, ok, msg):
    if not ok:
        raise QbmoeError(QBMOE_EINVAL, f"{what}: {msg}")


def _check_mxfp4(what, name, t, dims):
    import torch
    _need(what, isinstance(t, Mxfp4), f"{name} is an Mxfp4 (codes, scales)")
    _need(what, t.codes.dtype == torch.uint8 and t.scales.dtype == torch.uint8 and t.codes.is_contiguous() and
          t.scales.is_contiguous(), f"{name}'s codes and scales are contiguous uint8")
    _need(what, t.codes.dim() in dims and tuple(t.scales.shape) ==
          tuple(t.codes.shape[:-1]) + (t.codes.shape[-1] * 2 // BLOCK,) and t.codes.shape[-1] % (BLOCK // 2) == 0 and
          t.codes.shape[-1] > 0, f"{name} is codes [..., K/2] and scales [..., K/32], K a multiple of {BLOCK}")


def _row_stride(what, name, t, align):
    """Row stride of a matrix whose rows are contiguous."""
    _need(what, t.dim() == 2 and (t.stride(1) == 1 or t.shape[1] == 1) and
          (t.shape[0] <= 1 or (t.stride(0) >= t.shape[1] and t.stride(0) % align == 0)),
          f"{name} is a matrix with contiguous rows, their stride a multiple of {align} elements")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def mxfp4_quantize(x, values=False, stream=None):
    """MXFP4 form of x [..., K] (fp32 or bf16), K a multiple of 32.

    Returns an :class:`Mxfp4`, or with ``values`` the pair (Mxfp4, what the
    codes stand for, in x's type).  Each block of 32 takes the scale
    2^(floor(log2 max|x|) - 2); elements round to nearest, ties to even.  A matrix
    may have strided rows."""
    import torch
    what = "mxfp4_quantize"
    _need(what, x.dtype in (torch.float32, torch.bfloat16) and x.dim() >= 1, "x is fp32 or bf16 [..., K]")
    K = x.shape[-1]
    _need(what, K > 0 and K % BLOCK == 0, f"K is a multiple of {BLOCK}")
    align = 4 if x.dtype == torch.float32 else 8
    if x.dim() == 2:
        ld = _row_stride(what, "x", x, align)
    else:
        _need(what, x.is_contiguous(), "x is contiguous, or a matrix with contiguous rows")
        ld = K
    _check_device(what, x)
    rows = x.numel() // K
    with _allocating_on(stream):
        q = Mxfp4(torch.empty(x.shape[:-1] + (K // 2,), dtype=torch.uint8, device=x.device),
                  torch.empty(x.shape[:-1] + (K // BLOCK,), dtype=torch.uint8, device=x.device))
        v = torch.empty(x.shape, dtype=x.dtype, device=x.device) if values else None
        rc = load_library().moe_mxfp4_quantize(rows, K, QBMOE_F32 if x.dtype == torch.float32 else QBMOE_BF16, _p(x),
                                               ld, _p(q.codes), _p(q.scales), _p(v), _stream_ptr(stream))
    if rc:
        raise QbmoeError(rc, "moe_mxfp4_quantize")
    return (q, v) if values else q


def _groups(what, w, offsets):
    """Checked (E, N, K) of weights [N, K], or [E, N, K] with offsets."""
    import torch
    _check_mxfp4(what, "w", w, (2, 3))
    shape = w.shape
    E = shape[0] if len(shape) == 3 else 1
    _need(what, (len(shape) == 3) == (offsets is not None) or E == 1, "w is [E, N, K] with offsets, [N, K] without")
    _need(what, 1 <= E <= MAX_EXPERTS, f"1 to {MAX_EXPERTS} experts")
    _need(what, shape[-2] > 0 and shape[-2] % 8 == 0, "N is a multiple of 8")
    if offsets is not None:
        _need(what, offsets.dtype == torch.int32 and tuple(offsets.shape) == (E + 1,) and offsets.is_contiguous(),
              "offsets is contiguous int32 [E + 1]")
    return E, shape[-2], shape[-1]


def _workspace(lib, R, E, N, K, dev):
    import torch
    return torch.empty((max(lib.qbmoe_mxfp4_workspace_bytes(R, E, N, K), 256),), dtype=torch.uint8, device=dev)


def mxfp4_matmul(x, w: Mxfp4, offsets=None, stream=None):
    """y [R, N] bf16 = x w^T for MXFP4 weights w [N, K].

    x: an :class:`Mxfp4` [R, K], or fp32/bf16 rows, which are quantised first.
    Grouped: w [E, N, K] and offsets [E + 1] int32, the rows in expert order;
    rows that no expert owns are left unwritten."""
    import torch
    what = "mxfp4_matmul"
    if isinstance(x, Mxfp4):
        _check_mxfp4(what, "x", x, (2,))
        rows, kind, scales = x.codes, QBMOE_MXFP4, x.scales
        ld = x.shape[1]
    else:
        _need(what, x.dtype in (torch.float32, torch.bfloat16), "x is an Mxfp4 or fp32 or bf16 [R, K]")
        rows, scales = x, None
        kind, align = (QBMOE_F32, 4) if x.dtype == torch.float32 else (QBMOE_BF16, 8)
        ld = _row_stride(what, "x", x, align)
    R = rows.shape[0]
    E, N, K = _groups(what, w, offsets)
    _need(what, x.shape[1] == K, "x and w have the same K")
    _check_device(what, rows, scales, w.codes, w.scales, offsets)
    lib = load_library()
    with _allocating_on(stream):
        y = torch.empty((R, N), dtype=torch.bfloat16, device=rows.device)
        ws = _workspace(lib, R, E, N, K, y.device)
        rc = lib.moe_mxfp4_matmul(R, E, N, K, kind, _p(rows), ld, _p(scales), _p(w.codes), _p(w.scales), _p(offsets),
                                  _p(y), N, _p(ws), ws.numel(), _stream_ptr(stream))
    if rc:
        raise QbmoeError(rc, "moe_mxfp4_matmul")
    return y


def mxfp4_matmul_backward(dy, xq: Mxfp4, w: Mxfp4, offsets=None, need_dx=True, need_dw=True, dw_dtype=None,
                          stream=None):
    """Gradients (dx [R, K] bf16, dw [N, K] or [E, N, K]) of ``mxfp4_matmul(xq, w, offsets)``.

    dy [R, N] bf16 (rows may be strided); dw is fp32 unless dw_dtype says
    bf16, and zero for an expert without rows.  They are the gradients for the
    values that xq and w stand for; a trainer passes them straight through its
    quantisation.  need_dx / need_dw False: None in that place."""
    import torch
    what = "mxfp4_matmul_backward"
    _check_mxfp4(what, "xq", xq, (2,))
    R = xq.codes.shape[0]
    E, N, K = _groups(what, w, offsets)
    _need(what, xq.shape[1] == K, "xq and w have the same K")
    _need(what, dy.dtype == torch.bfloat16 and tuple(dy.shape) == (R, N), "dy is bf16 [R, N]")
    ld = _row_stride(what, "dy", dy, 8)
    dw_dtype = dw_dtype or torch.float32
    _need(what, dw_dtype in (torch.float32, torch.bfloat16), "dw is fp32 or bf16")
    _check_device(what, dy, xq.codes, xq.scales, w.codes, w.scales, offsets)
    lib, dev, dx, dw, rc = load_library(), dy.device, None, None, 0
    with _allocating_on(stream):
        ws = _workspace(lib, R, E, N, K, dev)
        if need_dx:
            dx = torch.empty((R, K), dtype=torch.bfloat16, device=dev)
            rc = lib.moe_mxfp4_dgrad(R, E, N, K, _p(dy), ld, _p(w.codes), _p(w.scales), _p(offsets), _p(dx), K,
                                     _p(ws), ws.numel(), _stream_ptr(stream))
            if rc:
                raise QbmoeError(rc, "moe_mxfp4_dgrad")
        if need_dw:
            dw = torch.empty(w.shape, dtype=dw_dtype, device=dev)
            rc = lib.moe_mxfp4_wgrad(R, E, N, K, _p(dy), ld, _p(xq.codes), _p(xq.scales), _p(offsets),
                                     QBMOE_F32 if dw_dtype == torch.float32 else QBMOE_BF16, _p(dw), _p(ws),
                                     ws.numel(), _stream_ptr(stream))
            if rc:
                raise QbmoeError(rc, "moe_mxfp4_wgrad")
    return dx, dw
