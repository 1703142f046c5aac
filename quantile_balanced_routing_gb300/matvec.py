"""MXFP4 weights with few rows, and the routed experts of a few tokens.

Argument checks and allocation around ``moe_mxfp4_matvec`` and
``moe_mxfp4_experts`` (see include/qbmoe.h for formulas and limits); every step
runs in libqbmoe's CUDA kernels.
"""
from __future__ import annotations

from . import (MATVEC_MAX_K, MAX_EXPERTS, MAX_ROUTES, MAX_ROWS, MAX_TOPK, QBMOE_BF16, QBMOE_F32, QBMOE_MXFP8,
               QbmoeError, _here, _p, _refuse, load_library)
from .mxfp4 import Mxfp4, _groups, _row_stride, _small, _start
from .rmsnorm import Mxfp8


def _input(what, x, K):
    """(rows' tensor, type code, scales, R, stride, address) of x [R, K]."""
    import torch
    if isinstance(x, Mxfp8):
        t, kind, scales = x.codes, QBMOE_MXFP8, _small(x.scales)
    else:
        t, kind, scales = x, QBMOE_BF16, None
        if t.dtype is not torch.bfloat16:
            _refuse(what, "x is an Mxfp8, or bf16")
    if t.dim() != 2 or t.shape[1] != K:
        _refuse(what, "x is [R, K] with the K of the weights")
    if K > MATVEC_MAX_K:
        _refuse(what, f"K is at most {MATVEC_MAX_K}")
    return t, kind, scales, t.shape[0], K if scales is not None else _row_stride(what, "x", t, 8), _start(what, "x", t)


def mxfp4_matvec(x, w: Mxfp4, offsets=None, out_dtype=None, stream=None):
    """y [R, N] = x w^T for few rows x and MXFP4 weights w [N, K].

    x has 8 or 16 bits, where :func:`mxfp4_matmul` takes 4-bit rows: an :class:`Mxfp8`
    [R, K], or bf16 (rows may be strided).  y is bf16, or fp32 with out_dtype.  Meant for
    few rows a matrix: its weights are read again for every 2 to 24 rows.  Larger calls hold
    bf16 elements within 2^-22 of the largest of their 32 neighbours, exactly down to 2^-14 of it,
    smaller calls exactly down to 2^-32.
    Grouped: w [E, N, K] and offsets [E + 1] int32, the rows in expert order;
    rows that no expert owns are left unwritten."""
    import torch
    if stream is not None:   # outputs and scratch are allocated on the stream that uses them
        with torch.cuda.stream(stream):
            return mxfp4_matvec(x, w, offsets, out_dtype)
    what = "mxfp4_matvec"
    E, N, K = _groups(what, w, offsets)
    t, kind, scales, R, ld, at = _input(what, x, K)
    if R > MAX_ROWS:
        _refuse(what, f"at most {MAX_ROWS} rows")
    f32 = out_dtype is torch.float32
    if not f32 and out_dtype is not None and out_dtype is not torch.bfloat16:
        _refuse(what, "y is bf16 or fp32")
    w_at = _start(what, "w", w.codes)
    cur = _here(what, t, scales, w.codes, w.scales, offsets)
    lib, dev, w_scales = load_library(), t.device, _small(w.scales)
    y = torch.empty((R, N), dtype=torch.float32 if f32 else torch.bfloat16, device=dev)
    nbytes = lib.qbmoe_mxfp4_matvec_workspace_bytes(R, N, K)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    rc = lib.moe_mxfp4_matvec(R, E, N, K, kind, at, ld, _p(scales), w_at, w_scales.data_ptr(), _p(offsets),
                              QBMOE_F32 if f32 else QBMOE_BF16, y.data_ptr(), N, _p(ws), nbytes, cur)
    if rc:
        raise QbmoeError(rc, "moe_mxfp4_matvec")
    return y


def mxfp4_experts(x, idx, w, gate: Mxfp4, up: Mxfp4, out: Mxfp4, gamma=None, eps=1e-6, beta1=4.0, beta2=25.0, stream=None):
    """Routed experts of a few tokens: [T, L] bf16.

    x [T, L]: an :class:`Mxfp8`, or bf16 (rows may be strided).  idx [T, k] int32 and w [T, k]
    fp32: each token's experts and their weights, as :func:`route_qb` returns them; an
    index outside [0, E) stands for no route.  gate and up MXFP4 [E, M, L], out [E, L, M].
    Each route's SiTU-GLU(x gate^T, x up^T) goes through out; a token's routes are
    summed by weight, and with gamma [L] fp32 the sum is RMS-normed and scaled: the routed
    part of :class:`LatentMoE`, with fp32 between its steps, of which the down product takes
    22 bits.  T k is at most 4096."""
    import torch
    if stream is not None:
        with torch.cuda.stream(stream):
            return mxfp4_experts(x, idx, w, gate, up, out, gamma, eps, beta1, beta2)
    what = "mxfp4_experts"
    if not isinstance(gate, Mxfp4) or not isinstance(up, Mxfp4) or not isinstance(out, Mxfp4):
        _refuse(what, "gate, up and out are Mxfp4")
    if len(gate.shape) != 3 or up.shape != gate.shape:
        _refuse(what, "gate and up are [E, M, L]")
    E, M, L = gate.shape
    if out.shape != (E, L, M):
        _refuse(what, "out is [E, L, M]")
    if E < 1 or E > MAX_EXPERTS or M % 32 or M < 32 or M > MATVEC_MAX_K:
        _refuse(what, f"1 to {MAX_EXPERTS} experts; M a multiple of 32, at most {MATVEC_MAX_K}")
    t, kind, scales, T, ld, at = _input(what, x, L)
    if idx.dtype is not torch.int32 or idx.dim() != 2 or idx.shape[0] != T or not idx.is_contiguous():
        _refuse(what, "idx is contiguous int32 [T, k]")
    k = idx.shape[1]
    if k < 1 or k > MAX_TOPK or T * k > MAX_ROUTES:
        _refuse(what, f"1 <= k <= {MAX_TOPK}, T k at most {MAX_ROUTES}")
    if w.dtype is not torch.float32 or w.shape != idx.shape or not w.is_contiguous():
        _refuse(what, "w is contiguous fp32 [T, k]")
    if gamma is not None and (gamma.dtype is not torch.float32 or gamma.shape != (L,) or not gamma.is_contiguous()):
        _refuse(what, "gamma is contiguous fp32 [L]")
    if not 0.0 <= eps < 2.0 ** 128 or not 1e-45 < beta1 or not 1e-45 < beta2 or not beta1 * beta2 <= 2.0 ** 127:
        _refuse(what, "eps is finite and not negative, beta1 and beta2 are positive, and beta1 beta2 is at most 2^127 (all of them as fp32)")
    g_at, u_at, o_at = _start(what, "gate", gate.codes), _start(what, "up", up.codes), _start(what, "out", out.codes)
    cur = _here(what, t, scales, idx, w, gate.codes, gate.scales, up.codes, up.scales, out.codes, out.scales, gamma)
    lib, dev = load_library(), t.device
    gs, us, os = _small(gate.scales), _small(up.scales), _small(out.scales)
    y = torch.empty((T, L), dtype=torch.bfloat16, device=dev)
    nbytes = lib.qbmoe_mxfp4_experts_workspace_bytes(T, k, L, M)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    rc = lib.moe_mxfp4_experts(T, k, E, L, M, kind, at, ld, _p(scales), idx.data_ptr(), w.data_ptr(), g_at,
                               gs.data_ptr(), u_at, us.data_ptr(), o_at, os.data_ptr(), beta1, beta2, _p(gamma), eps,
                               y.data_ptr(), L, ws.data_ptr(), nbytes, cur)
    if rc:
        raise QbmoeError(rc, "moe_mxfp4_experts")
    return y
