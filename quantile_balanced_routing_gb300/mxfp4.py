"""MXFP4 tensors: quantisation, product and its gradients.

Argument checks and allocation around ``moe_mxfp4_*`` (see include/qbmoe.h for
formats and formulas); every step runs in libqbmoe's CUDA kernels.  The codes
and scales are the layout :class:`LatentMoE` takes for MXFP4 experts.
"""
from __future__ import annotations

from . import MAX_EXPERTS, MAX_ROWS, QBMOE_BF16, QBMOE_F32, QBMOE_MXFP4, QbmoeError, _here, _p, _refuse, load_library

BLOCK = 32
_MAX_COLS, _MAX_STRIDE, _MAX_ELEMENTS = 1 << 24, 1 << 27, 1 << 40


class Mxfp4:
    """An MXFP4 tensor [..., K]: ``codes`` uint8 [..., K / 2], two E2M1 codes a
    byte (element 2i in the low nibble), and ``scales`` uint8 [..., K / 32], one
    E8M0 byte per 32 elements.  Checked when it is made, so that the calls that
    take it need not.  The tensors may be slices of larger ones; codes start on a
    16-byte boundary, as any row does, and scales that do not are copied by the calls."""
    __slots__ = ("codes", "scales", "shape")

    def __init__(self, codes, scales):
        import torch
        if codes.dtype is not torch.uint8 or scales.dtype is not torch.uint8 or not codes.is_contiguous() or \
                not scales.is_contiguous():
            _refuse("Mxfp4", "codes and scales are contiguous uint8")
        if codes.dim() < 1 or scales.dim() < 1:
            _refuse("Mxfp4", "codes [..., K/2] and scales [..., K/32]")
        (*lead, half), (*lead_s, blocks) = codes.shape, scales.shape
        if half == 0 or blocks * (BLOCK // 2) != half or lead != lead_s:
            _refuse("Mxfp4", f"codes [..., K/2] and scales [..., K/32], K a multiple of {BLOCK}")
        self.codes, self.scales, self.shape = codes, scales, (*lead, 2 * half)

    def __iter__(self):
        return iter((self.codes, self.scales))


def _made(codes, scales, shape):
    """An Mxfp4 of tensors known to be right."""
    q = object.__new__(Mxfp4)
    q.codes, q.scales, q.shape = codes, scales, shape
    return q


def _row_stride(what, name, t, align):
    """Elements between the rows of a matrix whose rows are contiguous."""
    ld, one = t.stride()
    rows, cols = t.shape
    if rows <= 1:
        ld = cols
    if rows == 0:            # no row to read: the strides may be anything
        return ld
    if (one != 1 and cols != 1) or ld < cols or ld % align:
        _refuse(what, f"{name} is a matrix with contiguous rows, their stride a multiple of {align} elements")
    return ld


def _start(what, name, t):
    """The address of a tensor that is read in 16-byte pieces."""
    p = t.data_ptr()
    if p & 15:
        _refuse(what, f"{name} starts on a 16-byte boundary")
    return p


def _small(t):
    """Scales or offsets that start on a 16-byte boundary: a copy of a slice that does not."""
    return t if t is None or not t.data_ptr() & 15 else t.clone()


def mxfp4_quantize(x, values=False, stream=None):
    """MXFP4 form of x [..., K] (fp32 or bf16), K a multiple of 32.

    Returns an :class:`Mxfp4`, or with ``values`` the pair (Mxfp4, what the
    codes stand for, in x's type).  Each block of 32 takes the scale
    2^(floor(log2 max|x|) - 2); elements round to nearest, ties to even.  A matrix
    may have strided rows."""
    import torch
    if stream is not None:   # outputs are allocated on the stream that writes them
        with torch.cuda.stream(stream):
            return mxfp4_quantize(x, values)
    what = "mxfp4_quantize"
    f32 = x.dtype is torch.float32
    if (not f32 and x.dtype is not torch.bfloat16) or x.dim() < 1:
        _refuse(what, "x is fp32 or bf16 [..., K]")
    K = x.shape[-1]
    if K == 0 or K % BLOCK or K > 0x7fffffff:
        _refuse(what, f"K is a multiple of {BLOCK}, at most 2^31 - 1")
    if x.numel() > _MAX_ELEMENTS:
        _refuse(what, "x has at most 2^40 elements")
    if x.dim() == 2:
        ld, lead, rows = _row_stride(what, "x", x, 4 if f32 else 8), (x.shape[0],), x.shape[0]
    else:
        if not x.is_contiguous():
            _refuse(what, "x is contiguous, or a matrix with contiguous rows")
        ld, lead, rows = K, tuple(x.shape[:-1]), x.numel() // K
    at = _start(what, "x", x)
    cur = _here(what, x)
    dev, empty = x.device, torch.empty
    codes = empty((*lead, K // 2), dtype=torch.uint8, device=dev)
    scales = empty((*lead, K // BLOCK), dtype=torch.uint8, device=dev)
    v = empty(x.shape, dtype=x.dtype, device=dev) if values else None
    rc = load_library().moe_mxfp4_quantize(rows, K, QBMOE_F32 if f32 else QBMOE_BF16, at, ld,
                                           codes.data_ptr(), scales.data_ptr(), _p(v), cur)
    if rc:
        raise QbmoeError(rc, "moe_mxfp4_quantize")
    q = _made(codes, scales, (*lead, K))
    return (q, v) if values else q


def _groups(what, w, offsets):
    """Checked (E, N, K) of weights [N, K], or [E, N, K] with offsets."""
    import torch
    if not isinstance(w, Mxfp4):
        _refuse(what, "w is an Mxfp4")
    shape = w.shape
    if len(shape) == 3 and offsets is not None:
        E, N, K = shape
    elif len(shape) == 2 and offsets is None:
        E, (N, K) = 1, shape
    else:
        _refuse(what, "w is [E, N, K] with offsets, [N, K] without")
    if E < 1 or E > MAX_EXPERTS:
        _refuse(what, f"1 to {MAX_EXPERTS} experts")
    if N == 0 or N % 8:
        _refuse(what, "N is a multiple of 8")
    if N > _MAX_COLS or K > _MAX_COLS or E * N > 0x7fffffff:
        _refuse(what, "N and K are at most 2^24, E N at most 2^31 - 1")
    if offsets is not None and (offsets.dtype is not torch.int32 or offsets.shape != (E + 1,) or
                                not offsets.is_contiguous()):
        _refuse(what, "offsets is contiguous int32 [E + 1]")
    return E, N, K


def mxfp4_matmul(x, w: Mxfp4, offsets=None, stream=None):
    """y [R, N] bf16 = x w^T for MXFP4 weights w [N, K].

    x: an :class:`Mxfp4` [R, K], or fp32/bf16 rows, which are quantised first: both
    operands have 4 bits, where :class:`LatentMoE` keeps its activations at bf16
    precision.  y carries no graph; :func:`mxfp4_matmul_backward` is its gradient.
    Grouped: w [E, N, K] and offsets [E + 1] int32, the rows in expert order;
    rows that no expert owns are left unwritten."""
    import torch
    if stream is not None:
        with torch.cuda.stream(stream):
            return mxfp4_matmul(x, w, offsets)
    what = "mxfp4_matmul"
    E, N, K = _groups(what, w, offsets)
    if isinstance(x, Mxfp4):
        shape = x.shape
        rows, kind, scales, ld = x.codes, QBMOE_MXFP4, x.scales, K
    else:
        shape, rows, scales = x.shape, x, None
        kind = QBMOE_F32 if x.dtype is torch.float32 else QBMOE_BF16
        if kind == QBMOE_BF16 and x.dtype is not torch.bfloat16:
            _refuse(what, "x is an Mxfp4, or fp32 or bf16")
    if len(shape) != 2 or shape[1] != K:
        _refuse(what, "x is [R, K] with the K of w")
    R = shape[0]
    if R > MAX_ROWS:
        _refuse(what, f"at most {MAX_ROWS} rows")
    if scales is None:
        ld = _row_stride(what, "x", x, 4 if kind == QBMOE_F32 else 8)
    x_at, w_at = _start(what, "x", rows), _start(what, "w", w.codes)
    cur = _here(what, rows, scales, w.codes, w.scales, offsets)
    lib, dev = load_library(), rows.device
    scales, w_scales, offsets = _small(scales), _small(w.scales), _small(offsets)
    y = torch.empty((R, N), dtype=torch.bfloat16, device=dev)
    ws, nbytes = None, 0
    if scales is None:
        nbytes = lib.qbmoe_mxfp4_workspace_bytes(R, K)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    rc = lib.moe_mxfp4_matmul(R, E, N, K, kind, x_at, ld, _p(scales), w_at, w_scales.data_ptr(), _p(offsets),
                              y.data_ptr(), N, _p(ws), nbytes, cur)
    if rc:
        raise QbmoeError(rc, "moe_mxfp4_matmul")
    return y


def mxfp4_matmul_backward(dy, xq: Mxfp4, w: Mxfp4, offsets=None, need_dx=True, need_dw=True, dw_dtype=None,
                          stream=None):
    """Gradients (dx [R, K] bf16, dw [N, K] or [E, N, K]) of ``mxfp4_matmul(xq, w, offsets)``.

    dy [R, N] bf16 (rows may be strided); dw is fp32 unless dw_dtype says
    bf16, and zero for an expert without rows; dx of rows that no expert owns is left
    unwritten.  They are the gradients for the
    values that xq and w stand for; a trainer passes them straight through its
    quantisation.  need_dx / need_dw False: None in that place."""
    import torch
    if stream is not None:
        with torch.cuda.stream(stream):
            return mxfp4_matmul_backward(dy, xq, w, offsets, need_dx, need_dw, dw_dtype)
    what = "mxfp4_matmul_backward"
    E, N, K = _groups(what, w, offsets)
    shape = xq.shape if isinstance(xq, Mxfp4) else ()
    if len(shape) != 2 or shape[1] != K:
        _refuse(what, "xq is [R, K] with the K of w")
    R = shape[0]
    if R > MAX_ROWS:
        _refuse(what, f"at most {MAX_ROWS} rows")
    if dy.dtype is not torch.bfloat16 or dy.shape != (R, N):
        _refuse(what, "dy is bf16 [R, N]")
    ld = _row_stride(what, "dy", dy, 8)
    if ld > _MAX_STRIDE:
        _refuse(what, "dy's rows are at most 2^27 elements apart")
    f32 = dw_dtype is None or dw_dtype is torch.float32
    if not f32 and dw_dtype is not torch.bfloat16:
        _refuse(what, "dw is fp32 or bf16")
    dy_at, x_at, w_at = _start(what, "dy", dy), _start(what, "xq", xq.codes), _start(what, "w", w.codes)
    cur = _here(what, dy, xq.codes, xq.scales, w.codes, w.scales, offsets)
    lib, dev, dx, dw, offsets = load_library(), dy.device, None, None, _small(offsets)
    if need_dx:
        w_scales = _small(w.scales)
        dx = torch.empty((R, K), dtype=torch.bfloat16, device=dev)
        rc = lib.moe_mxfp4_dgrad(R, E, N, K, dy_at, ld, w_at, w_scales.data_ptr(), _p(offsets), dx.data_ptr(), K, cur)
        if rc:
            raise QbmoeError(rc, "moe_mxfp4_dgrad")
    if need_dw:
        x_scales = _small(xq.scales)
        dw = torch.empty((N, K) if offsets is None else (E, N, K), dtype=torch.float32 if f32 else torch.bfloat16,
                         device=dev)
        nbytes = lib.qbmoe_mxfp4_wgrad_workspace_bytes(R, E, N, K)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
        rc = lib.moe_mxfp4_wgrad(R, E, N, K, dy_at, ld, x_at, x_scales.data_ptr(), _p(offsets),
                                 QBMOE_F32 if f32 else QBMOE_BF16, dw.data_ptr(), _p(ws), nbytes, cur)
        if rc:
            raise QbmoeError(rc, "moe_mxfp4_wgrad")
    return dx, dw
