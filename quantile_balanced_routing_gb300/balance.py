"""Router training: balance loss, per-expert counts and the logits' gradient.

Argument checks and allocation around ``moe_balance_loss`` and
``moe_router_backward`` (see include/qbmoe.h for the formulas); every step runs
in libqbmoe's CUDA kernels.  A call's host side is what a small batch costs, so
the checks are plain comparisons without intermediate objects.
"""
from __future__ import annotations

from typing import NamedTuple

from . import MAX_EXPERTS, MAX_ROWS, MAX_TOPK, QBMOE_BF16, QBMOE_F32, QbmoeError, _here, _p, _refuse, load_library


class BalanceLoss(NamedTuple):
    loss: "torch.Tensor"     # [S] fp32, per sequence
    counts: "torch.Tensor"   # [S, n] int32, routes of the sequence's valid tokens
    probs: "torch.Tensor"    # [S, n] fp32, mean share of the router's score
    tokens: "torch.Tensor"   # [S] int32, valid tokens


def _row_stride(what, name, t, n):
    """Elements between the rows of t [T, n]; torch leaves the stride of a single row free."""
    ld, one = t.stride()
    if t.shape[0] == 1:
        ld = n
    if one != 1 or ld < n:
        _refuse(what, f"{name}: a token's values are contiguous")
    return ld


def _router_args(what, logits, idx, seq_offsets, token_mask):
    """Checked (T, n, k, S, dtype code, row stride) of a routed batch."""
    import torch
    if logits.dim() != 2 or (logits.dtype is not torch.float32 and logits.dtype is not torch.bfloat16):
        _refuse(what, "logits are fp32 or bf16 [T, n]")
    T, n = logits.shape
    if T < 1 or T > MAX_ROWS or n < 2 or n > MAX_EXPERTS:
        _refuse(what, f"1 to at most {MAX_ROWS} tokens and 2 <= n <= {MAX_EXPERTS}")
    ld = _row_stride(what, "logits", logits, n)
    if idx.dtype is not torch.int32 or idx.dim() != 2 or idx.shape[0] != T or not idx.is_contiguous():
        _refuse(what, "idx is contiguous int32 [T, k]")
    k = idx.shape[1]
    if k < 1 or k > n or k > MAX_TOPK:
        _refuse(what, f"1 <= k <= min(n, {MAX_TOPK})")
    S = 1
    if seq_offsets is not None:
        if seq_offsets.dtype is not torch.int32 or seq_offsets.dim() != 1 or seq_offsets.shape[0] < 2 or \
                not seq_offsets.is_contiguous():
            _refuse(what, "seq_offsets is contiguous int32 [S + 1]")
        S = seq_offsets.shape[0] - 1
        if S > MAX_ROWS:
            _refuse(what, f"at most {MAX_ROWS} sequences")
    if token_mask is not None and (
            (token_mask.dtype is not torch.bool and token_mask.dtype is not torch.uint8) or token_mask.dim() != 1 or
            token_mask.shape[0] != T or not token_mask.is_contiguous()):
        _refuse(what, "token_mask is contiguous bool or uint8 [T]")
    return T, n, k, S, QBMOE_F32 if logits.dtype is torch.float32 else QBMOE_BF16, ld


def balance_loss(logits, idx, seq_offsets=None, token_mask=None, stream=None) -> BalanceLoss:
    """Balance loss of each sequence, with its per-expert counts and mean shares.

    logits [T, n] (fp32 or bf16, pre-sigmoid; rows may be strided), idx [T, k]
    int32 as returned by the router, seq_offsets [S + 1] int32 (None: one
    sequence), token_mask [T] bool, False for padding.  The caller weighs and
    sums ``loss``, which carries no graph; its gradient goes into
    :func:`router_backward`."""
    import torch
    if stream is not None:   # outputs and scratch are allocated on the stream that uses them
        with torch.cuda.stream(stream):
            return balance_loss(logits, idx, seq_offsets, token_mask)
    T, n, k, S, dt, ld = _router_args("balance_loss", logits, idx, seq_offsets, token_mask)
    cur = _here("balance_loss", logits, idx, seq_offsets, token_mask)
    lib, dev, empty = load_library(), logits.device, torch.empty
    r = BalanceLoss(empty(S, dtype=torch.float32, device=dev), empty((S, n), dtype=torch.int32, device=dev),
                    empty((S, n), dtype=torch.float32, device=dev), empty(S, dtype=torch.int32, device=dev))
    nbytes = lib.qbmoe_balance_workspace_bytes(T, n, S)
    ws = empty(nbytes, dtype=torch.uint8, device=dev)
    rc = lib.moe_balance_loss(T, n, k, S, dt, logits.data_ptr(), ld, idx.data_ptr(), _p(seq_offsets), _p(token_mask),
                              r.loss.data_ptr(), r.counts.data_ptr(), r.probs.data_ptr(), r.tokens.data_ptr(),
                              ws.data_ptr(), nbytes, cur)
    if rc:
        raise QbmoeError(rc, "moe_balance_loss")
    return r


def router_backward(logits, idx, dw=None, dloss=None, counts=None, tokens=None, seq_offsets=None, token_mask=None,
                    out=None, stream=None):
    """Gradient [T, n] (of the logits' type) of the router logits.

    dw [T, k] fp32: gradient of the mixture weights (the chosen scores
    renormalised); dloss [S] fp32: gradient of each sequence's balance loss,
    with the counts and tokens that :func:`balance_loss` returned.  Either may
    be None.  out may be the logits themselves."""
    import torch
    if stream is not None:
        with torch.cuda.stream(stream):
            return router_backward(logits, idx, dw, dloss, counts, tokens, seq_offsets, token_mask, out)
    what = "router_backward"
    T, n, k, S, dt, ld = _router_args(what, logits, idx, seq_offsets, token_mask)
    if dw is None and dloss is None:
        _refuse(what, "needs dw or dloss")
    if dw is not None and (dw.dtype is not torch.float32 or dw.shape != idx.shape or not dw.is_contiguous()):
        _refuse(what, "dw is contiguous fp32 [T, k]")
    if dloss is None:
        counts = tokens = None
    else:
        if counts is None or tokens is None:
            _refuse(what, "dloss needs counts and tokens")
        if dloss.dtype is not torch.float32 or dloss.shape != (S,) or not dloss.is_contiguous():
            _refuse(what, "dloss is contiguous fp32 [S]")
        if counts.dtype is not torch.int32 or counts.shape != (S, n) or not counts.is_contiguous():
            _refuse(what, "counts is contiguous int32 [S, n]")
        if tokens.dtype is not torch.int32 or tokens.shape != (S,) or not tokens.is_contiguous():
            _refuse(what, "tokens is contiguous int32 [S]")
    if out is not None and (out.dtype is not logits.dtype or out.shape != logits.shape):
        _refuse(what, "out is [T, n] of the logits' type")
    cur = _here(what, logits, idx, seq_offsets, token_mask, dw, dloss, counts, tokens, out)
    if out is None:
        out, ldg = torch.empty((T, n), dtype=logits.dtype, device=logits.device), n
    else:
        ldg = _row_stride(what, "out", out, n)
    rc = load_library().moe_router_backward(T, n, k, S, dt, logits.data_ptr(), ld, idx.data_ptr(), _p(seq_offsets),
                                            _p(token_mask), _p(dw), _p(dloss), _p(counts), _p(tokens), out.data_ptr(),
                                            ldg, cur)
    if rc:
        raise QbmoeError(rc, "moe_router_backward")
    return out
