"""Router training: balance loss, per-expert counts and the logits' gradient.

Argument checks and allocation around ``moe_balance_loss`` and
``moe_router_backward`` (see include/qbmoe.h for the formulas); every step runs
in libqbmoe's CUDA kernels.
"""
from __future__ import annotations

from typing import NamedTuple

from . import (MAX_EXPERTS, MAX_TOPK, QBMOE_BF16, QBMOE_EINVAL, QBMOE_F32, QbmoeError, _allocating_on, _check_device,
               _p, _stream_ptr, load_library)


class BalanceLoss(NamedTuple):
    loss: "torch.Tensor"     # [S] fp32, per sequence
    counts: "torch.Tensor"   # [S, n] int32, routes of the sequence's valid tokens
    probs: "torch.Tensor"    # [S, n] fp32, mean share of the router's score
    tokens: "torch.Tensor"   # [S] int32, valid tokens


def _router_args(what, logits, idx, seq_offsets, token_mask):
    """Checked (T, n, k, S, dtype code) of a routed batch."""
    import torch

    def need(ok, msg):
        if not ok:
            raise QbmoeError(QBMOE_EINVAL, f"{what}: {msg}")

    need(logits.dim() == 2 and logits.dtype in (torch.float32, torch.bfloat16), "logits are fp32 or bf16 [T, n]")
    T, n = logits.shape
    need(T >= 1 and 2 <= n <= MAX_EXPERTS, f"T >= 1 and 2 <= n <= {MAX_EXPERTS}")
    need(logits.stride(1) == 1 and (logits.stride(0) >= n or T == 1), "a token's logits are contiguous")
    need(idx.dtype == torch.int32 and idx.dim() == 2 and idx.shape[0] == T and idx.is_contiguous(),
         "idx is contiguous int32 [T, k]")
    k = idx.shape[1]
    need(1 <= k <= min(n, MAX_TOPK), f"1 <= k <= min(n, {MAX_TOPK})")
    S = 1
    if seq_offsets is not None:
        need(seq_offsets.dtype == torch.int32 and seq_offsets.dim() == 1 and seq_offsets.shape[0] >= 2 and
             seq_offsets.is_contiguous(), "seq_offsets is contiguous int32 [S + 1]")
        S = seq_offsets.shape[0] - 1
    if token_mask is not None:
        need(token_mask.dtype in (torch.bool, torch.uint8) and tuple(token_mask.shape) == (T,) and
             token_mask.is_contiguous(), "token_mask is contiguous bool or uint8 [T]")
    _check_device(what, logits, idx, seq_offsets, token_mask)
    return T, n, k, S, QBMOE_F32 if logits.dtype == torch.float32 else QBMOE_BF16


def _ld(t):
    return max(t.stride(0), t.shape[1])   # torch leaves the stride of a single row free


def balance_loss(logits, idx, seq_offsets=None, token_mask=None, stream=None) -> BalanceLoss:
    """Balance loss of each sequence, with its per-expert counts and mean shares.

    logits [T, n] (fp32 or bf16, pre-sigmoid; rows may be strided), idx [T, k]
    int32 as returned by the router, seq_offsets [S + 1] int32 (None: one
    sequence), token_mask [T] bool, False for padding.  The caller weighs and
    sums ``loss``; its gradient goes into :func:`router_backward`."""
    import torch
    T, n, k, S, dt = _router_args("balance_loss", logits, idx, seq_offsets, token_mask)
    lib, dev = load_library(), logits.device
    nbytes = lib.qbmoe_balance_workspace_bytes(T, n, S)
    with _allocating_on(stream):
        r = BalanceLoss(torch.empty((S,), dtype=torch.float32, device=dev),
                        torch.empty((S, n), dtype=torch.int32, device=dev),
                        torch.empty((S, n), dtype=torch.float32, device=dev),
                        torch.empty((S,), dtype=torch.int32, device=dev))
        ws = torch.empty((max(nbytes, 256),), dtype=torch.uint8, device=dev)
        rc = lib.moe_balance_loss(T, n, k, S, dt, _p(logits), _ld(logits), _p(idx), _p(seq_offsets), _p(token_mask),
                                  _p(r.loss), _p(r.counts), _p(r.probs), _p(r.tokens), _p(ws), ws.numel(),
                                  _stream_ptr(stream))
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
    what = "router_backward"
    T, n, k, S, dt = _router_args(what, logits, idx, seq_offsets, token_mask)

    def need(ok, msg):
        if not ok:
            raise QbmoeError(QBMOE_EINVAL, f"{what}: {msg}")

    need(dw is not None or dloss is not None, "needs dw or dloss")
    if dw is not None:
        need(dw.dtype == torch.float32 and tuple(dw.shape) == (T, k) and dw.is_contiguous(),
             "dw is contiguous fp32 [T, k]")
    if dloss is not None:
        need(counts is not None and tokens is not None, "dloss needs counts and tokens")
        need(dloss.dtype == torch.float32 and tuple(dloss.shape) == (S,) and dloss.is_contiguous(), "dloss is fp32 [S]")
        need(counts.dtype == torch.int32 and tuple(counts.shape) == (S, n) and counts.is_contiguous(),
             "counts is contiguous int32 [S, n]")
        need(tokens.dtype == torch.int32 and tuple(tokens.shape) == (S,) and tokens.is_contiguous(),
             "tokens is int32 [S]")
    else:
        counts = tokens = None
    if out is not None:
        need(out.dtype == logits.dtype and tuple(out.shape) == (T, n) and out.stride(1) == 1 and
             (out.stride(0) >= n or T == 1), "out is [T, n] of the logits' type, a token's gradient contiguous")
    _check_device(what, logits, dw, dloss, counts, tokens, out)
    with _allocating_on(stream):
        if out is None:
            out = torch.empty((T, n), dtype=logits.dtype, device=logits.device)
        rc = load_library().moe_router_backward(T, n, k, S, dt, _p(logits), _ld(logits), _p(idx), _p(seq_offsets),
                                                _p(token_mask), _p(dw), _p(dloss), _p(counts), _p(tokens), _p(out),
                                                _ld(out), _stream_ptr(stream))
    if rc:
        raise QbmoeError(rc, "moe_router_backward")
    return out
