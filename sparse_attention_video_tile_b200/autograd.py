"""Sliding Tile Attention with autograd, for finetuning.

The forward keeps each row's log-sum-exp; the backward gives dq, dk and dv over
the same tile windows ("Fast Video Generation with Sliding Tile Attention",
abstract and "Method details": attention restricted to a sliding window of whole
tiles; the review replies describe finetuning with it).  Every step runs in the
library's CUDA kernels through the C ABI:

    forward   raster q, k, v --tile reorder--> tiled --sta_attention_fwd_lse--> tiled out, lse
              tiled out --tile unorder--> raster out
    backward  raster dout --tile reorder--> tiled --sta_attention_bwd--> tiled dq, dk, dv
              --tile unorder--> raster dq, dk, dv

Raster tensors are either [B, heads, L, d] (``token_major=False``) or the
token-major [B, L, heads, d] (``token_major=True``), where the transposes are
part of the reorders.  The tiled q, k, v, output and log-sum-exp are kept for
the backward.  Tiles must hold a multiple of 128 tokens and the grid must be a
tile multiple (the backward kernel's blocking).  The backward is not itself
differentiable: a second derivative raises.

``sta_diff_attention`` (differential attention over the same windows, any grid),
``sta_layer_norm`` and ``sta_dropout`` are the other operators of such a block, each
with its backward in the library's kernels.
"""
from __future__ import annotations

from typing import Optional, Sequence

import torch
from torch.autograd.function import once_differentiable

from . import (sta_attention_bwd, sta_attention_fwd_lse, sta_diff_attention_bwd, sta_diff_forward, sta_dropout_forward,
               sta_layer_norm_bwd, sta_layer_norm_forward, sta_tile_reorder, sta_tile_reorder_tokens, sta_tile_unorder,
               sta_tile_unorder_tokens)


def _to_tiled(x, grid, tile, token_major: bool):
    if token_major:
        b, n, h, d = x.shape
        t = torch.empty((b, h, n, d), dtype=x.dtype, device=x.device)
        sta_tile_reorder_tokens(x, t, grid, tile)
    else:
        t = torch.empty_like(x)
        sta_tile_reorder(x, t, grid, tile)
    return t


def _from_tiled(t, grid, tile, token_major: bool):
    if token_major:
        b, h, n, d = t.shape
        x = torch.empty((b, n, h, d), dtype=t.dtype, device=t.device)
        sta_tile_unorder_tokens(t, x, grid, tile)
    else:
        x = torch.empty_like(t)
        sta_tile_unorder(t, x, grid, tile)
    return x


class STAttentionFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, grid, tile, windows, scale, token_major):
        qt, kt, vt = (_to_tiled(x.contiguous(), grid, tile, token_major) for x in (q, k, v))
        ot = torch.empty_like(qt)
        b, h, n, _ = qt.shape
        lse = torch.empty((b, h, n), dtype=torch.float32, device=qt.device)
        sta_attention_fwd_lse(qt, kt, vt, ot, lse, grid, tile, windows, scale)
        ctx.save_for_backward(qt, kt, vt, ot, lse)
        ctx.sta_args = (grid, tile, windows, scale, token_major)
        return _from_tiled(ot, grid, tile, token_major)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        qt, kt, vt, ot, lse = ctx.saved_tensors
        grid, tile, windows, scale, token_major = ctx.sta_args
        dot = _to_tiled(dout.to(torch.bfloat16).contiguous(), grid, tile, token_major)
        dq, dk, dv = (torch.empty_like(qt) for _ in range(3))
        sta_attention_bwd(qt, kt, vt, ot, dot, lse, dq, dk, dv, grid, tile, windows, scale)
        grads = tuple(_from_tiled(g, grid, tile, token_major) for g in (dq, dk, dv))
        return grads + (None, None, None, None, None)


def sta_attention(q, k, v, grid, tile, window_per_head: Sequence, scale: Optional[float] = None,
                  token_major: bool = False):
    """STA forward with a backward: bf16 CUDA tensors in raster order, [B, heads, L, d]
    or, with ``token_major``, [B, L, heads, d]; output in the same layout."""
    if scale is None:
        scale = 1.0 / float(q.shape[-1]) ** 0.5
    return STAttentionFunction.apply(q, k, v, tuple(grid), tuple(tile),
                                     [tuple(w) for w in window_per_head], float(scale), bool(token_major))


def _dense(x):
    """x as the kernels take it: contiguous from a 16-byte boundary.  A slice of rows of an odd
    width, or its gradient, is contiguous and starts anywhere; it is copied."""
    if x is None:
        return None
    x = x.contiguous()
    return x if x.data_ptr() % 16 == 0 else x.clone()


class STADiffAttentionFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, lam, grid, tile, windows, scale, token_major, save):
        q, k, v, lam = (_dense(x) for x in (q, k, v, lam))
        if not save:
            return sta_diff_forward(q, k, v, lam, grid, tile, windows, scale, token_major)
        out, out2, lse = sta_diff_forward(q, k, v, lam, grid, tile, windows, scale, token_major, save=True)
        ctx.save_for_backward(q, k, v, lam, out, out2, lse)
        ctx.sta_args = (grid, tile, windows, scale, token_major)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        q, k, v, lam, out, out2, lse = ctx.saved_tensors
        grid, tile, windows, scale, token_major = ctx.sta_args
        dq, dk, dv, dlam = (torch.empty_like(x) for x in (q, k, v, lam))
        sta_diff_attention_bwd(q, k, v, lam, out, out2, lse, _dense(dout.to(torch.bfloat16)), dq, dk, dv, dlam, grid,
                               tile, windows, scale, token_major)
        return dq, dk, dv, dlam, None, None, None, None, None, None


class STALayerNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, residual, dropout_p, rng):
        ctx.set_materialize_grads(False)   # h is often not used further: no zeros to write and read for its gradient
        x, residual, weight, bias = (_dense(t) for t in (x, residual, weight, bias))
        rng = rng.clone() if dropout_p > 0 else None   # the backward's mask, whatever becomes of the caller's state
        y, h, mean, rstd = sta_layer_norm_forward(x, weight, bias, eps, residual, dropout_p, rng)
        ctx.save_for_backward(x if h is None else h, mean, rstd, weight, rng)
        ctx.sta_args = (bias is not None, residual is not None, dropout_p, h is not None, None if bias is None else bias.dtype)
        return (y, h) if h is not None else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        h, mean, rstd, weight, rng = ctx.saved_tensors
        has_bias, has_res, p, _, bias_dtype = ctx.sta_args
        if dy is None and dh is None:
            return None, None, None, None, None, None, None
        dy = torch.zeros_like(h) if dy is None else _dense(dy.to(h.dtype))
        dh = None if dh is None else _dense(dh.to(h.dtype))
        want_w = weight is not None and ctx.needs_input_grad[1]
        want_b = has_bias and ctx.needs_input_grad[2]
        dx = torch.empty_like(h)
        dres = torch.empty_like(h) if has_res and p > 0 else None
        pd = weight.dtype if weight is not None else bias_dtype
        dw = torch.empty(h.shape[-1], dtype=pd, device=h.device) if want_w else None
        db = torch.empty(h.shape[-1], dtype=pd, device=h.device) if want_b else None
        sta_layer_norm_bwd(dy, h, mean, rstd, weight, dx, dres, dw, db, dh, p, rng)
        return dx, dw, db, None, ((dx if dres is None else dres) if has_res else None), None, None


class STADropoutFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dropout_p, rng):
        rng = rng.clone()
        ctx.save_for_backward(rng)
        ctx.dropout_p = dropout_p
        return sta_dropout_forward(_dense(x), dropout_p, rng)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        (rng,) = ctx.saved_tensors
        return sta_dropout_forward(_dense(dy), ctx.dropout_p, rng), None, None


def _check_dropout(dropout_p, rng):
    if not 0.0 <= dropout_p <= 1.0:   # NaN too
        raise ValueError(f"dropout_p must lie in 0 .. 1, got {dropout_p}")
    if dropout_p > 0 and not isinstance(rng, torch.Tensor):
        raise ValueError("dropout needs rng, an int64 CUDA tensor [seed, offset]")


def sta_layer_norm(x, weight=None, bias=None, eps: float = 1e-5, residual=None, dropout_p: float = 0.0, rng=None):
    """Layer norm over the last dimension of h = residual + dropout(x), with gradients:
    CUDA tensors in bf16, fp16 or fp32, weight and bias in the same type or fp32.
    Returns y, or (y, h) when there is a residual or dropout (h is the residual stream;
    its gradient flows back through the same kernel).  ``rng``: int64 CUDA tensor
    [seed, offset]; give each call of a step its own offset."""
    _check_dropout(dropout_p, rng)
    return STALayerNormFunction.apply(x, weight, bias, float(eps), residual, float(dropout_p), rng)


def sta_dropout(x, dropout_p: float, rng):
    """Dropout with gradients; the mask is a function of ``rng`` (int64 CUDA tensor
    [seed, offset]) and the element's place (rows over the last dimension), and is
    evaluated again in the backward."""
    _check_dropout(dropout_p, rng)
    if dropout_p == 0:
        return x
    return STADropoutFunction.apply(x, float(dropout_p), rng)


def sta_diff_attention(q, k, v, lam, grid, tile, window_per_head: Sequence, scale: Optional[float] = None,
                       token_major: bool = False, norm_weight=None, norm_bias=None, eps: float = 1e-5,
                       dropout_p: float = 0.0, rng=None):
    """Differential attention over tile windows with a backward: bf16 CUDA tensors in
    raster order, [B, heads, L, d] or, with ``token_major``, [B, L, heads, d]; output in
    the same layout.  out = (softmax(scale Q1 K1^T) - lam softmax(scale Q2 K2^T)) V with
    Q1, K1 the first d/2 columns of q and k, Q2, K2 the last d/2, ``lam`` fp32 [heads]
    (any function of learned vectors; it receives a gradient) and scale 1 / sqrt(d / 2)
    by default.  Grids that are not tile multiples are padded with masking.  The method keeps
    lam around 0.2 to 0.8; with |lam| above 10 the first map's dq and dk lose accuracy in
    proportion to it (17 times the usual error at 100), since their row sums come from the
    stored bf16 outputs.

    With ``norm_weight`` (and ``norm_bias``), both [d], every head's output row then
    goes through ``sta_layer_norm`` (a factor such as 1 - lambda_init belongs in the weight).
    The published method has an RMS norm there, without the mean and a bias: weights trained
    with that one give other numbers here.  With ``dropout_p`` > 0 the result
    goes through ``sta_dropout`` with ``rng``."""
    if scale is None:
        scale = 1.0 / float(q.shape[-1] // 2) ** 0.5
    _check_dropout(dropout_p, rng)
    # numbers of this call, whatever becomes of the caller's objects before the backward
    grid, tile, windows = tuple(map(int, grid)), tuple(map(int, tile)), [tuple(map(int, w)) for w in window_per_head]
    # here and not in the function's forward, where gradients are always off and needs_input_grad
    # says what requires them whether or not they are
    save = torch.is_grad_enabled() and any(x.requires_grad for x in (q, k, v, lam))
    out = STADiffAttentionFunction.apply(q, k, v, lam, grid, tile, windows, float(scale), bool(token_major), save)
    if norm_weight is not None or norm_bias is not None:
        out = sta_layer_norm(out, norm_weight, norm_bias, eps)
    return sta_dropout(out, dropout_p, rng) if dropout_p > 0 else out
