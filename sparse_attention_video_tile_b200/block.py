"""Binding of the operators around an attention block: differential attention over
tile windows, layer norm (with an optional dropout and residual sum in front) and
dropout.  Argument marshalling only, like the rest of the package: functions named
after a C entry point of ``include/sta.h`` write into tensors that the caller gives;
``sta_diff_forward``, ``sta_layer_norm_forward``, ``sta_layer_norm_backward`` and
``sta_dropout_forward`` allocate what they return.

All tensors of a call live on one CUDA device, which need not be the current one:
the kernels are launched there, on ``stream`` or that device's current stream.
"""
from __future__ import annotations

import contextlib
import functools
import math
from typing import Optional, Sequence

import numpy as np
import torch

from . import StaError, _check, _d3, _stream, _stream_context, _windows, load_library


_INT32_MAX = 2 ** 31 - 1
_CODES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}   # sta_dtype


def _dtype_code(dtype, name: str) -> int:
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, got {dtype}")
    return code


def _ptr(x, name: str, dtype=None, shape=None, optional: bool = False) -> Optional[int]:
    """Address of a contiguous CUDA tensor, checked against ``dtype`` and ``shape``."""
    if x is None and optional:
        return None
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dtype is not None and x.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {x.dtype}")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if shape is not None and x.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(x.shape)}")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return x.data_ptr()


class _On:
    """Runs the body on the tensors' device (they must share one) and on ``stream``; yields
    the raw stream handle.  Where both are current already, nothing is switched."""

    __slots__ = ("stream", "tensors", "stack")

    def __init__(self, stream, *tensors):
        for t in tensors:
            if t is not None and not isinstance(t, torch.Tensor):
                raise TypeError(f"expected a torch.Tensor, got {type(t).__name__}")
        self.stream, self.tensors, self.stack = stream, tensors, None

    def __enter__(self):
        dev = None
        for t in self.tensors:
            if t is not None:
                d = t.device
                if dev is None:
                    dev = d
                elif d != dev:
                    raise ValueError(f"tensors of one call must be on one device, got {dev} and {d}")
        if dev is None or dev.type != "cuda":
            raise ValueError("CUDA tensors are required")
        at = getattr(self.stream, "device", dev)   # a raw handle does not know its device
        if at != dev:   # the kernels would run there, on memory of another device
            raise ValueError(f"the stream is on {at}, the tensors are on {dev}")
        if self.stream is None and dev.index == torch.cuda.current_device():
            return torch._C._cuda_getCurrentRawStream(dev.index)
        with contextlib.ExitStack() as stack:
            stack.enter_context(torch.cuda.device(dev))
            stack.enter_context(_stream_context(self.stream))
            raw = _stream(self.stream)
            self.stack = stack.pop_all()
        return raw

    def __exit__(self, *exc):
        if self.stack is not None:
            return self.stack.__exit__(*exc)
        return False


def _workspace_ptr(ws, name: str):
    """Address and byte count of a caller's workspace tensor (any element type)."""
    if ws is None:
        return None, 0
    return _ptr(ws, name), ws.numel() * ws.element_size()


_GEOMETRIES = {}   # (grid, tile, windows) of plain numbers -> their C arguments


def _geometry(grid, tile, windows):
    """The C arguments of a (grid, tile, windows) triple, built once for each value.  Only
    numbers are kept: a tensor hashes by its identity, and its value can change."""
    key = (tuple(grid), tuple(tile), tuple(map(tuple, windows)))
    args = _GEOMETRIES.get(key)
    if args is None:
        args = _d3(key[0]), _d3(key[1]), _windows(key[2])
        if all(isinstance(x, (int, np.integer)) for part in (key[:2], key[2]) for t in part for x in t):
            if len(_GEOMETRIES) >= 64:
                _GEOMETRIES.clear()
            _GEOMETRIES[key] = args
    return args


# ------------------------------------------------------------------ layer norm and dropout

def _rows_cols(x, name: str):
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.dim() < 1:
        raise ValueError(f"{name} must have at least one dimension")
    cols = int(x.shape[-1])
    if cols > _INT32_MAX:   # a 32-bit argument of the library, which ctypes would cut
        raise ValueError(f"{name} must have fewer than 2^31 columns, got {cols}")
    return (int(x.numel()) // cols if cols else 0), cols


def _params(weight, bias, cols: int, dtype):
    """Pointers of the weight and the bias and the code of their element type."""
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise TypeError(f"weight and bias types differ: {weight.dtype}, {bias.dtype}")
    pd = weight.dtype if weight is not None else (bias.dtype if bias is not None else dtype)
    return (_ptr(weight, "weight", None, (cols,), True), _ptr(bias, "bias", None, (cols,), True), _dtype_code(pd, "weight"))


def _rng_ptr(rng):
    return _ptr(rng, "rng", torch.int64, (2,), optional=True)


def sta_layer_norm_fwd(x, weight, bias, y, eps: float = 1e-5, residual=None, h=None, mean=None, rstd=None,
                       dropout_p: float = 0.0, rng=None, stream=None) -> None:
    """y = layer norm of h = residual + dropout(x) over the last dimension of contiguous
    CUDA tensors (bf16, fp16 or fp32; weight and bias of the same type or fp32, each may
    be None).  ``h`` receives the sum, ``mean`` and ``rstd`` (fp32 [rows]) the row
    statistics.  ``rng``: int64 CUDA tensor [seed, offset], needed when ``dropout_p`` > 0."""
    rows, cols = _rows_cols(x, "x")
    code = _dtype_code(x.dtype, "x")
    with _On(stream, x, weight, bias, y, residual, h, mean, rstd, rng) as st:
        w, b, pcode = _params(weight, bias, cols, x.dtype)
        px = _ptr(x, "x")
        py = _ptr(y, "y", x.dtype, x.shape)
        pr = _ptr(residual, "residual", x.dtype, x.shape, optional=True)
        ph = _ptr(h, "h", x.dtype, x.shape, optional=True)
        pm = _ptr(mean, "mean", torch.float32, (rows,), optional=True)
        ps = _ptr(rstd, "rstd", torch.float32, (rows,), optional=True)
        _check(load_library().sta_layer_norm_fwd(px, pr, w, b, py, ph, pm, ps, rows, cols, code, pcode, float(eps),
                                                 float(dropout_p), _rng_ptr(rng), st), "sta_layer_norm_fwd")


def sta_layer_norm_forward(x, weight=None, bias=None, eps: float = 1e-5, residual=None, dropout_p: float = 0.0,
                           rng=None, stream=None):
    """``sta_layer_norm_fwd`` into new tensors: (y, h, mean, rstd).  ``h`` is None where
    it would be x itself (no residual and no dropout)."""
    rows, cols = _rows_cols(x, "x")
    code = _dtype_code(x.dtype, "x")
    with _On(stream, x, weight, bias, residual, rng) as st:   # new tensors need no checks of their own
        w, b, pcode = _params(weight, bias, cols, x.dtype)
        px, pr, prng = _ptr(x, "x"), _ptr(residual, "residual", x.dtype, x.shape, optional=True), _rng_ptr(rng)
        y = torch.empty_like(x)
        h = torch.empty_like(x) if residual is not None or dropout_p > 0 else None
        mean = torch.empty(rows, dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
        _check(load_library().sta_layer_norm_fwd(px, pr, w, b, y.data_ptr(), None if h is None else h.data_ptr(),
                                                 mean.data_ptr(), rstd.data_ptr(), rows, cols, code, pcode, float(eps),
                                                 float(dropout_p), prng, st), "sta_layer_norm_forward")
    return y, h, mean, rstd


@functools.lru_cache(maxsize=256)
def sta_layer_norm_bwd_workspace(rows: int, cols: int) -> int:
    """Bytes of workspace that ``sta_layer_norm_bwd`` needs when it makes a weight's or bias's gradient."""
    rows, cols = int(rows), int(cols)
    n = load_library().sta_layer_norm_bwd_workspace(rows, cols) if max(abs(rows) >> 32, abs(cols)) <= _INT32_MAX else -1
    if n < 0:
        raise StaError(4, "sta_layer_norm_bwd_workspace")
    return int(n)


def sta_layer_norm_bwd(dy, h, mean, rstd, weight, dx=None, dresidual=None, dweight=None, dbias=None, dh=None,
                       dropout_p: float = 0.0, rng=None, workspace=None, stream=None) -> None:
    """Backward of ``sta_layer_norm_fwd`` from the normalised ``h`` and its statistics:
    ``dresidual`` is the gradient of h (plus ``dh``, the gradient that reaches h by the
    residual stream), ``dx`` that gradient through the dropout mask; ``dweight`` and
    ``dbias`` are sums over the rows.  ``workspace`` (a CUDA tensor of at least
    ``sta_layer_norm_bwd_workspace`` bytes) is allocated when it is None."""
    rows, cols = _rows_cols(h, "h")
    code = _dtype_code(h.dtype, "h")
    with _On(stream, dy, h, mean, rstd, weight, dx, dresidual, dweight, dbias, dh, rng, workspace) as st:
        if workspace is None and (dweight is not None or dbias is not None):
            workspace = torch.empty(sta_layer_norm_bwd_workspace(rows, cols), dtype=torch.uint8, device=h.device)
        w, _, pcode = _params(weight, None, cols, h.dtype)
        dw, db, gcode = _params(dweight, dbias, cols, h.dtype)
        if weight is not None and (dweight is not None or dbias is not None) and pcode != gcode:
            raise TypeError("dweight and dbias must have the weight's type")
        if weight is None:
            pcode = gcode
        like = h.dtype, h.shape
        ptrs = [_ptr(dy, "dy", *like), _ptr(h, "h"), _ptr(mean, "mean", torch.float32, (rows,)),
                _ptr(rstd, "rstd", torch.float32, (rows,)), w, _ptr(dh, "dh", *like, optional=True),
                _ptr(dx, "dx", *like, optional=True), _ptr(dresidual, "dresidual", *like, optional=True), dw, db]
        pw, nw = _workspace_ptr(workspace, "workspace")
        _check(load_library().sta_layer_norm_bwd(*ptrs, rows, cols, code, pcode, float(dropout_p), _rng_ptr(rng), pw, nw,
                                                 st), "sta_layer_norm_bwd")


def sta_layer_norm_backward(dy, h, mean, rstd, weight=None, dh=None, bias: bool = True, dropout_p: float = 0.0,
                            rng=None, stream=None):
    """``sta_layer_norm_bwd`` into new tensors: (dx, dresidual, dweight, dbias).  Without
    dropout dresidual is dx itself; dweight is None without a weight, dbias without
    ``bias``.  Both have the weight's type (h's type without a weight)."""
    rows, cols = _rows_cols(h, "h")
    code = _dtype_code(h.dtype, "h")
    with _On(stream, dy, h, mean, rstd, weight, dh, rng) as st:   # new tensors need no checks of their own
        w, _, pcode = _params(weight, None, cols, h.dtype)
        like = h.dtype, h.shape
        ptrs = [_ptr(dy, "dy", *like), _ptr(h, "h"), _ptr(mean, "mean", torch.float32, (rows,)),
                _ptr(rstd, "rstd", torch.float32, (rows,)), w, _ptr(dh, "dh", *like, optional=True)]
        prng = _rng_ptr(rng)
        dx = torch.empty_like(h)
        dres = torch.empty_like(h) if dropout_p > 0 else None
        dw = db = ws = None
        if weight is not None:
            dw = torch.empty_like(weight)
        if bias:
            db = torch.empty(cols, dtype=h.dtype if weight is None else weight.dtype, device=h.device)
        size = 0
        if dw is not None or db is not None:
            size = sta_layer_norm_bwd_workspace(rows, cols)
            ws = torch.empty(size, dtype=torch.uint8, device=h.device)
        ptrs += [None if t is None else t.data_ptr() for t in (dx, dres, dw, db)]
        _check(load_library().sta_layer_norm_bwd(*ptrs, rows, cols, code, pcode, float(dropout_p), prng,
                                                 None if ws is None else ws.data_ptr(), size, st),
               "sta_layer_norm_backward")
    return dx, (dx if dres is None else dres), dw, db


def sta_dropout(x, y, dropout_p: float, rng, stream=None) -> None:
    """y = dropout of x: contiguous CUDA tensors (bf16, fp16 or fp32) of one shape, rows
    over the last dimension.  The mask is a function of ``rng`` (int64 CUDA tensor
    [seed, offset]) and the element's place; call it on the gradient with the same rng
    for the backward."""
    rows, cols = _rows_cols(x, "x")
    with _On(stream, x, y, rng) as st:
        _check(load_library().sta_dropout(_ptr(x, "x"), _ptr(y, "y", x.dtype, x.shape), rows, cols,
                                          _dtype_code(x.dtype, "x"), float(dropout_p), _rng_ptr(rng), st), "sta_dropout")


def sta_dropout_forward(x, dropout_p: float, rng, stream=None):
    """``sta_dropout`` into a new tensor."""
    rows, cols = _rows_cols(x, "x")
    code = _dtype_code(x.dtype, "x")
    with _On(stream, x, rng) as st:
        px, prng = _ptr(x, "x"), _rng_ptr(rng)
        y = torch.empty_like(x)
        _check(load_library().sta_dropout(px, y.data_ptr(), rows, cols, code, float(dropout_p), prng, st),
               "sta_dropout_forward")
    return y


# ------------------------------------------------------------------ differential attention

def _diff_dims(q, grid, token_major: bool, windows):
    if q.dim() != 4:
        raise ValueError("q must be [batch, heads, L, d], or [batch, L, heads, d] with token_major")
    a, b, c, d = q.shape
    B, Hn, L = (a, c, b) if token_major else (a, b, c)
    if max(B, Hn, d) > _INT32_MAX:   # 32-bit arguments of the library, which ctypes would cut
        raise ValueError(f"batch, heads and d must be below 2^31, got {B}, {Hn}, {d}")
    if L != grid[0] * grid[1] * grid[2]:
        raise ValueError("L must equal T*H*W")
    if len(windows) != Hn:
        raise ValueError("one window per head is required")
    return B, Hn, L, d


def sta_diff_attention_bwd_workspace(q, grid, tile, window_per_head, token_major: bool = False) -> int:
    """Bytes of workspace that ``sta_diff_attention_bwd`` needs for tensors shaped like q."""
    B, Hn, _, d = _diff_dims(q, grid, token_major, window_per_head)
    n = load_library().sta_diff_attention_bwd_workspace(B, Hn, d, *_geometry(grid, tile, window_per_head))
    if n < 0:
        raise StaError(10, "sta_diff_attention_bwd_workspace")
    return int(n)


def sta_diff_attention_fwd(q, k, v, lam, out, grid, tile, window_per_head: Sequence, scale: float, out2=None, lse=None,
                           token_major: bool = False, stream=None) -> None:
    """Differential attention over tile windows on raster-order bf16 CUDA tensors
    [B, heads, T*H*W, d] ([B, T*H*W, heads, d] with ``token_major``):
    out = (softmax(scale Q1 K1^T) - lam softmax(scale Q2 K2^T)) V, where Q1, K1 are the
    first d/2 columns of q and k, Q2, K2 the last d/2, and lam is fp32 [heads].
    ``out2`` (shaped like out) receives softmax(scale Q2 K2^T) V and ``lse`` (fp32
    [2, B, heads, L]) both maps' log-sum-exps, which the backward needs."""
    B, Hn, L, d = _diff_dims(q, grid, token_major, window_per_head)
    geo = _geometry(grid, tile, window_per_head)
    with _On(stream, q, k, v, lam, out, out2, lse) as st:
        shape = q.shape
        ptrs = [_ptr(q, "q", torch.bfloat16)] + [_ptr(t, n, torch.bfloat16, shape) for n, t in (("k", k), ("v", v))]
        ptrs.append(_ptr(lam, "lam", torch.float32, (Hn,)))
        ptrs.append(_ptr(out, "out", torch.bfloat16, shape))
        ptrs.append(_ptr(out2, "out2", torch.bfloat16, shape, optional=True))
        ptrs.append(_ptr(lse, "lse", torch.float32, (2, B, Hn, L), optional=True))
        _check(load_library().sta_diff_attention_fwd(*ptrs, B, Hn, d, int(bool(token_major)), *geo, float(scale), st),
               "sta_diff_attention_fwd")


def sta_diff_attention_bwd(q, k, v, lam, out, out2, lse, dout, dq, dk, dv, dlam, grid, tile, window_per_head: Sequence,
                           scale: float, token_major: bool = False, workspace=None, stream=None) -> None:
    """Backward of ``sta_diff_attention_fwd``: writes dq, dk, dv (bf16, laid out like q)
    and dlam (fp32 [heads]) from the forward's inputs, out, out2, lse and the output
    gradient dout.  ``workspace`` (at least ``sta_diff_attention_bwd_workspace`` bytes)
    is allocated when it is None."""
    B, Hn, L, d = _diff_dims(q, grid, token_major, window_per_head)
    geo = _geometry(grid, tile, window_per_head)
    with _On(stream, q, k, v, lam, out, out2, lse, dout, dq, dk, dv, dlam, workspace) as st:
        shape = q.shape
        bf = lambda t, n: _ptr(t, n, torch.bfloat16, shape)  # noqa: E731
        ptrs = [bf(q, "q"), bf(k, "k"), bf(v, "v"), _ptr(lam, "lam", torch.float32, (Hn,)), bf(out, "out"),
                bf(out2, "out2"), _ptr(lse, "lse", torch.float32, (2, B, Hn, L)), bf(dout, "dout"), bf(dq, "dq"),
                bf(dk, "dk"), bf(dv, "dv"), _ptr(dlam, "dlam", torch.float32, (Hn,))]
        if workspace is None:
            need = load_library().sta_diff_attention_bwd_workspace(B, Hn, d, *geo)
            if need > 0:
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        pw, nw = _workspace_ptr(workspace, "workspace")
        _check(load_library().sta_diff_attention_bwd(*ptrs, B, Hn, d, int(bool(token_major)), *geo, float(scale), pw, nw,
                                                     st),
               "sta_diff_attention_bwd")


def sta_diff_forward(q, k, v, lam, grid, tile, window_per_head: Sequence, scale: Optional[float] = None,
                     token_major: bool = False, save: bool = False, stream=None):
    """``sta_diff_attention_fwd`` into new tensors, allocated on ``stream``: out, or
    (out, out2, lse) with ``save`` (what the backward needs).  ``scale`` defaults to
    1 / sqrt(d / 2), d / 2 being the columns of one map."""
    B, Hn, L, d = _diff_dims(q, grid, token_major, window_per_head)
    sc = 1.0 / math.sqrt(d / 2) if scale is None else float(scale)
    geo = _geometry(grid, tile, window_per_head)
    with _On(stream, q, k, v, lam) as st:   # new tensors need no checks of their own
        shape = q.shape
        ptrs = [_ptr(q, "q", torch.bfloat16), _ptr(k, "k", torch.bfloat16, shape), _ptr(v, "v", torch.bfloat16, shape),
                _ptr(lam, "lam", torch.float32, (Hn,))]
        out = torch.empty_like(q)
        out2 = lse = None
        if save:
            out2 = torch.empty_like(q)
            lse = torch.empty((2, B, Hn, L), dtype=torch.float32, device=q.device)
        ptrs += [None if t is None else t.data_ptr() for t in (out, out2, lse)]
        _check(load_library().sta_diff_attention_fwd(*ptrs, B, Hn, d, int(bool(token_major)), *geo, sc, st),
               "sta_diff_forward")
    return (out, out2, lse) if save else out
