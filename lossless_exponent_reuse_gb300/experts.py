"""The mixture-of-experts layer next to the Allgather that rebuilds its weights.

Thin binding of the ``ciera_rmsnorm`` ... ``ciera_expert_mm_dw`` entry points
of libciera (include/ciera.h has the formulas): argument checks, outputs
allocated with torch unless given, and the current CUDA stream.  Every sum,
choice and product runs in libciera's sm_103a kernels; there is no CPU
fallback.

    norm       rmsnorm, rmsnorm_backward, quantize_rows
    route      route, route_backward
    combine    gather_rows, combine, combine_backward
    products   mm, mm_gated, mm_dx, mm_dw

The products take the experts' weights as strided views: ``bucket_views``
gives those of a flat bucket as ``SimulatedAllgather.step`` rebuilds it, so
that no weight is copied between the Allgather and the layer.  Matrices may
have any row stride; their last dimension must be contiguous.

Every call takes ``stream`` (a torch stream or a handle) as a keyword and runs
on the current one without it; what it allocates, outputs and scratch memory,
belongs to that stream or to the graph it is captured in, so that calls of
several threads, streams and replayed graphs may overlap.  ``status`` reads the
device's error word.  Nothing is registered with autograd: outputs carry no
history, and a training step makes the gradients' calls itself.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import NamedTuple, Optional, Tuple

import torch

from . import ciera

BF16 = 0
E4M3 = 1
F32 = 2
ROUTE_RENORMALIZE = 1
GATED = 1
ACCUMULATE = 2

_BF16, _F32, _E4M3, _I32 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int32


class Norm(NamedTuple):
    y: torch.Tensor                  # bf16, or e4m3 with scale
    scale: Optional[torch.Tensor]    # [rows] float32, or None
    h: torch.Tensor                  # x + residual (x itself without a residual)
    rstd: torch.Tensor               # [rows] float32


class Routing(NamedTuple):
    weights: torch.Tensor            # [tokens, topk] float32
    experts: torch.Tensor            # [tokens, topk] int32, -1: none
    slots: torch.Tensor              # [tokens, topk] int32 row in expert order, -1: none
    tokens: torch.Tensor             # [tokens * topk] int32 token of each row, -1: unused
    offsets: torch.Tensor            # [experts + 1] int32


def bucket_views(bucket: torch.Tensor, experts: int, dim: int, ff: int,
                 offset: int = 0) -> Tuple[torch.Tensor, torch.Tensor]:
    """(gate_up [experts, 2 ff, dim], down [experts, dim, ff]) as bf16 views of
    a flat bucket (bf16 or its uint16 bit patterns) that holds, from
    ``offset`` on, each expert's gate [ff, dim], up [ff, dim] and
    down [dim, ff] in turn (``workloads``' layout)."""
    if bucket.dim() != 1 or not bucket.is_contiguous() or bucket.element_size() != 2:
        raise ValueError("bucket must be a flat contiguous 16-bit tensor")
    if offset < 0 or bucket.numel() < offset + 3 * experts * dim * ff:
        raise ValueError(f"bucket holds {bucket.numel()} values, needs "
                         f"{offset + 3 * experts * dim * ff}")
    b = bucket.view(_BF16)
    at = b.storage_offset() + offset
    each = 3 * ff * dim
    return (b.as_strided((experts, 2 * ff, dim), (each, dim, 1), at),
            b.as_strided((experts, dim, ff), (each, ff, 1), at + 2 * ff * dim))


# ---- arguments -----------------------------------------------------------

_needs = {}           # (tokens, experts, dim): bytes
_workspaces = {}      # (device index, stream handle): scratch memory of its calls
_controls = {}        # device index: its control block's address
_functions = {}
_MAX_TOPK = 32        # the router's limit
_raw_stream = torch._C._cuda_getCurrentRawStream
_capturing = torch._C._cuda_isCurrentStreamCapturing
# Rows per expert above which a product's rows are gathered before it, by a
# launch of its own, instead of inside it (see ciera_expert_mm's row_tokens).
_GATHER_ROWS = 32


def _on_stream(fn):
    """Runs ``fn`` on its ``stream`` argument (a torch stream or a handle), so
    that what it allocates belongs to that stream too; None: the current one."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream))
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _scratch(index: int, stream: int, tokens: int, experts: int, dim: int) -> torch.Tensor:
    """Memory for one call of these sizes on the current stream, whose handle is
    ``stream``: calls on a stream follow one another and share it (the library
    keeps a call's launches together), a captured call has its graph's own."""
    need = _needs.get((tokens, experts, dim)) or _need(tokens, experts, dim)
    if _capturing():
        return torch.empty(need, dtype=torch.uint8, device=index)
    ws = _workspaces.get((index, stream))
    if ws is None or ws.numel() < need:
        ws = _workspaces[index, stream] = torch.empty(1 << (need - 1).bit_length(),
                                                      dtype=torch.uint8, device=index)
    return ws


def _need(tokens: int, experts: int, dim: int) -> int:
    need = ciera.lib().ciera_moe_workspace_bytes(tokens, experts, dim)
    if need == 0:
        raise ValueError(f"no workspace for {tokens} tokens, {experts} experts, {dim} columns")
    if len(_needs) < 4096:
        _needs[tokens, experts, dim] = need
    return need


def workspace(index: int, stream: int, tokens: int = 0, experts: int = 0,
              dim: int = 0) -> torch.Tensor:
    """A workspace for the C entry points' calls of these sizes on a stream
    handle of a device: the caller's own, zero-filled."""
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=index)):
        return torch.zeros(_need(tokens, experts, dim), dtype=torch.uint8, device=index)


def _control(index: int) -> int:
    """The device's control block, which all products share."""
    at = _controls.get(index)
    if at is None:
        got = ctypes.c_void_p()
        _call("ciera_moe_control", index, ctypes.byref(got))
        at = _controls[index] = got.value
    return at


@_on_stream
def status(device="cuda") -> int:
    """ciera_status of the device's products: waits for the stream; what other
    streams' calls and replayed graphs have reported by then counts too."""
    index = torch.empty(0, device=device).get_device()
    with torch.cuda.device(index):
        st = ciera.lib().ciera_status(_control(index), _raw_stream(index))
    if st == ciera.E_CUDA:
        raise ciera.CieraError(st, "ciera_status")
    return st


# The checks below are on every call's path: one test where all is well, and
# the words for what is wrong apart from it.

def _index(t, name: str) -> int:
    """Device index of the tensor that the others have to be with."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _placed(t, name: str, dtype, index: int) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != index:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, other tensors on cuda:{index}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _matrix(t, name: str, dtype, index: int, rows: Optional[int] = None,
            cols: Optional[int] = None) -> int:
    """Row stride of a matrix with contiguous rows (of one row: any)."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index:
        shape = t.shape
        if (len(shape) == 2 and (rows is None or shape[0] == rows)
                and (cols is None or shape[1] == cols)):
            stride, unit = t.stride()
            if unit == 1 or shape[1] <= 1:
                if shape[0] <= 1:
                    return shape[1]
                if stride >= shape[1]:
                    return stride
    _placed(t, name, dtype, index)
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, got {t.dim()}")
    if (rows is not None and t.shape[0] != rows) or (cols is not None and t.shape[1] != cols):
        want = ["any" if rows is None else rows, "any" if cols is None else cols]
        raise ValueError(f"{name} must be {want}, got {list(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    raise ValueError(f"{name}'s rows overlap")


def _array(t, name: str, dtype, index: int, *shape: int) -> int:
    """Pointer of a contiguous tensor of this shape."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index
            and t.shape == shape and t.is_contiguous()):
        return t.data_ptr()
    _placed(t, name, dtype, index)
    raise ValueError(f"{name} must be contiguous and {list(shape)}, got {list(t.shape)}")


def _stack(t, name: str, dtype, index: int) -> Tuple[int, int]:
    """Row and expert strides of [experts, rows, columns], contiguous rows."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index:
        shape = t.shape
        if len(shape) == 3:
            expert, row, unit = t.stride()
            if shape[1] <= 1:
                row = shape[2]
            if (unit == 1 or shape[2] <= 1) and row >= shape[2]:
                return row, expert if shape[0] > 1 else shape[1] * row
    _placed(t, name, dtype, index)
    if t.dim() != 3:
        raise ValueError(f"{name} must be [experts, rows, columns]")
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    raise ValueError(f"{name}'s rows overlap")


def _load(name: str):
    fn = _functions[name] = getattr(ciera.lib(), name)
    return fn


def _call(name: str, index: int, *args) -> None:
    fn = _functions.get(name) or _load(name)
    if index == torch._C._cuda_getDevice():
        st = fn(*args)
    else:
        with torch.cuda.device(index):
            st = fn(*args)
    if st != ciera.OK:
        raise ciera.CieraError(st, name)


# ---- norm ----------------------------------------------------------------

@_on_stream
def rmsnorm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
            eps: float = 1e-6, quantize: bool = False) -> Norm:
    """ciera_rmsnorm: the norm of x + residual (bf16 [rows, dim]), as bf16 or,
    with ``quantize``, as e4m3 with a scale per row."""
    index = _index(x, "x")
    x_stride = _matrix(x, "x", _BF16, index)
    rows, dim = x.shape
    w = _array(weight, "weight", _BF16, index, dim)
    device = x.device
    y = torch.empty((rows, dim), dtype=_E4M3 if quantize else _BF16, device=device)
    rstd = torch.empty(rows, dtype=_F32, device=device)
    scale = torch.empty(rows, dtype=_F32, device=device) if quantize else None
    if residual is None:
        h, res, res_stride, h_ptr = x, None, 0, None
    else:
        res_stride = _matrix(residual, "residual", _BF16, index, rows, dim)
        h = torch.empty((rows, dim), dtype=_BF16, device=device)
        res, h_ptr = residual.data_ptr(), h.data_ptr()
    _call("ciera_rmsnorm", index, x.data_ptr(), x_stride, res, res_stride, w, rows, dim, eps,
          y.data_ptr(), E4M3 if quantize else BF16, scale.data_ptr() if quantize else None,
          h_ptr, rstd.data_ptr(), _raw_stream(index))
    return Norm(y, scale, h, rstd)


@_on_stream
def rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, rstd: torch.Tensor,
                     weight: torch.Tensor,
                     dh: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """ciera_rmsnorm_backward: (dx, dweight) with dx the gradient of x and of
    the residual alike; ``dh`` is the gradient that reaches h through the next
    residual."""
    index = _index(dy, "dy")
    dy_stride = _matrix(dy, "dy", _BF16, index)
    rows, dim = dy.shape
    h_stride = _matrix(h, "h", _BF16, index, rows, dim)
    r = _array(rstd, "rstd", _F32, index, rows)
    w = _array(weight, "weight", _BF16, index, dim)
    dh_stride = 0 if dh is None else _matrix(dh, "dh", _BF16, index, rows, dim)
    s = _raw_stream(index)
    ws = _scratch(index, s, rows, 0, dim)
    dx = torch.empty((rows, dim), dtype=_BF16, device=dy.device)
    dweight = torch.empty(dim, dtype=_F32, device=dy.device)
    _call("ciera_rmsnorm_backward", index, dy.data_ptr(), dy_stride, h.data_ptr(), h_stride, r, w,
          None if dh is None else dh.data_ptr(), dh_stride, rows, dim, dx.data_ptr(),
          dweight.data_ptr(), ws.data_ptr(), ws.numel(), s)
    return dx, dweight


@_on_stream
def quantize_rows(x: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """ciera_quantize_rows: (e4m3, scale per row) of bf16 [..., dim] (weights,
    laid out once; several leading dimensions that no one row stride covers, as
    a bucket's views have them, are copied first)."""
    index = _index(x, "x")
    shape = x.shape
    flat = x if len(shape) == 2 else x.reshape(math.prod(shape[:-1]), *shape[-1:])
    stride = _matrix(flat, "x", _BF16, index)
    rows, dim = flat.shape
    y = torch.empty(shape, dtype=_E4M3, device=x.device)
    scale = torch.empty(shape[:-1], dtype=_F32, device=x.device)
    _call("ciera_quantize_rows", index, flat.data_ptr(), stride, rows, dim, y.data_ptr(),
          scale.data_ptr(), _raw_stream(index))
    return y, scale


# ---- route ---------------------------------------------------------------

def _logits(t) -> int:
    if not isinstance(t, torch.Tensor) or t.dtype not in (_BF16, _F32):
        raise ValueError("logits must be float32 or bfloat16")
    return F32 if t.dtype is _F32 else BF16


@_on_stream
def route(logits: torch.Tensor, topk: int, renormalize: bool = False,
          token_mask: Optional[torch.Tensor] = None) -> Routing:
    """ciera_route: the topk experts of each token and the expert order;
    ``token_mask`` (bool or uint8 per token), where false, routes nowhere."""
    kind = _logits(logits)
    index = _index(logits, "logits")
    stride = _matrix(logits, "logits", logits.dtype, index)
    tokens, experts = logits.shape
    topk = int(topk)
    if not 1 <= topk <= min(experts, _MAX_TOPK):
        raise ValueError(f"topk must be in 1..{min(experts, _MAX_TOPK)}, got {topk}")
    mask = None
    if token_mask is not None:
        if token_mask.dtype not in (torch.bool, torch.uint8):
            raise ValueError("token_mask must be bool or uint8")
        mask = _array(token_mask, "token_mask", token_mask.dtype, index, tokens)
    s = _raw_stream(index)
    ws = _scratch(index, s, tokens, experts, 0)
    device, pairs = logits.device, (tokens, topk)
    weights = torch.empty(pairs, dtype=_F32, device=device)
    chosen = torch.empty(pairs, dtype=_I32, device=device)
    slots = torch.empty(pairs, dtype=_I32, device=device)
    row_tokens = torch.empty(tokens * topk, dtype=_I32, device=device)
    offsets = torch.empty(experts + 1, dtype=_I32, device=device)
    _call("ciera_route", index, logits.data_ptr(), kind, stride, mask, tokens, experts, topk,
          ROUTE_RENORMALIZE if renormalize else 0, weights.data_ptr(), chosen.data_ptr(),
          slots.data_ptr(), row_tokens.data_ptr(), offsets.data_ptr(), ws.data_ptr(), ws.numel(),
          s)
    return Routing(weights, chosen, slots, row_tokens, offsets)


@_on_stream
def route_backward(dweights: torch.Tensor, weights: torch.Tensor, experts: torch.Tensor,
                   logits: torch.Tensor, renormalize: bool = False) -> torch.Tensor:
    """ciera_route_backward: the logits' gradient from the weights' (``weights``
    and ``experts`` as ``route`` returned them)."""
    kind = _logits(logits)
    index = _index(logits, "logits")
    stride = _matrix(logits, "logits", logits.dtype, index)
    tokens, n_experts = logits.shape
    if weights.dim() != 2:
        raise ValueError("weights must be [tokens, topk]")
    topk = weights.shape[1]
    w = _array(weights, "weights", _F32, index, tokens, topk)
    dw = _array(dweights, "dweights", _F32, index, tokens, topk)
    chosen = _array(experts, "experts", _I32, index, tokens, topk)
    dlogits = torch.empty((tokens, n_experts), dtype=logits.dtype, device=logits.device)
    _call("ciera_route_backward", index, dw, w, chosen, logits.data_ptr(), kind, stride, tokens,
          n_experts, topk, ROUTE_RENORMALIZE if renormalize else 0, dlogits.data_ptr(),
          _raw_stream(index))
    return dlogits


# ---- gather and combine ----------------------------------------------------

def _slots(t, index: int) -> Tuple[int, int]:
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError("slots must be [tokens, topk]")
    _array(t, "slots", _I32, index, *t.shape)
    return t.shape


@_on_stream
def combine(rows: torch.Tensor, slots: torch.Tensor,
            weights: Optional[torch.Tensor] = None) -> torch.Tensor:
    """ciera_combine: each token's weighted sum of its rows ([tokens, dim]
    bf16); without ``weights`` the plain sum, which is the gradient of
    gathering tokens into expert order."""
    index = _index(rows, "rows")
    stride = _matrix(rows, "rows", _BF16, index)
    tokens, topk = _slots(slots, index)
    w = None if weights is None else _array(weights, "weights", _F32, index, tokens, topk)
    n_rows, dim = rows.shape
    y = torch.empty((tokens, dim), dtype=_BF16, device=rows.device)
    _call("ciera_combine", index, rows.data_ptr(), stride, n_rows, slots.data_ptr(), w, tokens,
          topk, dim, y.data_ptr(), _raw_stream(index))
    return y


@_on_stream
def combine_backward(dy: torch.Tensor, rows: torch.Tensor, slots: torch.Tensor,
                     weights: torch.Tensor,
                     offsets: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """ciera_combine_backward: (drows, dweights)."""
    index = _index(rows, "rows")
    stride = _matrix(rows, "rows", _BF16, index)
    n_rows, dim = rows.shape
    tokens, topk = _slots(slots, index)
    dy_stride = _matrix(dy, "dy", _BF16, index, tokens, dim)
    w = _array(weights, "weights", _F32, index, tokens, topk)
    off, experts = _offsets(offsets, index)
    drows = torch.empty((n_rows, dim), dtype=_BF16, device=rows.device)
    dweights = torch.empty((tokens, topk), dtype=_F32, device=rows.device)
    _call("ciera_combine_backward", index, dy.data_ptr(), dy_stride, rows.data_ptr(), stride,
          n_rows, slots.data_ptr(), w, off, experts, tokens, topk, dim, drows.data_ptr(),
          dweights.data_ptr(), _raw_stream(index))
    return drows, dweights


def _gather(x, tokens, x_scale, stride, index, grain=1):
    """x[tokens], rows a multiple of ``grain`` elements apart, and their scales."""
    rows, dim = tokens.numel(), x.shape[1]
    y_stride = -(-dim // grain) * grain
    y = torch.empty((rows, y_stride), dtype=x.dtype, device=x.device)
    scale = None if x_scale is None else torch.empty(rows, dtype=_F32, device=x.device)
    _call("ciera_gather_rows_strided", index, x.data_ptr(), stride, x.shape[0],
          E4M3 if x.dtype is _E4M3 else BF16, None if x_scale is None else x_scale.data_ptr(),
          tokens.data_ptr(), rows, dim, y.data_ptr(), y_stride,
          None if scale is None else scale.data_ptr(), _raw_stream(index))
    return y, scale


@_on_stream
def gather_rows(x: torch.Tensor, tokens: torch.Tensor, x_scale: Optional[torch.Tensor] = None):
    """ciera_gather_rows: x[tokens] in expert order (bf16, or e4m3 with
    ``x_scale``: then (rows, scales)), zeros where tokens is -1.  A training
    step that needs the rows twice (``mm_gated``, then ``mm_dw``) gathers them
    once."""
    index = _index(x, "x")
    e4m3 = x_scale is not None
    stride = _matrix(x, "x", _E4M3 if e4m3 else _BF16, index)
    _tokens(tokens, index)
    if e4m3:
        _array(x_scale, "x_scale", _F32, index, x.shape[0])
    y, scale = _gather(x, tokens, x_scale, stride, index)
    return (y, scale) if e4m3 else y


# ---- products grouped by expert -------------------------------------------

def _offsets(t, index: int, experts: Optional[int] = None) -> Tuple[int, int]:
    """Pointer, and the number of experts."""
    if experts is None:
        if not isinstance(t, torch.Tensor) or t.numel() < 1:
            raise ValueError("offsets must hold experts + 1 values")
        experts = t.numel() - 1
    return _array(t, "offsets", _I32, index, experts + 1), experts


def _tokens(t, index: int) -> int:
    if not isinstance(t, torch.Tensor) or t.dim() != 1:
        raise ValueError("tokens must have one dimension")
    return _array(t, "tokens", _I32, index, t.shape[0])


def _forward(x, w, offsets, tokens, x_scale, w_scale, gated, keep):
    index = _index(x, "x")
    dtype = x.dtype
    e4m3 = dtype is _E4M3
    if not e4m3:
        dtype = _BF16
    x_stride = _matrix(x, "x", dtype, index)
    w_stride, w_expert_stride = _stack(w, "w", dtype, index)
    experts, features, k = w.shape
    x_rows = x.shape[0]
    if x.shape[1] != k:
        raise ValueError(f"x has {x.shape[1]} columns, w {k}")
    if gated and features % 2:
        raise ValueError("a gated product needs an even number of features (gate, then up)")
    if e4m3 != (x_scale is not None) or e4m3 != (w_scale is not None):
        raise ValueError("x_scale and w_scale go with e4m3 operands")
    xs = ws = None
    if e4m3:
        xs = _array(x_scale, "x_scale", _F32, index, x_rows)
        ws = _array(w_scale, "w_scale", _F32, index, experts, features)
    off, _ = _offsets(offsets, index, experts)
    rows, row_tokens = x_rows, None
    if tokens is not None:
        row_tokens = _tokens(tokens, index)
        rows = tokens.shape[0]
        if rows > _GATHER_ROWS * experts:
            x, x_scale = _gather(x, tokens, x_scale, x_stride, index, 16 if e4m3 else 8)
            x_stride, x_rows, row_tokens = x.shape[1], rows, None
            xs = x_scale.data_ptr() if e4m3 else None
    n = features // 2 if gated else features
    s = _raw_stream(index)
    y = torch.empty((rows, n), dtype=_BF16, device=x.device)
    pre = torch.empty((rows, features), dtype=_BF16, device=x.device) if keep else None
    _call("ciera_expert_mm", index, x.data_ptr(), x_stride, x_rows, row_tokens, w.data_ptr(),
          w_stride, w_expert_stride, xs, ws, off, rows, experts, n, k, E4M3 if e4m3 else BF16,
          GATED if gated else 0, y.data_ptr(), pre.data_ptr() if keep else None,
          _control(index), s)
    return y, pre


@_on_stream
def mm(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor,
       tokens: Optional[torch.Tensor] = None, x_scale: Optional[torch.Tensor] = None,
       w_scale: Optional[torch.Tensor] = None) -> torch.Tensor:
    """ciera_expert_mm: rows in expert order times each row's expert's weights
    (w [experts, n, k]); bf16, or e4m3 with ``x_scale`` (per row of x) and
    ``w_scale`` [experts, n].  With ``tokens`` row r is x[tokens[r]]."""
    return _forward(x, w, offsets, tokens, x_scale, w_scale, False, False)[0]


@_on_stream
def mm_gated(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor,
             tokens: Optional[torch.Tensor] = None, x_scale: Optional[torch.Tensor] = None,
             w_scale: Optional[torch.Tensor] = None, keep: bool = False):
    """ciera_expert_mm with CIERA_GATED: silu(gate) * up of w [experts, 2 n, k];
    with ``keep``, (h, pre) where pre [rows, 2 n] is what the gradient needs."""
    h, pre = _forward(x, w, offsets, tokens, x_scale, w_scale, True, keep)
    return (h, pre) if keep else h


@_on_stream
def mm_dx(dy: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor,
          gated: Optional[torch.Tensor] = None) -> torch.Tensor:
    """ciera_expert_mm_dx: gradient of the rows, [rows, k]; with ``gated`` (the
    ``pre`` that mm_gated kept) through the gated unit, [rows, 2 k]."""
    index = _index(dy, "dy")
    dy_stride = _matrix(dy, "dy", _BF16, index)
    w_stride, w_expert_stride = _stack(w, "w", _BF16, index)
    experts, n, k = w.shape
    rows = dy.shape[0]
    if dy.shape[1] != n:
        raise ValueError(f"dy has {dy.shape[1]} columns, w {n} features")
    off, _ = _offsets(offsets, index, experts)
    pre = None if gated is None else _array(gated, "gated", _BF16, index, rows, 2 * k)
    s = _raw_stream(index)
    dx = torch.empty((rows, k if gated is None else 2 * k), dtype=_BF16, device=dy.device)
    _call("ciera_expert_mm_dx", index, dy.data_ptr(), dy_stride, w.data_ptr(), w_stride,
          w_expert_stride, off, rows, experts, n, k, pre, dx.data_ptr(),
          _control(index), s)
    return dx


@_on_stream
def mm_dw(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor,
          tokens: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
          accumulate: bool = False) -> torch.Tensor:
    """ciera_expert_mm_dw: gradient of the weights, [experts, n, k], into
    ``out`` (bf16 or float32, for instance a view of a gradient bucket; bf16
    if not given), added to what it holds with ``accumulate``."""
    index = _index(dy, "dy")
    dy_stride = _matrix(dy, "dy", _BF16, index)
    x_stride = _matrix(x, "x", _BF16, index)
    rows, n = dy.shape
    off, experts = _offsets(offsets, index)
    k = x.shape[1]
    if tokens is not None:
        _tokens(tokens, index)
    if (x if tokens is None else tokens).shape[0] != rows:
        raise ValueError(f"dy has {rows} rows, x {(x if tokens is None else tokens).shape[0]}")
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = torch.empty((experts, n, k), dtype=_BF16, device=dy.device)
    elif not isinstance(out, torch.Tensor) or out.dtype not in (_BF16, _F32):
        raise ValueError("out must be bfloat16 or float32")
    out_stride, out_expert_stride = _stack(out, "out", out.dtype, index)
    if out.shape != (experts, n, k):
        raise ValueError(f"out must be {[experts, n, k]}, got {list(out.shape)}")
    # an expert behind the other, or each row's experts side by side
    if (experts > 1 and n and k and out_expert_stride < (n - 1) * out_stride + k
            and (out_expert_stride < k or out_stride < (experts - 1) * out_expert_stride + k)):
        raise ValueError("out's experts overlap")
    if tokens is not None:
        x, _ = _gather(x, tokens, None, x_stride, index, 8)
        x_stride = x.shape[1]
    s = _raw_stream(index)
    _call("ciera_expert_mm_dw", index, dy.data_ptr(), dy_stride, x.data_ptr(), x_stride, off, rows,
          experts, n, k, out.data_ptr(), out_stride, out_expert_stride,
          F32 if out.dtype is _F32 else BF16, ACCUMULATE if accumulate else 0,
          _control(index), s)
    return out
