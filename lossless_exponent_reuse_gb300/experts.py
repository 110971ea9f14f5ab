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
on the current one without it; what it allocates belongs to that stream.
Calls that need scratch memory share one workspace per device and stream
(``workspace``), created on first use and grown as needed; ``status`` reads
the error word the kernels leave there.
"""
from __future__ import annotations

import functools
from typing import NamedTuple, Optional, Tuple

import torch

from . import ciera

BF16 = 0
E4M3 = 1
F32 = 2
ROUTE_RENORMALIZE = 1
GATED = 1
ACCUMULATE = 2

_BF16, _F32, _E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


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

_workspaces = {}
_CONTROL_BYTES = 256
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


def _current(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def workspace(device, stream: int, tokens: int = 0, experts: int = 0, dim: int = 0):
    """The workspace of a device and stream handle, for calls of these sizes."""
    need = ciera.lib().ciera_moe_workspace_bytes(tokens, experts, dim)
    if need == 0:
        raise ValueError(f"no workspace for {tokens} tokens, {experts} experts, {dim} columns")
    key = (device, stream)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < need:
        old, ws = ws, torch.zeros(need, dtype=torch.uint8, device=device)
        if old is not None:  # a status not read yet
            ws[:_CONTROL_BYTES].copy_(old[:_CONTROL_BYTES])
        _workspaces[key] = ws
    return ws


@_on_stream
def status(device="cuda") -> int:
    """ciera_status of the stream's workspace: waits for the stream."""
    device = torch.empty(0, device=device).device
    s = _current(device)
    ws = _workspaces.get((device, s))
    return ciera.OK if ws is None else ciera.status(ws, stream=s)


def _matrix(t: torch.Tensor, name: str, dtype, shape=None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, got {t.dim()}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{name}'s rows overlap")
    return t


def _stride(t: torch.Tensor) -> int:
    """Row stride; that of a single row does not matter and may be anything."""
    return t.stride(-2) if t.shape[-2] > 1 else t.shape[-1]


def _array(t: torch.Tensor, name: str, dtype, shape) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {list(shape)}, got "
                         f"{t.dtype} {list(t.shape)}")
    return t


def _stack(t: torch.Tensor, name: str, dtype) -> torch.Tensor:
    """Experts' matrices [experts, rows, columns], contiguous rows."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [experts, rows, columns]")
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    if t.shape[1] > 1 and t.stride(1) < t.shape[2]:
        raise ValueError(f"{name}'s rows overlap")
    return t


def _same_device(*tensors) -> torch.device:
    device = tensors[0].device
    for t in tensors[1:]:
        if t is not None and t.device != device:
            raise ValueError(f"tensors on {device} and {t.device}")
    return device


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _call(name: str, device: torch.device, *args) -> None:
    if device.index == torch.cuda.current_device():
        st = getattr(ciera.lib(), name)(*args)
    else:
        with torch.cuda.device(device):
            st = getattr(ciera.lib(), name)(*args)
    if st != ciera.OK:
        raise ciera.CieraError(st, name)


# ---- norm ----------------------------------------------------------------

@_on_stream
def rmsnorm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
            eps: float = 1e-6, quantize: bool = False) -> Norm:
    """ciera_rmsnorm: the norm of x + residual (bf16 [rows, dim]), as bf16 or,
    with ``quantize``, as e4m3 with a scale per row."""
    _matrix(x, "x", _BF16)
    rows, dim = x.shape
    _array(weight, "weight", _BF16, (dim,))
    if residual is not None:
        _matrix(residual, "residual", _BF16, (rows, dim))
    device = _same_device(x, weight, residual)
    y = torch.empty((rows, dim), dtype=_E4M3 if quantize else _BF16, device=device)
    scale = torch.empty(rows, dtype=_F32, device=device) if quantize else None
    h = torch.empty((rows, dim), dtype=_BF16, device=device) if residual is not None else x
    rstd = torch.empty(rows, dtype=_F32, device=device)
    _call("ciera_rmsnorm", device, _ptr(x), _stride(x), _ptr(residual),
          0 if residual is None else _stride(residual), _ptr(weight), rows, dim, float(eps),
          _ptr(y), E4M3 if quantize else BF16, _ptr(scale),
          None if residual is None else _ptr(h), _ptr(rstd), _current(device))
    return Norm(y, scale, h, rstd)


@_on_stream
def rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, rstd: torch.Tensor,
                     weight: torch.Tensor, dh: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """ciera_rmsnorm_backward: (dx, dweight) with dx the gradient of x and of
    the residual alike; ``dh`` is the gradient that reaches h through the next
    residual."""
    _matrix(dy, "dy", _BF16)
    rows, dim = dy.shape
    _matrix(h, "h", _BF16, (rows, dim))
    _array(rstd, "rstd", _F32, (rows,))
    _array(weight, "weight", _BF16, (dim,))
    if dh is not None:
        _matrix(dh, "dh", _BF16, (rows, dim))
    device = _same_device(dy, h, rstd, weight, dh)
    s = _current(device)
    ws = workspace(device, s, tokens=rows, dim=dim)
    dx = torch.empty((rows, dim), dtype=_BF16, device=device)
    dweight = torch.empty(dim, dtype=_F32, device=device)
    _call("ciera_rmsnorm_backward", device, _ptr(dy), _stride(dy), _ptr(h), _stride(h),
          _ptr(rstd), _ptr(weight), _ptr(dh), 0 if dh is None else _stride(dh), rows, dim,
          _ptr(dx), _ptr(dweight), _ptr(ws), ws.numel(), s)
    return dx, dweight


@_on_stream
def quantize_rows(x: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """ciera_quantize_rows: (e4m3, scale per row) of bf16 [..., dim] whose
    leading dimensions, if several, are contiguous (weights, laid out once)."""
    flat = x if isinstance(x, torch.Tensor) and x.dim() == 2 else x.reshape(-1, x.shape[-1])
    _matrix(flat, "x", _BF16)
    rows, dim = flat.shape
    device = flat.device
    y = torch.empty(x.shape, dtype=_E4M3, device=device)
    scale = torch.empty(x.shape[:-1], dtype=_F32, device=device)
    _call("ciera_quantize_rows", device, _ptr(flat), _stride(flat), rows, dim, _ptr(y),
          _ptr(scale), _current(device))
    return y, scale


# ---- route ---------------------------------------------------------------

def _logits(t: torch.Tensor) -> int:
    if not isinstance(t, torch.Tensor) or t.dtype not in (_BF16, _F32):
        raise ValueError("logits must be float32 or bfloat16")
    _matrix(t, "logits", t.dtype)
    return F32 if t.dtype == _F32 else BF16


@_on_stream
def route(logits: torch.Tensor, topk: int, renormalize: bool = False,
          token_mask: Optional[torch.Tensor] = None) -> Routing:
    """ciera_route: the topk experts of each token and the expert order;
    ``token_mask`` (bool or uint8 per token), where false, routes nowhere."""
    kind = _logits(logits)
    tokens, experts = logits.shape
    if token_mask is not None:
        if token_mask.dtype not in (torch.bool, torch.uint8):
            raise ValueError("token_mask must be bool or uint8")
        _array(token_mask, "token_mask", token_mask.dtype, (tokens,))
    device = _same_device(logits, token_mask)
    s = _current(device)
    topk = int(topk)
    if not 1 <= topk <= experts:
        raise ValueError(f"topk must be in 1..{experts}, got {topk}")
    ws = workspace(device, s, tokens=tokens, experts=experts)
    weights = torch.empty((tokens, topk), dtype=_F32, device=device)
    chosen = torch.empty((tokens, topk), dtype=torch.int32, device=device)
    slots = torch.empty((tokens, topk), dtype=torch.int32, device=device)
    row_tokens = torch.empty(tokens * topk, dtype=torch.int32, device=device)
    offsets = torch.empty(experts + 1, dtype=torch.int32, device=device)
    _call("ciera_route", device, _ptr(logits), kind, _stride(logits), _ptr(token_mask), tokens,
          experts, topk, ROUTE_RENORMALIZE if renormalize else 0, _ptr(weights), _ptr(chosen),
          _ptr(slots), _ptr(row_tokens), _ptr(offsets), _ptr(ws), ws.numel(), s)
    return Routing(weights, chosen, slots, row_tokens, offsets)


@_on_stream
def route_backward(dweights: torch.Tensor, weights: torch.Tensor, experts: torch.Tensor,
                   logits: torch.Tensor, renormalize: bool = False) -> torch.Tensor:
    """ciera_route_backward: the logits' gradient from the weights' (``weights``
    and ``experts`` as ``route`` returned them)."""
    kind = _logits(logits)
    tokens, n_experts = logits.shape
    if weights.dim() != 2:
        raise ValueError("weights must be [tokens, topk]")
    shape = (tokens, weights.shape[1])
    _array(weights, "weights", _F32, shape)
    _array(dweights, "dweights", _F32, shape)
    _array(experts, "experts", torch.int32, shape)
    device = _same_device(logits, dweights, weights, experts)
    dlogits = torch.empty((tokens, n_experts), dtype=logits.dtype, device=device)
    _call("ciera_route_backward", device, _ptr(dweights), _ptr(weights), _ptr(experts),
          _ptr(logits), kind, _stride(logits), tokens, n_experts, shape[1],
          ROUTE_RENORMALIZE if renormalize else 0, _ptr(dlogits), _current(device))
    return dlogits


# ---- combine -------------------------------------------------------------

@_on_stream
def combine(rows: torch.Tensor, slots: torch.Tensor,
            weights: Optional[torch.Tensor] = None) -> torch.Tensor:
    """ciera_combine: each token's weighted sum of its rows ([tokens, dim]
    bf16); without ``weights`` the plain sum, which is the gradient of
    gathering tokens into expert order."""
    _matrix(rows, "rows", _BF16)
    if slots.dim() != 2:
        raise ValueError("slots must be [tokens, topk]")
    _array(slots, "slots", torch.int32, slots.shape)
    if weights is not None:
        _array(weights, "weights", _F32, slots.shape)
    device = _same_device(rows, slots, weights)
    tokens, topk = slots.shape
    n_rows, dim = rows.shape
    y = torch.empty((tokens, dim), dtype=_BF16, device=device)
    _call("ciera_combine", device, _ptr(rows), _stride(rows), n_rows, _ptr(slots),
          _ptr(weights), tokens, topk, dim, _ptr(y), _current(device))
    return y


@_on_stream
def combine_backward(dy: torch.Tensor, rows: torch.Tensor, slots: torch.Tensor,
                     weights: torch.Tensor, offsets: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """ciera_combine_backward: (drows, dweights)."""
    _matrix(rows, "rows", _BF16)
    n_rows, dim = rows.shape
    if slots.dim() != 2:
        raise ValueError("slots must be [tokens, topk]")
    tokens, topk = slots.shape
    _matrix(dy, "dy", _BF16, (tokens, dim))
    _array(slots, "slots", torch.int32, (tokens, topk))
    _array(weights, "weights", _F32, (tokens, topk))
    _offsets(offsets)
    device = _same_device(rows, dy, slots, weights, offsets)
    drows = torch.empty((n_rows, dim), dtype=_BF16, device=device)
    dweights = torch.empty((tokens, topk), dtype=_F32, device=device)
    _call("ciera_combine_backward", device, _ptr(dy), _stride(dy), _ptr(rows), _stride(rows),
          n_rows, _ptr(slots), _ptr(weights), _ptr(offsets), offsets.numel() - 1, tokens, topk,
          dim, _ptr(drows), _ptr(dweights), _current(device))
    return drows, dweights


# ---- products grouped by expert -------------------------------------------

def _offsets(t: torch.Tensor, experts: Optional[int] = None) -> torch.Tensor:
    n = t.numel() if experts is None else experts + 1
    if t.numel() < 1:
        raise ValueError("offsets must hold experts + 1 values")
    return _array(t, "offsets", torch.int32, (n,))


def _rows_of(x: torch.Tensor, tokens: Optional[torch.Tensor]) -> int:
    if tokens is None:
        return x.shape[0]
    if tokens.dim() != 1:
        raise ValueError("tokens must have one dimension")
    _array(tokens, "tokens", torch.int32, tokens.shape)
    return tokens.numel()


def _gather(x, tokens, x_scale, device):
    rows, dim = tokens.numel(), x.shape[1]
    y = torch.empty((rows, dim), dtype=x.dtype, device=device)
    scale = None if x_scale is None else torch.empty(rows, dtype=_F32, device=device)
    _call("ciera_gather_rows", device, _ptr(x), _stride(x), x.shape[0],
          E4M3 if x.dtype == _E4M3 else BF16, _ptr(x_scale), _ptr(tokens), rows, dim, _ptr(y),
          _ptr(scale), _current(device))
    return y, scale


@_on_stream
def gather_rows(x: torch.Tensor, tokens: torch.Tensor, x_scale: Optional[torch.Tensor] = None):
    """ciera_gather_rows: x[tokens] in expert order (bf16, or e4m3 with
    ``x_scale``: then (rows, scales)), zeros where tokens is -1.  A training
    step that needs the rows twice (``mm_gated``, then ``mm_dw``) gathers them
    once."""
    e4m3 = x_scale is not None
    _matrix(x, "x", _E4M3 if e4m3 else _BF16)
    _rows_of(x, tokens)
    if e4m3:
        _array(x_scale, "x_scale", _F32, (x.shape[0],))
    y, scale = _gather(x, tokens, x_scale, _same_device(x, tokens, x_scale))
    return (y, scale) if e4m3 else y


def _forward(x, w, offsets, tokens, x_scale, w_scale, gated, keep):
    e4m3 = isinstance(x, torch.Tensor) and x.dtype == _E4M3
    dtype = _E4M3 if e4m3 else _BF16
    _matrix(x, "x", dtype)
    _stack(w, "w", dtype)
    experts, features, k = w.shape
    if x.shape[1] != k:
        raise ValueError(f"x has {x.shape[1]} columns, w {k}")
    if gated and features % 2:
        raise ValueError("a gated product needs an even number of features (gate, then up)")
    if e4m3 != (x_scale is not None) or e4m3 != (w_scale is not None):
        raise ValueError("x_scale and w_scale go with e4m3 operands")
    if e4m3:
        _array(x_scale, "x_scale", _F32, (x.shape[0],))
        _array(w_scale, "w_scale", _F32, (experts, features))
    _offsets(offsets, experts)
    rows = _rows_of(x, tokens)
    n = features // 2 if gated else features
    device = _same_device(x, w, offsets, tokens, x_scale, w_scale)
    s = _current(device)
    if tokens is not None and rows > _GATHER_ROWS * experts:
        x, x_scale = _gather(x, tokens, x_scale, device)
        tokens = None
    y = torch.empty((rows, n), dtype=_BF16, device=device)
    pre = torch.empty((rows, features), dtype=_BF16, device=device) if keep else None
    _call("ciera_expert_mm", device, _ptr(x), _stride(x), x.shape[0], _ptr(tokens), _ptr(w),
          _stride(w), w.stride(0) if experts > 1 else features * k, _ptr(x_scale),
          _ptr(w_scale), _ptr(offsets), rows, experts, n, k, E4M3 if e4m3 else BF16,
          GATED if gated else 0, _ptr(y), _ptr(pre), _ptr(workspace(device, s)), s)
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
    _matrix(dy, "dy", _BF16)
    _stack(w, "w", _BF16)
    experts, n, k = w.shape
    rows = dy.shape[0]
    if dy.shape[1] != n:
        raise ValueError(f"dy has {dy.shape[1]} columns, w {n} features")
    _offsets(offsets, experts)
    if gated is not None:
        _array(gated, "gated", _BF16, (rows, 2 * k))
    device = _same_device(dy, w, offsets, gated)
    s = _current(device)
    dx = torch.empty((rows, k if gated is None else 2 * k), dtype=_BF16, device=device)
    _call("ciera_expert_mm_dx", device, _ptr(dy), _stride(dy), _ptr(w), _stride(w),
          w.stride(0) if experts > 1 else n * k, _ptr(offsets), rows, experts, n, k,
          _ptr(gated), _ptr(dx), _ptr(workspace(device, s)), s)
    return dx


@_on_stream
def mm_dw(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor,
          tokens: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
          accumulate: bool = False) -> torch.Tensor:
    """ciera_expert_mm_dw: gradient of the weights, [experts, n, k], into
    ``out`` (bf16 or float32, for instance a view of a gradient bucket; bf16
    if not given), added to what it holds with ``accumulate``."""
    _matrix(dy, "dy", _BF16)
    _matrix(x, "x", _BF16)
    rows, n = dy.shape
    if _rows_of(x, tokens) != rows:
        raise ValueError(f"dy has {rows} rows, x {_rows_of(x, tokens)}")
    _offsets(offsets)
    experts, k = offsets.numel() - 1, x.shape[1]
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = torch.empty((experts, n, k), dtype=_BF16, device=dy.device)
    elif not isinstance(out, torch.Tensor) or out.dtype not in (_BF16, _F32):
        raise ValueError("out must be bfloat16 or float32")
    _stack(out, "out", out.dtype)
    if tuple(out.shape) != (experts, n, k):
        raise ValueError(f"out must be {[experts, n, k]}, got {list(out.shape)}")
    if experts > 1 and n and k and out.stride(0) < (n - 1) * _stride(out) + k:
        raise ValueError("out's experts overlap")
    device = _same_device(dy, x, offsets, tokens, out)
    s = _current(device)
    if tokens is not None:
        x, _ = _gather(x, tokens, None, device)
    _call("ciera_expert_mm_dw", device, _ptr(dy), _stride(dy), _ptr(x), _stride(x),
          _ptr(offsets), rows, experts, n, k, _ptr(out), _stride(out), out.stride(0) if experts > 1 else n * k, F32 if out.dtype == _F32 else BF16,
          ACCUMULATE if accumulate else 0, _ptr(workspace(device, s)), s)
    return out
