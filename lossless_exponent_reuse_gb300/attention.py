"""The attention half of a layer whose weights the Allgather rebuilds.

Thin binding of the ``ciera_rotary`` ... ``ciera_attend`` entry points of
libciera (include/ciera.h has the formulas), next to ``experts``, whose manner
of checks, streams and scratch memory it shares.

    rotary     rotary_table, rotary, rotary_backward
    pages      page_pool, assign_pages, release_pages
    cache      page_cache, append
    attention  attend

A serving step of a batch: ``assign_pages`` gives the new tokens of each
request their places, ``append`` rotates queries and keys and writes keys and
values there, ``attend`` reads them; the first serves all layers of a step.
Tensors of heads, [tokens, heads, head_dim], and pages may have any strides; a
head's values must be contiguous.  Every call takes ``stream`` as ``experts``'
calls do; ``experts.status`` reads the error word that ``attend`` reports to.
Nothing is registered with autograd: ``rotary_backward`` is the gradient's call.
"""
from __future__ import annotations

import math
import struct
from typing import NamedTuple, Optional, Sequence, Union

import torch

from . import ciera, experts
from .experts import (BF16, E4M3, _BF16, _E4M3, _array, _call, _control, _I32, _index, _on_stream,
                      _placed, _raw_stream)

INTERLEAVED = 1
INVERSE = 2
_I64, _U8 = torch.int64, torch.uint8


class Rotary(NamedTuple):
    """Frequencies of ``pairs`` pairs: int64 2^-64ths of a turn per position,
    modulo 2^64; an amplitude; pairs (2i, 2i + 1), or (i, i + pairs)."""
    turns: torch.Tensor
    amplitude: float = 1.0
    interleaved: bool = False


class Cache(NamedTuple):
    """Pages of keys and values, [pages, page_size, heads, head_dim]: bf16, or
    e4m3 with a power of two per row, uint8 [pages, page_size, heads], biased
    by 127 (255: NaN)."""
    key: torch.Tensor
    value: torch.Tensor
    key_exponent: Optional[torch.Tensor] = None
    value_exponent: Optional[torch.Tensor] = None


class Pool(NamedTuple):
    table: torch.Tensor      # [requests, width] int32 pages, -1: none
    free: torch.Tensor       # [capacity] int32: the stack of free pages
    count: torch.Tensor      # [1] int32: how many of it are free


class Step(NamedTuple):
    offsets: torch.Tensor    # [requests + 1] int32: first new token of each
    context: torch.Tensor    # [requests] int32: keys with the new; 0: no pages were left
    lengths: torch.Tensor    # [requests] int32: the next step's ``cached``
    positions: torch.Tensor  # [tokens] int32
    slots: torch.Tensor      # [tokens] int32, -1: none
    pool: Pool               # with the new count


# ---- arguments -----------------------------------------------------------

_cache_words = struct.Struct("4Q17q").pack


def _heads(t, name: str, index: int, tokens: Optional[int] = None, dim: Optional[int] = None):
    """Shape and the strides of tokens and heads."""
    if isinstance(t, torch.Tensor) and t.dtype is _BF16 and t.get_device() == index:
        shape = t.shape
        if (len(shape) == 3 and (tokens is None or shape[0] == tokens)
                and (dim is None or shape[2] == dim)):
            token, head, unit = t.stride()
            if unit == 1 or shape[2] <= 1:
                return shape, token, head
    _placed(t, name, _BF16, index)
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim], got {list(t.shape)}")
    if (tokens is not None and t.shape[0] != tokens) or (dim is not None and t.shape[2] != dim):
        raise ValueError(f"{name} must be {['any' if tokens is None else tokens, 'any', dim]}, "
                         f"got {list(t.shape)}")
    raise ValueError(f"{name}'s heads must be contiguous")


def _rotary(r, index: int, dim: int):
    if not isinstance(r, Rotary):
        raise ValueError("rotary must be a Rotary (rotary_table)")
    turns = r.turns
    if not isinstance(turns, torch.Tensor) or turns.dim() != 1:
        raise ValueError("rotary.turns must have one dimension")
    pairs = turns.shape[0]
    if 2 * pairs > dim:
        raise ValueError(f"{pairs} pairs do not fit heads of {dim}")
    return _array(turns, "rotary.turns", _I64, index, pairs), pairs


def _side(t, exponent, name: str, dtype, index: int, shape):
    if t.dtype is not dtype or t.get_device() != index or t.shape != shape:
        _placed(t, f"cache.{name}", dtype, index)
        raise ValueError(f"cache.{name} must be {list(shape)}, got {list(t.shape)}")
    stride = t.stride()
    if stride[3] != 1 and shape[3] > 1:
        raise ValueError(f"cache.{name}'s rows must be contiguous")
    if exponent is None:
        return t.data_ptr(), 0, stride[:3], (0, 0, 0)
    _placed(exponent, f"cache.{name}_exponent", _U8, index)
    if exponent.shape != shape[:3]:
        raise ValueError(f"cache.{name}_exponent must be {list(shape[:3])}, "
                         f"got {list(exponent.shape)}")
    return t.data_ptr(), exponent.data_ptr(), stride[:3], exponent.stride()


def _cache(c, index: int):
    """The cache's shape, and its ciera_cache as bytes."""
    if not isinstance(c, Cache):
        raise ValueError("cache must be a Cache (page_cache)")
    key = c.key
    if not isinstance(key, torch.Tensor) or not isinstance(c.value, torch.Tensor) or key.dim() != 4:
        raise ValueError("cache.key and cache.value must be [pages, page_size, heads, head_dim]")
    dtype, shape = key.dtype, key.shape
    e4m3 = dtype is _E4M3
    if not e4m3 and dtype is not _BF16:
        raise ValueError(f"cache.key must be bfloat16 or float8_e4m3fn, got {dtype}")
    if e4m3 != (c.key_exponent is not None) or e4m3 != (c.value_exponent is not None):
        raise ValueError("exponents go with an e4m3 cache")
    if shape[1] < 1 or shape[0] * shape[1] > 2147483647:
        raise ValueError(f"a cache of {shape[0]} pages of {shape[1]} tokens is not taken")
    k, ke, ks, kes = _side(key, c.key_exponent, "key", dtype, index, shape)
    v, ve, vs, ves = _side(c.value, c.value_exponent, "value", dtype, index, shape)
    return shape, _cache_words(k, v, ke, ve, *ks, *vs, *kes, *ves, *shape, E4M3 if e4m3 else BF16)


def _table(t, name: str, index: int):
    """Pointer, row stride and shape of a block table."""
    stride = experts._matrix(t, name, _I32, index)
    return t.data_ptr(), stride, t.shape


# ---- rotary positions ------------------------------------------------------

def rotary_table(dim: int, base: float = 10000.0, interleaved: bool = False,
                 scaling: Optional[str] = None, factor: float = 1.0, original: int = 0,
                 bounds: Sequence[float] = (1.0, 32.0), amplitude: Optional[float] = None,
                 frequencies: Optional[Sequence[float]] = None,
                 device: Union[str, torch.device] = "cuda") -> Rotary:
    """The frequencies of the first ``dim`` values of a head: base^(-2i / dim)
    radians per position, i < dim / 2, or ``frequencies`` as given; for contexts
    ``factor`` times as long as the ``original`` one

      "linear"  all divided by factor
      "base"    the base raised, by factor^(dim / (dim - 2)): the slowest divided
                by factor, the fastest as it was
      "parts"   those that make fewer than bounds[0] turns in the original
                context divided by factor, those of bounds[1] and more as they
                were, and between the two linearly in the turns (a model that was
                tuned with a ramp in the pairs' index, between two rounded ends, wants
                its ``frequencies`` given).

    ``amplitude``: of the rotated values; 1, and for "parts" 1 + 0.1 ln factor,
    unless given.  Laid out once for many calls."""
    dim = int(dim)
    if dim < 0 or dim % 2:
        raise ValueError(f"dim must be even, got {dim}")
    if not (factor >= 1 and math.isfinite(factor)):
        raise ValueError(f"factor must be 1 or more, got {factor}")
    if scaling not in (None, "linear", "base", "parts"):
        raise ValueError(f"scaling must be None, 'linear', 'base' or 'parts', got {scaling!r}")
    if frequencies is None:
        if not (base > 0 and math.isfinite(base)):
            raise ValueError(f"base must be positive, got {base}")
        if scaling == "base" and dim > 2:
            base = base * factor ** (dim / (dim - 2))
        f = [base ** (-2 * i / dim) for i in range(dim // 2)]
    else:
        f = [float(w) for w in frequencies]
        if len(f) != dim // 2 or not all(math.isfinite(w) for w in f):
            raise ValueError(f"frequencies must be {dim // 2} finite numbers")
        if scaling == "base":
            raise ValueError("'base' makes frequencies of its own")
    if scaling == "linear":
        f = [w / factor for w in f]
    if scaling == "parts":
        low, high = bounds
        if original < 1 or not low < high:
            raise ValueError("'parts' needs the original context and bounds that rise")
        keep = [min(1.0, max(0.0, (original * abs(w) / (2 * math.pi) - low) / (high - low)))
                for w in f]
        f = [w * (k + (1 - k) / factor) for w, k in zip(f, keep)]
    if amplitude is None:
        amplitude = 1 + 0.1 * math.log(factor) if scaling == "parts" else 1.0
    whole = [round(w / (2 * math.pi) * 2.0 ** 64) % (1 << 64) for w in f]
    turns = torch.tensor([v - (1 << 64) if v >> 63 else v for v in whole], dtype=_I64)
    return Rotary(turns.to(device), float(amplitude), bool(interleaved))


def _rotate(x, positions, rotary, out, flags):
    index = _index(x, "x")
    shape, x_token, x_head = _heads(x, "x", index)
    tokens, heads, dim = shape
    turns, pairs = _rotary(rotary, index, dim)
    at = _array(positions, "positions", _I32, index, tokens)
    if out is None:
        out = torch.empty(shape, dtype=_BF16, device=x.device)
        y_token, y_head = heads * dim, dim
    else:
        got, y_token, y_head = _heads(out, "out", index, tokens, dim)
        if got != shape:
            raise ValueError(f"out must be {list(shape)}, got {list(got)}")
    if rotary.interleaved:
        flags |= INTERLEAVED
    _call("ciera_rotary", index, x.data_ptr(), x_token, x_head, at, turns, pairs, rotary.amplitude,
          tokens, heads, dim, out.data_ptr(), y_token, y_head, flags, _raw_stream(index))
    return out


@_on_stream
def rotary(x: torch.Tensor, positions: torch.Tensor, rotary: Rotary,
           out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """ciera_rotary: x [tokens, heads, head_dim] bf16 turned to its positions
    (int32 per token); ``out`` may be x itself."""
    return _rotate(x, positions, rotary, out, 0)


@_on_stream
def rotary_backward(dy: torch.Tensor, positions: torch.Tensor, rotary: Rotary,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """ciera_rotary with CIERA_INVERSE: the gradient of ``rotary``'s x."""
    return _rotate(dy, positions, rotary, out, INVERSE)


# ---- pages -----------------------------------------------------------------

def page_pool(pages: int, requests: int, width: int,
              device: Union[str, torch.device] = "cuda") -> Pool:
    """A pool whose ``pages`` pages are all free, for ``requests`` requests of
    at most ``width`` pages each."""
    return Pool(torch.full((requests, width), -1, dtype=_I32, device=device),
                torch.arange(pages - 1, -1, -1, dtype=_I32, device=device),
                torch.tensor([pages], dtype=_I32, device=device))


def _pool(pool, index: int):
    table, stride, shape = _table(pool.table, "pool.table", index)
    free = pool.free
    if not isinstance(free, torch.Tensor) or free.dim() != 1:
        raise ValueError("pool.free must have one dimension")
    return (table, stride, shape, _array(free, "pool.free", _I32, index, free.shape[0]),
            free.shape[0], _array(pool.count, "pool.count", _I32, index, 1))


@_on_stream
def assign_pages(pool: Pool, cached: torch.Tensor, new: torch.Tensor, tokens: int, page_size: int,
                 count: Optional[torch.Tensor] = None) -> Step:
    """ciera_assign_pages: places for ``new`` tokens (int32 per request) behind
    the ``cached`` ones, ``tokens`` or fewer in all; new pages are written to
    the pool's table in place.  ``count`` receives the number of pages left:
    pool.count itself for a pool that goes on from step to step without being
    handed on (a captured step), a new tensor if not given."""
    index = _index(pool.table, "pool.table")
    table, stride, (requests, width), free, capacity, old = _pool(pool, index)
    c = _array(cached, "cached", _I32, index, requests)
    n = _array(new, "new", _I32, index, requests)
    tokens = int(tokens)
    if tokens < 0 or page_size < 1:
        raise ValueError(f"{tokens} tokens in pages of {page_size} are not taken")
    out = torch.empty(3 * requests + 2 * tokens + 2, dtype=_I32, device=pool.table.device)
    offsets, context, lengths, positions, slots, left = out.split(
        [requests + 1, requests, requests, tokens, tokens, 1])
    if count is None:
        count = left
    left_at = _array(count, "count", _I32, index, 1)
    at = out.data_ptr()
    r, t = 4 * requests, 4 * tokens
    _call("ciera_assign_pages", index, c, n, requests, tokens, int(page_size), table, stride, width,
          free, capacity, old, left_at, at, at + r + 4, at + 2 * r + 4, at + 3 * r + 4,
          at + 3 * r + t + 4, _raw_stream(index))
    return Step(offsets, context, lengths, positions, slots, Pool(pool.table, pool.free, count))


@_on_stream
def release_pages(pool: Pool, lengths: torch.Tensor, done: torch.Tensor, page_size: int,
                  count: Optional[torch.Tensor] = None) -> Pool:
    """ciera_release_pages: the pages of requests whose ``done`` (bool or uint8)
    is set go back to the pool; table, stack and ``lengths`` change in place,
    ``count`` as in ``assign_pages``."""
    index = _index(pool.table, "pool.table")
    table, stride, (requests, width), free, capacity, old = _pool(pool, index)
    n = _array(lengths, "lengths", _I32, index, requests)
    if not isinstance(done, torch.Tensor) or done.dtype not in (torch.bool, _U8):
        raise ValueError("done must be bool or uint8")
    gone = _array(done, "done", done.dtype, index, requests)
    if page_size < 1:
        raise ValueError(f"page_size must be positive, got {page_size}")
    if count is None:
        count = torch.empty(1, dtype=_I32, device=pool.table.device)
    _call("ciera_release_pages", index, gone, n, requests, int(page_size), table, stride, width,
          free, capacity, old, _array(count, "count", _I32, index, 1), _raw_stream(index))
    return Pool(pool.table, pool.free, count)


# ---- cache -----------------------------------------------------------------

def page_cache(pages: int, page_size: int, heads: int, head_dim: int, e4m3: bool = False,
               device: Union[str, torch.device] = "cuda") -> Cache:
    """An empty cache, a head's rows of a page side by side."""
    sides = [torch.zeros((pages, heads, page_size, head_dim), dtype=_BF16, device=device)
             .to(_E4M3 if e4m3 else _BF16).transpose(1, 2) for _ in range(2)]
    if not e4m3:
        return Cache(*sides)
    return Cache(*sides, *(torch.zeros((pages, heads, page_size), dtype=_U8,
                                       device=device).transpose(1, 2) for _ in range(2)))


@_on_stream
def append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
           slots: torch.Tensor, rotary: Rotary, cache: Cache,
           out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """ciera_append: the rotated queries (``out``, which may be q itself); rotated
    keys, and values, go to their slots of the cache."""
    index = _index(q, "q")
    (tokens, heads, dim), q_token, q_head = _heads(q, "q", index)
    shape, words = _cache(cache, index)
    if shape[3] != dim:
        raise ValueError(f"q has heads of {dim}, the cache of {shape[3]}")
    k_shape, k_token, k_head = _heads(k, "k", index, tokens, dim)
    v_shape, v_token, v_head = _heads(v, "v", index, tokens, dim)
    if k_shape[1] != shape[2] or v_shape[1] != shape[2]:
        raise ValueError(f"k and v have {k_shape[1]} and {v_shape[1]} heads, the cache {shape[2]}")
    turns, pairs = _rotary(rotary, index, dim)
    at = _array(positions, "positions", _I32, index, tokens)
    to = _array(slots, "slots", _I32, index, tokens)
    if out is None:
        out = torch.empty((tokens, heads, dim), dtype=_BF16, device=q.device)
        out_token, out_head = heads * dim, dim
    else:
        got, out_token, out_head = _heads(out, "out", index, tokens, dim)
        if got[1] != heads:
            raise ValueError(f"out must be {[tokens, heads, dim]}, got {list(got)}")
    _call("ciera_append", index, q.data_ptr(), q_token, q_head, k.data_ptr(), k_token, k_head,
          v.data_ptr(), v_token, v_head, at, to, turns, pairs, rotary.amplitude, tokens, heads,
          out.data_ptr(), out_token, out_head, words, INTERLEAVED if rotary.interleaved else 0,
          _raw_stream(index))
    return out


# ---- attention -------------------------------------------------------------

_needs = {}           # (device index, q heads, heads, head_dim): bytes


def _need(index: int, *heads: int) -> int:
    with torch.cuda.device(index):
        need = ciera.lib().ciera_attend_workspace_bytes(*heads)
    if need == 0:
        raise ValueError("no attention of {} heads over {} heads of {}".format(*heads))
    if len(_needs) < 4096:
        _needs[(index, *heads)] = need
    return need


@_on_stream
def attend(q: torch.Tensor, cache: Cache, table: torch.Tensor, offsets: torch.Tensor,
           context: torch.Tensor, scale: Optional[float] = None,
           longest: Optional[int] = None) -> torch.Tensor:
    """ciera_attend: each request's new tokens (q [tokens, heads, head_dim] bf16,
    request r's from offsets[r] on) over its pages, of which ``context`` [requests]
    keys are there, the new ones last; each token sees the keys up to its own.
    ``scale``: head_dim^-0.5 if not given.  ``longest``: the most new tokens of a
    request, if the caller knows (1 for a step of single tokens): it chooses the
    faster kernel for the whole call, no result; guessed 1 where tokens are no more than
    requests."""
    index = _index(q, "q")
    (tokens, heads, dim), q_token, q_head = _heads(q, "q", index)
    shape, words = _cache(cache, index)
    if shape[3] != dim:
        raise ValueError(f"q has heads of {dim}, the cache of {shape[3]}")
    table_at, stride, (requests, width) = _table(table, "table", index)
    off = _array(offsets, "offsets", _I32, index, requests + 1)
    keys = _array(context, "context", _I32, index, requests)
    need = _needs.get((index, heads, shape[2], dim)) or _need(index, heads, shape[2], dim)
    if longest is None:
        longest = tokens if tokens > requests else 1
    s = _raw_stream(index)
    ws = experts._scratch_bytes(index, s, need)
    o = torch.empty((tokens, heads, dim), dtype=_BF16, device=q.device)
    _call("ciera_attend", index, q.data_ptr(), q_token, q_head, tokens, heads, words, table_at,
          stride, width, off, keys, requests, int(longest),
          dim ** -0.5 if scale is None else float(scale), o.data_ptr(), ws.data_ptr(), ws.numel(),
          _control(index), s)
    return o
