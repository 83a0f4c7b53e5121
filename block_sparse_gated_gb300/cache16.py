"""Rotary positions and the 16-bit paged K/V cache: torch-facing wrappers over
the C ABI (argument marshalling only).

The calls around a prefill over pages: ``cache16_write`` rotates queries and keys
by their positions and puts keys and values into the page pools that ``prefill``
reads through a block table, ``decode16`` attends to them with the tokens that
follow, and ``rotary`` rotates without a cache.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Sequence

import torch

from . import _native
from .api import _DTYPES, _nbytes, _on_device
from .cache4 import _BAD_TABLE, _I32, _call, _empty, _int32_vector, _strides

MAX_AXES = 4
_F32 = torch.float32


class KVCache16(NamedTuple):
    """Page pools of a 16-bit cache: views into memory that the caller owns.

    ``layout`` "phtd" (the default, and the faster one for single tokens: a head's
    tokens lie together): bf16 or fp16 [pages, Hkv, page_size, d]; "pthd": [pages,
    page_size, Hkv, d].  ``prefill`` takes the same pools:
    ``prefill(q, cache.k, cache.v, block_table=..., kv_layout=cache.layout)``."""
    k: torch.Tensor
    v: torch.Tensor
    layout: str = "phtd"


class Rope(NamedTuple):
    """A rotation: ``inv_freq`` float32 [pairs] on the device (a multiple of 8, at
    most half the head dimension; elements behind the last pair pass).  Pair j of
    a row is turned by position * inv_freq[j], with the position on axis
    ``axes[j]`` (None: one axis; at most 4, such as time, height and width).
    Pairs are elements j and j + pairs, or with ``interleaved`` 2j and 2j + 1."""
    inv_freq: torch.Tensor
    axes: Optional[Sequence[int]] = None
    interleaved: bool = False


def cache16_empty(num_pages: int, num_heads_kv: int, page_size: int, head_dim: int, *,
                  layout: str = "phtd", dtype=torch.bfloat16, device="cuda") -> KVCache16:
    """Pools of zeros for ``num_pages`` pages of ``page_size`` tokens (a multiple
    of 16; for a prefill over them, of 128) of ``num_heads_kv`` heads."""
    if layout not in ("phtd", "pthd"):
        raise ValueError(layout)
    if head_dim not in (64, 128) or page_size <= 0 or page_size % 16:
        raise ValueError("head_dim must be 64 or 128 and page_size a positive multiple of 16")
    if dtype not in _DTYPES:
        raise TypeError("expected bfloat16 or float16")
    inner = (num_heads_kv, page_size) if layout == "phtd" else (page_size, num_heads_kv)
    return KVCache16(*[torch.zeros(num_pages, *inner, head_dim, dtype=dtype, device=device)
                       for _ in range(2)], layout)


def _cache_fields(cache: KVCache16, block_table: torch.Tensor, device, batch: int):
    """The packed bsfa_cache16 of a call on ``device`` with ``batch`` sequences,
    its heads, head dimension and element type, and the tokens that a row of the
    block table can hold."""
    k, v, layout = cache
    shape = k.shape
    if len(shape) != 4:
        raise ValueError("page pools are 4-D")
    n, x, y, d = shape
    if layout == "phtd":
        heads, page, h, t = x, y, 1, 2
    elif layout == "pthd":
        heads, page, h, t = y, x, 2, 1
    else:
        raise ValueError(layout)
    index = device.index
    if device.type != "cuda" or not k.get_device() == v.get_device() == \
            block_table.get_device() == index:
        _on_device(device, k=k, v=v, block_table=block_table)
    a, b = k.stride(), v.stride()
    code = _DTYPES.get(k.dtype)
    if code is None or v.dtype is not k.dtype:
        raise TypeError("page pools are bfloat16 or float16, both of one type")
    if v.shape != shape or a[3] != 1 or b[3] != 1:
        raise ValueError("K and V pools must have one shape, with the head dimension contiguous")
    if block_table.dtype is not _I32 or block_table.dim() != 2:
        raise ValueError(_BAD_TABLE)
    rows, width = block_table.shape
    pitch, unit = block_table.stride()
    if unit != 1 and width > 1:
        raise ValueError(_BAD_TABLE)
    if rows < batch:
        raise ValueError("block_table has fewer rows than sequences")
    return _native.CACHE16.pack(
        k.data_ptr(), v.data_ptr(), a[0], a[h], a[t], b[0], b[h], b[t], n, page, heads, d,
        block_table.data_ptr(), pitch if rows > 1 else width, width, code), heads, d, code, \
        width * page


def _positions_fields(positions, num_axes: int, varlen: bool, batch: int, n: int, device):
    """Address and {axis, batch} strides of a call's positions."""
    want = (n,) if varlen else (batch, n)
    shape = tuple(positions.shape)
    if shape == want and num_axes == 1:
        strides = (0, *positions.stride())
    elif shape[1:] == want and num_axes <= shape[0] <= MAX_AXES:
        strides = positions.stride()
    else:
        raise ValueError(f"positions must be an int32 [axes, {', '.join(map(str, want))}] tensor")
    if positions.dtype is not _I32 or (strides[-1] != 1 and n > 1):
        raise ValueError("positions must be int32 with the positions of a sequence contiguous")
    if positions.get_device() != device.index:
        _on_device(device, positions=positions)
    return positions.data_ptr(), strides[0], 0 if varlen else strides[1]


def _rope_fields(rope: Rope, positions, inverse: bool, varlen: bool, batch: int, n: int, device):
    """The packed bsfa_rope of a call on n rows of each of ``batch`` sequences, or
    on n packed rows."""
    f, axes, interleaved = rope
    if f.dtype is not _F32 or f.dim() != 1 or not f.is_contiguous():
        raise ValueError("inv_freq must be a contiguous float32 [pairs] tensor")
    pairs = f.numel()
    if not 0 < pairs <= 64:
        raise ValueError("inv_freq must have 1 to 64 pairs")
    if f.get_device() != device.index:
        _on_device(device, inv_freq=f)
    if axes is None:
        code, num_axes = b"", 1
    else:
        if len(axes) != pairs or min(axes) < 0 or max(axes) >= MAX_AXES:
            raise ValueError(f"axes must name one of at most {MAX_AXES} axes for each pair")
        code, num_axes = bytes(axes), max(axes) + 1
    at = (0, 0, 0) if positions is None else \
        _positions_fields(positions, num_axes, varlen, batch, n, device)
    return _native.ROPE.pack(f.data_ptr(), *at, pairs, 1 if interleaved else 0,
                             1 if inverse else 0, num_axes, code)


_NONE = (0, 0, 0)


def _like(t, given, layout, varlen: bool, device):
    """Strides of a tensor that must have the shape and type of ``given``, whose
    shape, strides, type and strides {batch, head, token} these are."""
    shape, strides, dtype, s = given
    if t.dtype is not dtype:
        raise TypeError("all rows must share one element type")
    if t.shape != shape:
        raise ValueError("tensors of one kind must have one shape")
    if t.get_device() != device.index:
        _on_device(device, rows=t)
    a = t.stride()
    return s if a == strides else _strides(t, shape, a, layout, varlen)[0]


def _rows_fields(q, k, v, q_out, k_out, layout, cu_seqlens, start, device):
    """The packed bsfa_rows16 of a call (q, v and k_out may be None, and k where
    q is not), its number of sequences, rows (of each sequence or packed), KV
    heads, head dimension and element type, and whether the rows are packed."""
    varlen = cu_seqlens is not None
    if layout is None:
        layout = "htd" if varlen else "bhld"
    one = k if k is not None else q
    shape, dtype, index = one.shape, one.dtype, device.index
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError("expected a bfloat16 or float16 tensor")
    if device.type != "cuda" or one.get_device() != index:
        _on_device(device, rows=one)
    a = one.stride()
    s, h, n = _strides(one, shape, a, layout, varlen)
    d = shape[-1]
    given = (shape, a, dtype, s)
    qp = kp = vp = qo = ko = hq = hkv = 0
    qs = ks = vs = qos = kos = _NONE
    if k is not None:
        kp, ks, hkv = k.data_ptr(), s, h
        if v is not None:
            vp, vs = v.data_ptr(), _like(v, given, layout, varlen, device)
        if k_out is not None:
            ko, kos = k_out.data_ptr(), _like(k_out, given, layout, varlen, device)
        if q is not None:
            size = q.shape
            if q.dtype is not dtype:
                raise TypeError("all rows must share one element type")
            if q.get_device() != index:
                _on_device(device, rows=q)
            a = q.stride()
            s, h, m = _strides(q, size, a, layout, varlen)
            if m != n or size[-1] != d or len(size) != len(shape) or \
                    len(size) == 4 and size[0] != shape[0]:
                raise ValueError("Q, K and V shapes disagree")
            given = (size, a, dtype, s)
    if q is not None:
        qp, qs, hq = q.data_ptr(), s, h
        qo, qos = q_out.data_ptr(), _like(q_out, given, layout, varlen, device)
    cu = first = 0
    if varlen:
        if cu_seqlens.dtype is not _I32 or cu_seqlens.dim() != 1 or \
                not cu_seqlens.is_contiguous() or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must be a contiguous int32 [batch + 1] tensor")
        if cu_seqlens.get_device() != index:
            _on_device(device, cu_seqlens=cu_seqlens)
        batch, cu = cu_seqlens.numel() - 1, cu_seqlens.data_ptr()
    else:
        batch = 1 if len(shape) == 3 else shape[0]
    if start is not None:
        first = _int32_vector(start, batch, "start")
        if start.get_device() != index:
            _on_device(device, start=start)
    return _native.ROWS16.pack(qp, kp, vp, qo, ko, *qs, *ks, *vs, *qos, *kos, batch, hq, hkv, n, d,
                               cu, first, code), batch, n, hkv, d, code, varlen


def rotary(rope: Rope, q, k=None, *, positions=None, start=None, cu_seqlens=None, layout=None,
           inverse=False, out=None, stream=None):
    """Queries and keys rotated by their positions; returns (q', k'), k' None
    without k.  Batched: q [B, Hq, L, d] and k [B, Hkv, L, d] (layout "bhld") or
    [B, L, H, d] ("blhd"), or [H, L, d] for one sequence; varlen (cu_seqlens int32
    on the device): [H, T, d] ("htd") or [T, H, d] ("thd"), rows outside every
    sequence are left as they are.

    Row i of sequence b has the position start[b] + i on every axis (``start``
    int32 [B] on the device, None: 0), or what ``positions`` says: int32 [axes, B,
    L] batched, [axes, T] varlen, without the first dimension where there is one
    axis.  Angles are exact at any position; products are formed in fp32 and
    rounded once.

    ``inverse`` turns back.  It is also the gradient: of the rotated rows' it
    makes the rows'.  ``out``, a pair of tensors, may be (q, k) themselves; other
    tensors must not overlap them."""
    dev = q.device
    varlen = cu_seqlens is not None
    if out is None:
        q_out = torch.empty_like(q) if stream is None else _empty(stream, dev, q.shape, q.dtype)
        k_out = None if k is None else torch.empty_like(k) if stream is None else \
            _empty(stream, dev, k.shape, k.dtype)
    else:
        q_out, k_out = out
        if (k_out is None) != (k is None):
            raise ValueError("out must be a pair, with None where there is no k")
    r, batch, n, *_ = _rows_fields(q, k, None, q_out, k_out, layout, cu_seqlens, start, dev)
    f = _rope_fields(rope, positions, inverse, varlen, batch, n, dev)
    _call(_native.lib().bsfa_rotary, dev, stream, f, r)
    return q_out, k_out


def cache16_write(cache: KVCache16, k, v, block_table, *, rope: Optional[Rope] = None, q=None,
                  positions=None, start=None, cu_seqlens=None, layout=None, q_out=None,
                  stream=None):
    """Keys and values into the cache, the keys rotated on the way where there is
    a ``rope``, and with ``q`` the queries of the same tokens rotated beside them
    (returned: ``q_out``, else a new tensor; None without q).  Layouts, ``start``
    and ``positions`` as for ``rotary``.  Row i of sequence b becomes cache
    position start[b] + i, whatever its rotary positions are: token pos %
    page_size of page block_table[b, pos // page_size].  A position beyond the
    table, or an entry outside the pool, is dropped.  The positions of one call
    must differ."""
    dev = k.device
    if q is None:
        if q_out is not None:
            raise ValueError("q_out without q")
    elif rope is None:
        raise ValueError("q is only rotated: it needs a rope")
    elif q_out is None:
        q_out = torch.empty_like(q) if stream is None else _empty(stream, dev, q.shape, q.dtype)
    if rope is None and positions is not None:
        raise ValueError("positions without a rope")
    r, batch, n, heads, d, code, varlen = _rows_fields(q, k, v, q_out, None, layout, cu_seqlens,
                                                       start, dev)
    c, *have, _ = _cache_fields(cache, block_table, dev, batch)
    if have != [heads, d, code]:
        raise ValueError("K and V must have the cache's heads, head dimension and type")
    f = None if rope is None else _rope_fields(rope, positions, False, varlen, batch, n, dev)
    _call(_native.lib().bsfa_cache16_write, dev, stream, c, f, r)
    return q_out


def _decode_fields(q, cache, block_table, seqlens, out, device, *, layout, max_seqlen,
                   softmax_scale, causal, lse=0):
    """The packed bsfa_cache16 of a decode call, and the fields of its
    bsfa_decode4_params up to the workspace's address and size, and behind them."""
    if layout is None:
        layout = "bhld"
    shape = q.shape
    code = _DTYPES.get(q.dtype)
    if code is None:
        raise TypeError("expected a bfloat16 or float16 tensor")
    if out.shape != shape or out.dtype is not q.dtype:
        raise ValueError("q and out must have one shape and type")
    a, b = q.stride(), out.stride()
    qs, hq, n = _strides(q, shape, a, layout, False)
    os_ = qs if a == b else _strides(out, shape, b, layout, False)[0]
    batch = 1 if len(shape) == 3 else shape[0]
    c, heads, d, kind, most = _cache_fields(cache, block_table, device, batch)
    if shape[-1] != d or heads == 0 or hq % heads or kind != code:
        raise ValueError("q must have the cache's head dimension and type and a multiple of its "
                         "heads")
    if max_seqlen is None:
        max_seqlen = most
    elif max_seqlen > most:
        raise ValueError("block_table has too few pages per row for max_seqlen")
    return c, (q.data_ptr(), out.data_ptr(), *qs, *os_, batch, hq, n,
               _int32_vector(seqlens, batch, "seqlens"), int(max_seqlen),
               float(softmax_scale) if softmax_scale else 0.0, 1 if causal else 0, lse), code


def decode16(q, cache: KVCache16, block_table, seqlens, *, max_seqlen=None, softmax_scale=None,
             causal=True, layout=None, out=None, return_lse=False, workspace=None, stream=None):
    """Attention of new tokens over the 16-bit cache: q [B, Hq, n, d] (layout
    "bhld") or [B, n, Hq, d] ("blhd"), or [Hq, n, d] for one sequence, n = 1 for a
    decode step, of the cache's type.  The new tokens' own keys and values are in
    the cache already; ``seqlens`` (int32 [B] on the device) counts them.  Query i
    of sequence b attends to positions t <= seqlens[b] - n + i, or with
    ``causal=False`` to every t < seqlens[b].  Returns a dict with "out" and, on
    request, "lse" (float32 [Hq, B * n], natural log).  A query that sees nothing
    gives zeros and -inf.

    ``max_seqlen`` bounds the lengths (default: what the block table can hold;
    longer entries of seqlens are cut to it); the call reads lengths on the device
    only, so a captured graph stays right as they grow within it.  ``workspace``: at
    least ``decode16_workspace_bytes`` of device memory (0 where the lengths' bound
    and the batch are small), not shared by calls that may overlap (default:
    allocated for the call)."""
    dev = q.device
    if dev.type != "cuda" or not seqlens.get_device() == dev.index or \
            out is not None and out.device != dev or \
            workspace is not None and workspace.device != dev:
        _on_device(dev, out=out, seqlens=seqlens, workspace=workspace)
    if out is None:
        out = torch.empty_like(q) if stream is None else _empty(stream, dev, q.shape, q.dtype)
    res = {"out": out}
    lse = 0
    if return_lse:
        *b, h, n, _ = q.shape
        if layout == "blhd" and b:
            h, n = n, h
        res["lse"] = _empty(stream, dev, (h, b[0] * n if b else n), _F32)
        lse = res["lse"].data_ptr()
    c, fields, code = _decode_fields(q, cache, block_table, seqlens, out, dev, layout=layout,
                               max_seqlen=max_seqlen, softmax_scale=softmax_scale, causal=causal,
                               lse=lse)
    at = size = 0
    if workspace is not None:
        if not workspace.is_contiguous():
            raise ValueError("the workspace must be contiguous")
        at, size = workspace.data_ptr(), _nbytes(workspace)
    p = _native.DECODE4.pack(*fields, at, size, code)
    if workspace is None:
        size = _native.lib().bsfa_decode16_workspace_size(c, p)
        if size:
            workspace = _empty(stream, dev, (size,), torch.uint8)
            p = _native.DECODE4.pack(*fields, workspace.data_ptr(), size, code)
    _call(_native.lib().bsfa_decode16, dev, stream, c, p)
    return res


def decode16_workspace_bytes(q, cache: KVCache16, block_table, seqlens, *, max_seqlen=None,
                             layout=None) -> int:
    """Workspace bytes that decode16 needs for this call's shapes."""
    c, fields, code = _decode_fields(q, cache, block_table, seqlens, q, q.device, layout=layout,
                                     max_seqlen=max_seqlen, softmax_scale=None, causal=True)
    return int(_native.lib().bsfa_decode16_workspace_size(
        c, _native.DECODE4.pack(*fields, 0, 0, code)))
