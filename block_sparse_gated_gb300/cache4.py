"""The 4-bit K/V cache: torch-facing wrappers over the C ABI (argument
marshalling only).

``prefill`` leaves keys and values in 16 bits; ``cache4_write`` quantises them
into the pages of a ``KVCache4``, ``decode4`` attends to it with the tokens
that follow, and ``cache4_read`` gives the 16-bit rows back.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _native
from .api import _DTYPES, _check, _dtype_code, _nbytes, _on_device, _strides_bhtd

GROUP = 16  # elements that share a scale
_U8, _E4M3, _I32 = torch.uint8, torch.float8_e4m3fn, torch.int32
_BAD_TABLE = "block_table must be an int32 [batch, pages_per_sequence] tensor"


class KVCache4(NamedTuple):
    """Page pools of a 4-bit cache: views into memory that the caller owns.

    ``layout`` "phtd" (the default, and the faster one: a head's tokens lie
    together) or "pthd", as for the prefill's page pools.  In "phtd" order the
    codes are uint8 [pages, Hkv, page_size, d / 2] (two e2m1 codes to a byte,
    the even element in the low four bits) and the scales float8_e4m3fn
    [pages, Hkv, page_size, d / 16]; ``k_exp`` and ``v_exp`` are int32 [Hkv]
    or None (0).  Element i of a row stands for
    code[i] * scale[i // 16] * 2 ** exp.  Pages and heads may lie apart (any
    multiple of 16 bytes for the codes, of d / 16 for the scales)."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor
    k_exp: Optional[torch.Tensor] = None
    v_exp: Optional[torch.Tensor] = None
    layout: str = "phtd"


def cache4_empty(num_pages: int, num_heads_kv: int, page_size: int, head_dim: int, *,
                 layout: str = "phtd", k_exp=None, v_exp=None, device="cuda") -> KVCache4:
    """Pools for ``num_pages`` pages of ``page_size`` tokens (a multiple of 16)
    of ``num_heads_kv`` heads; every row stands for zeros."""
    if layout not in ("phtd", "pthd"):
        raise ValueError(layout)
    if head_dim not in (64, 128) or page_size <= 0 or page_size % 16:
        raise ValueError("head_dim must be 64 or 128 and page_size a positive multiple of 16")
    inner = (num_heads_kv, page_size) if layout == "phtd" else (page_size, num_heads_kv)
    codes = [torch.zeros(num_pages, *inner, head_dim // 2, dtype=torch.uint8, device=device)
             for _ in range(2)]
    scales = [torch.zeros(num_pages, *inner, head_dim // GROUP, dtype=torch.float8_e4m3fn,
                          device=device) for _ in range(2)]
    return KVCache4(*codes, *scales, k_exp, v_exp, layout)


def _bad_pool(cache, device):
    """Says what is wrong with a cache that _cache_fields found fault with."""
    _on_device(device, k=cache.k, v=cache.v, k_scale=cache.k_scale, v_scale=cache.v_scale,
               k_exp=cache.k_exp, v_exp=cache.v_exp)
    shape = tuple(cache.k.shape)
    for name, t, dtype, want in (
            ("k", cache.k, torch.uint8, shape), ("v", cache.v, torch.uint8, shape),
            ("k_scale", cache.k_scale, torch.float8_e4m3fn, shape[:3] + (shape[3] // 8,)),
            ("v_scale", cache.v_scale, torch.float8_e4m3fn, shape[:3] + (shape[3] // 8,))):
        if t.dtype != dtype or tuple(t.shape) != want or t.stride(3) != 1:
            raise ValueError(f"{name} must be a {dtype} {list(want)} tensor with rows contiguous")
    heads, _ = _heads_and_dim(cache)
    for name, e in (("k_exp", cache.k_exp), ("v_exp", cache.v_exp)):
        if e is not None and (e.dtype != torch.int32 or tuple(e.shape) != (heads,) or
                              not e.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous int32 [{heads}] tensor")
    raise ValueError("the cache's tensors disagree")


def _cache_fields(cache: KVCache4, block_table: torch.Tensor, device, batch: int):
    """The packed bsfa_cache4 of a call on ``device`` with ``batch`` sequences,
    and the tokens that a row of the block table can hold."""
    k, v, ks, vs, ke, ve, layout = cache
    heads, d = _heads_and_dim(cache)
    index = device.index
    shape = k.shape
    n, x, y, row = shape
    scales = (n, x, y, row // 8)
    a, b, e, f = k.stride(), v.stride(), ks.stride(), vs.stride()
    if not (k.dtype is v.dtype is _U8 and ks.dtype is vs.dtype is _E4M3 and v.shape == shape and
            ks.shape == scales and vs.shape == scales and a[3] == b[3] == e[3] == f[3] == 1 and
            k.get_device() == v.get_device() == ks.get_device() == vs.get_device() == index):
        _bad_pool(cache, device)
    ke_ptr = ve_ptr = 0
    if ke is not None:
        ke_ptr = _exponents(ke, heads, cache, device)
    if ve is not None:
        ve_ptr = _exponents(ve, heads, cache, device)
    if block_table.get_device() != index:
        _on_device(device, block_table=block_table)
    if block_table.dtype is not _I32 or block_table.dim() != 2:
        raise ValueError(_BAD_TABLE)
    rows, width = block_table.shape
    pitch, unit = block_table.stride()
    if unit != 1 and width > 1:
        raise ValueError(_BAD_TABLE)
    if rows < batch:
        raise ValueError("block_table has fewer rows than sequences")
    if layout == "phtd":
        return _native.CACHE4.pack(
            k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), ke_ptr, ve_ptr,
            a[0], a[1], a[2], b[0], b[1], b[2], e[0], e[1], e[2], f[0], f[1], f[2],
            n, y, heads, d, block_table.data_ptr(), pitch if rows > 1 else width,
            width), width * y
    return _native.CACHE4.pack(
        k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), ke_ptr, ve_ptr,
        a[0], a[2], a[1], b[0], b[2], b[1], e[0], e[2], e[1], f[0], f[2], f[1],
        n, x, heads, d, block_table.data_ptr(), pitch if rows > 1 else width, width), width * x


def _exponents(t, heads: int, cache, device):
    if not (t.dtype is _I32 and t.shape == (heads,) and t.is_contiguous() and
            t.get_device() == device.index):
        _bad_pool(cache, device)
    return t.data_ptr()


def _strides(t, shape, s, layout: str, varlen: bool):
    """Element strides {batch, head, token}, heads and tokens of a tensor of
    this shape and stride: _strides_bhtd for the layouts met most, without
    reading the tensor's attributes again."""
    if len(shape) == 4 and s[3] == 1 and not varlen:
        if layout == "bhld":
            return (s[0], s[1], s[2]), shape[1], shape[2]
        if layout == "blhd":
            return (s[0], s[2], s[1]), shape[2], shape[1]
    return _strides_bhtd(t, layout, varlen)


def _int32_vector(t, n: int, what: str):
    if t.dtype is not _I32 or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 [{n}] tensor")
    return t.data_ptr()


def _rows_fields(k, v, layout, cu_seqlens, start, heads: int, d: int, device):
    """The packed bsfa_cache4_rows of a call, and its number of sequences."""
    varlen = cu_seqlens is not None
    if layout is None:
        layout = "htd" if varlen else "bhld"
    shape = k.shape
    if v.shape != shape:
        raise ValueError("K and V shapes disagree")
    code = _DTYPES.get(k.dtype)
    if code is None:
        raise TypeError("expected a bfloat16 or float16 tensor")
    if v.dtype is not k.dtype:
        raise TypeError("K and V must share one element type")
    if device.type != "cuda" or not k.get_device() == v.get_device() == device.index:
        _on_device(device, k=k, v=v)
    a, b = k.stride(), v.stride()
    ks, hk, n = _strides(k, shape, a, layout, varlen)
    vs = ks if a == b else _strides(v, shape, b, layout, varlen)[0]
    if hk != heads or shape[-1] != d:
        raise ValueError("K and V must have the cache's heads and head dimension")
    cu = first = 0
    if varlen:
        if cu_seqlens.dtype is not _I32 or cu_seqlens.dim() != 1 or \
                not cu_seqlens.is_contiguous() or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must be a contiguous int32 [batch + 1] tensor")
        if cu_seqlens.get_device() != device.index:
            _on_device(device, cu_seqlens=cu_seqlens)
        batch, cu = cu_seqlens.numel() - 1, cu_seqlens.data_ptr()
    else:
        batch = 1 if len(shape) == 3 else shape[0]
    if start is not None:
        first = _int32_vector(start, batch, "start")
        if start.get_device() != device.index:
            _on_device(device, start=start)
    return _native.CACHE4_ROWS.pack(k.data_ptr(), v.data_ptr(), *ks, *vs, batch, n, cu, first,
                                    code), batch


def _heads_and_dim(cache: KVCache4):
    """KV heads and head dimension of a cache."""
    shape, layout = cache.k.shape, cache.layout
    if len(shape) != 4:
        raise ValueError("code pools are 4-D")
    if layout == "phtd":
        return shape[1], 2 * shape[3]
    if layout == "pthd":
        return shape[2], 2 * shape[3]
    raise ValueError(layout)


def _call(fn, device, stream, *args):
    """One library call on ``stream`` (default: the device's current one), with
    the tensors' device current."""
    index = device.index
    raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == index:
        status = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            status = fn(*args, raw)
    if status:
        _check(status, fn.__name__)


def _empty(stream, device, shape, dtype):
    """A tensor for a call on ``stream``: memory that this stream may write at
    once, and that is not handed out again while the caller's stream reads it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def cache4_write(cache: KVCache4, k, v, block_table, *, start=None, cu_seqlens=None, layout=None,
                 stream=None) -> None:
    """Quantise 16-bit keys and values into the cache.  Batched: k, v
    [B, Hkv, L, d] (layout "bhld") or [B, L, Hkv, d] ("blhd"), or [Hkv, L, d]
    for one sequence; varlen (cu_seqlens int32 on the device): [Hkv, T, d]
    ("htd") or [T, Hkv, d] ("thd").  Row i of sequence b becomes cache position
    start[b] + i (``start`` int32 [B] on the device, None: 0), which is token
    pos % page_size of page block_table[b, pos // page_size].  A position
    beyond the table, or an entry outside the pool, is dropped.  The positions
    of one call must differ.

    A group of 16 elements shares the scale e4m3(amax / 6), at least 2**-9 and
    at most 448; elements round to the nearest e2m1 value, ties to the even
    code.  A group that holds an infinity or a NaN reads back as NaN."""
    dev = k.device
    r, batch = _rows_fields(k, v, layout, cu_seqlens, start, *_heads_and_dim(cache), dev)
    c, _ = _cache_fields(cache, block_table, dev, batch)
    _call(_native.lib().bsfa_cache4_write, dev, stream, c, r)


def cache4_read(cache: KVCache4, block_table, *, seqlen=None, total=None, start=None,
                cu_seqlens=None, dtype=torch.bfloat16, layout=None, out=None, stream=None):
    """The 16-bit rows (k, v) of cache positions start[b] .. of each sequence.
    Batched: ``seqlen`` rows of each of block_table's sequences, [B, Hkv,
    seqlen, d] ("bhld") or [B, seqlen, Hkv, d] ("blhd"); varlen: ``total``
    packed rows, [Hkv, total, d] ("htd") or [total, Hkv, d] ("thd"), of which
    those outside every sequence are left as they are.  ``out``, a pair of such
    tensors, takes the place of the sizes and the type.  Positions that name no
    cache row read as zeros.  Values are rounded once, to ``dtype``."""
    varlen = cu_seqlens is not None
    heads, d = _heads_and_dim(cache)
    dev = cache.k.device
    if layout is None:
        layout = "htd" if varlen else "bhld"
    if out is None:
        n = total if varlen else seqlen
        if n is None or n < 0:
            raise ValueError("a varlen read needs total, a batched one seqlen")
        if layout == "bhld" and not varlen:
            shape = (block_table.shape[0], heads, n, d)
        elif layout == "blhd" and not varlen:
            shape = (block_table.shape[0], n, heads, d)
        elif layout == "htd" and varlen:
            shape = (heads, n, d)
        elif layout == "thd" and varlen:
            shape = (n, heads, d)
        else:
            raise ValueError(layout)
        if dtype not in _DTYPES:
            raise TypeError("expected bfloat16 or float16")
        k = _empty(stream, dev, shape, dtype)
        v = _empty(stream, dev, shape, dtype)
    else:
        k, v = out
    r, batch = _rows_fields(k, v, layout, cu_seqlens, start, heads, d, dev)
    c, _ = _cache_fields(cache, block_table, dev, batch)
    _call(_native.lib().bsfa_cache4_read, dev, stream, c, r)
    return k, v


def _decode_fields(q, cache, block_table, seqlens, out, device, *, layout, max_seqlen,
                   softmax_scale, causal, lse=0):
    """The packed bsfa_cache4 of a decode call, and a function of a workspace's
    address and size that gives its packed bsfa_decode4_params."""
    if layout is None:
        layout = "bhld"
    shape = q.shape
    if out.shape != shape or q.dtype is not out.dtype:
        raise ValueError("q and out must have one shape and type")
    code = _dtype_code(q)
    a, b = q.stride(), out.stride()
    qs, hq, n = _strides(q, shape, a, layout, False)
    os_ = qs if a == b else _strides(out, shape, b, layout, False)[0]
    heads, d = _heads_and_dim(cache)
    if shape[-1] != d or heads == 0 or hq % heads:
        raise ValueError("q must have the cache's head dimension and a multiple of its heads")
    batch = 1 if len(shape) == 3 else shape[0]
    c, most = _cache_fields(cache, block_table, device, batch)
    if max_seqlen is None:
        max_seqlen = most
    elif max_seqlen > most:
        raise ValueError("block_table has too few pages per row for max_seqlen")
    fixed = (q.data_ptr(), out.data_ptr(), *qs, *os_, batch, hq, n,
             _int32_vector(seqlens, batch, "seqlens"), int(max_seqlen),
             float(softmax_scale) if softmax_scale else 0.0, 1 if causal else 0, lse)
    return c, lambda ws, size: _native.DECODE4.pack(*fixed, ws, size, code)


def decode4(q, cache: KVCache4, block_table, seqlens, *, max_seqlen=None, softmax_scale=None,
            causal=True, layout=None, out=None, return_lse=False, workspace=None, stream=None):
    """Attention of new tokens over the 4-bit cache: q [B, Hq, n, d] (layout
    "bhld") or [B, n, Hq, d] ("blhd"), or [Hq, n, d] for one sequence, n = 1
    for a decode step.  The new tokens' own keys and values are in the cache
    already; ``seqlens`` (int32 [B] on the device) counts them.  Query i of
    sequence b attends to positions t <= seqlens[b] - n + i, or with
    ``causal=False`` to every t < seqlens[b].  Returns a dict with "out" and, on
    request, "lse" (float32 [Hq, B * n], natural log).  A query that sees
    nothing gives zeros and -inf.

    ``max_seqlen`` bounds the lengths (default: what the block table can hold;
    longer entries of seqlens are cut to it); the call reads lengths on the
    device only, so a captured graph stays right as they grow within it.
    ``workspace``: at least ``decode4_workspace_bytes`` of device memory (0 where
    the lengths' bound and the batch are small), not shared by calls that may
    overlap (default: allocated for the call)."""
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
        _, hq, n = _strides_bhtd(q, layout or "bhld", False)
        rows = n if q.dim() == 3 else q.shape[0] * n
        res["lse"] = _empty(stream, dev, (hq, rows), torch.float32)
        lse = res["lse"].data_ptr()
    c, fields = _decode_fields(q, cache, block_table, seqlens, out, dev, layout=layout,
                               max_seqlen=max_seqlen, softmax_scale=softmax_scale, causal=causal,
                               lse=lse)
    if workspace is None:
        need = _native.lib().bsfa_decode4_workspace_size(c, fields(0, 0))
        if need:
            workspace = _empty(stream, dev, (need,), torch.uint8)
    elif not workspace.is_contiguous():
        raise ValueError("the workspace must be contiguous")
    _call(_native.lib().bsfa_decode4, dev, stream, c,
          fields(0, 0) if workspace is None else fields(workspace.data_ptr(), _nbytes(workspace)))
    return res


def decode4_workspace_bytes(q, cache: KVCache4, block_table, seqlens, *, max_seqlen=None,
                            layout=None) -> int:
    """Workspace bytes that decode4 needs for this call's shapes."""
    c, fields = _decode_fields(q, cache, block_table, seqlens, q, q.device, layout=layout,
                               max_seqlen=max_seqlen, softmax_scale=None, causal=True)
    return int(_native.lib().bsfa_decode4_workspace_size(c, fields(0, 0)))
