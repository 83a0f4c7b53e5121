"""The 4-bit K/V cache: torch-facing wrappers over the C ABI (argument
marshalling only).

``prefill`` leaves keys and values in 16 bits; ``cache4_write`` quantises them
into the pages of a ``KVCache4``, ``decode4`` attends to it with the tokens
that follow, and ``cache4_read`` gives the 16-bit rows back.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import _native
from .api import _DTYPES, _check, _dtype_code, _nbytes, _on_device, _stream, _strides_bhtd

GROUP = 16  # elements that share a scale


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


def _pool(c, t: torch.Tensor, what: str, dtype, shape, order, field):
    if t.dtype != dtype or t.dim() != 4 or tuple(t.shape) != shape or t.stride(3) != 1:
        raise ValueError(f"{what} must be a {dtype} {list(shape)} tensor with rows contiguous")
    s = t.stride()
    getattr(c, field)[:] = s[0], s[order[0]], s[order[1]]
    return t.data_ptr()


def _cache_params(cache: KVCache4, block_table: torch.Tensor, device, batch: int):
    """The bsfa_cache4 of a call on ``device`` with ``batch`` sequences."""
    k = cache.k
    if cache.layout == "phtd":
        order = (1, 2)
    elif cache.layout == "pthd":
        order = (2, 1)
    else:
        raise ValueError(cache.layout)
    if k.dim() != 4:
        raise ValueError("code pools are 4-D")
    _on_device(device, k=k, v=cache.v, k_scale=cache.k_scale, v_scale=cache.v_scale,
               k_exp=cache.k_exp, v_exp=cache.v_exp, block_table=block_table)
    shape = tuple(k.shape)
    d = 2 * shape[3]
    scales = shape[:3] + (d // GROUP,)
    c = _native.Cache4()
    c.k = _pool(c, k, "k", torch.uint8, shape, order, "k_stride")
    c.v = _pool(c, cache.v, "v", torch.uint8, shape, order, "v_stride")
    c.k_scale = _pool(c, cache.k_scale, "k_scale", torch.float8_e4m3fn, scales, order,
                      "k_scale_stride")
    c.v_scale = _pool(c, cache.v_scale, "v_scale", torch.float8_e4m3fn, scales, order,
                      "v_scale_stride")
    c.num_pages, c.num_heads_kv, c.page_size = shape[0], shape[order[0]], shape[order[1]]
    c.head_dim = d
    for name, e in (("k_exp", cache.k_exp), ("v_exp", cache.v_exp)):
        if e is not None:
            if e.dtype != torch.int32 or tuple(e.shape) != (c.num_heads_kv,) or \
                    not e.is_contiguous():
                raise ValueError(f"{name} must be a contiguous int32 [{c.num_heads_kv}] tensor")
            setattr(c, name, e.data_ptr())
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or \
            (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError("block_table must be an int32 [batch, pages_per_sequence] tensor")
    rows, width = block_table.shape
    if rows < batch:
        raise ValueError("block_table has fewer rows than sequences")
    c.block_table, c.block_table_width = block_table.data_ptr(), width
    c.block_table_stride = block_table.stride(0) if rows > 1 else width
    return c


def _int32_vector(t, n: int, what: str):
    if t.dtype != torch.int32 or tuple(t.shape) != (n,) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 [{n}] tensor")
    return t.data_ptr()


def _rows_params(k, v, layout, cu_seqlens, start, heads: int, d: int):
    varlen = cu_seqlens is not None
    if layout is None:
        layout = "htd" if varlen else "bhld"
    r = _native.Cache4Rows()
    ks, Hk, L = _strides_bhtd(k, layout, varlen)
    vs, Hv, Lv = _strides_bhtd(v, layout, varlen)
    if k.shape != v.shape or (Hk, L) != (Hv, Lv):
        raise ValueError("K and V shapes disagree")
    if k.dtype != v.dtype:
        raise TypeError("K and V must share one element type")
    if Hk != heads or k.shape[-1] != d:
        raise ValueError("K and V must have the cache's heads and head dimension")
    r.k, r.v = k.data_ptr(), v.data_ptr()
    r.k_stride[:], r.v_stride[:] = ks, vs
    r.seqlen, r.dtype = L, _dtype_code(k)
    if varlen:
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or \
                not cu_seqlens.is_contiguous() or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must be a contiguous int32 [batch + 1] tensor")
        r.batch, r.cu_seqlens = cu_seqlens.numel() - 1, cu_seqlens.data_ptr()
    else:
        r.batch = 1 if k.dim() == 3 else k.shape[0]
    if start is not None:
        r.start = _int32_vector(start, r.batch, "start")
    return r


def _heads_and_dim(cache: KVCache4):
    if cache.k.dim() != 4:
        raise ValueError("code pools are 4-D")
    return cache.k.shape[1 if cache.layout == "phtd" else 2], 2 * cache.k.shape[3]


def _call(name, device, stream, *args):
    """One library call on ``stream`` (default: the device's current one), with
    the tensors' device current."""
    fn = getattr(_native.lib(), name)
    if torch.cuda.current_device() != device.index:
        with torch.cuda.device(device):
            _check(fn(*args, _stream(stream, device)), name)
    else:
        _check(fn(*args, _stream(stream, device)), name)


def _made_here(stream, device, *tensors):
    """Tensors allocated by a call that runs on ``stream``: their memory must
    not be handed out again before that stream is done with it."""
    if stream is not None and stream != torch.cuda.current_stream(device):
        for t in tensors:
            t.record_stream(stream)


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
    _on_device(dev, v=v, start=start, cu_seqlens=cu_seqlens)
    r = _rows_params(k, v, layout, cu_seqlens, start, *_heads_and_dim(cache))
    c = _cache_params(cache, block_table, dev, r.batch)
    _call("bsfa_cache4_write", dev, stream, ctypes.byref(c), ctypes.byref(r))


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
        if n is None or int(n) < 0:
            raise ValueError("a varlen read needs total, a batched one seqlen")
        if dtype not in _DTYPES:
            raise TypeError("expected bfloat16 or float16")
        shapes = {"bhld": (block_table.shape[0], heads, int(n), d),
                  "blhd": (block_table.shape[0], int(n), heads, d),
                  "htd": (heads, int(n), d), "thd": (int(n), heads, d)}
        if layout not in (("htd", "thd") if varlen else ("bhld", "blhd")):
            raise ValueError(layout)
        k, v = (torch.empty(shapes[layout], dtype=dtype, device=dev) for _ in range(2))
        if stream is not None:
            _made_here(stream, dev, k, v)
    else:
        k, v = out
    _on_device(dev, k=k, v=v, start=start, cu_seqlens=cu_seqlens)
    r = _rows_params(k, v, layout, cu_seqlens, start, heads, d)
    c = _cache_params(cache, block_table, dev, r.batch)
    _call("bsfa_cache4_read", dev, stream, ctypes.byref(c), ctypes.byref(r))
    return k, v


def _decode_params(q, cache, block_table, seqlens, out, *, layout, max_seqlen, softmax_scale,
                   causal):
    p = _native.Decode4Params()
    qs, Hq, n = _strides_bhtd(q, layout or "bhld", False)
    os_, Ho, no = _strides_bhtd(out, layout or "bhld", False)
    if q.shape != out.shape or q.dtype != out.dtype:
        raise ValueError("q and out must have one shape and type")
    heads, d = _heads_and_dim(cache)
    if q.shape[-1] != d or Hq % heads:
        raise ValueError("q must have the cache's head dimension and a multiple of its heads")
    p.batch = 1 if q.dim() == 3 else q.shape[0]
    c = _cache_params(cache, block_table, q.device, p.batch)
    p.q, p.o = q.data_ptr(), out.data_ptr()
    p.q_stride[:], p.o_stride[:] = qs, os_
    p.num_heads_q, p.q_len = Hq, n
    p.seqlens = _int32_vector(seqlens, p.batch, "seqlens")
    most = c.block_table_width * c.page_size
    p.max_seqlen = most if max_seqlen is None else int(max_seqlen)
    if p.max_seqlen > most:
        raise ValueError("block_table has too few pages per row for max_seqlen")
    p.softmax_scale = float(softmax_scale) if softmax_scale else 0.0
    p.causal = 1 if causal else 0
    p.dtype = _dtype_code(q)
    return p, c


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
    ``workspace``: at least ``decode4_workspace_bytes`` of device memory, not
    shared by calls that may overlap (default: allocated for the call)."""
    made = []
    if out is None:
        out = torch.empty_like(q)
        made.append(out)
    dev = q.device
    _on_device(dev, out=out, seqlens=seqlens)
    p, c = _decode_params(q, cache, block_table, seqlens, out, layout=layout,
                          max_seqlen=max_seqlen, softmax_scale=softmax_scale, causal=causal)
    res = {"out": out}
    if return_lse:
        lse = torch.empty((p.num_heads_q, p.batch * p.q_len), dtype=torch.float32, device=dev)
        p.lse = lse.data_ptr()
        res["lse"] = lse
        made.append(lse)
    need = _native.lib().bsfa_decode4_workspace_size(ctypes.byref(c), ctypes.byref(p))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        made.append(workspace)
    else:
        if not workspace.is_contiguous():
            raise ValueError("the workspace must be contiguous")
        _on_device(dev, workspace=workspace)
    p.workspace, p.workspace_bytes = workspace.data_ptr(), _nbytes(workspace)
    if stream is not None:
        _made_here(stream, dev, *made)
    _call("bsfa_decode4", dev, stream, ctypes.byref(c), ctypes.byref(p))
    return res


def decode4_workspace_bytes(q, cache: KVCache4, block_table, seqlens, *, max_seqlen=None,
                            layout=None) -> int:
    """Workspace bytes that decode4 needs for this call's shapes."""
    p, c = _decode_params(q, cache, block_table, seqlens, q, layout=layout,
                          max_seqlen=max_seqlen, softmax_scale=None, causal=True)
    return int(_native.lib().bsfa_decode4_workspace_size(ctypes.byref(c), ctypes.byref(p)))
