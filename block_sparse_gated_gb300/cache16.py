"""Rotary positions and the 16-bit paged K/V cache: torch-facing wrappers over
the C ABI (argument marshalling only, done in csrc/binding.cpp).

The calls around a prefill over pages: ``cache16_write`` rotates queries and keys
by their positions and puts keys and values into the page pools that ``prefill``
reads through a block table, ``decode16`` attends to them with the tokens that
follow, and ``rotary`` rotates without a cache.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Sequence

import torch

from . import _native
from .api import _DTYPES


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

    ``inverse`` turns back.  It is also the gradient, of the rotated rows' it
    makes the rows', and what autograd takes for q and k that require one (zero
    for rows outside every sequence; frequencies have none).  ``out``, a pair of
    tensors, may be (q, k) themselves; other tensors must not overlap them, and it
    takes no part in a recorded graph."""
    f, axes, interleaved = rope
    q_out, k_out = (None, None) if out is None else out
    return _native.binding().rotary(f, axes, interleaved, q, k, positions, start, cu_seqlens,
                                    layout, inverse, q_out, k_out, stream)


class _Rotary(torch.autograd.Function):
    """Recorded rotations: arguments as the binding's, and ``zeros``, whether packed
    rows outside every sequence are zeros rather than left as they are."""

    @staticmethod
    def forward(ctx, q, k, f, axes, interleaved, positions, start, cu_seqlens, layout, inverse,
                zeros, stream):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(f, positions, start, cu_seqlens)
        ctx.how = axes, interleaved, layout, inverse
        out = None, None
        if zeros and cu_seqlens is not None:
            out = torch.zeros_like(q), None if k is None else torch.zeros_like(k)
        q1, k1 = _native.binding().rotary(f, axes, interleaved, q, k, positions, start, cu_seqlens,
                                          layout, inverse, *out, stream)
        ctx.mark_non_differentiable(*[y for y, needed in zip((q1, k1), ctx.needs_input_grad)
                                      if y is not None and not needed])
        return q1, k1

    @staticmethod
    def backward(ctx, *grads):
        f, positions, start, cu_seqlens = ctx.saved_tensors
        axes, interleaved, layout, inverse = ctx.how
        # Dense and aligned, whatever made them (a sum's gradient has strides of zero).
        g = [x.contiguous() for x in grads if x is not None]
        g = [x.clone() if x.data_ptr() % 16 else x for x in g]
        if not g:
            return (None,) * 12
        turned = iter(_Rotary.apply(g[0], g[1] if len(g) > 1 else None, f, axes, interleaved,
                                    positions, start, cu_seqlens, layout, not inverse, True, None))
        return *[None if x is None else next(turned) for x in grads], *(None,) * 10


def _rotary_recorded(f, axes, interleaved, q, k, positions, start, cu_seqlens, layout, inverse,
                     q_out, k_out, stream):
    """What the binding's rotary calls for rows that require a gradient."""
    return _Rotary.apply(q, k, f, axes, interleaved, positions, start, cu_seqlens, layout, inverse,
                         False, stream)


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
    must differ, and k and v must not overlap the pools.  No gradient passes
    through a cache: tensors that require one are refused while gradients are
    recorded (``rotary`` has one)."""
    k_pool, v_pool, kv_layout = cache
    f, axes, interleaved = (None, None, False) if rope is None else rope
    return _native.binding().cache16_write(k_pool, v_pool, kv_layout, k, v, block_table, f, axes,
                                           interleaved, q, positions, start, cu_seqlens, layout,
                                           q_out, stream)


def decode16(q, cache: KVCache16, block_table, seqlens, *, max_seqlen=None, softmax_scale=None,
             causal=True, layout=None, out=None, return_lse=False, workspace=None, stream=None):
    """Attention of new tokens over the 16-bit cache: q [B, Hq, n, d] (layout
    "bhld") or [B, n, Hq, d] ("blhd"), or [Hq, n, d] for one sequence, n = 1 for a
    decode step, of the cache's type.  The new tokens' own keys and values are in
    the cache already; ``seqlens`` (int32 [B] on the device) counts them.  Query i
    of sequence b attends to positions t <= seqlens[b] - n + i, or with
    ``causal=False`` to every t < seqlens[b].  Returns a dict with "out" and, on
    request, "lse" (float32 [Hq, B * n], natural log).  A query that sees nothing
    gives zeros and -inf.  ``out`` may be q itself.  No gradient is recorded.

    ``max_seqlen`` bounds the lengths (default: what the block table can hold;
    longer entries of seqlens are cut to it); the call reads lengths on the device
    only, so a captured graph stays right as they grow within it.  ``workspace``: at
    least ``decode16_workspace_bytes`` of device memory (0 where the lengths' bound
    and the batch are small), not shared by calls that may overlap (default:
    allocated for the call)."""
    k, v, kv_layout = cache
    return _native.binding().decode16(q, k, v, kv_layout, block_table, seqlens, max_seqlen,
                                      softmax_scale, causal, layout, out, return_lse, workspace,
                                      stream)


def decode16_workspace_bytes(q, cache: KVCache16, block_table, seqlens, *, max_seqlen=None,
                             layout=None) -> int:
    """Workspace bytes that decode16 needs for this call's shapes."""
    k, v, kv_layout = cache
    return _native.binding().decode16_workspace(q, k, v, kv_layout, block_table, seqlens,
                                                max_seqlen, layout)
