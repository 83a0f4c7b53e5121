"""Helpers of the tests of rotary positions and the 16-bit cache."""
from __future__ import annotations

import math

import numpy as np
import torch

from oracle import cache4_oracle as co
from oracle import rotary_oracle as ro
from tests import cache4_util as c4


def inv_freq(pairs: int, base: float = 10000.0) -> torch.Tensor:
    return (base ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float()


def rotated(x: torch.Tensor, pos, freq: torch.Tensor, *, axes=None, interleaved=False,
            inverse=False):
    """(fp64 rows, error bound) of rotating x [.., L, d] at pos [A, L].

    The kernel's sines and cosines are off by less than 2^-22: the reduced angle, at most pi / 4, by
    three roundings (2^-24 of it each), their polynomials by the two last roundings (2^-24 of a
    number up to 1 each) and 2^-29 of what they leave out, and 2 pi * (2^-33 + (1 + f) |p| 2^-64)
    of the reduction, which is below 2^-29 for |p| < 2^31 and f <= 1.  A product and a sum add
    2^-24 of (|a| + |b|) each.  Together less than 2^-21 of |a| + |b|; then the one rounding to
    the type, half a step of the result, or of its least subnormal."""
    y = x.cpu().double().numpy()
    f = freq.double().numpy()
    want = ro.rotate(y, pos, f, axes=axes, interleaved=interleaved, inverse=inverse)
    info = torch.finfo(x.dtype)
    near = ro.size(y, len(f), interleaved=interleaved) * 2.0 ** -21
    tol = near + (np.abs(want) + near) * info.eps / 2 + (near > 0) * info.smallest_normal * info.eps
    return want, tol


def check_rotated(got: torch.Tensor, x: torch.Tensor, pos, freq, **kw) -> None:
    want, tol = rotated(x, pos, freq, **kw)
    err = np.abs(got.cpu().double().numpy() - want)
    assert (err <= tol).all(), f"off by {np.nanmax(err / np.maximum(tol, 1e-300)):.2f} bounds"


def rand(shape, dtype, seed, device="cpu", scale=1.0) -> torch.Tensor:
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).to(device)


def i32(x, device) -> torch.Tensor:
    return torch.tensor(x, dtype=torch.int32, device=device)


def random_cache(bsfa, lens, page, heads, d, dtype, seed, device, *, layout="phtd",
                 fill=float("nan"), block=None, positive=False):
    """A cache whose rows of every sequence hold gaussians and all other rows ``fill``.  Returns
    (cache, table, [(k, v) fp64 [heads, L, d] per sequence]).  ``block``: the rows repeat that
    many tokens, each sequence from another place in them.  ``positive``: values in [0.75, 1.25]."""
    rng = np.random.default_rng(seed)
    table, pool = c4.table_for(lens, page, rng)
    pools, rows = [], [[] for _ in lens]
    n = block or max(sum(lens), 1)
    for i in range(2):
        x = rng.standard_normal((n, heads, d))
        if i == 0:
            x *= 0.5 + np.abs(rng.standard_normal((heads, d)))
        elif positive:
            x = rng.uniform(0.75, 1.25, x.shape)
        x = torch.from_numpy(x).to(dtype)
        wide = x.double().numpy().transpose(1, 0, 2)
        p = torch.full((pool, page, heads, d), fill, dtype=dtype)
        at = 0
        for b, L in enumerate(lens):
            t = np.arange(L)
            src = (t + 977 * b) % n if block else t + at
            at += L
            p[torch.from_numpy(table[b, t // page]).long(), torch.from_numpy(t % page)] = \
                x[torch.from_numpy(src)]
            rows[b].append(wide[:, src])
        p = p if layout == "pthd" else p.transpose(1, 2).contiguous()
        pools.append(p.to(device))
    return bsfa.KVCache16(*pools, layout), torch.from_numpy(table).to(device), \
        [tuple(kv) for kv in rows]


def bounds(out, lse, weighted, flat, span, dtype, d, tokens):
    """Largest errors that the kernel's arithmetic allows, elementwise.

    Score: products of two 16-bit numbers are exact in fp32; d of them are added (each addition
    off by at most 2^-23 of the running magnitude, which span bounds), and scaling, the row's
    offset and 2^x add a few units: delta.

    Weights go into the products as two 16-bit numbers.  The first is off by half a step (bf16
    2^-8, fp16 2^-11), the second by half a step of that.  fp16's subnormals add 2^-25 a token
    where the largest weight is at least 2^5, so 2^-30 of the sum of weights.

    Sums: 32 products of a tile, each cut off by at most 2^-23 (2^-18 in all), then one addition
    in fp32 for each of a warp's tiles, rounded (2^-24 each), and at most 512 parts, for O and for
    the sum of weights.  The result is rounded once to dtype."""
    half = torch.finfo(dtype).eps / 2
    delta = span * (d + 8) * 2.0 ** -23 + 2.0 ** -20
    sums = 2.0 ** -18 + (2 * (tokens / 16) + 64) * 2.0 ** -24
    tiny = torch.finfo(dtype).smallest_normal * half
    o = np.abs(out) * half + weighted * (half ** 2 + 2 * sums + 2 * delta[..., None]) + \
        flat * 2.0 ** -30 + tiny
    return o * 1.01, delta + sums + np.abs(np.where(np.isfinite(lse), lse, 0.0)) * 2.0 ** -21


def check_decode(res, q, rows, lens, dtype, d, *, sigma=None, causal=True):
    """Every output row of every sequence against the oracle; q [B, Hq, n, d]."""
    sigma = 1 / math.sqrt(d) if sigma is None else sigma
    got = res["out"].detach().cpu().double().numpy()
    got_lse = res["lse"].cpu().double().numpy() if "lse" in res else None
    n = q.shape[2]
    worst = 0.0
    for b, (k, v) in enumerate(rows):
        out, lse, weighted, flat, span = co.attend(q[b].detach().cpu().double().numpy(),
                                                   k[:, :lens[b]], v[:, :lens[b]], sigma=sigma,
                                                   causal=causal)
        tol, tol_lse = bounds(out, lse, weighted, flat, span, dtype, d, lens[b])
        err = np.abs(got[b] - out)
        assert (err <= tol).all(), f"sequence {b}: {(err / tol).max():.2f} of the bound"
        worst = max(worst, float((err / tol).max(initial=0.0)))
        if got_lse is not None:
            y = got_lse[:, b * n:(b + 1) * n]
            seen = np.isfinite(lse)
            assert (np.isneginf(y) == ~seen).all()
            assert (np.abs(y[seen] - lse[seen]) <= tol_lse[seen]).all(), f"sequence {b}: lse"
    return worst


def wide_pieces(lens, max_len, *, heads_kv=1, row_tiles=1, sms=152):
    """How a call of more than 32 query rows per KV head is cut over the CTAs: (units per CTA,
    [(sequence, KV head and row tile, first CTA, last CTA) per segment]).  A segment is its tiles
    of 128 tokens and six units beside them."""
    def units(n):
        return 6 + math.ceil(max(0, min(n, max_len)) / 128)
    per_b = heads_kv * row_tiles
    total = per_b * sum(units(n) for n in lens)
    grid = min(sms, len(lens) * per_b * units(max_len))
    per_cta = max(1, math.ceil(total / grid))
    segments, at = [], 0
    for b, n in enumerate(lens):
        for s in range(per_b):
            segments.append((b, s, at // per_cta, (at + units(n) - 1) // per_cta))
            at += units(n)
    return per_cta, segments


def shared(table, batch):
    """The table of ``batch`` sequences that take turns in the pages of a few."""
    return table.repeat(math.ceil(batch / table.shape[0]), 1)[:batch].contiguous()
