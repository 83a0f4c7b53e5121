"""Helpers of the 4-bit cache tests: pools with pages in random order, the
oracle's view of a call, and the error bound of the attention kernel."""
from __future__ import annotations

import math

import numpy as np
import torch

from oracle import cache4_oracle as co

CASES_HEADS = {"mha": (2, 2), "gqa4": (8, 2), "odd": (9, 3)}


def table_for(lens, page, rng, spare=3):
    """int32 [B, most + 1] block table with pages in random order (unused
    entries far outside the pool) and the pool's size."""
    need = [math.ceil(x / page) for x in lens]
    pool = sum(need) + spare
    order = iter(rng.permutation(pool).tolist())
    table = np.full((len(lens), max(need, default=0) + 1), 1 << 30, dtype=np.int32)
    for b, n in enumerate(need):
        for j in range(n):
            table[b, j] = next(order)
    return table, pool


def random_cache(bsfa, lens, page, heads, d, seed, device, *, layout="phtd", exps=False,
                 scale=1.0, fill=0xFF):
    """A cache whose rows of every sequence hold quantised gaussians and all
    other rows ``fill`` bytes (0xff: NaN scales).  Returns (cache, table,
    [(k, v) fp64 [heads, L, d] per sequence])."""
    rng = np.random.default_rng(seed)
    table, pool = table_for(lens, page, rng)
    codes = [np.full((pool, heads, page, d // 2), fill, np.uint8) for _ in range(2)]
    scales = [np.full((pool, heads, page, d // 16), fill, np.uint8) for _ in range(2)]
    exp = [rng.integers(-6, 4, heads).astype(np.int32) if exps else np.zeros(heads, np.int32)
           for _ in range(2)]
    rows = []
    for b, L in enumerate(lens):
        kv = []
        for i in range(2):
            x = rng.standard_normal((heads, L, d)) * scale
            if i == 0:
                x *= 0.5 + np.abs(rng.standard_normal((heads, 1, d)))
            out = np.empty_like(x)
            for h in range(heads):
                c, s = co.quantise(x[h] * 2.0 ** exp[i][h], exp[i][h])
                c = co.pack(c)
                out[h] = co.values(c, s, exp[i][h])
                for t in range(L):
                    pg = table[b, t // page]
                    codes[i][pg, h, t % page], scales[i][pg, h, t % page] = c[t], s[t]
            kv.append(out)
        rows.append(tuple(kv))
    t = [torch.from_numpy(c) for c in codes] + [torch.from_numpy(s) for s in scales]
    if layout == "pthd":
        t = [x.transpose(1, 2).contiguous() for x in t]
    t = [x.to(device) for x in t]
    t[2:] = [x.view(torch.float8_e4m3fn) for x in t[2:]]
    e = [torch.from_numpy(x).to(device) if exps else None for x in exp]
    return bsfa.KVCache4(*t, *e, layout), torch.from_numpy(table).to(device), rows


def long_cache(bsfa, lens, page, heads, d, seed, device, *, layout="phtd", block=4000,
               positive=False):
    """random_cache() for long sequences: the rows of every sequence repeat one
    quantised block of ``block`` tokens, each sequence from another place in it,
    and no row is set by itself.  ``positive``: values in [0.75, 1.25]."""
    rng = np.random.default_rng(seed)
    table, pool = table_for(lens, page, rng)
    out, rows = [], [[] for _ in lens]
    for i in range(2):
        x = rng.standard_normal((heads, block, d))
        if i == 0:
            x *= 0.5 + np.abs(rng.standard_normal((heads, 1, d)))
        elif positive:
            x = rng.uniform(0.75, 1.25, x.shape)
        code, byte = co.quantise(x)
        code = co.pack(code)
        stands = co.values(code, byte)
        codes = np.full((pool, page, heads, d // 2), 0xFF, np.uint8)
        scales = np.full((pool, page, heads, d // 16), 0xFF, np.uint8)
        for b, L in enumerate(lens):
            t = np.arange(L)
            src = (t + 977 * b) % block
            at = (table[b, t // page], t % page)
            codes[at] = code[:, src].transpose(1, 0, 2)
            scales[at] = byte[:, src].transpose(1, 0, 2)
            rows[b].append(stands[:, src])
        out.append((codes, scales))
    t = [torch.from_numpy(out[i][j]).to(device) for j in range(2) for i in range(2)]
    if layout == "phtd":
        t = [y.transpose(1, 2).contiguous() for y in t]
    t[2:] = [y.view(torch.float8_e4m3fn) for y in t[2:]]
    return bsfa.KVCache4(*t, None, None, layout), torch.from_numpy(table).to(device), \
        [tuple(kv) for kv in rows]


def widen(table, page, tokens=70000):
    """The same table with unused columns up to a capacity of ``tokens``: the
    bound that a call works with when it is given none.  With the default a call
    cuts the batch into equal pieces instead of giving each sequence a cluster."""
    more = -(-tokens // page) - table.shape[1]
    pad = torch.full((table.shape[0], max(0, more)), 1 << 30, dtype=torch.int32,
                     device=table.device)
    return torch.cat([table, pad], 1)


def query_error(q, k, sigma):
    """Largest score error [Hq, n] from holding query rows q [Hq, n, d] in fp16,
    over keys k [Hkv, L, d].  The kernel scales a row by the power of two that
    brings its largest element into [2^14, 2^15) (by 2^126 at most).  An element
    that stays at 2^-14 or above is exact: bf16 has 8 bits, fp16 11.  One below
    is rounded to a multiple of 2^-24, so it is off by 2^-25 at most."""
    amax = np.abs(q).max(-1)
    up = np.minimum(14 - np.floor(np.log2(np.where(amax > 0, amax, 1.0))), 126)
    most = np.abs(k).sum(-1).max(-1, initial=0.0).repeat(q.shape[0] // k.shape[0])
    return 2.0 ** (-25 - up) * most[:, None] * sigma


def bounds(out, lse, weighted, flat, span, dtype, d, query=0.0):
    """Largest errors that the kernel's arithmetic allows, elementwise.

    Score: products are exact; d of them are added in fp32 (each addition off by
    at most 2^-23 of the running magnitude, which span bounds), and scaling,
    the subtraction of the reference and 2^x add a few units: delta.  Queries
    whose elements differ in size by more than 2^28 are not exact in fp16: query
    is what query_error() allows for that.

    Weights p are rounded to fp16: by 2^-11 of themselves, and below its normal
    range by 2^-25.  The largest weight of a row is at least 2^5: p carries
    2^10, and the reference is raised where a score passes it by 2^5.  So the
    sum of weights is at least 2^5, a small weight is off by at most 2^-30 of
    it, whatever the others are, and an output by 2^-30 sum |v| (that sum is
    not bounded by sum p |v|: the heavy tokens' values may be zero).

    Sums run in fp32, and the result is rounded once to dtype."""
    delta = span * (d + 8) * 2.0 ** -23 + 2.0 ** -20 + query
    half = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal * half
    o = np.abs(out) * half + weighted * (2.0 ** -11 + 2.0 ** -16 + 2 * delta[..., None]) + \
        flat * 2.0 ** -30 + tiny
    return o * 1.01, delta + np.abs(np.where(np.isfinite(lse), lse, 0.0)) * 2.0 ** -21


def check_decode(res, q, rows, lens, dtype, d, *, sigma=None, causal=True, uneven=False):
    """Every output row of every sequence against the oracle; q [B, Hq, n, d].
    ``uneven``: with query_error()."""
    sigma = 1 / math.sqrt(d) if sigma is None else sigma
    got = res["out"].detach().cpu().double().numpy()
    got_lse = res["lse"].cpu().double().numpy() if "lse" in res else None
    n = q.shape[2]
    worst = 0.0
    for b, (k, v) in enumerate(rows):
        qq = q[b].detach().cpu().double().numpy()
        out, lse, weighted, flat, span = co.attend(qq, k[:, :lens[b]], v[:, :lens[b]],
                                                   sigma=sigma, causal=causal)
        query = query_error(qq, k[:, :lens[b]], sigma) if uneven else 0.0
        tol, tol_lse = bounds(out, lse, weighted, flat, span, dtype, d, query)
        err = np.abs(got[b] - out)
        assert (err <= tol).all(), f"sequence {b}: {(err / tol).max():.2f} of the bound"
        worst = max(worst, float((err / tol).max(initial=0.0)))
        if got_lse is not None:
            y = got_lse[:, b * n:(b + 1) * n]
            seen = np.isfinite(lse)
            assert (np.isneginf(y) == ~seen).all()
            assert (np.abs(y[seen] - lse[seen]) <= tol_lse[seen]).all(), f"sequence {b}: lse"
    return worst
