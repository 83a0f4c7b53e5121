"""fp64 oracle of the 4-bit K/V cache: what a written row stands for, and
attention of new tokens over cached rows.  numpy only; nothing of the package.

A row is d e2m1 codes and one e4m3 scale per 16 elements; see quantise().
"""
from __future__ import annotations

import numpy as np

GROUP = 16
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _e4m3_values() -> np.ndarray:
    """The values of bytes 0x00 .. 0x7e (0x7f is NaN)."""
    v = []
    for byte in range(0x7F):
        e, m = byte >> 3, byte & 7
        v.append(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(v)


E4M3 = _e4m3_values()


def nearest(table: np.ndarray, x: np.ndarray) -> np.ndarray:
    """Index of the table's entry (ascending) nearest to each x >= 0, a tie to
    the even index, beyond the last one the last."""
    hi = np.searchsorted(table, x).clip(0, len(table) - 1)
    lo = (hi - 1).clip(0)
    dl, dh = x - table[lo], table[hi] - x  # exact: few significant bits each
    pick_lo = (dl < dh) | ((dl == dh) & (lo % 2 == 0))
    return np.where((x >= table[-1]) | ~pick_lo, hi, lo)


def quantise(x: np.ndarray, exp=0):
    """x [..., d] (fp64, exactly the 16-bit inputs) -> codes [..., d] (0..15),
    scale bytes [..., d / 16].  Groups that are not finite: codes 0, 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    finite = np.isfinite(g).all(-1)
    g = np.where(finite[..., None], g, 0.0) * 2.0 ** -float(exp)
    byte = np.maximum(nearest(E4M3, np.abs(g).max(-1) / 6), 1)
    code = nearest(E2M1, np.abs(g) / E4M3[byte][..., None])
    code = np.where((g < 0) & (code > 0), code + 8, code)
    code = np.where(finite[..., None], code, 0)
    return code.reshape(x.shape).astype(np.uint8), np.where(finite, byte, 0x7F).astype(np.uint8)


def pack(code: np.ndarray) -> np.ndarray:
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def values(packed: np.ndarray, byte: np.ndarray, exp=0) -> np.ndarray:
    """fp64 values of packed codes [..., d / 2] and scale bytes [..., d / 16]."""
    code = np.stack([packed & 15, packed >> 4], -1)
    code = code.reshape(*packed.shape[:-1], 2 * packed.shape[-1])
    x = E2M1[code & 7] * np.where(code >= 8, -1.0, 1.0)
    s = np.append(E4M3, np.nan)[byte & 0x7F] * np.where(byte >= 0x80, -1.0, 1.0)
    return x * np.repeat(s, GROUP, -1) * 2.0 ** float(exp)


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, *, sigma: float, causal=True):
    """One sequence: q [Hq, n, d], k and v [Hkv, L, d] -> out [Hq, n, d], lse
    [Hq, n], and for error bounds weighted [Hq, n, d] (sum of p |v|), flat
    [Hq, n, d] (sum of |v|) and span [Hq, n] (the largest sum of |q k| sigma),
    each over the visible keys."""
    Hq, n, d = q.shape
    Hkv, L = k.shape[:2]
    out, lse = np.zeros((Hq, n, d)), np.full((Hq, n), -np.inf)
    weighted, flat, span = np.zeros((Hq, n, d)), np.zeros((Hq, n, d)), np.zeros((Hq, n))
    for h in range(Hq):
        kh, vh = k[h // (Hq // Hkv)], v[h // (Hq // Hkv)]
        for i in range(n):
            m = max(0, L - n + i + 1) if causal else L
            if m == 0:
                continue
            s = kh[:m] @ q[h, i] * sigma
            top = s.max()
            with np.errstate(invalid="ignore"):
                p = np.exp(s - top)
            out[h, i] = p @ vh[:m] / p.sum()
            weighted[h, i] = p @ np.abs(vh[:m]) / p.sum()
            flat[h, i] = np.abs(vh[:m]).sum(0)
            lse[h, i] = top + np.log(p.sum())
            span[h, i] = (np.abs(kh[:m]) @ np.abs(q[h, i])).max() * sigma
    return out, lse, weighted, flat, span
