"""fp64 oracle of rotary positions.  numpy only; nothing of the package."""
from __future__ import annotations

import numpy as np


def rotate(x: np.ndarray, pos: np.ndarray, inv_freq: np.ndarray, *, axes=None, interleaved=False,
           inverse=False) -> np.ndarray:
    """x [.., L, d] (fp64, exactly the 16-bit inputs) turned by the integer positions pos [A, L]:
    pair j by pos[axes[j]] * inv_freq[j] (inv_freq exactly the fp32 values).  The angle is formed
    from whole turns taken off in extended precision, so that it is good at any position."""
    P = len(inv_freq)
    axes = np.zeros(P, dtype=int) if axes is None else np.asarray(axes)
    two_pi = 2 * np.longdouble("3.14159265358979323846264338327950288")
    angle = np.asarray(pos)[axes].T.astype(np.longdouble) * inv_freq.astype(np.longdouble)
    angle = (angle - np.floor(angle / two_pi) * two_pi).astype(np.float64)  # [L, P]
    c, s = np.cos(angle), np.sin(angle) * (-1.0 if inverse else 1.0)
    y = x.copy()
    first, second = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if interleaved else \
        (slice(0, P), slice(P, 2 * P))
    a, b = x[..., first], x[..., second]
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    return y


def size(x: np.ndarray, P: int, *, interleaved=False) -> np.ndarray:
    """|a| + |b| at both elements of every pair, 0 at the others: what a rotation's error is
    relative to."""
    y = np.zeros_like(x)
    first, second = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if interleaved else \
        (slice(0, P), slice(P, 2 * P))
    both = np.abs(x[..., first]) + np.abs(x[..., second])
    y[..., first] = y[..., second] = both
    return y
