"""Helpers of the tests of rotary positions and the 16-bit cache."""
from __future__ import annotations

import numpy as np
import torch

from oracle import rotary_oracle as ro


def inv_freq(pairs: int, base: float = 10000.0) -> torch.Tensor:
    return (base ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float()


def rotated(x: torch.Tensor, pos, freq: torch.Tensor, *, axes=None, interleaved=False,
            inverse=False):
    """(fp64 rows, error bound) of rotating x [.., L, d] at pos [A, L].

    The kernel's sines and cosines are off by less than 2^-22: one unit in the last place of a
    number up to 1 (2^-24), twice that for the function's own bound, the reduced angle's rounding
    (2^-25 of at most pi / 4) and 2 pi * (2^-33 + (1 + f) |p| 2^-64) of the reduction, which is
    below 2^-29 for |p| < 2^31 and f <= 1.  A product and a sum add 2^-24 of (|a| + |b|) each.
    Together less than 2^-21 of |a| + |b|; then the one rounding to the type, half a step of the
    result, or of its least subnormal."""
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
