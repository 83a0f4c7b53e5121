"""Numbers at the ends of their types' range: frequencies of many turns to a token."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from tests import cache16_util as cu

pytestmark = pytest.mark.gpu

HF = torch.float16


def _bsfa():
    import block_sparse_gated_gb300 as b
    return b


def _pi():
    """pi to 2^-300, by Machin's formula in integers."""
    one = 1 << 320

    def arctan_of_inverse(n):
        total, power, k = 0, one // n, 0
        while power:
            total += (-1) ** k * power // (2 * k + 1)
            power //= n * n
            k += 1
        return total
    return Fraction(4 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239)), one)


@pytest.mark.parametrize("exponent", [40, 55, 56, 57, 58, 59])
def test_frequencies_of_many_turns(cuda_device, exponent):
    """The angle is within (1 + f) |position| 2^-64 + 2^-33 turns of the exact one, which is far
    less than a turn for these; no shift of the frequency's bits may lose them."""
    b = _bsfa()
    freq = (torch.tensor([1.0, 1.17, 1.26, 1.39, 1.55, 1.62, 1.81, 1.94]) * 2.0 ** exponent).float()
    pos = [0, 1, 2, 3] if exponent < 59 else [0, 1]
    x = torch.zeros(1, 1, len(pos), 64, dtype=HF, device=cuda_device)
    x[..., :8] = 1.0  # (1, 0) turns into (cos, sin)
    got, _ = b.rotary(b.Rope(freq.to(cuda_device)), x,
                      positions=cu.i32([pos], cuda_device))
    got = got[0, 0].double().cpu().numpy()
    turn = 2 * _pi()
    for i, p in enumerate(pos):
        for j, f in enumerate(freq.tolist()):
            part = Fraction(f) * p / turn
            angle = 2 * np.pi * float(part - int(part))
            off = 2 * np.pi * ((1 + f) * p * 2.0 ** -64 + 2.0 ** -33)
            # the angle's, the sine's and cosine's (2^-21), and half a step of fp16
            tol = off + 2.0 ** -21 + 2.0 ** -11
            assert abs(got[i, j] - np.cos(angle)) <= tol, (p, f)
            assert abs(got[i, 8 + j] - np.sin(angle)) <= tol, (p, f)
