"""Numbers at the ends of their types' range: frequencies of many turns to a token, and values
whose sums no fp32 number would hold."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from tests import cache16_util as cu
from tests.cache4_util import widen

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


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


def _scaled(cache, rows, power):
    """The cache and its rows with values times 2^power, the largest cut to what bf16 holds."""
    most = torch.finfo(BF).max
    v = (cache.v.double() * 2.0 ** power).clamp(-most, most).to(BF)
    back = [(k, np.clip(x * 2.0 ** power, -most, most)) for k, x in rows]
    return cache._replace(v=v), back


# What runs: one CTA a segment, a cluster of sixteen, pieces, CTAs of one warp; then more than 32
# rows over pieces and over segments within a CTA.
PATHS = [([250, 1, 0, 17], (8, 2, 1), 256), ([4000], (8, 2, 1), 4096),
         ([700, 1, 0, 1301], (12, 1, 1), 70000), ([3, 60, 101, 0] * 100, (8, 4, 1), 112),
         ([700, 1, 0, 1301], (40, 1, 1), 70000), ([300, 517, 90] * 80, (20, 1, 2), 640)]


@pytest.mark.parametrize("power", [126, 110, -90])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("path", range(len(PATHS)))
def test_values_of_any_size(cuda_device, path, d, power):
    """A weighted mean of finite bf16 values is finite, and as exact as any other."""
    b = _bsfa()
    lens, (Hq, Hkv, n), bound = PATHS[path]
    few = lens[:4]  # the others repeat them
    cache, table, rows = cu.random_cache(b, few, 32, Hkv, d, BF, path, cuda_device, fill=0.0)
    cache, rows = _scaled(cache, rows, power)
    table = widen(cu.shared(table, len(lens)), 32, bound)
    q = cu.rand((len(few), Hq, n, d), BF, path, cuda_device, 1.5)
    pick = torch.arange(len(lens)) % len(few)
    lens = [few[i] for i in pick.tolist()]
    res = b.decode16(q[pick.to(cuda_device)], cache, table, cu.i32(lens, cuda_device),
                     max_seqlen=bound, return_lse=True)
    some = sorted(set(range(0, len(lens), 7)) | set(range(4)) & set(range(len(lens))))
    lse = res["lse"].view(Hq, len(lens), n)
    for i in some:
        cu.check_decode({"out": res["out"][i:i + 1], "lse": lse[:, i]}, q[i % len(few)][None],
                        [rows[i % len(few)]], [lens[i]], BF, d)


@pytest.mark.parametrize("rows", [4, 40])
@pytest.mark.parametrize("length", [1, 16, 1000, 1 << 17])
def test_flat_rows_of_the_largest_values(cuda_device, rows, length):
    """Every token has the same weight and the largest value there is: so has the mean."""
    b = _bsfa()
    most = torch.finfo(BF).max
    pages = max(1, -(-length // 512))
    cache = b.cache16_empty(pages, 1, 512, 128, device=cuda_device)
    cache.v.fill_(most)
    cache.v[..., 1::2] = -most
    table = torch.arange(pages, dtype=torch.int32, device=cuda_device)[None]
    q = torch.zeros(1, rows, 1, 128, dtype=BF, device=cuda_device)
    out = b.decode16(q, cache, table, cu.i32([length], cuda_device))["out"]
    want = torch.full_like(out, most)
    want[..., 1::2] = -most
    # bf16 numbers are 2^-8 apart at least, and the mean's other errors below half of that
    assert torch.equal(out, want)
