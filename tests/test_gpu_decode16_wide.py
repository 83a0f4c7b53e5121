"""Calls of more than 32 query rows per KV head where a CTA holds whole segments or long pieces
of them: what a warpgroup adds up over many tiles, the join of the two within a CTA, and numbers
that are not finite there.  Each test says, from the lengths, what its pieces are."""
import math
import time

import numpy as np
import pytest
import torch

from oracle import cache4_oracle as co
from tests import cache16_util as cu

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
RUN = 64  # tiles that a warpgroup sums before it adds them in memory


def _bsfa():
    import block_sparse_gated_gb300 as b
    return b


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _call(few, batch, heads, d, dtype, device, *, page=64, seed=3, block=None, scale=1.5, **kw):
    """``batch`` sequences that repeat those of the lengths ``few`` (their pages are shared, their
    queries the same): the call's arguments, what the oracle needs, and the pieces."""
    b = _bsfa()
    Hq, Hkv, n = heads
    cache, table, rows = cu.random_cache(b, few, page, Hkv, d, dtype, seed, device, block=block,
                                         **kw)
    table = cu.shared(table, batch)
    lens = [few[i % len(few)] for i in range(batch)]
    q = cu.rand((len(few), Hq, n, d), dtype, seed, device, scale)
    q = q.repeat(math.ceil(batch / len(few)), 1, 1, 1)[:batch].contiguous()
    row_tiles = math.ceil(Hq // Hkv * n / 128)
    pieces = cu.wide_pieces(lens, table.shape[1] * page, heads_kv=Hkv, row_tiles=row_tiles,
                            sms=_sms())
    return q, cache, table, cu.i32(lens, device), lens, rows, pieces


def _whole(segments):
    return [s for s in segments if s[2] == s[3]]


def _check(res, q, rows, lens, dtype, d, some):
    B, Hq, n = q.shape[:3]
    lse = res["lse"].view(Hq, B, n)
    for i in some:
        cu.check_decode({"out": res["out"][i:i + 1], "lse": lse[:, i]}, q[i:i + 1],
                        [rows[i % len(rows)]], [lens[i]], dtype, d)


@pytest.mark.parametrize("d,dtype", [(64, HF), (128, BF), (64, BF), (128, HF)])
@pytest.mark.parametrize("heads", [(40, 1, 1), (20, 1, 3), (32, 2, 8), (50, 1, 5)])
def test_segments_within_a_cta(cuda_device, d, dtype, heads):
    """Sequences of one tile to eight, most of them within one CTA, whose two warpgroups share
    their tiles."""
    few = [1000, 129, 700, 1, 256, 0, 1024]
    q, cache, table, n32, lens, rows, (per_cta, segments) = _call(few, 210, heads, d, dtype,
                                                                  cuda_device)
    whole = [s for s in _whole(segments) if lens[s[0]] > 128]
    assert per_cta >= 14 and len(whole) > 30
    res = _bsfa().decode16(q, cache, table, n32, return_lse=True)
    _check(res, q, rows, lens, dtype, d, range(0, 210, 5))


@pytest.mark.parametrize("d,dtype", [(64, HF), (128, BF)])
@pytest.mark.parametrize("few", [[17000], [40000], [33000, 16385, 900, 16384]])
def test_more_tiles_than_a_warpgroup_sums_at_once(cuda_device, d, dtype, few):
    """Pieces of 134 tiles and more: sums that go to memory in the middle of a segment, of whole
    ones and of parts, up to exactly 64 and 65 tiles to a warpgroup."""
    batch = 160 if len(few) == 1 else 260
    q, cache, table, n32, lens, rows, (per_cta, segments) = _call(
        few, batch, (12, 1, 4), d, dtype, cuda_device, block=4000)
    assert per_cta > 2 * RUN + 6
    long = [s for s in segments if math.ceil(lens[s[0]] / 128) > 2 * RUN]
    assert [s for s in long if s[2] != s[3]]
    assert _whole(long)
    res = _bsfa().decode16(q, cache, table, n32, return_lse=True)
    _check(res, q, rows, lens, dtype, d, range(0, batch, 37))
    # The others repeat these; where they are cut differs, so that sums differ by their roundings.
    first = res["out"][:len(few)].float()
    again = res["out"].view(-1, len(few), *first.shape[1:]).float()
    assert bool(((again - first).abs() <= first.abs() * torch.finfo(dtype).eps * 2 + 1e-3).all())


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
def test_sums_of_values_of_one_sign(cuda_device, dtype, d):
    """The tensor cores cut off what they add to a sum: at most 2^-23 of it (a step of fp32) at
    each of the 16 steps of a tile, over 64 tiles, so 2^-13 of O, and always toward zero.  Weights
    leave 2^-16, the sums in memory and in the join 2^-18.  The one rounding is monotone, so the
    result lies between the roundings of what those allow."""
    L, batch = 40000, 160
    q, cache, table, n32, lens, rows, (per_cta, _) = _call(
        [L], batch, (48, 1, 1), d, dtype, cuda_device, block=4000, positive=True, scale=0.3)
    assert per_cta > 2 * RUN + 6
    res = _bsfa().decode16(q, cache, table, n32, return_lse=True)
    k, v = rows[0][0][0], rows[0][1][0]
    s = q[0, :, 0].cpu().double().numpy() @ k.T / math.sqrt(d)
    p = np.exp(s - s.max(1, keepdims=True))
    want = torch.from_numpy((p / p.sum(1, keepdims=True)) @ v)
    got = res["out"][:, :, 0].cpu()
    near = 2.0 ** -16 + 2.0 ** -18
    assert bool((got >= (want * (1 - 2.0 ** -13 - near)).to(dtype)).all())
    assert bool((got <= (want * (1 + near)).to(dtype)).all())


def _bad_in(cache, table, seq, token, element, number, page=64):
    at = (table[seq, token // page].item(), slice(None), token % page, element)
    was = cache.v[at].clone()
    cache.v[at] = number
    return at, was


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("d,dtype", [(64, HF), (128, BF)])
@pytest.mark.parametrize("few,batch", [([1000, 700], 200), ([16800], 160)])
def test_values_that_are_not_finite_within_a_cta(cuda_device, bad, d, dtype, few, batch):
    """A value poisons its element of the queries that see the token, in every sequence that holds
    it, and nothing else, down to the bit, in whole segments and in cut ones, with results in a
    tensor of their own or in place of the queries."""
    b = _bsfa()
    n, L = 3, few[0]
    q, cache, table, n32, lens, rows, (per_cta, segments) = _call(
        few, batch, (18, 1, n), d, dtype, cuda_device, block=4000 if L > 4000 else None)
    holds = torch.tensor([i % len(few) == 0 for i in range(batch)], device=cuda_device)
    mine = [s for s in segments if s[0] % len(few) == 0]
    assert len(_whole(mine)) >= 5 and len(mine) > len(_whole(mine))
    clean = b.decode16(q, cache, table, n32, return_lse=True)
    for token, first in ((L - 2, 1), (L - 1, 2), (100, 0)):  # seen by queries `first` and later
        at, was = _bad_in(cache, table, 0, token, 37, bad)
        got = b.decode16(q, cache, table, n32, return_lse=True)
        place = q.clone()
        b.decode16(place, cache, table, n32, out=place)
        cache.v[at] = was
        hit = torch.zeros_like(got["out"], dtype=torch.bool)
        hit[holds, :, first:, 37] = True
        x = got["out"][hit]
        assert bool((torch.isnan(x) if math.isnan(bad) else x == bad).all())
        assert torch.equal(got["lse"], clean["lse"])
        again = hit.clone()
        again[holds, :, :, 37] = True  # formed anew, from weights in fp32
        assert torch.equal(got["out"][~again], clean["out"][~again])
        same = torch.equal(torch.nan_to_num(got["out"].float(), nan=1e9),
                           torch.nan_to_num(place.float(), nan=1e9))
        assert same
        got["out"][hit] = clean["out"][hit]
        _check(got, q, rows, lens, dtype, d, range(0, batch, 23))


def test_pages_and_lengths_of_rows_that_are_formed_anew(cuda_device):
    """Beside a value that is not a number and not seen by all: entries outside the pool read as
    zero keys and values there too, and both orders of tokens and heads, two KV heads and three
    tiles of rows are walked right."""
    b = _bsfa()
    for layout, d, dtype in (("pthd", 64, BF), ("phtd", 128, HF)):
        few = [900, 300, 120]
        Hq, n = 10, 60
        q, cache, table, n32, lens, rows, (_, segments) = _call(
            few, 120, (Hq, 2, n), d, dtype, cuda_device, page=48, layout=layout)
        for i, L in enumerate(few):
            token = L - 2
            page = table[i, token // 48].item()
            at = (page, slice(None), token % 48) if layout == "phtd" else (page, token % 48)
            cache.v[at][..., 5] = float("nan")
        for i in range(0, 120, 3):  # the third page of the first one's histories
            table[i, 2] = -1
        rows[0] = tuple(x.copy() for x in rows[0])
        for x in rows[0]:
            x[:, 96:144] = 0.0
        assert _whole(segments)
        got = b.decode16(q, cache, table, n32, return_lse=True)
        out = got["out"]
        seen = torch.zeros_like(out, dtype=torch.bool)
        seen[:, :, n - 2:, 5] = True
        assert bool(torch.isnan(out[seen]).all()) and bool(torch.isfinite(out[~seen]).all())
        for x in rows:  # the rows that see it are compared in their other elements alone
            x[1][:, -2, 5] = 0.0
        for i in (0, 1, 2, 60, 61, 62, 117, 118, 119):
            part = {"out": out[i:i + 1].clone(),
                    "lse": got["lse"].view(Hq, 120, n)[:, i]}
            clean = rows[i % 3]
            exact = co.attend(q[i].cpu().double().numpy(), *clean, sigma=1 / math.sqrt(d))[0]
            part["out"][0, :, n - 2:, 5] = torch.from_numpy(exact[:, n - 2:, 5]).to(out)
            cu.check_decode(part, q[i:i + 1], [clean], [lens[i]], dtype, d)


def test_values_that_are_not_finite_in_long_histories(cuda_device):
    """Hundreds of thousands of tokens to a CTA, their last value not a number and hidden from one
    query, their first ones seen by all: no wait runs out, and rows beside them are what they
    were."""
    from block_sparse_gated_gb300 import api
    b = _bsfa()
    L, batch, d, page = 1 << 18, 160, 64, 256
    q, cache, table, n32, lens, rows, (per_cta, segments) = _call(
        [L], batch, (20, 1, 2), d, BF, cuda_device, page=page, block=4000)
    assert per_cta > 2000 and _whole(segments)
    assert api.device_error() == 0
    clean = b.decode16(q, cache, table, n32, return_lse=True)
    cache.v[table[0, L // page - 1].item(), 0, page - 1, 3] = float("nan")
    cache.v[table[0, 0].item(), 0, 2, 16:] = float("inf")
    torch.cuda.synchronize()
    began = time.time()
    got = b.decode16(q, cache, table, n32, return_lse=True)
    torch.cuda.synchronize()
    print(f"{time.time() - began:.3f} s")
    assert api.device_error() == 0
    out = got["out"]
    assert bool((out[..., 16:] == float("inf")).all())
    assert bool(torch.isnan(out[:, :, 1, 3]).all())
    same = [0, 1, 2] + list(range(4, 16))
    assert torch.equal(out[..., same], clean["out"][..., same])
    assert torch.equal(got["lse"], clean["lse"])
    # Formed anew: each side within its bound, a rounding and 2^-13, of the same mean.
    was = clean["out"][:, :, 0, 3].float()
    size = float(np.abs(rows[0][1][0, :, 3]).mean())
    assert bool(((out[:, :, 0, 3].float() - was).abs() <= was.abs() * 2.0 ** -7 +
                 size * 2.0 ** -11).all())


@pytest.mark.parametrize("heads", [(40, 1, 1), (32, 2, 12)])
def test_every_segment_has_its_place_in_the_join(cuda_device, heads):
    """The table that the join reads is written whole by every call, whatever the workspace held:
    sequence, head and row tile, the first CTA and, of segments that are cut, the last."""
    b = _bsfa()
    few, d = [1000, 0, 5000, 129], 128
    q, cache, table, n32, lens, rows, (per_cta, segments) = _call(few, 60, heads, d, BF,
                                                                  cuda_device)
    need = b.decode16_workspace_bytes(q, cache, table, n32)
    slots = 2 * 160 * 128 * 2  # two parts to each of two warpgroups of 160 CTAs, 128 rows
    at = slots * d * 4 + slots * 8
    for fill in (0x00, 0x7F, 0xFF):
        ws = torch.full((need,), fill, dtype=torch.uint8, device=cuda_device)
        res = b.decode16(q, cache, table, n32, workspace=ws, return_lse=True)
        jobs = ws[at:at + 16 * len(segments)].view(torch.int32).view(-1, 4).cpu().tolist()
        for job, (seq, seg, first, last) in zip(jobs, segments):
            assert job == [seq, seg, first, last if last != first else -1]
        _check(res, q, rows, lens, BF, d, range(0, 60, 7))


def test_no_wait_ran_out(cuda_device):
    from block_sparse_gated_gb300 import api
    assert api.device_error() == 0
