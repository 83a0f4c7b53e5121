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


def _bad_in(cache, table, seq, token, element, number, page=64):
    at = (table[seq, token // page].item(), slice(None), token % page, element)
    was = cache.v[at].clone()
    cache.v[at] = number
    return at, was


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
