"""Attention of new tokens over the 16-bit cache against the fp64 oracle, with
the elementwise bound that the kernel's arithmetic allows."""
import math

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


def _queries(B, Hq, n, d, dtype, seed, device, scale=1.0):
    return cu.rand((B, Hq, n, d), dtype, seed, device, scale)


_i32 = cu.i32

# (heads q, heads kv, query tokens): rows of one KV head 1 .. 70, so that every
# width of the query row tile and more than one tile of them occur.
HEADS = [(2, 2, 1), (8, 2, 1), (8, 1, 1), (9, 3, 2), (12, 1, 1), (4, 1, 4), (8, 2, 5), (6, 2, 8),
         (32, 1, 1), (10, 1, 3), (8, 1, 5), (14, 1, 5)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("bound", [256, 1400, 70000])
def test_against_the_oracle(cuda_device, d, heads, bound):
    """Ragged batches, an empty sequence among them, by one CTA each, shared by clusters and cut
    into pieces; rows past each end hold NaN."""
    b = _bsfa()
    Hq, Hkv, n = heads
    lens = [1, 0, 16, 250, 17] if bound == 256 else [700, 1, 0, 64, 1301, 129]
    page, layout = (16, "pthd") if (Hq + d) % 3 == 0 else (48, "phtd")
    dtype = BF if n % 2 else HF
    cache, table, rows = cu.random_cache(b, lens, page, Hkv, d, dtype, 10 * Hq + n, cuda_device,
                                         layout=layout)
    q = _queries(len(lens), Hq, n, d, dtype, Hq, cuda_device, 1.5)
    table = widen(table, page, bound)
    res = b.decode16(q, cache, table, _i32(lens, cuda_device), return_lse=True, max_seqlen=bound)
    cu.check_decode(res, q, rows, lens, dtype, d)


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 63, 64, 65, 127, 256, 257, 511, 1000])
def test_every_kind_of_length(cuda_device, length):
    """One sequence at tile, unit and page borders: cut into pieces, shared by a cluster, by one
    CTA."""
    b = _bsfa()
    cache, table, rows = cu.random_cache(b, [length], 32, 2, 128, BF, length, cuda_device)
    q = _queries(1, 8, 1, 128, BF, length, cuda_device, 2.0)
    wide = widen(table, 32)
    for most in (70000, 1024, 64, length):
        if most < length:
            continue
        res = b.decode16(q, cache, wide, _i32([length], cuda_device), return_lse=True,
                         max_seqlen=most)
        cu.check_decode(res, q, rows, [length], BF, 128)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n", [1, 3, 33, 100])
def test_queries_longer_than_the_cache(cuda_device, causal, n):
    """Rows that see nothing give zeros and -inf; without the causal mask every row sees the
    whole cache."""
    b = _bsfa()
    lens = [2, 90, 0, 40]
    cache, table, rows = cu.random_cache(b, lens, 16, 2, 64, HF, n, cuda_device)
    q = _queries(4, 4, n, 64, HF, n, cuda_device)
    for t in (table, widen(table, 16)):
        res = b.decode16(q, cache, t, _i32(lens, cuda_device), causal=causal, return_lse=True)
        cu.check_decode(res, q, rows, lens, HF, 64, causal=causal)
    if causal and n > 2:
        assert not res["out"][0, :, :n - 2].any()
        assert bool(torch.isneginf(res["lse"][:, :n - 2]).all())


def test_layouts_strides_and_scale(cuda_device):
    """q and out as [B, n, Hq, d], as slices, with gaps, one sequence in 3-D; pools whose keys and
    values lie in one allocation."""
    b = _bsfa()
    lens, d = [77, 300], 128
    cache, table, rows = cu.random_cache(b, lens, 64, 2, d, BF, 5, cuda_device)
    both = torch.stack([cache.k, cache.v], 1)
    cache = b.KVCache16(both[:, 0], both[:, 1])
    n32 = _i32(lens, cuda_device)
    big = _queries(2, 5, 12, d + 8, BF, 3, cuda_device)  # [B, tokens, heads + 4, d + 8]
    q = big[:, 1:4, 2:10, 8:]
    out = torch.full((2, 6, 10, d), 3.0, dtype=BF, device=cuda_device)
    res = b.decode16(q, cache, table, n32, layout="blhd", out=out[:, 2:5, 1:9],
                     softmax_scale=0.21, return_lse=True)
    cu.check_decode({"out": res["out"].transpose(1, 2), "lse": res["lse"]}, q.transpose(1, 2),
                    rows, lens, BF, d, sigma=float(np.float32(0.21)))
    keep = torch.ones(2, 6, 10, dtype=torch.bool, device=cuda_device)
    keep[:, 2:5, 1:9] = False
    assert bool((out[keep] == 3.0).all())
    one = b.decode16(q[1].transpose(0, 1), cache, table[1:], n32[1:], softmax_scale=0.21)["out"]
    assert one.shape == (8, 3, d)
    two = b.decode16(q[1:].transpose(1, 2).contiguous(), cache, table[1:], n32[1:],
                     softmax_scale=0.21)["out"][0]
    assert torch.equal(one, two)


def test_lengths_beyond_the_bound_are_cut(cuda_device):
    """Entries of seqlens past max_seqlen, past the table or below zero."""
    b = _bsfa()
    lens = [400, 400, 400, 400]
    cache, table, rows = cu.random_cache(b, lens, 16, 1, 64, BF, 8, cuda_device)
    q = _queries(4, 4, 1, 64, BF, 8, cuda_device)
    given = _i32([400, 1 << 30, -5, -(1 << 31)], cuda_device)
    res = b.decode16(q, cache, table[:, :25], given, max_seqlen=390, return_lse=True)
    cu.check_decode(res, q, rows, [390, 390, 0, 0], BF, 64)


def test_no_length_at_all(cuda_device):
    """A bound of 0, or a table of no pages: every query sees nothing, whatever seqlens says."""
    b = _bsfa()
    cache, table, _ = cu.random_cache(b, [40, 40], 16, 2, 128, HF, 8, cuda_device)
    q = _queries(2, 8, 3, 128, HF, 8, cuda_device)
    n32 = _i32([40, 7], cuda_device)
    for t, most in ((table, 0), (table[:, :0], None)):
        res = b.decode16(q, cache, t, n32, max_seqlen=most, return_lse=True)
        assert not res["out"].any() and bool(torch.isneginf(res["lse"]).all())
    none = b.decode16(q[:, :, :0], cache, table, n32, return_lse=True)
    assert none["out"].shape == (2, 8, 0, 128) and none["lse"].shape == (8, 0)


@pytest.mark.parametrize("cut", [True, False])
def test_the_largest_batch(cuda_device, cut):
    """4096 sequences of 0 to 3 tokens and one of 500; one more is refused."""
    b = _bsfa()
    lens = [int(x) for x in np.random.default_rng(5).integers(0, 4, 4096)]
    lens[2222] = 500
    cache, table, rows = cu.random_cache(b, lens, 16, 1, 64, BF, 2, cuda_device)
    table = widen(table, 16) if cut else table
    q = _queries(4097, 2, 1, 64, BF, 2, cuda_device)
    n32 = _i32(lens + [1], cuda_device)
    res = b.decode16(q[:4096], cache, table, n32[:4096], return_lse=True)
    cu.check_decode(res, q[:4096], rows, lens, BF, 64)
    with pytest.raises(b.BsfaError, match="unsupported"):
        b.decode16(q, cache, torch.cat([table, table[:1]]), n32)


@pytest.mark.parametrize("batch,length,d", [(1, 4097, 128), (2, 3000, 64), (19, 600, 128),
                                            (40, 550, 64), (75, 513, 128), (3, 16000, 64)])
def test_few_sequences_of_some_length(cuda_device, batch, length, d):
    """Clusters of 8 down to 1, and the lengths' bounds between them and the cut."""
    b = _bsfa()
    rng = np.random.default_rng(batch)
    lens = [length] + [int(x) for x in rng.integers(0, length + 1, batch - 1)]
    lens = [x if i < 4 else x % 100 for i, x in enumerate(lens)]
    cache, table, rows = cu.random_cache(b, lens, 32, 2, d, HF, 6, cuda_device)
    q = _queries(batch, 8, 1, d, HF, 6, cuda_device, 1.5)
    res = b.decode16(q, cache, table, _i32(lens, cuda_device), max_seqlen=length, return_lse=True)
    cu.check_decode(res, q, rows, lens, HF, d)


def test_entries_outside_the_pool_read_as_zero_rows(cuda_device):
    """A position whose page does not exist is a zero key and a zero value."""
    b = _bsfa()
    lens = [200]
    cache, table, rows = cu.random_cache(b, lens, 16, 2, 128, BF, 12, cuda_device)
    table[0, 3], table[0, 7], table[0, 12] = -1, cache.k.shape[0], 1 << 30
    for k in rows[0]:
        for j in (3, 7, 12):
            k[:, 16 * j:16 * j + 16] = 0.0
    q = _queries(1, 4, 1, 128, BF, 12, cuda_device)
    res = b.decode16(q, cache, table, _i32(lens, cuda_device), return_lse=True)
    cu.check_decode(res, q, rows, lens, BF, 128)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["value", "key"])
@pytest.mark.parametrize("d,heads", [(64, (2, 1)), (128, (2, 1)), (64, (5, 1)), (128, (16, 1))])
@pytest.mark.parametrize("cut", [True, False])
def test_numbers_that_are_not_finite_reach_only_the_queries_that_see_them(cuda_device, bad, where,
                                                                         d, heads, cut):
    """A value poisons its element of the queries that see the token (an infinity makes it an
    infinity), a NaN key everything of them, a key with an infinity what the formula says; no
    other query or element changes."""
    b = _bsfa()
    L, n = 85, 6
    cache, table, rows = cu.random_cache(b, [L], 32, 1, d, BF, 3, cuda_device)
    # (96 rows with a long bound are another kernel's, below.)
    table = widen(table, 32) if cut and heads[0] < 16 else table
    q = _queries(1, heads[0], n, d, BF, 3, cuda_device)
    n32 = _i32([L], cuda_device)
    clean = b.decode16(q, cache, table, n32, return_lse=True)
    pool = cache.v if where == "value" else cache.k
    for t, first in ((82, 3), (4, 0)):  # 82 is seen by queries i with 82 <= 85 - 6 + i
        page, row = table[0, t // 32].item(), t % 32
        was = pool[page, 0, row, 37].clone()
        pool[page, 0, row, 37] = bad
        got = b.decode16(q, cache, table, n32, return_lse=True)
        pool[page, 0, row, 37] = was
        hit = torch.zeros_like(clean["out"], dtype=torch.bool)
        if where == "value":
            hit[:, :, first:, 37] = True
            assert torch.equal(got["lse"], clean["lse"])
            x = got["out"][hit]
            assert bool((torch.isnan(x) if math.isnan(bad) else x == bad).all())
        else:
            # +inf scores give NaN (inf - inf), -inf scores weigh nothing
            sign = torch.sign(q[:, :, :, 37].float()) * (1 if bad > 0 else -1)
            rows_hit = torch.zeros(1, heads[0], n, dtype=torch.bool, device=cuda_device)
            rows_hit[:, :, first:] = True
            if not math.isnan(bad):
                k, v = rows[0][0].copy(), rows[0][1]
                k[:, t] = 0.0  # rows with a score of -inf: as if the token were not there
                gone = rows_hit & (sign < 0)
                rows_hit = rows_hit & (sign > 0)
                qq, o = q.double().cpu().numpy(), got["out"].double().cpu().numpy()
                for h, i in zip(*np.nonzero(gone[0].cpu().numpy())):
                    s = (k[0] @ qq[0, h, i]) / math.sqrt(d)
                    s[t], s[L - n + i + 1:] = -np.inf, -np.inf
                    p = np.exp(s - s.max())
                    err = np.abs(o[0, h, i] - p @ v[0] / p.sum())
                    assert err.max() <= 0.02  # a weight of the missing token would be 1/85 and up
                hit |= gone[..., None]  # compared above
                got["out"][gone] = float("nan")
            hit |= rows_hit[..., None]
            assert bool(torch.isnan(got["out"][hit]).all())
        assert torch.equal(got["out"][~hit], clean["out"][~hit])


def test_queries_that_are_not_finite(cuda_device):
    """A row with a NaN or an infinity beside keys of both signs gives NaN; rows beside it are
    untouched."""
    b = _bsfa()
    lens = [120]
    for wide in (False, True):
        cache, table, rows = cu.random_cache(b, lens, 16, 1, 64, BF, 3, cuda_device)
        table = widen(table, 16) if wide else table
        q = _queries(1, 8, 1, 64, BF, 2, cuda_device)
        clean = b.decode16(q, cache, table, _i32(lens, cuda_device))["out"]
        bad = q.clone()
        bad[0, 1, 0, 7], bad[0, 4, 0, 9] = float("nan"), float("inf")
        got = b.decode16(bad, cache, table, _i32(lens, cuda_device))["out"]
        nan = torch.isnan(got).all(-1)[0, :, 0].tolist()
        assert nan == [i in (1, 4) for i in range(8)]
        rest = [0, 2, 3, 5, 6, 7]
        assert torch.equal(got[0, rest], clean[0, rest])


def test_sharp_and_flat_rows(cuda_device):
    """Scores that rise along the sequence by thousands (the offset moves at every tile), fall,
    or are all equal."""
    b = _bsfa()
    L, d = 900, 64
    for dtype in (BF, HF):
        cache, table, rows = cu.random_cache(b, [L], 16, 1, d, dtype, 14, cuda_device)
        q = torch.zeros(1, 4, 1, d, dtype=dtype, device=cuda_device)
        q[0, 0], q[0, 1], q[0, 3] = 400.0, -400.0, 3.0
        for t in (table, widen(table, 16)):
            res = b.decode16(q, cache, t, _i32([L], cuda_device), return_lse=True)
            cu.check_decode(res, q, rows, [L], dtype, d)


def test_weights_far_apart(cuda_device):
    """One token takes nearly all of the weight and its value is zero: what is left comes from
    weights of 2^-20 and less."""
    b = _bsfa()
    L, d = 333, 128
    for dtype in (BF, HF):
        cache, table, rows = cu.random_cache(b, [L], 48, 1, d, dtype, 4, cuda_device)
        q = torch.ones(1, 4, 1, d, dtype=dtype, device=cuda_device)
        t = 170
        at = (table[0, t // 48].item(), 0, t % 48)
        cache.k[at], cache.v[at] = 2.5, 0.0
        rows[0][0][:, t], rows[0][1][:, t] = 2.5, 0.0
        for w in (table, widen(table, 48)):
            res = b.decode16(q, cache, w, _i32([L], cuda_device), return_lse=True)
            cu.check_decode(res, q, rows, [L], dtype, d)


def test_runs_repeat_bit_for_bit_whatever_the_workspace_holds(cuda_device):
    b = _bsfa()
    lens = [3000, 10, 777]
    cache, table, rows = cu.random_cache(b, lens, 64, 2, 128, BF, 4, cuda_device)
    table = widen(table, 64)
    q = _queries(3, 16, 1, 128, BF, 4, cuda_device)
    n32 = _i32(lens, cuda_device)
    need = b.decode16_workspace_bytes(q, cache, table, n32)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=cuda_device)
    first = b.decode16(q, cache, table, n32, workspace=ws, return_lse=True)
    cu.check_decode(first, q, rows, lens, BF, 128)
    for fill in (0x00, 0x3C, 0xFF):
        ws.fill_(fill)
        again = b.decode16(q, cache, table, n32, workspace=ws, return_lse=True)
        assert torch.equal(again["out"], first["out"]) and torch.equal(again["lse"], first["lse"])
    with pytest.raises(b.BsfaError, match="workspace"):
        b.decode16(q, cache, table, n32, workspace=ws[:need - 256])


@pytest.mark.parametrize("cut", [True, False])
def test_graphs_follow_the_lengths_and_streams_do_not_mix(cuda_device, cut):
    """A captured call reads the lengths at replay; two graphs with workspaces of their own run
    on two streams at once."""
    b = _bsfa()
    lens = [2000, 1500]
    cache, table, rows = cu.random_cache(b, lens, 32, 2, 64, HF, 21, cuda_device)
    table = widen(table, 32) if cut else table
    q = [_queries(2, 8, 1, 64, HF, s, cuda_device) for s in (1, 2)]
    n32 = [_i32(lens, cuda_device) for _ in range(2)]
    need = b.decode16_workspace_bytes(q[0], cache, table, n32[0])
    assert (need > 0) == cut
    ws = [torch.empty(need, dtype=torch.uint8, device=cuda_device) for _ in range(2)]
    outs = [torch.empty_like(x) for x in q]
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.decode16(q[i], cache, table, n32[i], out=outs[i], workspace=ws[i])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for now in ([2000, 1500], [3, 900], [0, 1], [1024, 64]):
        for t in n32:
            t.copy_(_i32(now, cuda_device))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                for _ in range(3):
                    g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            cu.check_decode({"out": outs[i]}, q[i], rows, now, HF, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = b.decode16(q[0], cache, table, n32[0], stream=side)
    side.synchronize()
    assert torch.equal(r["out"], outs[0])


def test_results_on_another_stream_have_memory_of_their_own(cuda_device):
    """Memory that the current stream has given back but still writes is not what a call on
    another stream returns its results in."""
    b = _bsfa()
    cache, table, rows = cu.random_cache(b, [500], 32, 2, 128, BF, 9, cuda_device)
    q = _queries(1, 8, 1, 128, BF, 9, cuda_device)
    n32 = _i32([500], cuda_device)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        old = [torch.empty_like(q) for _ in range(4)]
        torch.cuda._sleep(20_000_000)  # about 10 ms
        for t in old:
            t.fill_(7.0)
        del old, t
        r = b.decode16(q, cache, table, n32, stream=side, return_lse=True)
        torch.cuda.synchronize()
        cu.check_decode(r, q, rows, [500], BF, 128)


@pytest.mark.parametrize("cut", [True, False])
def test_a_batch_of_many_short_and_one_long(cuda_device, cut):
    """300 sequences, many of them in one piece and one over many pieces."""
    b = _bsfa()
    lens = [int(x) for x in np.random.default_rng(1).integers(0, 40, 299)] + [5000]
    cache, table, rows = cu.random_cache(b, lens, 16, 1, 64, BF, 2, cuda_device)
    table = widen(table, 16) if cut else table
    q = _queries(300, 2, 1, 64, BF, 2, cuda_device)
    res = b.decode16(q, cache, table, _i32(lens, cuda_device), return_lse=True)
    cu.check_decode(res, q, rows, lens, BF, 64)


@pytest.mark.parametrize("layout", ["phtd", "pthd"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,n", [(8, 1), (32, 1), (16, 2), (64, 1), (24, 2), (64, 3)])
def test_many_short_sequences(cuda_device, layout, d, Hq, n):
    """800 segments, more than are resident at once, for 1 to 24 query rows of a KV head."""
    b = _bsfa()
    rng = np.random.default_rng(Hq + d)
    lens = [int(x) for x in rng.integers(0, 101, 100)]
    cache, table, rows = cu.random_cache(b, lens, 16, 8, d, BF, 3, cuda_device, layout=layout)
    q = _queries(100, Hq, n, d, BF, Hq, cuda_device, 1.5)
    res = b.decode16(q, cache, table, _i32(lens, cuda_device), return_lse=True)
    cu.check_decode(res, q, rows, lens, BF, d)


@pytest.mark.parametrize("length,Hq,d,layout", [
    (70000, 4, 128, "phtd"), (70000, 12, 64, "pthd"), (70000, 32, 128, "pthd"),
    (150000, 4, 64, "phtd"), (150000, 8, 128, "phtd")])
def test_a_history_of_hundreds_of_parts(cuda_device, length, Hq, d, layout):
    """One sequence of one KV head: hundreds of parts for one block of the join to add."""
    b = _bsfa()
    cache, table, rows = cu.random_cache(b, [length], 64, 1, d, BF, Hq, cuda_device,
                                         layout=layout, block=4000)
    q = _queries(1, Hq, 1, d, BF, Hq, cuda_device, 1.5)
    res = b.decode16(q, cache, table, _i32([length], cuda_device), return_lse=True)
    cu.check_decode(res, q, rows, [length], BF, d)


@pytest.mark.parametrize("Hq,n,d,longest", [(2, 1, 128, 20000), (12, 1, 64, 20000),
                                            (4, 5, 128, 40000), (4, 1, 64, 131000)])
def test_one_long_history_among_many_short_ones(cuda_device, Hq, n, d, longest):
    """300 short sequences make few parts the rule; the long one has many, which one warp per
    row adds 32 at a time."""
    b = _bsfa()
    lens = [int(x) for x in np.random.default_rng(Hq).integers(0, 40, 300)]
    lens.insert(123, longest)
    cache, table, rows = cu.random_cache(b, lens, 16, 1, d, HF, Hq, cuda_device, block=4000)
    q = _queries(301, Hq, n, d, HF, Hq, cuda_device, 1.5)
    res = b.decode16(q, cache, table, _i32(lens, cuda_device), return_lse=True)
    cu.check_decode(res, q, rows, lens, HF, d)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_sums_of_a_million_values_of_one_sign(cuda_device, dtype):
    """320 histories of 2^20 tokens, read from the same pages, each the work of about one CTA:
    the tensor cores' sums do not fall behind."""
    b = _bsfa()
    L, d, B = 1 << 20, 64, 320
    cache, table, rows = cu.random_cache(b, [L], 256, 1, d, dtype, 5, cuda_device, positive=True,
                                         block=4000)
    q = _queries(1, 1, 1, d, dtype, 5, cuda_device, 0.3)
    res = b.decode16(q.repeat(B, 1, 1, 1), cache, table.repeat(B, 1), _i32([L] * B, cuda_device),
                     return_lse=True)
    s = rows[0][0][0] @ q[0, 0, 0].cpu().double().numpy() / 8
    p = np.exp(s - s.max())
    want = rows[0][1][0].T @ (p / p.sum())
    off = res["out"][:, 0, 0].cpu().double().numpy() / want - 1
    # One rounding, and before it 2^-16 of the weights' and at most 2^14 additions to a sum of
    # a warp, each off by 2^-24 and as often up as down.
    half = torch.finfo(dtype).eps / 2
    assert abs(off).max() <= half + 2.0 ** -16 + 2.0 ** -14
    assert abs(off.mean()) <= 3 * half / math.sqrt(3 * 64) + 2.0 ** -15


def test_offsets_beyond_32_bits(cuda_device):
    """Pages more than 4 GiB apart."""
    b = _bsfa()
    d, page, L = 128, 32, 70
    small, table, rows = cu.random_cache(b, [L], page, 2, d, BF, 5, cuda_device)
    P, step = small.k.shape[0], (1 << 31) + 4096  # elements
    raw = torch.empty((P - 1) * step + 65536, dtype=BF, device=cuda_device)
    views = [raw.as_strided(small.k.shape, (step, page * d, d, 1), at) for at in (0, 16384)]
    for v, x in zip(views, small[:2]):
        v.copy_(x)
    q = _queries(1, 8, 1, d, BF, 5, cuda_device)
    for t in (table, widen(table, page)):
        res = b.decode16(q, b.KVCache16(*views), t, _i32([L], cuda_device), return_lse=True)
        cu.check_decode(res, q, rows, [L], BF, d)


@pytest.mark.parametrize("layout", ["phtd", "pthd"])
@pytest.mark.parametrize("stride", [0, 1, 8])
def test_pools_of_one_page_and_one_head(cuda_device, layout, stride):
    """The strides of dimensions of one element say nothing."""
    b = _bsfa()
    cache, table, rows = cu.random_cache(b, [40], 48, 1, 128, BF, 6, cuda_device, layout=layout)
    page = table[0, 0].item()
    head = 1 if layout == "phtd" else 2
    odd = []
    for t in cache[:2]:
        t = t[page:page + 1]
        odd.append(t.as_strided(t.shape, [stride if i in (0, head) else s
                                          for i, s in enumerate(t.stride())]))
    q = _queries(1, 4, 1, 128, BF, 6, cuda_device)
    res = b.decode16(q, b.KVCache16(*odd, layout), _i32([[0]], cuda_device), _i32([40], cuda_device),
                     return_lse=True)
    cu.check_decode(res, q, rows, [40], BF, 128)


def test_prefill_over_pages_then_decode_as_they_are_used(cuda_device):
    """A prompt's keys and values rotated into pages, its prefill over them, then tokens one at a
    time: each is rotated, written and attends to everything before it.  Prefill and decode agree
    with the formula over what the pages hold, and with each other."""
    b = _bsfa()
    Hq, Hkv, L, steps, d, page = 8, 2, 300, 5, 128, 128
    total = L + steps
    fused = cu.rand((1, total, Hq + 2 * Hkv, d), BF, 31, cuda_device)  # one projection
    q, k, v = fused.split([Hq, Hkv, Hkv], 2)
    rope = b.Rope(cu.inv_freq(64).to(cuda_device))
    pages = math.ceil(total / page)
    cache = b.cache16_empty(pages, Hkv, page, d, device=cuda_device)
    table = torch.arange(pages, dtype=torch.int32, device=cuda_device).flip(0)[None].contiguous()
    kw = dict(rope=rope, layout="blhd")
    q2 = b.cache16_write(cache, k[:, :L], v[:, :L], table, q=q[:, :L], **kw)
    over = dict(mode="none", block_table=table, kv_layout=cache.layout)
    first = b.prefill(q2, cache.k, cache.v, layout="blhd", **over)["out"]
    n32 = _i32([L], cuda_device)
    outs, turned = [], [q2]
    for i in range(L, total):
        now = slice(i, i + 1)
        turned.append(b.cache16_write(cache, k[:, now], v[:, now], table, q=q[:, now], start=n32,
                                      **kw))
        n32 += 1
        outs.append(b.decode16(turned[-1], cache, table, n32, layout="blhd")["out"])
    qs = torch.cat(turned, 1).transpose(1, 2).contiguous()
    want_q, want_k = b.rotary(rope, q, k, layout="blhd")
    assert torch.equal(qs, want_q.transpose(1, 2))
    flat = [p[table[0].long()].transpose(1, 2).reshape(-1, Hkv, d)[:total].transpose(0, 1)
            for p in (cache.k, cache.v)]
    assert torch.equal(flat[0], want_k[0].transpose(0, 1))
    assert torch.equal(flat[1], v[0].transpose(0, 1))
    rows = [tuple(x.cpu().double().numpy() for x in flat)]
    for j, o in enumerate(outs):
        cu.check_decode({"out": o.transpose(1, 2)}, qs[:, :, L + j:L + j + 1], rows, [L + j + 1],
                        BF, d)
    chunk = b.decode16(qs, cache, table, n32, return_lse=True)
    cu.check_decode(chunk, qs, rows, [total], BF, d)
    whole = b.prefill(qs, cache.k, cache.v, return_lse=True, **over)
    # the prefill rounds its weights to bf16, which is within the rounding of its result
    assert (whole["out"].float() - chunk["out"].float()).abs().max().item() < 2e-2
    assert (whole["lse"] - chunk["lse"]).abs().max().item() < 2e-3
    assert (first.transpose(1, 2).float() - chunk["out"][:, :, :L].float()).abs().max() < 2e-2


def test_a_launch_that_failed_leaves_no_error_behind(cuda_device):
    """The runtime refuses a launch on the legacy stream while this thread captures a blocking
    stream; the calls after it answer for themselves."""
    import ctypes
    b = _bsfa()
    cache, table, rows = cu.random_cache(b, [100], 16, 2, 64, BF, 5, cuda_device)
    q = _queries(1, 4, 1, 64, BF, 5, cuda_device)
    n32, out = _i32([100], cuda_device), torch.empty_like(q)
    rope = b.Rope(cu.inv_freq(32).to(cuda_device))
    spare = torch.empty_like(q)
    b.decode16(q, cache, table, n32, out=out)
    torch.cuda.synchronize()
    with open("/proc/self/maps") as f:  # the runtime that torch has loaded
        rt = ctypes.CDLL(next(line.split()[-1] for line in f if "libcudart" in line))
    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert rt.cudaStreamCreate(ctypes.byref(stream)) == 0
    assert rt.cudaStreamBeginCapture(stream, 0) == 0
    legacy, seen = torch.cuda.default_stream(), []
    try:
        for call in (lambda: b.decode16(q, cache, table, n32, out=out, stream=legacy),
                     lambda: b.rotary(rope, q, out=(spare, None), stream=legacy)):
            try:
                call()
            except b.BsfaError as e:
                seen.append(e.status)
    finally:
        rt.cudaStreamEndCapture(stream, ctypes.byref(graph))
        rt.cudaGetLastError()
        rt.cudaStreamDestroy(stream)
    assert seen == [3, 3]
    b.rotary(rope, q, out=(spare, None))
    cu.check_decode(b.decode16(q, cache, table, n32), q, rows, [100], BF, 64)


# Calls of more than 32 query rows of a KV head, (heads q, heads kv, query tokens): 33 to 300 rows.
MANY = [(33, 1, 1), (16, 2, 5), (16, 1, 8), (64, 1, 1), (32, 2, 8), (128, 1, 1), (43, 1, 3),
        (10, 2, 60)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", MANY)
@pytest.mark.parametrize("page,layout", [(16, "phtd"), (48, "pthd"), (128, "phtd")])
def test_many_query_rows(cuda_device, d, heads, page, layout):
    """Rows by the hundred, in tiles of 128, over sequences that lie within a CTA and over such
    that are cut; an empty one among them, NaN past each end."""
    b = _bsfa()
    Hq, Hkv, n = heads
    lens = [1300, 1, 0, 129, 700, 3000]
    dtype = BF if n % 2 else HF
    cache, table, rows = cu.random_cache(b, lens, page, Hkv, d, dtype, Hq + n, cuda_device,
                                         layout=layout)
    q = _queries(len(lens), Hq, n, d, dtype, Hq, cuda_device, 1.5)
    for t in (table, widen(table, page)):
        res = b.decode16(q, cache, t, _i32(lens, cuda_device), return_lse=True)
        cu.check_decode(res, q, rows, lens, dtype, d)


@pytest.mark.parametrize("d,dtype", [(64, HF), (128, BF)])
@pytest.mark.parametrize("lens", [[40000], [9000, 20, 1500, 17000], [1100] * 40, [2100, 0] * 60])
def test_many_query_rows_over_long_and_many_sequences(cuda_device, d, dtype, lens):
    """More tiles than a warpgroup sums at once, pieces that hold several sequences."""
    b = _bsfa()
    cache, table, rows = cu.random_cache(b, lens, 64, 1, d, dtype, 3, cuda_device, block=4000)
    q = _queries(len(lens), 12, 4, d, dtype, 5, cuda_device, 1.5)
    res = b.decode16(q, cache, table, _i32(lens, cuda_device), return_lse=True)
    some = list(range(len(lens)))[:6]
    lse = res["lse"].view(12, len(lens), 4)
    for i in some:
        cu.check_decode({"out": res["out"][i:i + 1], "lse": lse[:, i]}, q[i:i + 1], rows[i:i + 1],
                        lens[i:i + 1], dtype, d)


def test_many_query_rows_of_the_largest_batch(cuda_device):
    """4096 sequences of 0 to 3 tokens and one of 700, queries inside a larger tensor."""
    b = _bsfa()
    lens = [int(x) for x in np.random.default_rng(5).integers(0, 4, 4096)]
    lens[2222] = 700
    cache, table, rows = cu.random_cache(b, lens, 16, 1, 64, BF, 2, cuda_device)
    q = _queries(4096, 42, 1, 80, BF, 2, cuda_device)[:, 1:41, :, 8:72]
    res = b.decode16(q, cache, table, _i32(lens, cuda_device), return_lse=True)
    lse = res["lse"].view(40, 4096, 1)
    for i in [0, 1, 2, 2221, 2222, 2223, 4094, 4095] + list(range(100, 4000, 300)):
        cu.check_decode({"out": res["out"][i:i + 1], "lse": lse[:, i]}, q[i:i + 1], rows[i:i + 1],
                        lens[i:i + 1], BF, 64)
    empty = torch.tensor([x == 0 for x in lens], device=cuda_device)
    assert not res["out"][empty].any() and bool(res["out"][~empty].any(-1).all())


@pytest.mark.parametrize("causal", [True, False])
def test_many_queries_longer_than_the_cache(cuda_device, causal):
    """Tiles of rows of which some or all see nothing."""
    b = _bsfa()
    lens = [2, 190, 0, 40]
    cache, table, rows = cu.random_cache(b, lens, 16, 2, 64, HF, 4, cuda_device)
    q = _queries(4, 4, 100, 64, HF, 4, cuda_device)
    res = b.decode16(q, cache, widen(table, 16), _i32(lens, cuda_device), causal=causal,
                     return_lse=True)
    cu.check_decode(res, q, rows, lens, HF, 64, causal=causal)


@pytest.mark.parametrize("d", [64, 128])
def test_many_query_rows_over_pages_that_do_not_exist(cuda_device, d):
    b = _bsfa()
    lens = [1500]
    cache, table, rows = cu.random_cache(b, lens, 32, 1, d, BF, 12, cuda_device)
    for j, bad in ((3, -1), (7, cache.k.shape[0]), (40, 1 << 30)):
        table[0, j] = bad
        for k in rows[0]:
            k[:, 32 * j:32 * j + 32] = 0.0
    q = _queries(1, 40, 1, d, BF, 12, cuda_device)
    res = b.decode16(q, cache, table, _i32(lens, cuda_device), return_lse=True)
    cu.check_decode(res, q, rows, lens, BF, d)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("d", [64, 128])
def test_many_query_rows_beside_values_that_are_not_finite(cuda_device, bad, d):
    """A value poisons its element of the queries that see the token; all else stays within
    the bound of what it is without it."""
    b = _bsfa()
    L, n = 1200, 7
    cache, table, rows = cu.random_cache(b, [L], 32, 1, d, BF, 3, cuda_device)
    q = _queries(1, 6, n, d, BF, 3, cuda_device)
    n32 = _i32([L], cuda_device)
    for t, first in ((L - 4, 3), (100, 0)):  # L - 4 is seen by queries i with L - 4 <= L - 7 + i
        at = (table[0, t // 32].item(), 0, t % 32, 37)
        was = cache.v[at].clone()
        cache.v[at] = bad
        got = b.decode16(q, cache, table, n32, return_lse=True)
        cache.v[at] = was
        hit = torch.zeros_like(got["out"], dtype=torch.bool)
        hit[:, :, first:, 37] = True
        x = got["out"][hit]
        assert bool((torch.isnan(x) if math.isnan(bad) else x == bad).all())
        clean = b.decode16(q, cache, table, n32)["out"]
        hit[:, :, :, 37] = True
        assert torch.equal(got["out"][~hit], clean[~hit])
        got["out"][:, :, first:, 37] = clean[:, :, first:, 37]
        cu.check_decode(got, q, rows, [L], BF, d)


def test_many_query_rows_of_keys_and_queries_that_are_not_numbers(cuda_device):
    b = _bsfa()
    L = 1200
    cache, table, rows = cu.random_cache(b, [L], 32, 1, 64, BF, 3, cuda_device)
    q = _queries(1, 40, 2, 64, BF, 3, cuda_device)
    n32 = _i32([L], cuda_device)
    clean = b.decode16(q, cache, table, n32)["out"]
    page, row = table[0, (L - 1) // 32].item(), (L - 1) % 32
    cache.k[page, 0, row, 5] = float("nan")  # the last token, seen by the last queries
    got = b.decode16(q, cache, table, n32)["out"]
    assert bool(torch.isnan(got[:, :, 1]).all()) and torch.equal(got[:, :, 0], clean[:, :, 0])
    cache.k[page, 0, row, 5] = 0.0
    clean = b.decode16(q, cache, table, n32)["out"]
    bad = q.clone()
    bad[0, 7, 0, 3] = float("nan")
    got = b.decode16(bad, cache, table, n32)["out"]
    assert bool(torch.isnan(got[0, 7, 0]).all())
    got[0, 7, 0] = clean[0, 7, 0]
    assert torch.equal(got, clean)


def test_many_query_rows_sharp_and_flat(cuda_device):
    """Scores that rise along the sequence by thousands, fall, or are all equal."""
    b = _bsfa()
    L, d = 3000, 64
    for dtype in (BF, HF):
        cache, table, rows = cu.random_cache(b, [L], 16, 1, d, dtype, 14, cuda_device)
        q = torch.zeros(1, 40, 1, d, dtype=dtype, device=cuda_device)
        q[0, 0:10], q[0, 10:20], q[0, 30:] = 400.0, -400.0, 3.0
        res = b.decode16(q, cache, table, _i32([L], cuda_device), return_lse=True)
        cu.check_decode(res, q, rows, [L], dtype, d)


def test_many_query_rows_in_graphs_with_strides_and_two_streams(cuda_device):
    """Captured calls follow the lengths, side by side, with outputs inside larger tensors."""
    b = _bsfa()
    lens = [2500, 1500]
    cache, table, rows = cu.random_cache(b, lens, 32, 2, 64, HF, 21, cuda_device)
    q = [_queries(2, 80, 1, 64, HF, s, cuda_device) for s in (1, 2)]
    n32 = [_i32(lens, cuda_device) for _ in range(2)]
    need = b.decode16_workspace_bytes(q[0], cache, table, n32[0])
    assert need > 0
    ws = [torch.full((need,), 0xFF, dtype=torch.uint8, device=cuda_device) for _ in range(2)]
    outs = [torch.full((2, 82, 1, 80), 7.0, dtype=HF, device=cuda_device) for _ in range(2)]
    graphs = []
    for i in range(2):
        b.decode16(q[i], cache, table, n32[i], out=outs[i][:, 1:81, :, 8:72], workspace=ws[i])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.decode16(q[i], cache, table, n32[i], out=outs[i][:, 1:81, :, 8:72], workspace=ws[i])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for now in ([2500, 1500], [3, 1400], [0, 1], [1024, 64]):
        for t in n32:
            t.copy_(_i32(now, cuda_device))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                for _ in range(3):
                    g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            part = outs[i][:, 1:81, :, 8:72]
            cu.check_decode({"out": part}, q[i], rows, now, HF, 64)
            again = part.clone()
            graphs[i].replay()
            torch.cuda.synchronize()
            assert torch.equal(part, again)
            keep = outs[i].clone()
            keep[:, 1:81, :, 8:72] = 7.0
            assert bool((keep == 7.0).all())
    with pytest.raises(b.BsfaError, match="workspace"):
        b.decode16(q[0], cache, table, n32[0], workspace=ws[0][:need - 256])


@pytest.mark.parametrize("heads", [(8, 2, 2), (40, 1, 2)])
@pytest.mark.parametrize("cut", [True, False])
def test_results_in_place_of_the_queries(cuda_device, heads, cut):
    """Also beside a value that is not a number and that some queries do not see."""
    b = _bsfa()
    Hq, Hkv, n = heads
    lens = [700, 3, 0, 1200]
    cache, table, rows = cu.random_cache(b, lens, 32, Hkv, 64, BF, 6, cuda_device)
    table = widen(table, 32) if cut else table
    q = _queries(4, Hq, n, 64, BF, 6, cuda_device)
    n32 = _i32(lens, cuda_device)
    for bad in (None, float("nan")):
        if bad is not None:  # in the last token of the first sequence
            cache.v[table[0, 699 // 32].item(), :, 699 % 32, 3] = bad
        want = b.decode16(q, cache, table, n32, return_lse=True)
        mine = q.clone()
        got = b.decode16(mine, cache, table, n32, out=mine, return_lse=True)
        assert got["out"] is mine
        for x, y in zip(want.values(), got.values()):
            assert torch.equal(torch.nan_to_num(x.float(), nan=1e9), torch.nan_to_num(y.float(), nan=1e9))
        if bad is None:
            cu.check_decode(got, q, rows, lens, BF, 64)
    assert bool(torch.isnan(want["out"][0, :, 1, 3]).all())
    assert bool(torch.isfinite(want["out"][0, :, 0]).all())


def test_first_calls_within_a_capture(cuda_device):
    """A process whose first call of each kernel is captured."""
    import subprocess
    import sys
    code = """
import torch, block_sparse_gated_gb300 as b
dev = torch.device("cuda:0")
x = torch.randn(2, 48, 1, 64, device=dev).bfloat16()
k = torch.randn(2, 1, 600, 64, device=dev).bfloat16()
cache = b.cache16_empty(20, 1, 64, 64)
table = torch.arange(20, dtype=torch.int32, device=dev).view(2, 10)
n = torch.full((2,), 600, dtype=torch.int32, device=dev)
rope = b.Rope(torch.rand(32, device=dev))
def calls():
    b.cache16_write(cache, k, k, table, rope=rope)
    q, _ = b.rotary(rope, x, start=n - 1)
    return [b.decode16(q[:, :h], cache, table, n)["out"] for h in (1, 16, 48)]
g = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g):
    got = calls()
g.replay()
want = calls()
torch.cuda.synchronize()
assert all(torch.equal(a, c) for a, c in zip(got, want)) and bool(got[2].any())
print("same")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.stdout.strip() == "same", r.stdout + r.stderr


def test_captures_with_copies_forks_and_joins(cuda_device):
    """A decode step whose calls follow copies, each other, other streams' calls and other
    kernels in one graph, replayed back to back on changing data: each sees all before it."""
    b = _bsfa()
    Hq, Hkv, d, page, L = 8, 2, 64, 32, 600
    cache = b.cache16_empty(2 * 32, Hkv, page, d, device=cuda_device)
    other = b.cache16_empty(2 * 32, Hkv, page, d, device=cuda_device)
    table = torch.randperm(64, generator=torch.Generator().manual_seed(1)).to(
        device=cuda_device, dtype=torch.int32).view(2, 32)
    rope = b.Rope(cu.inv_freq(32).to(cuda_device))
    src = [cu.rand((3, 2, h, 1, d), BF, s, cuda_device) for s, h in ((1, Hq), (2, Hkv), (3, Hkv))]
    seen = [cu.rand((2, Hkv, L, d), BF, s, cuda_device) for s in (4, 5)]
    q, k, v = (torch.zeros_like(x[0]) for x in src)
    n32, step = _i32([L, L - 70], cuda_device), torch.zeros(1, dtype=torch.int64, device=cuda_device)
    outs = [torch.zeros(4, 2, Hq, 1, d, dtype=BF, device=cuda_device) for _ in range(2)]
    side = torch.cuda.Stream()

    def body(out):
        for x, y in zip((q, k, v), src):
            x.copy_(y.index_select(0, step % 3)[0])
        # A fork: the second cache on a side stream, which a copy and the first cache's call feed.
        q1 = b.cache16_write(cache, k, v, table, q=q, rope=rope, start=n32)
        at = n32.clone()  # the side stream's own: n32 moves on meanwhile
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            q2 = b.cache16_write(other, k, v, table, q=q, rope=rope, start=at)
        at.record_stream(side)
        n32.add_(1)
        out[0].copy_(b.decode16(q1, cache, table, n32)["out"])
        torch.cuda.current_stream().wait_stream(side)  # a join: two calls before the next
        q2.record_stream(torch.cuda.current_stream())
        back, _ = b.rotary(rope, q2, start=n32 - 1, inverse=True)
        turned, _ = b.rotary(rope, back, start=n32 - 1)
        b.decode16(turned, other, table, n32, max_seqlen=700, out=out[1])
        wide = turned.repeat(1, 5, 1, 1)
        out[2:4].copy_(b.decode16(wide, other, table, n32)["out"][:, :2 * Hq].view(2, 2, Hq, 1, d)
                       .transpose(0, 1))
        out.mul_(0.5)
        step.add_(1)

    def reset():
        for c in (cache, other):
            c.k.zero_(), c.v.zero_()
            b.cache16_write(c, *seen, table, rope=rope)
        n32.copy_(_i32([L, L - 70], cuda_device))
        step.zero_()

    reset()
    want = []
    for _ in range(9):
        body(outs[0])
        torch.cuda.synchronize()
        want.append(outs[0].clone())
    reset()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        body(outs[1])
    reset()
    got = []
    for _ in range(9):  # no waits between the replays
        g.replay()
        got.append(outs[1].clone())
    torch.cuda.synchronize()
    for x, y in zip(want, got):
        assert torch.equal(x, y) and bool(x.any())
    reset()
    for i in range(9):  # nor between calls
        body(outs[0])
        assert torch.equal(outs[0], want[i])


def test_calls_from_several_threads(cuda_device):
    """Each thread on a stream of its own, the same caches read by all."""
    from concurrent.futures import ThreadPoolExecutor
    b = _bsfa()
    lens = [900, 50]
    cache, table, rows = cu.random_cache(b, lens, 32, 2, 64, HF, 6, cuda_device)
    table = widen(table, 32)
    n32 = _i32(lens, cuda_device)
    qs = [_queries(2, 8 * (1 + 9 * (i % 2)), 1, 64, HF, i, cuda_device) for i in range(6)]
    torch.cuda.synchronize()

    def work(q):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                r = b.decode16(q, cache, table, n32, return_lse=True)
        s.synchronize()
        return r

    with ThreadPoolExecutor(6) as ex:
        for q, r in zip(qs, ex.map(work, qs)):
            cu.check_decode(r, q, rows, lens, HF, 64)


def test_the_waits_of_many_query_rows_did_not_run_out(cuda_device):
    from block_sparse_gated_gb300 import api
    assert api.device_error() == 0
