"""Attention of new tokens over the 4-bit cache against the fp64 oracle, with
the elementwise bound that the kernel's arithmetic allows."""
import math

import numpy as np
import pytest
import torch

from tests import cache4_util as cu

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def _bsfa():
    import block_sparse_gated_gb300 as b
    return b


def _queries(B, Hq, n, d, dtype, seed, device, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(B, Hq, n, d, generator=g) * scale).to(dtype).to(device)


def _i32(x, device):
    return torch.tensor(x, dtype=torch.int32, device=device)


# (heads q, heads kv, query tokens): rows of one KV head 1 .. 70, so that every
# width of the query row tile and more than one tile of them occur.
HEADS = [(2, 2, 1), (8, 2, 1), (8, 1, 1), (9, 3, 2), (12, 1, 1), (4, 1, 4), (8, 2, 5), (6, 2, 8),
         (32, 1, 1), (10, 1, 3), (8, 1, 5), (14, 1, 5)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("bound", [256, 1400, 70000])
def test_against_the_oracle(cuda_device, d, heads, bound):
    """Ragged batches, an empty sequence among them, shared by clusters of four
    and eight and cut into pieces; rows past each end hold NaN scales."""
    b = _bsfa()
    Hq, Hkv, n = heads
    lens = [1, 0, 16, 250, 17] if bound == 256 else [700, 1, 0, 64, 1301, 129]
    page, layout = (16, "pthd") if (Hq + d) % 3 == 0 else (48, "phtd")
    dtype = BF if n % 2 else HF
    cache, table, rows = cu.random_cache(b, lens, page, Hkv, d, 10 * Hq + n, cuda_device,
                                         layout=layout, exps=Hkv == 2)
    q = _queries(len(lens), Hq, n, d, dtype, Hq, cuda_device, 1.5)
    table = cu.widen(table, page, bound)
    res = b.decode4(q, cache, table, _i32(lens, cuda_device), return_lse=True, max_seqlen=bound)
    cu.check_decode(res, q, rows, lens, dtype, d)


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 63, 64, 65, 127, 256, 257, 511, 1000])
def test_every_kind_of_length(cuda_device, length):
    """One sequence at tile, unit and page borders: cut into pieces, shared by a
    cluster, by one CTA."""
    b = _bsfa()
    cache, table, rows = cu.random_cache(b, [length], 32, 2, 128, length, cuda_device)
    q = _queries(1, 8, 1, 128, BF, length, cuda_device, 2.0)
    wide = cu.widen(table, 32)
    for most in (70000, 1024, 64, length):
        if most < length:
            continue
        res = b.decode4(q, cache, wide, _i32([length], cuda_device), return_lse=True,
                        max_seqlen=most)
        cu.check_decode(res, q, rows, [length], BF, 128)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n", [1, 3, 33, 100])
def test_queries_longer_than_the_cache(cuda_device, causal, n):
    """Rows that see nothing give zeros and -inf; without the causal mask every
    row sees the whole cache."""
    b = _bsfa()
    lens = [2, 90, 0, 40]
    cache, table, rows = cu.random_cache(b, lens, 16, 2, 64, n, cuda_device)
    q = _queries(4, 4, n, 64, HF, n, cuda_device)
    for t in (table, cu.widen(table, 16)):
        res = b.decode4(q, cache, t, _i32(lens, cuda_device), causal=causal, return_lse=True)
        cu.check_decode(res, q, rows, lens, HF, 64, causal=causal)
    if causal and n > 2:
        assert not res["out"][0, :, :n - 2].any()
        assert bool(torch.isneginf(res["lse"][:, :n - 2]).all())


def test_layouts_strides_and_scale(cuda_device):
    """q and out as [B, n, Hq, d], as slices, with gaps, one sequence in 3-D."""
    b = _bsfa()
    lens, d = [77, 300], 128
    cache, table, rows = cu.random_cache(b, lens, 64, 2, d, 5, cuda_device)
    n32 = _i32(lens, cuda_device)
    big = _queries(2, 5, 12, d + 8, BF, 3, cuda_device)  # [B, tokens, heads + 4, d + 8]
    q = big[:, 1:4, 2:10, 8:]
    out = torch.full((2, 6, 10, d), 3.0, dtype=BF, device=cuda_device)
    res = b.decode4(q, cache, table, n32, layout="blhd", out=out[:, 2:5, 1:9], softmax_scale=0.21,
                    return_lse=True)
    cu.check_decode({"out": res["out"].transpose(1, 2), "lse": res["lse"]}, q.transpose(1, 2),
                    rows, lens, BF, d, sigma=float(np.float32(0.21)))
    keep = torch.ones(2, 6, 10, dtype=torch.bool, device=cuda_device)
    keep[:, 2:5, 1:9] = False
    assert bool((out[keep] == 3.0).all())
    one = b.decode4(q[1].transpose(0, 1), cache, table[1:], n32[1:], softmax_scale=0.21)["out"]
    assert one.shape == (8, 3, d)
    two = b.decode4(q[1:].transpose(1, 2).contiguous(), cache, table[1:], n32[1:],
                    softmax_scale=0.21)["out"][0]
    assert torch.equal(one, two)


def test_lengths_beyond_the_bound_are_cut(cuda_device):
    """Entries of seqlens past max_seqlen, past the table or below zero."""
    b = _bsfa()
    lens = [400, 400, 400, 400]
    cache, table, rows = cu.random_cache(b, lens, 16, 1, 64, 8, cuda_device)
    q = _queries(4, 4, 1, 64, BF, 8, cuda_device)
    given = _i32([400, 1 << 30, -5, -(1 << 31)], cuda_device)
    res = b.decode4(q, cache, table[:, :25], given, max_seqlen=390, return_lse=True)
    cu.check_decode(res, q, rows, [390, 390, 0, 0], BF, 64)


def test_no_length_at_all(cuda_device):
    """A bound of 0: every query sees nothing, whatever seqlens says."""
    b = _bsfa()
    cache, table, _ = cu.random_cache(b, [40, 40], 16, 2, 128, 8, cuda_device)
    q = _queries(2, 8, 3, 128, HF, 8, cuda_device)
    res = b.decode4(q, cache, table, _i32([40, 7], cuda_device), max_seqlen=0, return_lse=True)
    assert not res["out"].any() and bool(torch.isneginf(res["lse"]).all())
    none = b.decode4(q[:, :, :0], cache, table, _i32([40, 7], cuda_device), return_lse=True)
    assert none["out"].shape == (2, 8, 0, 128) and none["lse"].shape == (8, 0)


@pytest.mark.parametrize("cut", [True, False])
def test_the_largest_batch(cuda_device, cut):
    """4096 sequences of 0 to 3 tokens and one of 500; one more is refused."""
    b = _bsfa()
    lens = [int(x) for x in np.random.default_rng(5).integers(0, 4, 4096)]
    lens[2222] = 500
    cache, table, rows = cu.random_cache(b, lens, 16, 1, 64, 2, cuda_device)
    table = cu.widen(table, 16) if cut else table
    q = _queries(4097, 2, 1, 64, BF, 2, cuda_device)
    n32 = _i32(lens + [1], cuda_device)
    res = b.decode4(q[:4096], cache, table, n32[:4096], return_lse=True)
    cu.check_decode(res, q[:4096], rows, lens, BF, 64)
    with pytest.raises(b.BsfaError, match="unsupported"):
        b.decode4(q, cache, torch.cat([table, table[:1]]), n32)


@pytest.mark.parametrize("batch,length,d", [(1, 4097, 128), (2, 3000, 64), (19, 600, 128),
                                            (40, 550, 64), (75, 513, 128), (3, 16000, 64)])
def test_few_sequences_of_some_length(cuda_device, batch, length, d):
    """Wide CTAs in clusters of 8 down to 1, and the lengths' bounds between
    them and the cut."""
    b = _bsfa()
    rng = np.random.default_rng(batch)
    lens = [length] + [int(x) for x in rng.integers(0, length + 1, batch - 1)]
    lens = [x if i < 4 else x % 100 for i, x in enumerate(lens)]
    cache, table, rows = cu.random_cache(b, lens, 32, 2, d, 6, cuda_device)
    q = _queries(batch, 8, 1, d, HF, 6, cuda_device, 1.5)
    res = b.decode4(q, cache, table, _i32(lens, cuda_device), max_seqlen=length, return_lse=True)
    cu.check_decode(res, q, rows, lens, HF, d)


def test_entries_outside_the_pool_read_as_zero_rows(cuda_device):
    """A position whose page does not exist is a zero key and a zero value."""
    b = _bsfa()
    lens = [200]
    cache, table, rows = cu.random_cache(b, lens, 16, 2, 128, 12, cuda_device)
    table[0, 3], table[0, 7], table[0, 12] = -1, cache.k.shape[0], 1 << 30
    for k in rows[0]:
        for j in (3, 7, 12):
            k[:, 16 * j:16 * j + 16] = 0.0
    q = _queries(1, 4, 1, 128, BF, 12, cuda_device)
    res = b.decode4(q, cache, table, _i32(lens, cuda_device), return_lse=True)
    cu.check_decode(res, q, rows, lens, BF, 128)


@pytest.mark.parametrize("where", ["value", "key"])
@pytest.mark.parametrize("d", [64, 128])
def test_nan_rows_reach_only_the_queries_that_see_them(cuda_device, where, d):
    """A group stored as NaN: a value poisons its 16 elements of the queries
    that see the token, a key everything of them; no other query or element."""
    b = _bsfa()
    L, n = 85, 6
    cache, table, rows = cu.random_cache(b, [L], 32, 1, d, 3, cuda_device)
    table = cu.widen(table, 32) if d == 64 else table
    q = _queries(1, 2, n, d, BF, 3, cuda_device)
    clean = b.decode4(q, cache, table, _i32([L], cuda_device), return_lse=True)
    t, group = 82, 2  # seen by queries i with 82 <= 85 - 6 + i, that is i >= 3
    pool = cache.v_scale if where == "value" else cache.k_scale
    pool.view(torch.uint8)[table[0, t // 32].item(), 0, t % 32, group] = 0x7F
    got = b.decode4(q, cache, table, _i32([L], cuda_device), return_lse=True)
    nan = torch.isnan(got["out"])
    want = torch.zeros_like(nan)
    if where == "value":
        want[:, :, 3:, 32:48] = True
        assert torch.equal(got["lse"], clean["lse"])
    else:
        want[:, :, 3:] = True
    assert torch.equal(nan, want)
    assert torch.equal(got["out"][~want], clean["out"][~want])
    # the same token in an older place, seen by all
    pool.view(torch.uint8)[table[0, 0].item(), 0, 4, group] = 0x7F
    got = b.decode4(q, cache, table, _i32([L], cuda_device))
    nan = torch.isnan(got["out"])
    assert bool(nan[..., 32:48].all()) and bool(nan.all()) == (where == "key")


def test_infinite_and_huge_queries(cuda_device):
    """A row with an infinity or a NaN gives NaN (its scores are not numbers);
    rows beside it are untouched; rows of any finite size are exact."""
    b = _bsfa()
    lens = [120]
    cache, table, rows = cu.random_cache(b, lens, 16, 1, 64, 3, cuda_device)
    q = _queries(1, 8, 1, 64, BF, 2, cuda_device)
    clean = b.decode4(q, cache, table, _i32(lens, cuda_device))["out"]
    bad = q.clone()
    bad[0, 1, 0, 7], bad[0, 4, 0, 9] = float("nan"), float("inf")
    got = b.decode4(bad, cache, table, _i32(lens, cuda_device))["out"]
    nan = torch.isnan(got).all(-1)[0, :, 0].tolist()
    assert nan == [i in (1, 4) for i in range(8)]
    assert torch.equal(got[0, [0, 2, 3, 5, 6, 7]], clean[0, [0, 2, 3, 5, 6, 7]])
    for power in (-60, -20, 20, 60):  # the score is the same: q up, sigma down
        r = b.decode4(q * 2.0 ** power, cache, table, _i32(lens, cuda_device),
                      softmax_scale=2.0 ** -power / 8, return_lse=True)
        assert torch.equal(r["out"], clean)


def test_sharp_and_flat_rows(cuda_device):
    """Scores that rise along the sequence by thousands (the reference moves at
    every tile), fall, or are all equal."""
    b = _bsfa()
    L, d = 900, 64
    cache, table, rows = cu.random_cache(b, [L], 16, 1, d, 14, cuda_device)
    q = torch.zeros(1, 4, 1, d, dtype=BF, device=cuda_device)
    q[0, 0] = 400.0
    q[0, 1] = -400.0
    q[0, 2] = 0.0
    q[0, 3] = 3.0
    for t in (table, cu.widen(table, 16)):
        res = b.decode4(q, cache, t, _i32([L], cuda_device), return_lse=True)
        cu.check_decode(res, q, rows, [L], BF, d)


def test_runs_repeat_bit_for_bit_whatever_the_workspace_holds(cuda_device):
    b = _bsfa()
    from block_sparse_gated_gb300 import cache4
    lens = [3000, 10, 777]
    cache, table, rows = cu.random_cache(b, lens, 64, 2, 128, 4, cuda_device)
    table = cu.widen(table, 64)
    q = _queries(3, 16, 1, 128, BF, 4, cuda_device)
    n32 = _i32(lens, cuda_device)
    need = cache4.decode4_workspace_bytes(q, cache, table, n32)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=cuda_device)
    first = b.decode4(q, cache, table, n32, workspace=ws, return_lse=True)
    cu.check_decode(first, q, rows, lens, BF, 128)
    for fill in (0x00, 0x3C, 0xFF):
        ws.fill_(fill)
        again = b.decode4(q, cache, table, n32, workspace=ws, return_lse=True)
        assert torch.equal(again["out"], first["out"]) and torch.equal(again["lse"], first["lse"])
    with pytest.raises(b.BsfaError, match="workspace"):
        b.decode4(q, cache, table, n32, workspace=ws[:need - 256])


@pytest.mark.parametrize("cut", [True, False])
def test_graphs_follow_the_lengths_and_streams_do_not_mix(cuda_device, cut):
    """A captured call reads the lengths at replay; two graphs with workspaces
    of their own run on two streams at once."""
    b = _bsfa()
    from block_sparse_gated_gb300 import cache4
    lens = [2000, 1500]
    cache, table, rows = cu.random_cache(b, lens, 32, 2, 64, 21, cuda_device)
    table = cu.widen(table, 32) if cut else table
    q = [_queries(2, 8, 1, 64, HF, s, cuda_device) for s in (1, 2)]
    n32 = [_i32(lens, cuda_device) for _ in range(2)]
    need = cache4.decode4_workspace_bytes(q[0], cache, table, n32[0])
    assert (need > 0) == cut
    ws = [torch.empty(need, dtype=torch.uint8, device=cuda_device) for _ in range(2)]
    outs = [torch.empty_like(x) for x in q]
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.decode4(q[i], cache, table, n32[i], out=outs[i], workspace=ws[i])
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
    r = b.decode4(q[0], cache, table, n32[0], stream=side)
    side.synchronize()
    assert torch.equal(r["out"], outs[0])


def test_results_on_another_stream_have_memory_of_their_own(cuda_device):
    """Memory that the current stream has given back but still writes is not what
    a call on another stream returns its results in."""
    b = _bsfa()
    cache, table, rows = cu.random_cache(b, [500], 32, 2, 128, 9, cuda_device)
    q = _queries(1, 8, 1, 128, BF, 9, cuda_device)
    n32 = _i32([500], cuda_device)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        old = [torch.empty_like(q), torch.empty(1, 2, 500, 128, dtype=BF, device=cuda_device),
               torch.empty(1, 2, 500, 128, dtype=BF, device=cuda_device)]
        torch.cuda._sleep(20_000_000)  # about 10 ms
        for t in old:
            t.fill_(7.0)
        del old, t
        r = b.decode4(q, cache, table, n32, stream=side, return_lse=True)
        k, v = b.cache4_read(cache, table, seqlen=500, stream=side)
        torch.cuda.synchronize()
        cu.check_decode(r, q, rows, [500], BF, 128)
        assert np.array_equal(k[0].cpu().double().numpy(), rows[0][0])
        assert np.array_equal(v[0].cpu().double().numpy(), rows[0][1])


@pytest.mark.parametrize("cut", [True, False])
def test_a_batch_of_many_short_and_one_long(cuda_device, cut):
    """300 sequences, many of them in one piece and one over many pieces."""
    b = _bsfa()
    lens = [int(x) for x in np.random.default_rng(1).integers(0, 40, 299)] + [5000]
    cache, table, rows = cu.random_cache(b, lens, 16, 1, 64, 2, cuda_device)
    table = cu.widen(table, 16) if cut else table
    q = _queries(300, 2, 1, 64, BF, 2, cuda_device)
    res = b.decode4(q, cache, table, _i32(lens, cuda_device), return_lse=True)
    cu.check_decode(res, q, rows, lens, BF, 64)


def test_prefill_then_decode_as_they_are_used(cuda_device):
    """A prompt's prefill, its keys and values into the cache, then tokens one
    at a time: each is written and attends to everything before it.  The same
    rows read back and given to the prefill agree with the cache's attention
    over all of them."""
    b = _bsfa()
    Hq, Hkv, L, steps, d, page = 8, 2, 300, 5, 128, 128
    g = torch.Generator().manual_seed(31)
    total = L + steps
    q, k, v = (torch.randn(1, h, total, d, generator=g).to(BF).to(cuda_device)
               for h in (Hq, Hkv, Hkv))
    pages = math.ceil(total / page)
    cache = b.cache4_empty(pages, Hkv, page, d, device=cuda_device)
    table = torch.arange(pages, dtype=torch.int32, device=cuda_device).flip(0)[None].contiguous()
    b.prefill(q[:, :, :L], k[:, :, :L], v[:, :, :L], mode="none")
    b.cache4_write(cache, k[:, :, :L], v[:, :, :L], table)
    n32 = _i32([L], cuda_device)
    outs = []
    for i in range(L, total):
        b.cache4_write(cache, k[:, :, i:i + 1], v[:, :, i:i + 1], table, start=n32)
        n32 += 1
        outs.append(b.decode4(q[:, :, i:i + 1], cache, table, n32)["out"])
    kr, vr = b.cache4_read(cache, table, seqlen=total)
    rows = [(kr[0].cpu().double().numpy(), vr[0].cpu().double().numpy())]
    for j, o in enumerate(outs):
        cu.check_decode({"out": o}, q[:, :, L + j:L + j + 1], rows, [L + j + 1], BF, d)
    whole = b.prefill(q, kr, vr, mode="none", return_lse=True)
    chunk = b.decode4(q, cache, table, n32, return_lse=True)
    cu.check_decode(chunk, q, rows, [total], BF, d)
    # two kernels, each within bf16's rounding and the weights' of the truth
    assert (whole["out"].float() - chunk["out"].float()).abs().max().item() < 2e-2
    assert (whole["lse"] - chunk["lse"]).abs().max().item() < 2e-3
    assert torch.equal(chunk["out"][:, :, -1:], outs[-1]) or \
        (chunk["out"][:, :, -1:].float() - outs[-1].float()).abs().max().item() < 2e-2


# Rows of one KV head for each width of the row tile: 4, 8, 12, 20, 32.
WIDTHS = [(8, 2, 1), (16, 2, 1), (12, 1, 1), (4, 1, 5), (32, 1, 1)]


@pytest.mark.parametrize("layout", ["phtd", "pthd"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", WIDTHS)
@pytest.mark.parametrize("bound", [256, 1400, 70000])
def test_both_page_orders_at_every_row_width(cuda_device, layout, d, heads, bound):
    """Pages laid out head first and token first, whatever the heads, by CTAs of
    four and of sixteen warps in clusters and by cut pieces."""
    b = _bsfa()
    Hq, Hkv, n = heads
    lens = [0, 250, 1, 33] if bound == 256 else [1301, 129, 0, 700, 16]
    cache, table, rows = cu.random_cache(b, lens, 32, Hkv, d, Hq + d, cuda_device, layout=layout)
    q = _queries(len(lens), Hq, n, d, HF if d == 64 else BF, Hq, cuda_device, 1.5)
    res = b.decode4(q, cache, cu.widen(table, 32, bound), _i32(lens, cuda_device),
                    max_seqlen=bound, return_lse=True)
    cu.check_decode(res, q, rows, lens, HF if d == 64 else BF, d)


@pytest.mark.parametrize("layout", ["phtd", "pthd"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,n", [(8, 1), (32, 1), (16, 2), (64, 1), (24, 2)])
def test_many_short_sequences(cuda_device, layout, d, Hq, n):
    """800 segments, more than are resident at once: CTAs of two warps, for one,
    four, eight and six query rows of a KV head."""
    b = _bsfa()
    rng = np.random.default_rng(Hq + d)
    lens = [int(x) for x in rng.integers(0, 101, 100)]
    cache, table, rows = cu.random_cache(b, lens, 16, 8, d, 3, cuda_device, layout=layout)
    q = _queries(100, Hq, n, d, BF, Hq, cuda_device, 1.5)
    res = b.decode4(q, cache, table, _i32(lens, cuda_device), return_lse=True)
    cu.check_decode(res, q, rows, lens, BF, d)


@pytest.mark.parametrize("length,Hq,d,layout", [
    (70000, 4, 128, "phtd"), (70000, 12, 64, "pthd"), (70000, 32, 128, "pthd"),
    (150000, 4, 64, "phtd"), (150000, 8, 128, "phtd")])
def test_a_history_of_hundreds_of_parts(cuda_device, length, Hq, d, layout):
    """One sequence of one KV head, four units to a CTA: 276 and 588 parts for one
    block of the join to add."""
    b = _bsfa()
    cache, table, rows = cu.long_cache(b, [length], 64, 1, d, Hq, cuda_device, layout=layout)
    q = _queries(1, Hq, 1, d, BF, Hq, cuda_device, 1.5)
    res = b.decode4(q, cache, table, _i32([length], cuda_device), return_lse=True)
    cu.check_decode(res, q, rows, [length], BF, d)


@pytest.mark.parametrize("Hq,n,d,longest", [(2, 1, 128, 20000), (12, 1, 64, 20000),
                                            (4, 5, 128, 40000), (4, 1, 64, 131000)])
def test_one_long_history_among_many_short_ones(cuda_device, Hq, n, d, longest):
    """300 short sequences make few parts the rule; the long one has 46 to 256,
    which one warp per row adds 32 at a time."""
    b = _bsfa()
    lens = [int(x) for x in np.random.default_rng(Hq).integers(0, 40, 300)]
    lens.insert(123, longest)
    cache, table, rows = cu.long_cache(b, lens, 16, 1, d, Hq, cuda_device)
    q = _queries(301, Hq, n, d, HF, Hq, cuda_device, 1.5)
    res = b.decode4(q, cache, table, _i32(lens, cuda_device), return_lse=True)
    cu.check_decode(res, q, rows, lens, HF, d)


@pytest.mark.parametrize("dtype,power", [(BF, 18), (BF, 22), (BF, 26), (BF, 30), (HF, 15)])
@pytest.mark.parametrize("heads", [(4, 1), (8, 1)])
def test_queries_of_very_different_elements(cuda_device, dtype, power, heads):
    """A row's largest element meets only zeros in the keys, so that the scores
    come from elements that are 2^18 to 2^30 times smaller (in fp16 from 2^-9
    beside 2^15)."""
    b = _bsfa()
    L, d = 300, 128
    cache, table, rows = cu.random_cache(b, [L], 32, 1, d, power, cuda_device)
    cache.k[..., 0] &= 0xF0  # element 0
    rows[0][0][..., 0] = 0.0
    q = _queries(1, heads[0], 1, d, dtype, power, cuda_device, 2.0 ** -9 if dtype == HF else 1.5)
    q[..., 0] = 2.0 ** power
    for t in (table, cu.widen(table, 32)):
        res = b.decode4(q, cache, t, _i32([L], cuda_device), return_lse=True)
        cu.check_decode(res, q, rows, [L], dtype, d, uneven=True)


@pytest.mark.parametrize("power", [-90, -105, -115, -122, -126, -130])
def test_tiny_queries_and_a_large_scale(cuda_device, power):
    """Query rows down to bf16's subnormals, with the softmax scale that makes
    their scores ordinary: they are scaled without losing a bit."""
    b = _bsfa()
    L, d = 200, 64
    cache, table, rows = cu.random_cache(b, [L], 16, 1, d, 7, cuda_device)
    q = (_queries(1, 8, 1, d, BF, 7, "cpu", 1.5).float() * 2.0 ** power).to(BF).to(cuda_device)
    assert q.any()
    sigma = 2.0 ** -power / 8
    for t in (table, cu.widen(table, 16)):
        res = b.decode4(q, cache, t, _i32([L], cuda_device), softmax_scale=sigma, return_lse=True)
        cu.check_decode(res, q, rows, [L], BF, d, sigma=sigma)


def test_zero_keys_of_a_head_with_a_large_exponent(cuda_device):
    """Scores of zero stay zero where the factor from products to scores passes
    fp32's range (queries of 2^120, keys in units of 2^100): equal weights."""
    b = _bsfa()
    L, d, page = 40, 64, 16
    big = torch.tensor([100], dtype=torch.int32, device=cuda_device)
    cache = b.cache4_empty(3, 1, page, d, k_exp=big, device=cuda_device)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=cuda_device)
    g = torch.Generator().manual_seed(3)
    v = torch.randn(1, 1, L, d, generator=g).to(BF).to(cuda_device)
    b.cache4_write(cache, torch.zeros_like(v), v, table)
    _, v = b.cache4_read(cache, table, seqlen=L)
    rows = [(np.zeros((1, L, d)), v[0].cpu().double().numpy())]
    q = (_queries(1, 4, 1, d, BF, 3, cuda_device) * 2.0 ** 120)
    res = b.decode4(q, cache, table, _i32([L], cuda_device), return_lse=True)
    cu.check_decode(res, q, rows, [L], BF, d)


def test_a_launch_that_failed_leaves_no_error_behind(cuda_device):
    """The runtime refuses a launch on the legacy stream while this thread
    captures a blocking stream; the calls after it answer for themselves."""
    import ctypes
    b = _bsfa()
    cache, table, rows = cu.random_cache(b, [100], 16, 2, 64, 5, cuda_device)
    q = _queries(1, 4, 1, 64, BF, 5, cuda_device)
    n32, out = _i32([100], cuda_device), torch.empty_like(q)
    x = torch.zeros(1, 2, 10, 64, dtype=BF, device=cuda_device)
    b.decode4(q, cache, table, n32, out=out)
    torch.cuda.synchronize()
    with open("/proc/self/maps") as f:  # the runtime that torch has loaded
        rt = ctypes.CDLL(next(line.split()[-1] for line in f if "libcudart" in line))
    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert rt.cudaStreamCreate(ctypes.byref(stream)) == 0
    assert rt.cudaStreamBeginCapture(stream, 0) == 0
    try:
        with pytest.raises(b.BsfaError) as e:
            b.decode4(q, cache, table, n32, out=out, stream=torch.cuda.default_stream())
    finally:
        rt.cudaStreamEndCapture(stream, ctypes.byref(graph))
        rt.cudaGetLastError()
        rt.cudaStreamDestroy(stream)
    assert e.value.status == 3
    spare = b.cache4_empty(1, 2, 16, 64, device=cuda_device)
    b.cache4_write(spare, x, x, torch.zeros(1, 1, dtype=torch.int32, device=cuda_device))
    cu.check_decode(b.decode4(q, cache, table, n32), q, rows, [100], BF, 64)


@pytest.mark.parametrize("layout", ["phtd", "pthd"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", [(4, 1), (8, 1), (12, 1), (4, 5), (32, 1)])
def test_pieces_of_more_than_one_run(cuda_device, layout, d, heads):
    """650 histories of 20000 to 40000 tokens, read from the same pages: a CTA's
    piece of a history is longer than what is summed at once, with histories that
    begin and end within pieces."""
    b = _bsfa()
    Hq, n = heads
    rng = np.random.default_rng(Hq + d)
    cache, table, rows = cu.long_cache(b, [40000], 64, 1, d, Hq, cuda_device, layout=layout)
    lens = [int(x) for x in rng.integers(20000, 40001, 650)]
    q = _queries(650, Hq, n, d, HF, Hq, cuda_device, 1.5)
    res = b.decode4(q, cache, table.repeat(650, 1), _i32(lens, cuda_device), return_lse=True)
    some = [0, 1, 314, 649]
    lse = res["lse"].view(Hq, 650, n)
    for i in some:
        cu.check_decode({"out": res["out"][i:i + 1], "lse": lse[:, i]}, q[i:i + 1], rows,
                        [lens[i]], HF, d)


def test_sums_of_a_million_values_of_one_sign(cuda_device):
    """640 histories of 2^20 tokens, read from the same pages, each the work of
    about one CTA: the tensor cores' sums do not fall behind."""
    b = _bsfa()
    L, d, B = 1 << 20, 64, 640
    cache, table, rows = cu.long_cache(b, [L], 256, 1, d, 5, cuda_device, positive=True)
    q = _queries(1, 1, 1, d, HF, 5, cuda_device, 0.3)
    res = b.decode4(q.repeat(B, 1, 1, 1), cache, table.repeat(B, 1), _i32([L] * B, cuda_device),
                    return_lse=True)
    cu.check_decode({"out": res["out"][:1], "lse": res["lse"][:, :1]}, q, rows, [L], HF, d)
    # The others are the same sum, cut elsewhere.  Output and weights are rounded to
    # fp16 (2^-11 each), and a run of 256 tiles is 512 products added, each cut by less
    # than 2^-23 of the sum (2^-14).  In the mean over 64 elements the roundings leave
    # 2^-11 / sqrt(3 * 64) beside that.
    want = rows[0][1][0].T @ _softmax(rows[0][0][0] @ q[0, 0, 0].cpu().double().numpy() / 8)
    off = res["out"][:, 0, 0].cpu().double().numpy() / want - 1
    assert abs(off).max() <= 2 * 2.0 ** -11 + 2.0 ** -14
    assert abs(off.mean()) <= 3 * 2.0 ** -11 / math.sqrt(3 * 64) + 2.0 ** -14


def _softmax(s):
    p = np.exp(s - s.max())
    return p / p.sum()


def test_graphs_follow_the_lengths_over_more_than_one_run(cuda_device):
    """A captured call whose bound allows long pieces, replayed for long histories
    and for short ones, with another call on another stream beside it."""
    b = _bsfa()
    from block_sparse_gated_gb300 import cache4
    B, d = 650, 64
    cache, table, rows = cu.long_cache(b, [30000], 64, 1, d, 8, cuda_device)
    table = table.repeat(B, 1)
    q = [_queries(B, 4, 1, d, HF, s, cuda_device) for s in (1, 2)]
    n32 = _i32([30000] * B, cuda_device)
    need = cache4.decode4_workspace_bytes(q[0], cache, table, n32)
    outs, graphs, ws = [torch.empty_like(x) for x in q], [], []
    for i in range(2):
        ws.append(torch.empty(need, dtype=torch.uint8, device=cuda_device))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.decode4(q[i], cache, table, n32, out=outs[i], workspace=ws[i])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    rng = np.random.default_rng(8)
    for lo, hi in ((25000, 30001), (0, 40), (0, 30001)):
        now = [int(x) for x in rng.integers(lo, hi, B)]
        n32.copy_(_i32(now, cuda_device))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            for j in (0, 77, 649):
                cu.check_decode({"out": outs[i][j:j + 1]}, q[i][j:j + 1], rows, [now[j]], HF, d)
