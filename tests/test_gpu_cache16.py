"""Rotary positions and writes into the 16-bit cache against the fp64 oracle:
every row, whole pools (rows that no token names keep what they held), and
calls as they are made in earnest."""
import itertools

import numpy as np
import pytest
import torch

from tests import cache16_util as cu
from tests import cache4_util as c4

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def _bsfa():
    import block_sparse_gated_gb300 as b
    return b


def _axes(pairs, n):
    """Pairs of n axes in turn, the first axis with the odd ones out."""
    return None if n == 1 else tuple(int(j * n // pairs) for j in range(pairs))


# (heads q, heads kv, d, pairs, axes, interleaved)
SHAPES = [(8, 2, 128, 64, 1, False), (4, 4, 64, 32, 1, True), (3, 1, 128, 24, 3, False),
          (5, 5, 64, 8, 2, True), (7, 1, 128, 64, 4, True), (1, 1, 64, 24, 1, False),
          (40, 8, 128, 56, 3, True), (2, 2, 64, 16, 2, False)]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("layout", ["bhld", "blhd", "htd", "thd"])
@pytest.mark.parametrize("shape", SHAPES)
def test_rotary_against_the_oracle(cuda_device, shape, layout, inverse):
    """Batched and packed rows, positions by a start or given; packed rows outside the sequences
    stay as they are."""
    b = _bsfa()
    Hq, Hkv, d, P, A, inter = shape
    dtype = BF if (Hq + d) % 3 else HF
    lens = [37] * 3 if layout in ("bhld", "blhd") else [5, 0, 70, 1]
    varlen = layout in ("htd", "thd")
    lead, tail = (3, 4) if varlen else (0, 0)
    total = lead + sum(lens) + tail
    rng = np.random.default_rng(Hq + P)
    start = rng.integers(0, 5000, len(lens))
    own = np.concatenate([s + np.arange(n) for s, n in zip(start, lens)])
    given = rng.integers(-50, 200000, (A, total)) if A > 1 or Hq % 2 else None
    freq = cu.inv_freq(P)
    kw = dict(layout=layout, inverse=inverse)
    if varlen:
        kw["cu_seqlens"] = cu.i32(np.cumsum([lead] + lens).tolist(), cuda_device)
    if given is None:
        kw["start"] = cu.i32(start.tolist(), cuda_device)
    else:
        p = cu.i32(given.tolist(), cuda_device)
        kw["positions"] = p if varlen else p.view(A, 3, 37)
        if A == 1 and Hq % 3 == 0:
            kw["positions"] = kw["positions"][0]
    flat = [cu.rand((h, total, d), dtype, seed) for seed, h in ((1, Hq), (2, Hkv))]

    def lay(x):
        if layout == "htd":
            return x
        if layout == "thd":
            return x.transpose(0, 1).contiguous()
        x = x.view(x.shape[0], 3, 37, d).transpose(0, 1).contiguous()
        return x if layout == "bhld" else x.transpose(1, 2).contiguous()

    def back(y):
        if layout == "htd":
            return y
        if layout == "thd":
            return y.transpose(0, 1)
        y = y if layout == "bhld" else y.transpose(1, 2)
        return y.transpose(0, 1).reshape(y.shape[1], total, d)

    q, k = (lay(x).to(cuda_device) for x in flat)
    out = tuple(torch.full_like(x, 7.0) for x in (q, k))
    rope = b.Rope(freq.to(cuda_device), _axes(P, A), inter)
    res = b.rotary(rope, q, k, out=out, **kw)
    assert res[0] is out[0] and res[1] is out[1]
    inside = slice(lead, total - tail)
    pos = own[None].repeat(A, 0) if given is None else given[:, inside]
    for x, y in zip(flat, out):
        y = back(y).cpu()
        cu.check_rotated(y[:, inside], x[:, inside], pos, freq, axes=_axes(P, A),
                         interleaved=inter, inverse=inverse)
        assert torch.equal(y[:, inside, 2 * P:], x[:, inside, 2 * P:])
        assert bool((y[:, :lead] == 7.0).all() and (y[:, total - tail:] == 7.0).all())
    fresh = b.rotary(rope, q, **kw)
    assert fresh[1] is None
    assert torch.equal(back(fresh[0])[:, inside], back(out[0])[:, inside])
    b.rotary(rope, q, k, out=(q, k), **kw)  # in place
    for x, y in zip((q, k), out):
        assert torch.equal(back(x)[:, inside], back(y)[:, inside])


@pytest.mark.parametrize("length,batch", [(1, 1), (1, 300), (2, 1), (15, 2), (17, 1), (4097, 1)])
def test_rotary_of_every_kind_of_length(cuda_device, length, batch):
    """One token to thousands, by blocks of one head and by blocks of many."""
    b = _bsfa()
    freq = cu.inv_freq(64)
    q = cu.rand((batch, 9, length, 128), BF, 1, cuda_device)
    start = cu.i32([7 * i for i in range(batch)], cuda_device)
    got, _ = b.rotary(b.Rope(freq.to(cuda_device)), q, start=start)
    for i in (0, batch // 2, batch - 1):
        cu.check_rotated(got[i], q[i], 7 * i + np.arange(length)[None], freq)


@pytest.mark.parametrize("far", [1 << 17, 1 << 24, 1 << 30, (1 << 31) - 64, -(1 << 31)])
def test_positions_far_away(cuda_device, far):
    """Angles of positions that fp32 does not hold, from a start and given."""
    b = _bsfa()
    freq = cu.inv_freq(32)
    q = cu.rand((1, 2, 64, 64), HF, 3, cuda_device)
    pos = far + np.arange(64)[None]
    rope = b.Rope(freq.to(cuda_device))
    got, _ = b.rotary(rope, q, positions=cu.i32(pos.tolist(), cuda_device))
    cu.check_rotated(got[0], q[0], pos, freq)
    other, _ = b.rotary(rope, q, start=cu.i32([far], cuda_device))
    assert torch.equal(got, other)


def test_frequencies_of_every_size(cuda_device):
    """Zero, subnormal, above one, negative; an infinity or a NaN gives NaN in its pair alone."""
    b = _bsfa()
    freq = torch.tensor([0.0, 1e-42, 1e-30, 1e-7, 1.0, -0.5, 3.1415927, 100.0], dtype=torch.float32)
    q = cu.rand((1, 1, 500, 64), HF, 5, cuda_device)
    got, _ = b.rotary(b.Rope(freq.to(cuda_device)), q)
    cu.check_rotated(got[0], q[0], np.arange(500)[None], freq)
    freq[2], freq[5] = float("inf"), float("nan")
    bad, _ = b.rotary(b.Rope(freq.to(cuda_device)), q)
    nan = torch.isnan(bad)
    want = torch.zeros_like(nan)
    want[..., [2, 5, 10, 13]] = True
    assert torch.equal(nan, want) and torch.equal(bad[~want], got[~want])


def test_rows_that_are_not_finite(cuda_device):
    """An infinity or a NaN reaches its own pair and nothing else."""
    b = _bsfa()
    rope = b.Rope(cu.inv_freq(16).to(cuda_device))
    q = cu.rand((1, 2, 40, 64), BF, 5, cuda_device)
    clean, _ = b.rotary(rope, q)
    bad = q.clone()
    bad[0, 0, 3, 5], bad[0, 1, 9, 30], bad[0, 1, 9, 50] = float("nan"), float("inf"), float("inf")
    got, _ = b.rotary(rope, bad)
    off = ~torch.isfinite(got)
    want = torch.zeros_like(off)
    want[0, 0, 3, [5, 21]] = want[0, 1, 9, [14, 30, 50]] = True
    assert torch.equal(off, want) and torch.equal(got[~want], clean[~want])
    assert got[0, 1, 9, 50] == float("inf")


def test_the_gradient_against_differences(cuda_device):
    """The inverse call gives the transpose: <g, R (x + e) - R (x - e)> / 2 = <R^T g, e>."""
    b = _bsfa()
    freq = cu.inv_freq(24)
    rope = b.Rope(freq.to(cuda_device), _axes(24, 3), True)
    pos = cu.i32(np.random.default_rng(2).integers(0, 900, (3, 2, 30)).tolist(), cuda_device)
    x, e, g = (cu.rand((2, 3, 30, 64), HF, s, cuda_device) for s in (1, 2, 3))
    grad, _ = b.rotary(rope, g, positions=pos, inverse=True)
    up, _ = b.rotary(rope, x + e, positions=pos)
    down, _ = b.rotary(rope, x - e, positions=pos)
    lhs = (g.double() * (up.double() - down.double())).sum() / 2
    rhs = (grad.double() * e.double()).sum()
    # Each of the n terms of either sum carries a rounding or two of half a step, 2^-11 of a
    # number of size |x| + |e|, times |g| or |e|: independent, so sqrt(n) of them and six sigma.
    n = x.numel()
    size = 6 * 4 * 2.0 ** -11 * n ** 0.5
    assert abs((lhs - rhs).item()) < size and abs(rhs.item()) > 0
    # and it undoes the rotation to two roundings
    again, _ = b.rotary(rope, b.rotary(rope, x, positions=pos)[0], positions=pos, inverse=True)
    two = x.double().abs().max().item() * 2 * 2 ** 0.5 * 2.0 ** -10
    assert (again.double() - x.double()).abs().max().item() < two


def _pool(cache):
    """Both pools as [pages, heads, page, d] arrays of 16-bit patterns."""
    out = []
    for t in (cache.k, cache.v):
        t = t if cache.layout == "phtd" else t.transpose(1, 2)
        out.append(t.contiguous().view(torch.int16).cpu().numpy())
    return out


LENS = [[1], [0, 17, 1, 130], [33, 64, 0, 0, 5], [300]]


@pytest.mark.parametrize("lens,page,layout,rows,dtype,d,pairs,axes", [
    (LENS[0], 16, "phtd", "htd", BF, 128, 64, 1),
    (LENS[1], 48, "pthd", "thd", HF, 64, 32, 3),
    (LENS[1], 16, "phtd", "thd", BF, 128, 24, 1),
    (LENS[2], 64, "pthd", "htd", BF, 64, 0, 1),
    (LENS[2], 32, "phtd", "htd", HF, 128, 64, 2),
    (LENS[3], 256, "pthd", "thd", HF, 128, 40, 1),
    (LENS[3], 80, "phtd", "bhld", BF, 64, 8, 1),
    ([21, 21, 21], 32, "pthd", "blhd", HF, 128, 64, 3),
    ([21, 21, 21], 128, "phtd", "blhd", BF, 64, 0, 1),
    ([1, 1, 1, 1, 1], 16, "phtd", "bhld", BF, 128, 64, 1),
])
@pytest.mark.parametrize("queries", [False, True])
def test_write_whole_pools(cuda_device, lens, page, layout, rows, dtype, d, pairs, axes, queries):
    """A call fills exactly the rows it names, at any start, with what ``rotary`` makes of the
    keys and the values as they are; without a rope, the keys as they are."""
    b = _bsfa()
    rng = np.random.default_rng(len(lens) * page + d)
    Hq, H, B = 6, 3, len(lens)
    start = rng.integers(0, 2 * page, B).astype(np.int32)
    table, pool = c4.table_for([s + n for s, n in zip(start, lens)], page, rng)
    cache = b.cache16_empty(pool, H, page, d, layout=layout, dtype=dtype, device=cuda_device)
    for t in cache[:2]:
        t.fill_(7.0)
    before = _pool(cache)
    varlen = rows in ("htd", "thd")
    lead, tail = (4, 7) if varlen else (0, 0)
    total = lead + sum(lens) + tail
    flat = [cu.rand((h, total, d), dtype, s) for s, h in ((1, Hq), (2, H), (3, H))]

    def lay(y):  # [H, total, d] -> the call's layout
        if rows == "htd":
            return y
        if rows == "thd":
            return y.transpose(0, 1).contiguous()
        y = y.reshape(y.shape[0], B, lens[0], d).transpose(0, 1).contiguous()  # bhld
        return y if rows == "bhld" else y.transpose(1, 2).contiguous()

    q, k, v = (lay(y).to(cuda_device) for y in flat)
    offsets = np.cumsum([lead] + lens).astype(np.int32)
    kw = dict(start=torch.from_numpy(start).to(cuda_device), layout=rows)
    if varlen:
        kw["cu_seqlens"] = torch.from_numpy(offsets).to(cuda_device)
    tab = torch.from_numpy(table).to(cuda_device)
    turn = {}
    if pairs:
        turn["rope"] = b.Rope(cu.inv_freq(pairs).to(cuda_device), _axes(pairs, axes))
        if axes > 1:
            p = cu.i32(rng.integers(0, 4000, (axes, total)).tolist(), cuda_device)
            turn["positions"] = p if varlen else p.view(axes, B, lens[0])
    elif queries:
        pytest.skip("queries are only rotated")
    turned = k
    if pairs:
        rope = turn["rope"]
        q2, turned = b.rotary(rope, q, k, out=(q.clone(), k.clone()), **kw,
                              **{n: x for n, x in turn.items() if n != "rope"})
    if queries:
        q_out = q.clone()
        assert b.cache16_write(cache, k, v, tab, q=q, q_out=q_out, **turn, **kw) is q_out
        assert torch.equal(q_out, q2)
    else:
        assert b.cache16_write(cache, k, v, tab, **turn, **kw) is None
    want = before
    for i, x in enumerate((turned, v)):
        x = x.view(torch.int16).cpu()
        for bb, h in itertools.product(range(B), range(H)):
            for t in range(lens[bb]):
                pos, r = int(start[bb]) + t, int(offsets[bb]) + t
                at = {"htd": (h, r), "thd": (r, h), "bhld": (bb, h, t), "blhd": (bb, t, h)}[rows]
                want[i][table[bb, pos // page], h, pos % page] = x[at].numpy()
    for x, y in zip(_pool(cache), want):
        assert np.array_equal(x, y)


def test_slices_of_one_projection(cuda_device):
    """Queries, keys and values beside each other in one tensor, and pools whose pages lie
    apart (keys and values interleaved in one allocation)."""
    b = _bsfa()
    Hq, H, L, d, page, pool = 4, 2, 75, 128, 32, 8
    fused = cu.rand((2, L, (Hq + 2 * H) * d), BF, 9, cuda_device).view(2, L, Hq + 2 * H, d)
    q, k, v = fused[:, :, :Hq], fused[:, :, Hq:Hq + H], fused[:, :, Hq + H:]
    both = torch.zeros(pool, 2, H, page, d, dtype=BF, device=cuda_device)
    cache = b.KVCache16(both[:, 0], both[:, 1])
    table = cu.i32([[6, 0, 3], [2, 7, 1]], cuda_device)
    rope = b.Rope(cu.inv_freq(64).to(cuda_device))
    got = b.cache16_write(cache, k, v, table, rope=rope, q=q, layout="blhd")
    plain = b.cache16_empty(pool, H, page, d, device=cuda_device)
    ref = b.cache16_write(plain, k.contiguous(), v.contiguous(), table, rope=rope,
                          q=q.contiguous(), layout="blhd")
    assert torch.equal(cache.k, plain.k) and torch.equal(cache.v, plain.v)
    assert torch.equal(got, ref)
    keep = v.clone()
    b.rotary(rope, q, k, out=(q, k), layout="blhd")  # within the projection
    assert torch.equal(q, ref) and torch.equal(v, keep)


def test_positions_that_name_no_row(cuda_device):
    """Entries outside the pool and positions beyond the table or before 0: the write is
    dropped, the queries are rotated all the same."""
    b = _bsfa()
    H, d, page = 1, 64, 16
    cache = b.cache16_empty(2, H, page, d, dtype=HF, device=cuda_device)
    for t in cache[:2]:
        t.fill_(3.0)
    rope = b.Rope(cu.inv_freq(32).to(cuda_device))
    x, q = (cu.rand((3, h, 64, d), HF, h, cuda_device) for h in (H, 2))
    bad = cu.i32([[-1, 2, 1 << 30, -(1 << 31)]] * 3, cuda_device)
    start = cu.i32([0, 64, -200], cuda_device)
    far = cu.i32([64, (1 << 31) - 1, -(1 << 31)], cuda_device)
    good = torch.zeros(3, 4, dtype=torch.int32, device=cuda_device)
    for table, at in ((bad, start), (good, far)):
        got = b.cache16_write(cache, x, x, table, rope=rope, q=q, start=at)
        assert torch.equal(got, b.rotary(rope, q, start=at)[0])
    none = torch.zeros(3, 0, dtype=torch.int32, device=cuda_device)  # a table of no pages
    b.cache16_write(cache, x, x, none)
    assert bool((cache.k == 3.0).all() and (cache.v == 3.0).all())
    # the end of a table: rows before it are kept, rows after it dropped
    b.cache16_write(cache, x[:1], x[:1], cu.i32([[1]], cuda_device), start=cu.i32([10], cuda_device))
    assert torch.equal(cache.k[1, 0, 10:], x[0, 0, :6]) and bool((cache.k[0] == 3.0).all())
    assert bool((cache.k[1, 0, :10] == 3.0).all())


def test_packed_offsets_far_below_zero(cuda_device):
    """Rows whose place in their sequence passes 2^31: their positions lie beyond the table."""
    b = _bsfa()
    cache = b.cache16_empty(1, 1, 16, 64, device=cuda_device)
    x = torch.ones(1, 8, 64, dtype=BF, device=cuda_device)
    b.cache16_write(cache, x, x, cu.i32([[0]], cuda_device),
                    cu_seqlens=cu.i32([-(1 << 31), 8], cuda_device),
                    start=cu.i32([(1 << 31) - 1], cuda_device))
    assert not cache.k.any() and not cache.v.any()


def test_calls_of_no_rows(cuda_device):
    b = _bsfa()
    cache = b.cache16_empty(1, 2, 16, 64, device=cuda_device)
    rope = b.Rope(cu.inv_freq(32).to(cuda_device))
    table = cu.i32([[0]], cuda_device)
    for B, L in ((1, 0), (0, 3)):
        q, k = (torch.ones(B, h, L, 64, dtype=BF, device=cuda_device) for h in (4, 2))
        assert b.rotary(rope, q, k)[0].shape == q.shape
        assert b.cache16_write(cache, k, k, table, rope=rope, q=q).shape == q.shape
    empty = cu.i32([0, 0, 0], cuda_device)  # packed sequences without rows
    k = torch.ones(2, 5, 64, dtype=BF, device=cuda_device)
    b.cache16_write(cache, k, k, table.expand(2, 1).contiguous(), cu_seqlens=empty)
    assert not cache.k.any()


def test_the_largest_batch(cuda_device):
    """One token of each of 4096 sequences, batched and packed; one more is refused."""
    b = _bsfa()
    g = torch.Generator().manual_seed(12)
    k, v = cu.rand((2, 4097, 1, 1, 64), HF, 12, cuda_device)
    start = torch.randint(0, 32, (4097,), generator=g, dtype=torch.int32).to(cuda_device)
    table = torch.randperm(8194, generator=g).to(torch.int32).view(4097, 2).to(cuda_device)
    rope = b.Rope(cu.inv_freq(32).to(cuda_device))
    n = 4096
    turned = b.rotary(rope, k[:n], start=start[:n])[0]
    page, row = table.long().gather(1, start.long()[:, None] // 16)[:n, 0], start.long()[:n] % 16
    for packed in (False, True):
        cache = b.cache16_empty(8194, 1, 16, 64, dtype=HF, device=cuda_device)
        if packed:
            b.cache16_write(cache, k[:n].view(1, n, 64), v[:n].view(1, n, 64), table, rope=rope,
                            start=start[:n],
                            cu_seqlens=torch.arange(n + 1, dtype=torch.int32, device=cuda_device))
        else:
            b.cache16_write(cache, k[:n], v[:n], table, rope=rope, start=start[:n])
        assert torch.equal(cache.k[page, 0, row], turned[:, 0, 0])
        assert torch.equal(cache.v[page, 0, row], v[:n, 0, 0])
        assert cache.v.abs().sum(-1).count_nonzero().item() == n
    with pytest.raises(b.BsfaError, match="unsupported"):
        b.cache16_write(cache, k, v, table)


def test_streams_and_graphs(cuda_device):
    """A side stream, and a captured write replayed at other positions on new data; results on
    another stream have memory of their own."""
    b = _bsfa()
    H, L, d, page = 2, 100, 128, 32
    xs = [cu.rand((1, H, L, d), BF, s, cuda_device) for s in range(3)]
    rope = b.Rope(cu.inv_freq(64).to(cuda_device))
    table = cu.i32([[2, 0, 3, 1, 5, 4, 6]], cuda_device)
    starts = [cu.i32([s], cuda_device) for s in (0, 11, 100)]

    def pools():
        return b.cache16_empty(7, H, page, d, device=cuda_device)

    refs = []
    for x, s in zip(xs, starts):
        c = pools()
        q = b.cache16_write(c, x, x, table, rope=rope, q=x, start=s)
        refs.append((q, c.k, c.v))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    c = pools()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        old = [torch.empty_like(xs[0]) for _ in range(3)]
        torch.cuda._sleep(20_000_000)  # about 10 ms
        for t in old:
            t.fill_(7.0)
        del old, t
        q = b.cache16_write(c, xs[1], xs[1], table, rope=rope, q=xs[1], start=starts[1],
                            stream=side)
        r, _ = b.rotary(rope, xs[2], start=starts[2], stream=side)
        torch.cuda.synchronize()
        assert torch.equal(q, refs[1][0]) and torch.equal(c.k, refs[1][1])
        assert torch.equal(r, refs[2][0])
    src, at, c = xs[0].clone(), starts[0].clone(), pools()
    out = torch.empty_like(src)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.cache16_write(c, src, src, table, rope=rope, q=src, start=at, q_out=out)
    for x, s, ref in zip(xs, starts, refs):
        src.copy_(x)
        at.copy_(s)
        c.k.zero_(), c.v.zero_()
        graph.replay()
        assert torch.equal(out, ref[0]) and torch.equal(c.k, ref[1]) and torch.equal(c.v, ref[2])


def test_offsets_beyond_32_bits(cuda_device):
    """Pages more than 4 GiB apart, and rows of a batch as far from each other."""
    b = _bsfa()
    H, d, page, L = 1, 128, 32, 70
    step = (1 << 31) + 4096  # elements
    raw = torch.empty(2 * step + 65536, dtype=BF, device=cuda_device)
    k_pool = raw.as_strided((3, H, page, d), (step, page * d, d, 1))
    v_pool = raw.as_strided((3, H, page, d), (step, page * d, d, 1), 8192)
    cache = b.KVCache16(k_pool, v_pool)
    small = b.cache16_empty(3, H, page, d, device=cuda_device)
    table = cu.i32([[2, 0, 1]], cuda_device)
    k, v = cu.rand((2, 1, H, L, d), BF, 6, cuda_device)
    q = raw.as_strided((3, 1, 5, d), (step, d, d, 1), 32768)
    q.copy_(cu.rand((3, 1, 5, d), BF, 8, cuda_device))
    rope = b.Rope(cu.inv_freq(64).to(cuda_device))
    for c in (cache, small):
        c.k.zero_(), c.v.zero_()
        b.cache16_write(c, k, v, table, rope=rope)
    assert torch.equal(cache.k, small.k) and torch.equal(cache.v, small.v)
    want, _ = b.rotary(rope, q.contiguous())
    b.rotary(rope, q, out=(q, None))
    assert torch.equal(q, want)


@pytest.mark.parametrize("layout", ["phtd", "pthd"])
@pytest.mark.parametrize("stride", [0, 1, 8])
def test_pools_of_one_page_and_one_head(cuda_device, layout, stride):
    """The strides of dimensions of one element say nothing."""
    b = _bsfa()
    k, v = cu.rand((2, 1, 1, 40, 128), BF, 6, cuda_device)
    table = cu.i32([[0]], cuda_device)
    plain = b.cache16_empty(1, 1, 48, 128, layout=layout, device=cuda_device)
    raw = b.cache16_empty(1, 1, 48, 128, layout=layout, device=cuda_device)
    head = 1 if layout == "phtd" else 2
    odd = raw._replace(**{n: t.as_strided(t.shape, [stride if i in (0, head) else s
                                                    for i, s in enumerate(t.stride())])
                          for n, t in zip(("k", "v"), raw)})
    for c in (plain, odd):
        b.cache16_write(c, k, v, table)
    assert torch.equal(plain.k, raw.k) and torch.equal(plain.v, raw.v)
    assert torch.equal(raw.k.view(48, 128)[:40], k[0, 0])


def test_a_4_bit_cache_of_rotated_keys(cuda_device):
    """The rotation on its own, before a 4-bit cache is written."""
    b = _bsfa()
    q, k, v = (cu.rand((1, h, 90, 64), BF, h, cuda_device) for h in (4, 2, 2))
    rope = b.Rope(cu.inv_freq(32).to(cuda_device))
    table = cu.i32([[0, 1, 2]], cuda_device)
    q2, k2 = b.rotary(rope, q, k)
    cache = b.cache4_empty(3, 2, 32, 64, device=cuda_device)
    b.cache4_write(cache, k2, v, table)
    r, _ = b.cache4_read(cache, table, seqlen=90)
    # e2m1's steps are at most 1/3 of the group's largest value apart
    assert (r - k2).abs().max().item() <= k2.abs().max().item() / 6 * 1.1
    out = b.decode4(q2[:, :, -1:], cache, table, cu.i32([90], cuda_device))["out"]
    assert bool(torch.isfinite(out).all())
