"""Writing the 4-bit K/V cache and reading it back: codes and scales bit for
bit against the fp64 oracle, whole pools (rows that no token names keep what
they held), and every refusal that needs a device tensor."""
import itertools

import numpy as np
import pytest
import torch

from oracle import cache4_oracle as co
from tests import cache4_util as cu

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def _bsfa():
    import block_sparse_gated_gb300 as b
    return b


def _as_u8(t):
    return t.view(torch.uint8).cpu().numpy()


def _patterns(dtype, n, seed):
    """Random 16-bit patterns as a tensor of ``dtype``, finite ones only."""
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.integers(0, 1 << 16, n, dtype=np.uint16).view(np.int16)).view(dtype)
    return torch.where(torch.isfinite(x), x, torch.zeros_like(x))


def _same_codes(got, want, scale):
    """Equal codes, a zero's sign aside."""
    g = np.stack([got & 15, got >> 4], -1)
    w = np.stack([want & 15, want >> 4], -1)
    g, w = np.where(g == 8, 0, g), np.where(w == 8, 0, w)
    return np.array_equal(g, w)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kind", ["bits", "gauss", "ties", "borders"])
@pytest.mark.parametrize("d", [64, 128])
def test_codes_and_scales_equal_the_oracle(cuda_device, dtype, kind, d):
    """Values over the whole range of the type, gaussians of many scales,
    elements halfway between two codes, and largest magnitudes halfway between
    two scales."""
    b = _bsfa()
    T, H, page = 512, 2, 64
    rng = np.random.default_rng(d)
    if kind == "bits":
        x = _patterns(dtype, 2 * H * T * d, 1).view(2, H, T, d)
    elif kind == "gauss":
        x = rng.standard_normal((2, H, T, d)) * 2.0 ** rng.integers(-14, 9, (2, H, T, 1))
        x = torch.from_numpy(x).to(dtype)
    else:
        # a group: its largest element, then small multiples of its scale
        g = np.zeros((2 * H * T * d // 16, 16))
        byte = rng.integers(8, 0x7E, len(g))
        s = co.E4M3[byte]
        if kind == "borders":  # a / 6 halfway between the scales byte, byte + 1
            g[:, 0] = 6 * (s + co.E4M3[byte + 1 - (byte == 0x7E)]) / 2
            g[:, 1:] = g[:, :1] * rng.random((len(g), 15))
        else:
            g[:, 0] = 6 * s
            mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
            g[:, 1:] = s[:, None] * rng.choice(mids, (len(g), 15))
        g *= rng.choice([-1.0, 1.0], g.shape)
        x = torch.from_numpy(g.reshape(2, H, T, d)).to(dtype)
    k, v = x.to(cuda_device)
    cache = b.cache4_empty(T // page, H, page, d, device=cuda_device)
    table = torch.arange(T // page, dtype=torch.int32, device=cuda_device)[None]
    b.cache4_write(cache, k, v, table)
    for y, codes, scales in ((x[0], cache.k, cache.k_scale), (x[1], cache.v, cache.v_scale)):
        want, byte = co.quantise(y.double().numpy())
        got = codes.transpose(0, 1).reshape(H, T, d // 2).cpu().numpy()
        got_s = _as_u8(scales).transpose(1, 0, 2, 3).reshape(H, T, d // 16)
        assert np.array_equal(got_s, byte)
        assert _same_codes(got, co.pack(want), byte)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_groups_that_are_not_finite_read_as_nan(cuda_device, dtype):
    b = _bsfa()
    x = torch.randn(1, 40, 128, generator=torch.Generator().manual_seed(3)).to(dtype)
    for t, bad in enumerate([float("nan"), float("inf"), -float("inf")]):
        x[0, 3 * t, 16 * t + 5] = bad
    x = x.to(cuda_device)
    cache = b.cache4_empty(1, 1, 48, 128, device=cuda_device)
    table = torch.zeros(1, 1, dtype=torch.int32, device=cuda_device)
    b.cache4_write(cache, x, x, table)
    k, _ = b.cache4_read(cache, table, seqlen=40, dtype=dtype)
    nan = torch.isnan(k[0, 0]).cpu().view(40, 8, 16)
    want = (~torch.isfinite(x[0])).cpu().view(40, 8, 16).any(-1, keepdim=True).expand(40, 8, 16)
    assert torch.equal(nan, want)


def _pool_state(cache):
    """Codes and scale bytes of both pools as [pages, heads, page, row] arrays."""
    out = []
    for t in (cache.k, cache.k_scale, cache.v, cache.v_scale):
        a = _as_u8(t)
        out.append(a if cache.layout == "phtd" else a.transpose(0, 2, 1, 3))
    return out


LENS = [[1], [0, 17, 1, 130], [33, 64, 0, 0, 5], [300]]


@pytest.mark.parametrize("lens,page,layout,rows,dtype,d,exps", [
    (LENS[0], 16, "phtd", "htd", BF, 128, False),
    (LENS[1], 48, "pthd", "thd", HF, 64, True),
    (LENS[1], 16, "phtd", "thd", BF, 128, True),
    (LENS[2], 64, "pthd", "htd", BF, 64, False),
    (LENS[2], 32, "phtd", "htd", HF, 128, True),
    (LENS[3], 256, "pthd", "thd", HF, 128, False),
    (LENS[3], 80, "phtd", "bhld", BF, 64, True),
    ([21, 21, 21], 32, "pthd", "blhd", HF, 128, True),
    ([1, 1, 1, 1, 1], 16, "phtd", "bhld", BF, 128, False),
])
def test_write_and_read_whole_pools(cuda_device, lens, page, layout, rows, dtype, d, exps):
    """A call fills exactly the rows it names, at any start, and a read gives
    them back; packed rows outside the sequences stay as they are."""
    b = _bsfa()
    rng = np.random.default_rng(len(lens) * page + d)
    H, B = 3, len(lens)
    start = rng.integers(0, 2 * page, B).astype(np.int32)
    table, pool = cu.table_for([s + n for s, n in zip(start, lens)], page, rng)
    exp = [torch.tensor([-3, 0, 5], dtype=torch.int32, device=cuda_device) if exps else None] * 2
    cache = b.cache4_empty(pool, H, page, d, layout=layout, k_exp=exp[0], v_exp=exp[1],
                           device=cuda_device)
    for t in cache[:4]:
        t.view(torch.uint8).fill_(0xA5)
    before = [a.copy() for a in _pool_state(cache)]
    e = [-3, 0, 5] if exps else [0, 0, 0]
    varlen = rows in ("htd", "thd")
    lead, tail = (4, 7) if varlen else (0, 0)
    total = lead + sum(lens) + tail
    x = (rng.standard_normal((2, H, total, d)) * 2.0 ** rng.integers(-4, 4, (2, 1, total, 1)))
    x = torch.from_numpy(x).to(dtype)

    def lay(y):  # [H, total, d] -> the call's layout
        if rows == "htd":
            return y
        if rows == "thd":
            return y.transpose(0, 1).contiguous()
        y = y.reshape(H, B, lens[0], d).transpose(0, 1).contiguous()  # bhld
        return y if rows == "bhld" else y.transpose(1, 2).contiguous()

    k, v = (lay(y).to(cuda_device) for y in x)
    offsets = np.cumsum([lead] + lens).astype(np.int32)
    kw = dict(start=torch.from_numpy(start).to(cuda_device), layout=rows)
    if varlen:
        kw["cu_seqlens"] = torch.from_numpy(offsets).to(cuda_device)
    tab = torch.from_numpy(table).to(cuda_device)
    b.cache4_write(cache, k, v, tab, **kw)
    want = before
    stands = np.full((2, H, total, d), np.nan)
    for i, bb, h in itertools.product(range(2), range(B), range(H)):
        for t in range(lens[bb]):
            pos = int(start[bb]) + t
            c, s = co.quantise(x[i, h, offsets[bb] + t].double().numpy(), e[h])
            want[2 * i][table[bb, pos // page], h, pos % page] = co.pack(c)
            want[2 * i + 1][table[bb, pos // page], h, pos % page] = s
            stands[i, h, offsets[bb] + t] = co.values(co.pack(c), s, e[h])
    got = _pool_state(cache)
    for i in range(2):
        assert np.array_equal(got[2 * i + 1], want[2 * i + 1])
        named = want[2 * i] != 0xA5
        assert _same_codes(got[2 * i][named], want[2 * i][named], None)
        assert np.array_equal(got[2 * i][~named], want[2 * i][~named])
    # read: a rectangle or packed rows, into tensors that hold a sentinel
    out = tuple(torch.full_like(y, 7.0) for y in (k, v))
    r = b.cache4_read(cache, tab, out=out, **kw)
    assert r[0] is out[0]
    for i in range(2):
        y = lay(torch.from_numpy(stands[i]))
        y = torch.where(torch.isnan(y), torch.full_like(y, 7.0), y).to(dtype)
        assert torch.equal(out[i].cpu(), y)
    if not varlen:
        fresh = b.cache4_read(cache, tab, seqlen=lens[0], dtype=dtype, **kw)
        assert torch.equal(fresh[0], out[0]) and torch.equal(fresh[1], out[1])


def test_rows_with_gaps_between_them(cuda_device):
    """Inputs and outputs that are slices of larger tensors, and pools whose
    pages lie apart (keys and values interleaved in one allocation)."""
    b = _bsfa()
    H, L, d, page, pool = 2, 75, 128, 32, 4
    gen = torch.Generator().manual_seed(9)
    big = torch.randn(2, L + 9, 3 * H, d + 16, generator=gen).to(BF).to(cuda_device)
    k, v = big[:, 4:L + 4, H:2 * H, 8:d + 8], big[:, 4:L + 4, 2 * H:, 8:d + 8]
    codes = torch.zeros(2 * pool, 2, H, page, d // 2, dtype=torch.uint8, device=cuda_device)
    scales = torch.zeros(2 * pool, 2, H, page, d // 16, dtype=torch.uint8, device=cuda_device)
    scales = scales.view(torch.float8_e4m3fn)
    cache = b.KVCache4(codes[:, 0], codes[:, 1], scales[:, 0], scales[:, 1])
    table = torch.tensor([[6, 0, 3], [2, 7, 1]], dtype=torch.int32, device=cuda_device)
    b.cache4_write(cache, k, v, table, layout="blhd")
    plain = b.cache4_empty(2 * pool, H, page, d, device=cuda_device)
    b.cache4_write(plain, k.contiguous(), v.contiguous(), table, layout="blhd")
    assert torch.equal(cache.k, plain.k) and torch.equal(cache.v, plain.v)
    out = torch.full_like(big, 5.0)
    ko, vo = out[:, 4:L + 4, H:2 * H, 8:d + 8], out[:, 4:L + 4, 2 * H:, 8:d + 8]
    b.cache4_read(cache, table, out=(ko, vo), layout="blhd")
    ref = b.cache4_read(plain, table, seqlen=L, layout="blhd")
    assert torch.equal(ko, ref[0]) and torch.equal(vo, ref[1])
    ko.fill_(5.0), vo.fill_(5.0)
    assert bool((out == 5.0).all())


def test_positions_that_name_no_row(cuda_device):
    """Entries outside the pool and positions beyond the table or before 0: a
    write is dropped, a read gives zeros."""
    b = _bsfa()
    H, d, page = 1, 64, 16
    cache = b.cache4_empty(2, H, page, d, device=cuda_device)
    for t in cache[:4]:
        t.view(torch.uint8).fill_(0x33)
    before = [t.view(torch.uint8).clone() for t in cache[:4]]
    x = torch.randn(3, H, 64, d, generator=torch.Generator().manual_seed(1)).to(HF).to(cuda_device)
    bad = torch.tensor([[-1, 2, 1 << 30, -(1 << 31)]] * 3, dtype=torch.int32, device=cuda_device)
    start = torch.tensor([0, 64, -200], dtype=torch.int32, device=cuda_device)
    b.cache4_write(cache, x, x, bad, start=start)
    far = torch.tensor([64, (1 << 31) - 1, -(1 << 31)], dtype=torch.int32, device=cuda_device)
    good = torch.zeros(3, 4, dtype=torch.int32, device=cuda_device)
    b.cache4_write(cache, x, x, good, start=far)
    assert all(torch.equal(t.view(torch.uint8), u) for t, u in zip(cache[:4], before))
    for table, at in ((bad, start), (good, far)):
        k, v = b.cache4_read(cache, table, seqlen=64, start=at, dtype=HF)
        assert not k.any() and not v.any()
    # the end of a table: rows before it are kept, rows after it dropped
    b.cache4_write(cache, x[:1], x[:1], torch.tensor([[1]], dtype=torch.int32, device=cuda_device),
                   start=torch.tensor([10], dtype=torch.int32, device=cuda_device))
    k, _ = b.cache4_read(cache, torch.tensor([[1]], dtype=torch.int32, device=cuda_device),
                         seqlen=8, start=torch.tensor([10], dtype=torch.int32, device=cuda_device),
                         dtype=HF)
    want = co.values(*[f(y) for f, y in zip((co.pack, np.array),
                                           co.quantise(x[0, 0, :6].double().cpu().numpy()))])
    assert np.array_equal(k[0, 0, :6].double().cpu().numpy(), want)
    assert not k[0, 0, 6:].any()
    assert torch.equal(cache.k[0], before[0][0])


def test_exponent_range_and_rounding_to_the_output_type(cuda_device):
    """Exponents are clamped to [-100, 100]; a value beyond the output type's
    normal range is rounded once (fp16 subnormals) or overflows to infinity."""
    b = _bsfa()
    page = 16
    x = torch.randn(4, 16, 64, generator=torch.Generator().manual_seed(2)).to(BF).to(cuda_device)
    exps = torch.tensor([-127, 100, -16, 4000], dtype=torch.int32, device=cuda_device)
    one = b.cache4_empty(1, 4, page, 64, device=cuda_device)
    table = torch.zeros(1, 1, dtype=torch.int32, device=cuda_device)
    b.cache4_write(one, x, x, table)
    cache = one._replace(k_exp=exps, v_exp=exps)
    for dtype in (BF, HF):
        k, _ = b.cache4_read(cache, table, seqlen=16, dtype=dtype)
        base = b.cache4_read(one, table, seqlen=16, dtype=BF)[0].double()
        f = torch.exp2(exps.clamp(-100, 100).double())[None, :, None, None]
        # through fp32: exact, so still one rounding
        assert torch.equal(k, (base * f).float().to(dtype))


def test_the_largest_batch(cuda_device):
    """One token of each of 4096 sequences, batched and packed."""
    b = _bsfa()
    g = torch.Generator().manual_seed(12)
    x = torch.randn(2, 4096, 1, 1, 64, generator=g).to(HF)
    k, v = x.to(cuda_device)
    start = torch.randint(0, 32, (4096,), generator=g, dtype=torch.int32).to(cuda_device)
    table = torch.randperm(8192, generator=g).to(torch.int32).view(4096, 2).to(cuda_device)
    got = []
    for packed in (False, True):
        cache = b.cache4_empty(8192, 1, 16, 64, device=cuda_device)
        kw = {"start": start}
        if packed:
            kw["cu_seqlens"] = torch.arange(4097, dtype=torch.int32, device=cuda_device)
            b.cache4_write(cache, k.view(1, 4096, 64), v.view(1, 4096, 64), table, **kw)
            got.append(b.cache4_read(cache, table, total=4096, dtype=HF, **kw)[0].view(4096, 64))
        else:
            b.cache4_write(cache, k, v, table, **kw)
            got.append(b.cache4_read(cache, table, seqlen=1, dtype=HF, **kw)[0].view(4096, 64))
        page, row = table.long().gather(1, start.long()[:, None] // 16)[:, 0], start.long() % 16
        codes, scale = cache.k[page, 0, row].cpu().numpy(), _as_u8(cache.k_scale)
        want, byte = co.quantise(x[0].view(4096, 64).double().numpy())
        assert _same_codes(codes, co.pack(want), None)
        assert np.array_equal(scale[page.cpu().numpy(), 0, row.cpu().numpy()], byte)
    assert torch.equal(got[0], got[1])


def test_streams_and_graphs(cuda_device):
    """A side stream, and a captured write-and-read replayed on new data."""
    b = _bsfa()
    H, L, d, page = 2, 100, 128, 32
    gen = torch.Generator().manual_seed(4)
    xs = [torch.randn(1, H, L, d, generator=gen).to(BF).to(cuda_device) for _ in range(3)]
    cache = b.cache4_empty(4, H, page, d, device=cuda_device)
    table = torch.tensor([[2, 0, 3, 1]], dtype=torch.int32, device=cuda_device)
    refs = []
    for x in xs:
        b.cache4_write(cache, x, x, table)
        refs.append(b.cache4_read(cache, table, seqlen=L)[0].clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b.cache4_write(cache, xs[1], xs[1], table, stream=side)
    k, _ = b.cache4_read(cache, table, seqlen=L, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(k, refs[1])
    src = xs[0].clone()
    out = (torch.empty_like(src), torch.empty_like(src))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.cache4_write(cache, src, src, table)
        b.cache4_read(cache, table, out=out)
    for x, ref in zip(xs, refs):
        src.copy_(x)
        graph.replay()
        assert torch.equal(out[0], ref) and torch.equal(out[1], ref)


def test_offsets_beyond_32_bits(cuda_device):
    """Pages more than 4 GiB apart."""
    b = _bsfa()
    H, d, page, L = 1, 128, 32, 70
    step = (1 << 31) + 4096
    raw = torch.empty(2 * step + 65536, dtype=torch.uint8, device=cuda_device)
    codes = raw.as_strided((3, H, page, d // 2), (step, page * d // 2, d // 2, 1))
    codes_v = raw.as_strided((3, H, page, d // 2), (step, page * d // 2, d // 2, 1), 8192)
    scales = raw.as_strided((3, H, page, d // 16), (step, page * d // 16, d // 16, 1), 16384)
    scales_v = raw.as_strided((3, H, page, d // 16), (step, page * d // 16, d // 16, 1), 32768)
    f8 = torch.float8_e4m3fn
    cache = b.KVCache4(codes, codes_v, scales.view(f8), scales_v.view(f8))
    small = b.cache4_empty(3, H, page, d, device=cuda_device)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=cuda_device)
    x = torch.randn(2, 1, H, L, d, generator=torch.Generator().manual_seed(6)).to(BF)
    k, v = x.to(cuda_device)
    q = torch.randn(1, 4, 1, d, generator=torch.Generator().manual_seed(7)).to(BF).to(cuda_device)
    n = torch.tensor([L], dtype=torch.int32, device=cuda_device)
    for c in (cache, small):
        b.cache4_write(c, k, v, table)
    for a, e in zip(b.cache4_read(cache, table, seqlen=L), b.cache4_read(small, table, seqlen=L)):
        assert torch.equal(a, e)
    assert torch.equal(b.decode4(q, cache, table, n)["out"], b.decode4(q, small, table, n)["out"])


def test_packed_offsets_far_below_zero(cuda_device):
    """Rows whose place in their sequence passes 2^31: their positions lie beyond
    the table, whatever the start."""
    b = _bsfa()
    cache = b.cache4_empty(1, 1, 16, 64, device=cuda_device)
    table = torch.zeros(1, 1, dtype=torch.int32, device=cuda_device)
    x = torch.ones(1, 8, 64, dtype=BF, device=cuda_device)
    where = dict(cu_seqlens=torch.tensor([-(1 << 31), 8], dtype=torch.int32, device=cuda_device),
                 start=torch.tensor([(1 << 31) - 1], dtype=torch.int32, device=cuda_device))
    b.cache4_write(cache, x, x, table, **where)
    assert not cache.k.any()
    cache.k.fill_(0x22), cache.k_scale.view(torch.uint8).fill_(0x38)
    k, _ = b.cache4_read(cache, table, total=8, **where)
    assert not k.any()


@pytest.mark.parametrize("layout", ["phtd", "pthd"])
@pytest.mark.parametrize("stride", [0, 1, 8])
def test_pools_of_one_page_and_one_head(cuda_device, layout, stride):
    """The strides of dimensions of one element say nothing."""
    b = _bsfa()
    L, d, page = 40, 128, 48
    g = torch.Generator().manual_seed(6)
    k, v = torch.randn(2, 1, 1, L, d, generator=g).to(BF).to(cuda_device)
    q = torch.randn(1, 4, 1, d, generator=g).to(BF).to(cuda_device)
    table = torch.zeros(1, 1, dtype=torch.int32, device=cuda_device)
    n32 = torch.tensor([L], dtype=torch.int32, device=cuda_device)
    plain = b.cache4_empty(1, 1, page, d, layout=layout, device=cuda_device)
    raw = b.cache4_empty(1, 1, page, d, layout=layout, device=cuda_device)
    head = 1 if layout == "phtd" else 2
    odd = raw._replace(**{n: t.as_strided(t.shape, [stride if i in (0, head) else s
                                                    for i, s in enumerate(t.stride())])
                          for n, t in zip(("k", "v", "k_scale", "v_scale"), raw)})
    got = []
    for c in (plain, odd):
        b.cache4_write(c, k, v, table)
        got.append((*b.cache4_read(c, table, seqlen=L), b.decode4(q, c, table, n32)["out"]))
    assert all(torch.equal(x, y) for x, y in zip(*got))
    for x, y in zip(plain[:4], raw[:4]):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_a_table_of_no_pages(cuda_device):
    """A block table of width 0 names no row: nothing is written, rows read as
    zeros, and a query sees nothing."""
    b = _bsfa()
    cache = b.cache4_empty(2, 2, 16, 64, device=cuda_device)
    table = torch.zeros(3, 0, dtype=torch.int32, device=cuda_device)
    x = torch.ones(3, 2, 5, 64, dtype=BF, device=cuda_device)
    b.cache4_write(cache, x, x, table)
    assert not any(t.view(torch.uint8).any() for t in cache[:4])
    k, v = b.cache4_read(cache, table, seqlen=5)
    assert not k.any() and not v.any()
    q = torch.ones(3, 4, 1, 64, dtype=BF, device=cuda_device)
    res = b.decode4(q, cache, table, torch.tensor([0, 7, 1], dtype=torch.int32, device=cuda_device),
                    return_lse=True)
    assert not res["out"].any() and bool(torch.isneginf(res["lse"]).all())
