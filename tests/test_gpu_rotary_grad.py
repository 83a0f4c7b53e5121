"""The gradient of rotated rows, by autograd, and the versions of tensors written in place."""
import pytest
import torch

from tests import cache16_util as cu

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def _bsfa():
    import block_sparse_gated_gb300 as b
    return b


def _plain(x, pos, freq, interleaved):
    """x [.., L, d] rotated at pos [.., L] in fp64, by elementary operations of torch."""
    P = freq.numel()
    a = pos.double()[..., None] * freq.double()
    c, s = a.cos(), a.sin()
    pairs = x[..., :2 * P]
    u, v = (pairs[..., 0::2], pairs[..., 1::2]) if interleaved else pairs.split(P, -1)
    y, z = u * c - v * s, v * c + u * s
    y = torch.stack([y, z], -1).flatten(-2) if interleaved else torch.cat([y, z], -1)
    return torch.cat([y, x[..., 2 * P:]], -1)


@pytest.mark.parametrize("layout", ["bhld", "blhd"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_gradients_of_queries_and_keys(cuda_device, layout, interleaved, inverse):
    """Against the plain formula's in 64 bits, for gradients of the rotated rows that are dense,
    broadcast, and given to one of the two only."""
    b = _bsfa()
    freq = cu.inv_freq(24)
    rope = b.Rope(freq.to(cuda_device), None, interleaved)
    start = cu.i32([5, 1000], cuda_device)
    shape = {"bhld": lambda h: (2, h, 37, 64), "blhd": lambda h: (2, 37, h, 64)}[layout]
    q = cu.rand(shape(6), HF, 1, cuda_device).requires_grad_()
    k = cu.rand(shape(2), HF, 2, cuda_device).requires_grad_()
    pos = (start[:, None] + torch.arange(37, device=cuda_device)) * (-1 if inverse else 1)
    pos = pos[:, None] if layout == "bhld" else pos[:, :, None]
    q64, k64 = (x.detach().double().requires_grad_() for x in (q, k))
    kw = dict(start=start, layout=layout, inverse=inverse)

    def close(got, want):
        # One rounding of a rotation, half a step of it, and 2^-21 of |a| + |b| before it.
        tol = want.abs() * 2.0 ** -11 + want.abs().max() * 2.0 ** -20 + 2.0 ** -24
        assert got.dtype == HF and bool(((got.double() - want).abs() <= tol).all())

    freq64 = freq.to(cuda_device)
    for x, x64, other in ((q, q64, k), (k, k64, q)):
        g = cu.rand(x.shape, HF, 3, cuda_device)
        want = torch.autograd.grad(_plain(x64, pos, freq64, interleaved), x64, g.double())[0]
        turned = b.rotary(rope, q, k, **kw)
        close(torch.autograd.grad(turned[0 if x is q else 1], x, g)[0], want)
        assert turned[0].requires_grad and turned[1].requires_grad
        wide = torch.ones((), dtype=HF, device=cuda_device).expand(x.shape)  # as of a sum
        want = torch.autograd.grad(_plain(x64, pos, freq64, interleaved), x64, wide.double())[0]
        turned = b.rotary(rope, q, k, **kw)
        close(torch.autograd.grad(turned[0 if x is q else 1], x, wide)[0], want)
    # Both at once, into .grad; the rotated rows are those of a call without a graph.
    turned = b.rotary(rope, q, k, **kw)
    with torch.no_grad():
        plain = b.rotary(rope, q, k, **kw)
    assert not plain[0].requires_grad
    assert all(torch.equal(x.detach(), y) for x, y in zip(turned, plain))
    (turned[0].float().square().sum() + turned[1].float().square().sum()).backward()
    for x in (q, k):  # lengths do not change as rows turn: the gradient of the squares is 2 x
        off = (x.grad.double() - 2 * x.detach().double()).abs()
        # two roundings and the doubled gradient's own
        size = x.detach().double().abs().max()
        assert bool((off <= 3 * 2 * size * 2 ** 0.5 * 2.0 ** -11).all())
    # One of the two without a gradient, and no keys at all.
    turned = b.rotary(rope, q.detach(), k, **kw)
    assert torch.autograd.grad(turned[1].float().sum(), k)[0].shape == k.shape
    alone = b.rotary(rope, q, **kw)
    assert alone[1] is None
    assert torch.autograd.grad(alone[0].float().sum(), q)[0].shape == q.shape


@pytest.mark.parametrize("layout", ["htd", "thd"])
def test_gradients_of_packed_rows(cuda_device, layout):
    """Rows outside every sequence have no part in the result: their gradient is zero.  Positions
    on three axes."""
    b = _bsfa()
    freq = cu.inv_freq(32)
    axes = [j % 3 for j in range(32)]
    rope = b.Rope(freq.to(cuda_device), axes)
    T, cu_seqlens = 60, cu.i32([4, 4, 30, 51], cuda_device)
    positions = torch.randint(0, 500, (3, T), device=cuda_device, dtype=torch.int32)
    q = cu.rand((3, T, 64) if layout == "htd" else (T, 3, 64), BF, 1, cuda_device).requires_grad_()
    kw = dict(positions=positions, cu_seqlens=cu_seqlens, layout=layout)
    g = cu.rand(q.shape, BF, 2, cuda_device)
    turned, _ = b.rotary(rope, q, **kw)
    got = torch.autograd.grad(turned, q, g)[0]
    rows = got if layout == "htd" else got.transpose(0, 1)
    g = g if layout == "htd" else g.transpose(0, 1)
    inside = slice(4, 51)
    assert not rows[:, :4].any() and not rows[:, 51:].any()
    cu.check_rotated(rows[:, inside], g[:, inside], positions.cpu().numpy()[:, inside], freq,
                     axes=axes, inverse=True)


def test_gradients_of_gradients_and_of_changed_positions(cuda_device):
    """The gradient's own gradient is the rotation; a position tensor changed between the two
    passes is told, not used."""
    b = _bsfa()
    rope = b.Rope(cu.inv_freq(32).to(cuda_device))
    q = cu.rand((1, 2, 9, 64), BF, 1, cuda_device).requires_grad_()
    start = cu.i32([3], cuda_device)
    g = cu.rand(q.shape, BF, 2, cuda_device).requires_grad_()
    turned, _ = b.rotary(rope, q, start=start)
    back = torch.autograd.grad(turned, q, g, create_graph=True)[0]
    h = cu.rand(q.shape, BF, 3, cuda_device)
    again = torch.autograd.grad(back, g, h)[0]
    assert torch.equal(again, b.rotary(rope, h, start=start)[0])
    turned, _ = b.rotary(rope, q, start=start)
    start += 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        turned.float().sum().backward()


def test_gradients_of_queries_that_are_keys(cuda_device):
    """One tensor given twice gets both gradients."""
    b = _bsfa()
    rope = b.Rope(cu.inv_freq(32).to(cuda_device))
    x = cu.rand((1, 2, 9, 64), BF, 1, cuda_device).requires_grad_()
    a, c = b.rotary(rope, x, x)
    g, h = (cu.rand(x.shape, BF, s, cuda_device) for s in (2, 3))
    got = torch.autograd.grad([a, c], x, [g, h])[0]
    one, two = (b.rotary(rope, y, inverse=True)[0] for y in (g, h))
    assert torch.equal(got, one + two)


def test_gradients_within_a_captured_graph(cuda_device):
    """Both passes captured, replayed on other data."""
    b = _bsfa()
    rope = b.Rope(cu.inv_freq(32).to(cuda_device))
    q = cu.rand((2, 4, 50, 64), BF, 1, cuda_device).requires_grad_()
    g = cu.rand(q.shape, BF, 2, cuda_device)

    def both():
        turned, _ = b.rotary(rope, q)
        return turned, torch.autograd.grad(turned, q, g)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    with torch.no_grad():
        q.copy_(cu.rand(q.shape, BF, 3, cuda_device))
        g.copy_(cu.rand(q.shape, BF, 4, cuda_device))
    graph.replay()
    want = both()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_a_gradient_step_by_differences(cuda_device):
    """The loss's change along a direction is the gradient's product with it: L(x) = <w, R x> is
    linear, so the difference is exact up to the roundings of the rotated rows."""
    b = _bsfa()
    rope = b.Rope(cu.inv_freq(32).to(cuda_device))
    x, e, w = (cu.rand((2, 3, 30, 64), HF, s, cuda_device) for s in (1, 2, 3))
    x.requires_grad_()
    turned, _ = b.rotary(rope, x)
    grad = torch.autograd.grad((turned.double() * w.double()).sum(), x)[0]
    with torch.no_grad():
        up, down = b.rotary(rope, x + e)[0], b.rotary(rope, x - e)[0]
    lhs = (w.double() * (up.double() - down.double())).sum() / 2
    rhs = (grad.double() * e.double()).sum()
    # As in the test of the inverse call: sqrt(n) roundings of half a step, six sigma.
    assert abs((lhs - rhs).item()) < 6 * 4 * 2.0 ** -11 * x.numel() ** 0.5
    assert abs(rhs.item()) > 0


def test_writes_in_place_are_counted(cuda_device):
    """What a call writes has a new version, so that a graph that keeps the old contents is told;
    tensors made for inference have none."""
    b = _bsfa()
    rope = b.Rope(cu.inv_freq(32).to(cuda_device))
    q, k = (cu.rand((1, h, 40, 64), BF, h, cuda_device) for h in (4, 2))
    cache = b.cache16_empty(3, 2, 16, 64, device=cuda_device)
    table = torch.arange(3, dtype=torch.int32, device=cuda_device)[None]
    n32 = cu.i32([40], cuda_device)
    out = [torch.empty_like(x) for x in (q, k)]

    def versions():
        return [x._version for x in (*out, cache.k, cache.v, q, k)]

    was = versions()
    b.rotary(rope, q, k, out=out)
    assert versions() == [was[0] + 1, was[1] + 1, *was[2:]]
    b.cache16_write(cache, k, k, table, rope=rope, q=q, q_out=out[0])
    assert versions() == [was[0] + 2, was[1] + 1, was[2] + 1, was[3] + 1, *was[4:]]
    b.decode16(q, cache, table, n32, out=out[0])
    assert versions() == [was[0] + 3, was[1] + 1, was[2] + 1, was[3] + 1, *was[4:]]
    w = torch.ones(q.shape, device=cuda_device, dtype=BF, requires_grad=True)
    y = w * out[0]
    b.rotary(rope, q, out=(out[0], None))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    with torch.inference_mode():
        made = [torch.empty_like(q), torch.empty_like(k)]
        store = b.cache16_empty(3, 2, 16, 64, device=cuda_device)
        b.rotary(rope, q, k, out=made)
    b.rotary(rope, q, k, out=made)
    b.cache16_write(store, k, k, table, rope=rope)
    assert torch.equal(made[0], b.rotary(rope, q)[0])
