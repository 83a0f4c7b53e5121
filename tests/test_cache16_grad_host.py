"""What rotary positions and cache writes refuse of tensors that require a gradient, without a
GPU: the check comes before the one of the device."""
import pytest
import torch

BF = torch.bfloat16


@pytest.fixture(scope="module")
def b():
    from block_sparse_gated_gb300 import build
    build.build()
    import block_sparse_gated_gb300
    return block_sparse_gated_gb300


def _rows(h, grad=False):
    return torch.zeros(1, h, 5, 64, dtype=BF, requires_grad=grad)


def test_rotary_with_a_gradient_has_no_out(b):
    rope = b.Rope(torch.ones(32))
    q, k = _rows(4), _rows(2)
    for x, y, out in ((_rows(4, True), k, (q.clone(), k.clone())),
                      (q, _rows(2, True), (q.clone(), k.clone())),
                      (q, k, (_rows(4, True), k.clone())),
                      (_rows(4, True), None, (q.clone(), None))):
        with pytest.raises(ValueError, match="out has no gradient"):
            b.rotary(rope, x, y, out=out)
        with torch.no_grad(), pytest.raises(ValueError, match="must be CUDA tensors"):
            b.rotary(rope, x, y, out=out)


def test_rotary_with_a_gradient_is_checked_like_any_call(b):
    rope = b.Rope(torch.ones(32))
    q = _rows(4, True)
    with pytest.raises(ValueError, match="must be CUDA tensors"):
        b.rotary(rope, q)
    with pytest.raises(ValueError, match="shapes disagree"):
        b.rotary(rope, q, torch.zeros(2, 2, 5, 64, dtype=BF))
    with pytest.raises(TypeError, match="k must be a tensor"):
        b.rotary(rope, q, 3)
    with pytest.raises(ValueError, match="inv_freq"):
        b.rotary(b.Rope(torch.ones(32, dtype=torch.float64)), q)


def test_frequencies_have_no_gradient(b):
    """The angles' gradient is not formed: asking for it is refused, not answered with none."""
    rope = b.Rope(torch.ones(32, requires_grad=True))
    with pytest.raises(ValueError, match="inv_freq has no gradient"):
        b.rotary(rope, _rows(4))
    with torch.no_grad(), pytest.raises(ValueError, match="must be CUDA tensors"):
        b.rotary(rope, _rows(4))


def test_cache_writes_record_no_gradient(b):
    cache = b.cache16_empty(1, 2, 16, 64, device="cpu")
    table = torch.zeros(1, 1, dtype=torch.int32)
    rope = b.Rope(torch.ones(32))
    q, k, v = _rows(4), _rows(2), _rows(2)
    for kw in (dict(k=_rows(2, True), v=v), dict(k=k, v=_rows(2, True)),
               dict(k=k, v=v, q=_rows(4, True), rope=rope),
               dict(k=k, v=v, q=q, rope=rope, q_out=_rows(4, True)),
               dict(k=k, v=v, rope=b.Rope(torch.ones(32, requires_grad=True)))):
        k1, v1 = kw.pop("k"), kw.pop("v")
        with pytest.raises(ValueError, match="records no gradient"):
            b.cache16_write(cache, k1, v1, table, **kw)
        with torch.no_grad(), pytest.raises(ValueError, match="must be CUDA tensors"):
            b.cache16_write(cache, k1, v1, table, **kw)
