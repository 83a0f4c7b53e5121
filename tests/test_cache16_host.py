"""Rotary positions and the 16-bit cache without a GPU: the C structs' layout, what
the library and the binding refuse before anything is launched, and the fp64
oracle against hand-written values."""
import ctypes
import os
import subprocess
import tempfile

import numpy as np
import pytest
import torch

from oracle import rotary_oracle as ro
from tests import cache16_util as cu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 5
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def lib():
    from block_sparse_gated_gb300 import _native, build
    build.build()
    return _native.lib()


def _native():
    from block_sparse_gated_gb300 import _native
    return _native


def _bsfa():
    import block_sparse_gated_gb300 as b
    return b


def _set(s, kw):
    for n, x in kw.items():
        setattr(s, n, x)
    return s


def _cache(**kw):
    """A valid descriptor of "phtd" pools whose pointers are never read."""
    c = _native().Cache16()
    c.k = c.v = c.block_table = 1 << 20
    c.k_stride[:] = c.v_stride[:] = (2 * 64 * 128, 64 * 128, 128)
    c.num_pages, c.page_size, c.num_heads_kv, c.head_dim = 10, 64, 2, 128
    c.block_table_stride = c.block_table_width = 4
    return _set(c, kw)


def _rope(**kw):
    r = _native().Rope()
    r.inv_freq, r.pairs, r.num_axes = 1 << 20, 64, 1
    return _set(r, kw)


def _rows(**kw):
    r = _native().Rows16()
    r.q = r.k = r.v = r.q_out = r.k_out = 1 << 20
    for s in (r.q_stride, r.q_out_stride):
        s[:] = (8 * 100 * 128, 100 * 128, 128)
    for s in (r.k_stride, r.v_stride, r.k_out_stride):
        s[:] = (2 * 100 * 128, 100 * 128, 128)
    r.batch, r.num_heads_q, r.num_heads_kv, r.seqlen, r.head_dim = 3, 8, 2, 100, 128
    return _set(r, kw)


def test_struct_layouts_match_the_header():
    src = r'''
#include <stddef.h>
#include <stdio.h>
#include "bsfa.h"
int main(void) {
  printf("%zu %zu %zu %zu ", sizeof(bsfa_cache16), offsetof(bsfa_cache16, num_pages),
         offsetof(bsfa_cache16, block_table), offsetof(bsfa_cache16, dtype));
  printf("%zu %zu %zu %zu ", sizeof(bsfa_rope), offsetof(bsfa_rope, position_stride),
         offsetof(bsfa_rope, num_axes), offsetof(bsfa_rope, axis));
  printf("%zu %zu %zu %zu %d\n", sizeof(bsfa_rows16), offsetof(bsfa_rows16, k_out_stride),
         offsetof(bsfa_rows16, cu_seqlens), offsetof(bsfa_rows16, dtype), BSFA_ROPE_MAX_AXES);
  return 0;
}
'''
    with tempfile.TemporaryDirectory() as tmp:
        c, exe = os.path.join(tmp, "probe.c"), os.path.join(tmp, "probe")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        got = tuple(map(int, subprocess.run([exe], capture_output=True, text=True,
                                            check=True).stdout.split()))
    from block_sparse_gated_gb300 import cache16
    n = _native()
    C, P, R = n.Cache16, n.Rope, n.Rows16
    assert (n.CACHE16.size, n.ROPE.size, n.ROWS16.size) == tuple(map(ctypes.sizeof, (C, P, R)))
    assert got == (ctypes.sizeof(C), C.num_pages.offset, C.block_table.offset, C.dtype.offset,
                   ctypes.sizeof(P), P.position_stride.offset, P.num_axes.offset, P.axis.offset,
                   ctypes.sizeof(R), R.k_out_stride.offset, R.cu_seqlens.offset, R.dtype.offset,
                   cache16.MAX_AXES)


def _write(lib, c, rope, r):
    by = [None if x is None else ctypes.byref(x) for x in (c, rope, r)]
    return lib.bsfa_cache16_write(*by, None)


def _rotary(lib, rope, r):
    return lib.bsfa_rotary(None if rope is None else ctypes.byref(rope),
                           None if r is None else ctypes.byref(r), None)


def _decode(**kw):
    p = _native().Decode4Params()
    p.q = p.o = p.seqlens = 1 << 20
    p.q_stride[:] = p.o_stride[:] = (8 * 128, 128, 128)
    p.batch, p.num_heads_q, p.q_len, p.max_seqlen = 3, 8, 1, 256
    return _set(p, kw)


@pytest.mark.parametrize("change,status", [
    (dict(head_dim=96), UNSUPPORTED), (dict(page_size=24), UNSUPPORTED),
    (dict(page_size=0), INVALID), (dict(num_pages=0), INVALID), (dict(num_heads_kv=0), INVALID),
    (dict(block_table_width=5), INVALID), (dict(block_table_width=-1), INVALID),
    (dict(block_table_width=(1 << 24) + 1, block_table_stride=1 << 25), UNSUPPORTED),
    (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(block_table=0), INVALID),
    (dict(k=(1 << 20) + 8), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED),
])
def test_cache_descriptors_that_are_refused(lib, change, status):
    r = _rows(head_dim=change.get("head_dim", 128))
    want = UNSUPPORTED if "head_dim" in change else status
    assert _write(lib, _cache(**change), _rope(pairs=32), r) == want
    c, p = _cache(**change), _decode()
    assert lib.bsfa_decode16(ctypes.byref(c), ctypes.byref(p), None) == status


def test_cache_strides_that_are_refused(lib):
    for field, i, bad in (("k_stride", 0, 64 * 128 + 4), ("v_stride", 2, 0), ("k_stride", 1, -64),
                          ("v_stride", 2, 1 << 24), ("k_stride", 2, 1 << 24)):
        c = _cache()
        getattr(c, field)[i] = bad
        assert _write(lib, c, _rope(), _rows()) == UNSUPPORTED
        p = _decode()
        assert lib.bsfa_decode16(ctypes.byref(c), ctypes.byref(p), None) == UNSUPPORTED


def test_decode_parameters_that_are_refused(lib):
    c = ctypes.byref(_cache())
    size = lib.bsfa_decode16_workspace_size
    for change, status in ((dict(num_heads_q=7), INVALID), (dict(num_heads_q=0), INVALID),
                           (dict(batch=-1), INVALID), (dict(q_len=-1), INVALID),
                           (dict(max_seqlen=-1), INVALID), (dict(max_seqlen=257), INVALID),
                           (dict(dtype=3), UNSUPPORTED), (dict(dtype=1), INVALID),
                           (dict(batch=4097), UNSUPPORTED), (dict(q_len=1 << 27), UNSUPPORTED),
                           (dict(batch=4096, q_len=1 << 22), UNSUPPORTED)):
        p = _decode(**change)
        assert lib.bsfa_decode16(c, ctypes.byref(p), None) == status, change
        assert size(c, ctypes.byref(p)) == 0, change
    long = _cache(block_table_width=2000, block_table_stride=2000)
    c2 = ctypes.byref(long)  # a bound this long needs a workspace
    need = size(c2, ctypes.byref(_decode(max_seqlen=100000)))
    assert need > 0 and size(c2, ctypes.byref(_decode(max_seqlen=256))) == 0
    for change, status in ((dict(q=0), INVALID), (dict(seqlens=0), INVALID),
                           (dict(o=(1 << 20) + 8), UNSUPPORTED), (dict(), WORKSPACE),
                           (dict(workspace=128, workspace_bytes=1 << 30), WORKSPACE),
                           (dict(workspace=1 << 20, workspace_bytes=0), WORKSPACE),
                           (dict(workspace=1 << 20, workspace_bytes=need - 1), WORKSPACE)):
        p = _decode(max_seqlen=100000, **change)
        assert lib.bsfa_decode16(c2, ctypes.byref(p), None) == status, change
    p = _decode(max_seqlen=100000)
    p.q_stride[1] = 4
    assert lib.bsfa_decode16(c2, ctypes.byref(p), None) == UNSUPPORTED
    p = _decode(max_seqlen=100000)
    p.q_stride[2] = 3  # the only token's stride says nothing
    assert lib.bsfa_decode16(c2, ctypes.byref(p), None) == WORKSPACE
    for empty in (dict(batch=0), dict(q_len=0)):
        p = _decode(q=0, o=0, **empty)
        assert lib.bsfa_decode16(c, ctypes.byref(p), None) == OK
    assert lib.bsfa_decode16(None, ctypes.byref(p), None) == INVALID
    assert lib.bsfa_decode16(c, None, None) == INVALID


def test_strides_of_one_element_dimensions_say_nothing(lib):
    """A pool of one page and one head is not refused for strides that no call multiplies by
    anything but 0; of two, it is."""
    for pages, heads, status in ((1, 1, WORKSPACE), (2, 1, UNSUPPORTED), (1, 2, UNSUPPORTED)):
        c = _cache(num_pages=pages, num_heads_kv=heads, block_table_width=2000,
                   block_table_stride=2000)
        for s in (c.k_stride, c.v_stride):
            if pages == 1:
                s[0] = 1
            if heads == 1:
                s[1] = 0
        if pages == 2:
            c.k_stride[0] = 4
        if heads == 2:
            c.v_stride[1] = 0
        p = _decode(max_seqlen=100000)  # long enough to need the workspace it lacks
        assert lib.bsfa_decode16(ctypes.byref(c), ctypes.byref(p), None) == status


def test_ropes_that_are_refused(lib):
    far = _rope(num_axes=2)
    far.axis[63] = 2
    for rope, status in ((None, INVALID), (_rope(pairs=0), INVALID), (_rope(pairs=12), UNSUPPORTED),
                         (_rope(pairs=72), UNSUPPORTED), (_rope(num_axes=0), INVALID),
                         (_rope(num_axes=5), UNSUPPORTED), (far, INVALID),
                         (_rope(inv_freq=0), INVALID)):
        assert _rotary(lib, rope, _rows()) == status
        if rope is not None:
            assert _write(lib, _cache(), rope, _rows()) == status
    assert _rotary(lib, _rope(pairs=64), _rows(head_dim=64)) == UNSUPPORTED
    assert _write(lib, _cache(), _rope(inverse=1), _rows()) == INVALID
    assert _write(lib, _cache(), None, _rows()) == INVALID  # queries and nothing to turn them by


def test_rows_that_are_refused(lib):
    both = ((dict(batch=-1), INVALID), (dict(seqlen=-1), INVALID), (dict(batch=4097), UNSUPPORTED),
            (dict(dtype=2), UNSUPPORTED), (dict(batch=4096, seqlen=1 << 20), UNSUPPORTED),
            (dict(head_dim=96), UNSUPPORTED), (dict(num_heads_q=0), INVALID),
            (dict(num_heads_q=4097), UNSUPPORTED), (dict(num_heads_kv=-2), INVALID),
            (dict(num_heads_kv=4097), UNSUPPORTED),
            (dict(q=(1 << 20) + 2), UNSUPPORTED), (dict(k=(1 << 20) + 8), UNSUPPORTED),
            (dict(q_out=0), INVALID), (dict(q_out=(1 << 20) + 4), UNSUPPORTED))
    for change, status in both:
        assert _rotary(lib, _rope(), _rows(**change)) == status, change
        assert _write(lib, _cache(), _rope(), _rows(**change)) == status, change
    for change, status in ((dict(k_out=0), INVALID), (dict(k_out=(1 << 20) + 8), UNSUPPORTED),
                           (dict(q=0, k=0), INVALID)):
        assert _rotary(lib, _rope(), _rows(**change)) == status, change
    for change, status in ((dict(k=0), INVALID), (dict(v=0), INVALID),
                           (dict(v=(1 << 20) + 8), UNSUPPORTED), (dict(num_heads_kv=3), INVALID),
                           (dict(head_dim=64), INVALID), (dict(dtype=1), INVALID)):
        assert _write(lib, _cache(), _rope(pairs=32), _rows(**change)) == status, change
    for field in ("q_stride", "k_stride", "q_out_stride"):
        r = _rows()
        getattr(r, field)[2] = 100  # rows off the 16-byte grid
        assert _write(lib, _cache(), _rope(), r) == UNSUPPORTED
        assert _rotary(lib, _rope(), r) == UNSUPPORTED
    assert _rotary(lib, _rope(), None) == INVALID
    assert _write(lib, None, _rope(), _rows()) == INVALID
    assert _write(lib, _cache(), _rope(), None) == INVALID
    for empty in (dict(batch=0), dict(seqlen=0)):  # no-ops, whatever the pointers
        r = _rows(q=0, k=0, v=0, **empty)
        assert _rotary(lib, _rope(inv_freq=0), r) == OK
        assert _write(lib, _cache(), None, r) == OK


@pytest.mark.parametrize("source", ["bsfa_cache16", "inst_decode16_d64_bf16", "inst_decode16_d64_f16",
                                    "inst_decode16_d128_bf16", "inst_decode16_d128_f16"])
def test_kernels_do_not_spill(lib, source):
    """The compiler warns of registers that it spills to local memory."""
    from block_sparse_gated_gb300 import build
    log = os.path.join(build.OBJDIR, source + ".o.log")
    if not os.path.exists(log):
        pytest.skip("the library was built without a log")
    with open(log) as f:
        assert "are spilled" not in f.read()


def test_binding_refuses_host_tensors():
    b = _bsfa()
    cache = b.cache16_empty(2, 2, 16, 64, device="cpu")
    x = torch.zeros(1, 2, 16, 64, dtype=BF)
    table = torch.zeros(1, 2, dtype=torch.int32)
    rope = b.Rope(cu.inv_freq(32))
    with pytest.raises(ValueError, match="CUDA"):
        b.cache16_write(cache, x, x, table)
    with pytest.raises(ValueError, match="CUDA"):
        b.rotary(rope, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        b.decode16(x, cache, table, torch.zeros(1, dtype=torch.int32))


class Cuda:  # stands for the host tensors' device
    type, index = "cuda", -1  # get_device() of a host tensor


def test_binding_checks_what_the_library_cannot_see(monkeypatch):
    """Shapes, types and extents, on host tensors with the residency check
    taken out (no call reaches the library)."""
    from block_sparse_gated_gb300 import cache16 as m
    b, n, dev = _bsfa(), _native(), Cuda()
    monkeypatch.setattr(m, "_on_device", lambda *a, **k: None)
    cache = b.cache16_empty(4, 2, 32, 128, device="cpu")
    table = torch.zeros(3, 2, dtype=torch.int32)

    packed, *rest = m._cache_fields(cache, table, dev, 3)
    c = n.Cache16.from_buffer_copy(packed)
    assert rest == [2, 128, 0, 64]
    assert (c.num_pages, c.num_heads_kv, c.page_size, c.head_dim, c.dtype) == (4, 2, 32, 128, 0)
    assert (c.k, c.v, c.block_table) == (cache.k.data_ptr(), cache.v.data_ptr(), table.data_ptr())
    assert tuple(c.k_stride) == (2 * 32 * 128, 32 * 128, 128)
    other = b.cache16_empty(4, 2, 32, 128, layout="pthd", dtype=HF, device="cpu")
    c = n.Cache16.from_buffer_copy(m._cache_fields(other, table, dev, 3)[0])
    assert (tuple(c.v_stride), c.page_size, c.dtype) == ((32 * 2 * 128, 128, 2 * 128), 32, 1)
    wide = torch.zeros(3, 9, dtype=torch.int32)[:, :2]
    c = n.Cache16.from_buffer_copy(m._cache_fields(cache, wide, dev, 3)[0])
    assert (c.block_table_stride, c.block_table_width) == (9, 2)
    for bad in (cache._replace(v=cache.v[:2]), cache._replace(k=cache.k[0]),
                cache._replace(layout="thpd"),
                cache._replace(k=cache.k.transpose(2, 3).contiguous().transpose(2, 3))):
        with pytest.raises(ValueError):
            m._cache_fields(bad, table, dev, 3)
    for bad in (cache._replace(k=cache.k.half()), cache._replace(v=cache.v.float())):
        with pytest.raises(TypeError):
            m._cache_fields(bad, table, dev, 3)
    for bad in (table.long(), table[0], torch.zeros(2, 3, dtype=torch.int32).t()):
        with pytest.raises(ValueError, match="block_table"):
            m._cache_fields(cache, bad, dev, 3)
    with pytest.raises(ValueError, match="fewer rows"):
        m._cache_fields(cache, table, dev, 4)

    q, k = torch.zeros(3, 8, 10, 128, dtype=BF), torch.zeros(3, 2, 10, 128, dtype=BF)
    packed, *rest = m._rows_fields(q, k, k, q, None, None, None, None, dev)
    r = n.Rows16.from_buffer_copy(packed)
    assert rest == [3, 10, 2, 128, 0, False]
    assert (r.batch, r.num_heads_q, r.num_heads_kv, r.seqlen, r.head_dim) == (3, 8, 2, 10, 128)
    assert (r.q, r.k, r.v, r.q_out, r.k_out) == (q.data_ptr(), k.data_ptr(), k.data_ptr(),
                                                 q.data_ptr(), None)
    assert tuple(r.q_out_stride) == (8 * 10 * 128, 10 * 128, 128)
    assert tuple(r.k_out_stride) == (0, 0, 0)
    at, off = torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    t = torch.zeros(10, 8, 128, dtype=HF)
    packed, *rest = m._rows_fields(t, t[:, :2], None, t, t[:, :2], "thd", off, at, dev)
    r = n.Rows16.from_buffer_copy(packed)
    assert rest == [3, 10, 2, 128, 1, True]
    assert (tuple(r.k_stride), r.start, r.cu_seqlens) == ((0, 128, 8 * 128), at.data_ptr(),
                                                         off.data_ptr())
    for args in ((q, k[:, :, :9], None, q, None), (q, k[:2], None, q, None),
                 (q, k[..., :64], None, q, None), (q, k, k[:, :1], q, None),
                 (q, k, None, q[:, :4], None), (q, k[0], None, q, None)):
        with pytest.raises(ValueError):
            m._rows_fields(*args, None, None, None, dev)
    for args in ((q, k.half(), None, q, None), (q.float(), None, None, q.float(), None)):
        with pytest.raises(TypeError):
            m._rows_fields(*args, None, None, None, dev)
    with pytest.raises(ValueError, match="start"):
        m._rows_fields(q, k, k, q, None, None, None, at[:2], dev)
    with pytest.raises(ValueError, match="cu_seqlens"):
        m._rows_fields(t, None, None, t, None, "thd", off.long(), None, dev)
    with pytest.raises(ValueError, match="layout|bhdl"):
        m._rows_fields(q, k, k, q, None, "bhdl", None, None, dev)

    f = cu.inv_freq(64)
    axes = (0,) * 20 + (1,) * 20 + (2,) * 24

    def rope(r, positions=None, varlen=False, batch=3, rows=10, inverse=False):
        return n.Rope.from_buffer_copy(m._rope_fields(r, positions, inverse, varlen, batch, rows,
                                                      dev))

    x = rope(b.Rope(f))
    assert (x.inv_freq, x.positions, x.pairs, x.num_axes) == (f.data_ptr(), None, 64, 1)
    assert (x.interleaved, x.inverse, bytes(x.axis)) == (0, 0, bytes(64))
    p = torch.zeros(3, 3, 10, dtype=torch.int32)
    x = rope(b.Rope(f, axes, True), p, inverse=True)
    assert (x.num_axes, x.interleaved, x.inverse, x.positions) == (3, 1, 1, p.data_ptr())
    assert tuple(x.position_stride) == (30, 10) and bytes(x.axis) == bytes(axes)
    x = rope(b.Rope(f), p[0])
    assert tuple(x.position_stride) == (0, 10)
    x = rope(b.Rope(f, axes), p[:, :1].expand(3, 3, 10))  # one sequence's positions for all
    assert tuple(x.position_stride) == (30, 0)
    x = rope(b.Rope(f, axes), p[:, 0], varlen=True)
    assert tuple(x.position_stride) == (30, 0)
    for r, kw in ((b.Rope(f[::2]), {}), (b.Rope(f.double()), {}), (b.Rope(f[:0]), {}),
                  (b.Rope(torch.zeros(65)), {}), (b.Rope(f, axes[:63]), {}),
                  (b.Rope(f, (4,) * 64), {}), (b.Rope(f, (-1,) * 64), {}),
                  (b.Rope(f, axes), dict(positions=p[:2])), (b.Rope(f, axes), dict(positions=p[0])),
                  (b.Rope(f), dict(positions=p[0].long())), (b.Rope(f), dict(positions=p[0, :2])),
                  (b.Rope(f), dict(positions=torch.zeros(10, 3, dtype=torch.int32).t())),
                  (b.Rope(f), dict(positions=torch.zeros(5, 3, 10, dtype=torch.int32)))):
        with pytest.raises(ValueError):
            rope(r, **kw)
    q1, lens = torch.zeros(3, 8, 1, 128, dtype=BF), torch.zeros(3, dtype=torch.int32)

    def decode(*a, **kw):
        kw = dict(dict(layout=None, max_seqlen=None, softmax_scale=None, causal=True), **kw)
        _, fields, code = m._decode_fields(*a, dev, **kw)
        return n.Decode4Params.from_buffer_copy(n.DECODE4.pack(*fields, 4096, 77, code))

    d = decode(q1, cache, table, lens, q1, lse=512, softmax_scale=0.5)
    assert (d.batch, d.num_heads_q, d.q_len, d.max_seqlen, d.dtype, d.causal) == (3, 8, 1, 64, 0, 1)
    assert (d.q, d.o, d.seqlens, d.lse) == (q1.data_ptr(), q1.data_ptr(), lens.data_ptr(), 512)
    assert (d.workspace, d.workspace_bytes, d.softmax_scale) == (4096, 77, 0.5)
    for bad, what in (((q1[:, :7], cache, table, lens, q1[:, :7]), "heads"),
                      ((q1, cache, table, lens, q1.half()), "shape and type"),
                      ((q1.half(), cache, table, lens, q1.half()), "type"),
                      ((q1, cache, table, lens.long(), q1), "seqlens")):
        with pytest.raises(ValueError, match=what):
            decode(*bad)
    with pytest.raises(ValueError, match="pages"):
        decode(q1, cache, table, lens, q1, max_seqlen=65)
    with pytest.raises(ValueError, match="rope"):
        b.cache16_write(cache, k, k, table, q=q)
    with pytest.raises(ValueError, match="rope"):
        b.cache16_write(cache, k, k, table, positions=p[0])
    with pytest.raises(ValueError, match="q_out"):
        b.cache16_write(cache, k, k, table, rope=b.Rope(f), q_out=q)
    with pytest.raises(ValueError, match="pair"):
        b.rotary(b.Rope(f), q, out=(q, k))
    with pytest.raises(ValueError, match="cache's"):
        m.cache16_write(cache, q, q, table, rope=b.Rope(f))


def test_cache_allocation_checks():
    b = _bsfa()
    kw = dict(num_pages=1, num_heads_kv=1, page_size=16, head_dim=64, device="cpu")
    for bad in (dict(page_size=24), dict(page_size=0), dict(head_dim=96), dict(layout="htpd")):
        with pytest.raises(ValueError):
            b.cache16_empty(**dict(kw, **bad))
    with pytest.raises(TypeError):
        b.cache16_empty(**kw, dtype=torch.float32)


# ------------------------------------------------------------------ the oracle
def test_oracle_rotation_by_hand():
    """A quarter turn and a third of one, of both kinds of pairs, and back."""
    x = np.array([[1.0, 2.0, 3.0, 4.0, 9.0]])
    f = np.array([np.pi / 2, np.pi / 3])
    y = ro.rotate(x, np.array([[1]]), f)
    h = np.sqrt(3) / 2
    assert np.allclose(y, [[-3, 2 * 0.5 - 4 * h, 1, 4 * 0.5 + 2 * h, 9]])
    y = ro.rotate(x, np.array([[1]]), f, interleaved=True)
    assert np.allclose(y, [[-2, 1, 3 * 0.5 - 4 * h, 4 * 0.5 + 3 * h, 9]])
    assert np.allclose(ro.rotate(y, np.array([[1]]), f, interleaved=True, inverse=True), x)
    y = ro.rotate(x, np.array([[1], [0]]), f, axes=[1, 0])  # the first pair by axis 1: not at all
    assert np.allclose(y, [[1, 2 * 0.5 - 4 * h, 3, 4 * 0.5 + 2 * h, 9]])
    assert np.allclose(ro.size(x, 2), [[4, 6, 4, 6, 0]])
    assert np.allclose(ro.size(x, 2, interleaved=True), [[3, 3, 7, 7, 0]])


def test_the_reduction_of_angles_in_integers():
    """The kernel's phase, restated in Python's integers: s * p modulo 2^64 with s made
    from the float's bits is p * f / 2 pi modulo a turn."""
    from fractions import Fraction
    pi = Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)
    whole = 0xA2F9836E4E441529
    assert whole == int(2 ** 66 / (2 * pi))
    rng = np.random.default_rng(1)
    for f in np.concatenate([np.float32(10000.0) ** -rng.random(200).astype(np.float32),
                             np.float32([1, 2, 3.75, 255, 1e-7, 1e-30, 1e-42])]):
        bits = int(np.float32(f).view(np.uint32))
        e = max(1, bits >> 23)
        m = (bits & 0x7FFFFF) | (0x800000 if bits >> 23 else 0)
        step = (m * whole >> (152 - e)) % 2 ** 64 if e <= 152 else (m * whole << (e - 152)) % 2 ** 64
        for p in (0, 1, -1, 131071, 2 ** 30, -2 ** 31, 2 ** 31 - 1):
            turns = Fraction(float(f)) * p / (2 * pi)
            off = abs(Fraction((step * p) % 2 ** 64, 2 ** 64) - turns % 1)
            assert min(off, 1 - off) <= (1 + Fraction(float(f))) * abs(p) * Fraction(1, 2 ** 64)
