"""The 4-bit cache without a GPU: the C structs' layout, what the library and
the binding refuse before anything is launched, and the fp64 oracle's own
format against hand-written values."""
import ctypes
import os
import re
import subprocess
import tempfile

import numpy as np
import pytest
import torch

from oracle import cache4_oracle as co

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 5


@pytest.fixture(scope="module")
def lib():
    from block_sparse_gated_gb300 import _native, build
    build.build()
    return _native.lib()


def _native():
    from block_sparse_gated_gb300 import _native
    return _native


def _cache(**kw):
    """A valid descriptor of "phtd" pools whose pointers are never read."""
    c = _native().Cache4()
    c.k = c.v = c.k_scale = c.v_scale = c.block_table = 1 << 20
    c.k_stride[:] = c.v_stride[:] = (2 * 64 * 64, 64 * 64, 64)
    c.k_scale_stride[:] = c.v_scale_stride[:] = (2 * 64 * 8, 64 * 8, 8)
    c.num_pages, c.page_size, c.num_heads_kv, c.head_dim = 10, 64, 2, 128
    c.block_table_stride = c.block_table_width = 4
    for n, x in kw.items():
        setattr(c, n, x)
    return c


def _rows(**kw):
    r = _native().Cache4Rows()
    r.k = r.v = 1 << 20
    r.k_stride[:] = r.v_stride[:] = (2 * 100 * 128, 100 * 128, 128)
    r.batch, r.seqlen = 3, 100
    for n, x in kw.items():
        setattr(r, n, x)
    return r


def _decode(**kw):
    p = _native().Decode4Params()
    p.q = p.o = p.seqlens = 1 << 20
    p.q_stride[:] = p.o_stride[:] = (8 * 128, 128, 128)
    p.batch, p.num_heads_q, p.q_len, p.max_seqlen = 3, 8, 1, 256
    for n, x in kw.items():
        setattr(p, n, x)
    return p


def test_struct_layouts_match_the_header():
    src = r'''
#include <stddef.h>
#include <stdio.h>
#include "bsfa.h"
int main(void) {
  printf("%zu %zu %zu %zu ", sizeof(bsfa_cache4), offsetof(bsfa_cache4, k_scale_stride),
         offsetof(bsfa_cache4, block_table), offsetof(bsfa_cache4, block_table_width));
  printf("%zu %zu %zu ", sizeof(bsfa_cache4_rows), offsetof(bsfa_cache4_rows, cu_seqlens),
         offsetof(bsfa_cache4_rows, dtype));
  printf("%zu %zu %zu %zu\n", sizeof(bsfa_decode4_params), offsetof(bsfa_decode4_params, seqlens),
         offsetof(bsfa_decode4_params, lse), offsetof(bsfa_decode4_params, dtype));
  return 0;
}
'''
    with tempfile.TemporaryDirectory() as tmp:
        c, exe = os.path.join(tmp, "probe.c"), os.path.join(tmp, "probe")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        got = tuple(map(int, subprocess.run([exe], capture_output=True, text=True,
                                            check=True).stdout.split()))
    n = _native()
    C, R, P = n.Cache4, n.Cache4Rows, n.Decode4Params
    assert (n.CACHE4.size, n.CACHE4_ROWS.size, n.DECODE4.size) == tuple(map(ctypes.sizeof,
                                                                           (C, R, P)))
    assert got == (ctypes.sizeof(C), C.k_scale_stride.offset, C.block_table.offset,
                   C.block_table_width.offset, ctypes.sizeof(R), R.cu_seqlens.offset,
                   R.dtype.offset, ctypes.sizeof(P), P.seqlens.offset, P.lse.offset,
                   P.dtype.offset)


@pytest.mark.parametrize("change,status", [
    (dict(head_dim=96), UNSUPPORTED), (dict(page_size=24), UNSUPPORTED),
    (dict(page_size=0), INVALID), (dict(num_pages=0), INVALID), (dict(num_heads_kv=0), INVALID),
    (dict(num_heads_kv=4097), UNSUPPORTED), (dict(block_table_width=5), INVALID),
    (dict(block_table_width=-1), INVALID),
    (dict(block_table_width=(1 << 24) + 1, block_table_stride=1 << 25), UNSUPPORTED),
    (dict(k=0), INVALID), (dict(v_scale=0), INVALID), (dict(block_table=0), INVALID),
    (dict(k=(1 << 20) + 8), UNSUPPORTED), (dict(k_scale=(1 << 20) + 4), UNSUPPORTED),
])
def test_cache_descriptors_that_are_refused(lib, change, status):
    """Every entry point refuses them, before the workspace is looked at."""
    c = _cache(**change)
    for fn, arg in ((lib.bsfa_cache4_write, _rows()), (lib.bsfa_cache4_read, _rows()),
                    (lib.bsfa_decode4, _decode())):
        assert fn(ctypes.byref(c), ctypes.byref(arg), None) == status


def test_cache_strides_that_are_refused(lib):
    for field, i, bad in (("k_stride", 0, 64 * 64 + 8), ("v_stride", 2, 0), ("k_stride", 1, -64),
                          ("k_scale_stride", 0, 1020), ("v_scale_stride", 2, 4),
                          ("k_stride", 0, 1 << 34), ("v_scale_stride", 0, 1 << 34),
                          ("v_stride", 2, 1 << 25), ("k_scale_stride", 2, 1 << 25)):
        c = _cache()
        getattr(c, field)[i] = bad
        p, r = _decode(), _rows()
        assert lib.bsfa_decode4(ctypes.byref(c), ctypes.byref(p), None) == UNSUPPORTED
        assert lib.bsfa_cache4_read(ctypes.byref(c), ctypes.byref(r), None) == UNSUPPORTED


def test_strides_of_one_element_dimensions_say_nothing(lib):
    """A pool of one page and one head is not refused for strides that no call
    multiplies by anything but 0; of two, it is."""
    for pages, heads, status in ((1, 1, WORKSPACE), (2, 1, UNSUPPORTED), (1, 2, UNSUPPORTED)):
        c = _cache(num_pages=pages, num_heads_kv=heads, block_table_width=2000,
                   block_table_stride=2000)
        for s in (c.k_stride, c.v_stride, c.k_scale_stride, c.v_scale_stride):
            if pages == 1:
                s[0] = 1
            if heads == 1:
                s[1] = 0
        if pages == 2:
            c.k_stride[0] = 8
        if heads == 2:
            c.v_scale_stride[1] = 0
        p = _decode(max_seqlen=100000)  # long enough to need the workspace it lacks
        assert lib.bsfa_decode4(ctypes.byref(c), ctypes.byref(p), None) == status


def test_rows_that_are_refused(lib):
    c = ctypes.byref(_cache())
    for change, status in ((dict(batch=-1), INVALID), (dict(seqlen=-1), INVALID),
                           (dict(batch=4097), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED),
                           (dict(batch=4096, seqlen=1 << 20), UNSUPPORTED),
                           (dict(k=0), INVALID), (dict(v=(1 << 20) + 2), UNSUPPORTED)):
        r = _rows(**change)
        assert lib.bsfa_cache4_write(c, ctypes.byref(r), None) == status, change
        assert lib.bsfa_cache4_read(c, ctypes.byref(r), None) == status, change
    r = _rows()
    r.k_stride[2] = 100  # rows off the 16-byte grid
    assert lib.bsfa_cache4_write(c, ctypes.byref(r), None) == UNSUPPORTED
    assert lib.bsfa_cache4_write(None, ctypes.byref(r), None) == INVALID
    assert lib.bsfa_cache4_write(c, None, None) == INVALID
    for empty in (dict(batch=0), dict(seqlen=0)):  # no-ops, whatever the pointers
        r = _rows(k=0, v=0, **empty)
        assert lib.bsfa_cache4_read(c, ctypes.byref(r), None) == OK


def test_decode_parameters_that_are_refused(lib):
    c = ctypes.byref(_cache())
    size = lib.bsfa_decode4_workspace_size
    for change, status in ((dict(num_heads_q=7), INVALID), (dict(num_heads_q=0), INVALID),
                           (dict(batch=-1), INVALID), (dict(q_len=-1), INVALID),
                           (dict(max_seqlen=-1), INVALID), (dict(max_seqlen=257), INVALID),
                           (dict(dtype=3), UNSUPPORTED), (dict(batch=4097), UNSUPPORTED),
                           (dict(q_len=1 << 27), UNSUPPORTED),
                           (dict(batch=4096, q_len=1 << 22), UNSUPPORTED)):
        p = _decode(**change)
        assert lib.bsfa_decode4(c, ctypes.byref(p), None) == status, change
        assert size(c, ctypes.byref(p)) == 0, change
    long = _cache(block_table_width=2000, block_table_stride=2000)
    c2 = ctypes.byref(long)  # a bound this long needs a workspace
    need = size(c2, ctypes.byref(_decode(max_seqlen=100000)))
    assert need > 0 and size(c2, ctypes.byref(_decode(max_seqlen=4096))) == 0
    for change, status in ((dict(q=0), INVALID), (dict(seqlens=0), INVALID),
                           (dict(o=(1 << 20) + 8), UNSUPPORTED), (dict(), WORKSPACE),
                           (dict(workspace=128, workspace_bytes=1 << 30), WORKSPACE),
                           (dict(workspace=1 << 20, workspace_bytes=0), WORKSPACE),
                           (dict(workspace=1 << 20, workspace_bytes=need - 1), WORKSPACE)):
        p = _decode(max_seqlen=100000, **change)
        assert lib.bsfa_decode4(c2, ctypes.byref(p), None) == status, change
    p = _decode(max_seqlen=100000)
    p.q_stride[1] = 4
    assert lib.bsfa_decode4(c2, ctypes.byref(p), None) == UNSUPPORTED
    p = _decode(max_seqlen=100000)
    p.q_stride[2] = 3  # the only token's stride says nothing
    assert lib.bsfa_decode4(c2, ctypes.byref(p), None) == WORKSPACE
    for empty in (dict(batch=0), dict(q_len=0)):
        p = _decode(q=0, o=0, **empty)
        assert lib.bsfa_decode4(c, ctypes.byref(p), None) == OK


@pytest.mark.parametrize("source", ["bsfa_cache4", "bsfa_decode4"])
def test_kernels_do_not_spill(lib, source):
    """The compiler warns of registers that it spills to local memory."""
    from block_sparse_gated_gb300 import build
    log = os.path.join(build.OBJDIR, source + ".o.log")
    if not os.path.exists(log):
        pytest.skip("the library was built without a log")
    with open(log) as f:
        assert "are spilled" not in f.read()


def _bsfa():
    import block_sparse_gated_gb300 as b
    return b


def test_binding_refuses_host_tensors():
    b = _bsfa()
    cache = b.cache4_empty(2, 2, 16, 64, device="cpu")
    x = torch.zeros(1, 2, 16, 64, dtype=torch.bfloat16)
    table = torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        b.cache4_write(cache, x, x, table)
    with pytest.raises(ValueError, match="CUDA"):
        b.cache4_read(cache, table, seqlen=4)
    with pytest.raises(ValueError, match="CUDA"):
        b.decode4(x, cache, table, torch.zeros(1, dtype=torch.int32))


def test_binding_checks_what_the_library_cannot_see(monkeypatch):
    """Shapes, types and extents, on host tensors with the residency check
    taken out (no call reaches the library)."""
    from block_sparse_gated_gb300 import cache4 as m
    b = _bsfa()
    monkeypatch.setattr(m, "_on_device", lambda *a, **k: None)
    cache = b.cache4_empty(4, 2, 32, 128, device="cpu")
    table = torch.zeros(3, 2, dtype=torch.int32)
    n = _native()

    def descriptor(*a):
        return n.Cache4.from_buffer_copy(m._cache_fields(*a)[0])

    class Cuda:  # stands for the host tensors' device
        type, index = "cuda", -1  # get_device() of a host tensor

    dev = Cuda()

    def rows(*a):
        return n.Cache4Rows.from_buffer_copy(m._rows_fields(*a, Cuda())[0])

    def decode(*a, **kw):
        return n.Decode4Params.from_buffer_copy(m._decode_fields(*a, dev, **kw)[1](4096, 77))

    c = descriptor(cache, table, dev, 3)
    assert (c.num_pages, c.num_heads_kv, c.page_size, c.head_dim) == (4, 2, 32, 128)
    assert (c.k, c.v_scale, c.k_exp) == (cache.k.data_ptr(), cache.v_scale.data_ptr(), None)
    assert tuple(c.k_stride) == (2 * 32 * 64, 32 * 64, 64)
    assert c.block_table == table.data_ptr()
    assert (c.block_table_stride, c.block_table_width) == (2, 2)
    other = b.cache4_empty(4, 2, 32, 128, layout="pthd", device="cpu")
    assert tuple(descriptor(other, table, dev, 3).v_scale_stride) == (32 * 2 * 8, 8, 2 * 8)
    wide = torch.zeros(3, 9, dtype=torch.int32)[:, :2]
    c = descriptor(cache, wide, dev, 3)
    assert (c.block_table_stride, c.block_table_width) == (9, 2)
    exps = torch.zeros(2, dtype=torch.int32)
    c = descriptor(cache._replace(k_exp=exps, v_exp=exps), table, dev, 3)
    assert c.k_exp == c.v_exp == exps.data_ptr()
    for bad in (cache._replace(v=cache.v[:2]), cache._replace(k_scale=cache.k_scale[..., :4]),
                cache._replace(k=cache.k.to(torch.int8)),
                cache._replace(v_scale=cache.v_scale.view(torch.uint8)),
                cache._replace(k_scale=cache.k_scale[0]), cache._replace(k=cache.k[0]),
                cache._replace(k_exp=torch.zeros(3, dtype=torch.int32)),
                cache._replace(v_exp=torch.zeros(2)), cache._replace(layout="thpd"),
                cache._replace(k=cache.k.transpose(2, 3).contiguous().transpose(2, 3))):
        with pytest.raises(ValueError):
            descriptor(bad, table, dev, 3)
    for bad in (table.long(), table[0], torch.zeros(2, 3, dtype=torch.int32).t()):
        with pytest.raises(ValueError, match="block_table"):
            descriptor(cache, bad, dev, 3)
    with pytest.raises(ValueError, match="fewer rows"):
        descriptor(cache, table, dev, 4)
    k = torch.zeros(3, 2, 10, 128, dtype=torch.bfloat16)
    ok = (None, None, None, 2, 128)
    r = rows(k, k, *ok)
    assert (r.batch, r.seqlen, r.dtype, r.cu_seqlens, r.start) == (3, 10, 0, None, None)
    assert tuple(r.v_stride) == (2 * 10 * 128, 10 * 128, 128) and r.v == k.data_ptr()
    at = torch.zeros(3, dtype=torch.int32)
    cu = torch.zeros(4, dtype=torch.int32)
    r = rows(k[0].half(), k[0].half(), "htd", cu, at, 2, 128)
    assert (r.batch, r.seqlen, r.dtype) == (3, 10, 1)
    assert (r.cu_seqlens, r.start) == (cu.data_ptr(), at.data_ptr())
    with pytest.raises(ValueError, match="disagree"):
        rows(k, k[:, :, :9], *ok)
    with pytest.raises(TypeError):
        rows(k, k.half(), *ok)
    with pytest.raises(TypeError):
        rows(k.float(), k.float(), *ok)
    with pytest.raises(ValueError, match="heads"):
        rows(k[..., :64], k[..., :64], *ok)
    with pytest.raises(ValueError, match="start"):
        rows(k, k, None, None, torch.zeros(2, dtype=torch.int32), 2, 128)
    with pytest.raises(ValueError, match="cu_seqlens"):
        rows(k[0], k[0], None, torch.zeros(2), None, 2, 128)
    with pytest.raises(ValueError, match="seqlen"):
        m.cache4_read(cache, table)
    with pytest.raises(ValueError, match="total"):
        m.cache4_read(cache, table, seqlen=3, cu_seqlens=torch.zeros(2, dtype=torch.int32))
    q = torch.zeros(3, 8, 1, 128, dtype=torch.bfloat16)
    lens = torch.zeros(3, dtype=torch.int32)
    kw = dict(layout=None, max_seqlen=None, softmax_scale=None, causal=True)
    p = decode(q, cache, table, lens, q, lse=512, **kw)
    assert (p.batch, p.num_heads_q, p.q_len, p.max_seqlen) == (3, 8, 1, 64)
    assert (p.q, p.o, p.seqlens, p.lse) == (q.data_ptr(), q.data_ptr(), lens.data_ptr(), 512)
    assert (p.workspace, p.workspace_bytes, p.dtype, p.causal) == (4096, 77, 0, 1)
    p = decode(q.half(), cache, table, lens, q.half(),
               **dict(kw, softmax_scale=0.5, causal=False, max_seqlen=9))
    assert (p.dtype, p.causal, p.max_seqlen, p.softmax_scale) == (1, 0, 9, 0.5)
    with pytest.raises(ValueError, match="heads"):
        decode(q[:, :7], cache, table, lens, q[:, :7], **kw)
    with pytest.raises(ValueError, match="shape and type"):
        decode(q, cache, table, lens, q.half(), **kw)
    with pytest.raises(ValueError, match="seqlens"):
        decode(q, cache, table, lens.long(), q, **kw)
    with pytest.raises(ValueError, match="pages"):
        decode(q, cache, table, lens, q, **dict(kw, max_seqlen=65))


def test_cache_allocation_checks():
    b = _bsfa()
    for bad in (dict(page_size=24), dict(page_size=0), dict(head_dim=96), dict(layout="htpd")):
        kw = dict(num_pages=1, num_heads_kv=1, page_size=16, head_dim=64, device="cpu")
        kw.update(bad)
        with pytest.raises(ValueError):
            b.cache4_empty(**kw)


def test_the_workspace_size_is_reached_from_the_package():
    b = _bsfa()
    from block_sparse_gated_gb300 import cache4
    assert b.decode4_workspace_bytes is cache4.decode4_workspace_bytes


# ------------------------------------------------------------------ the oracle
def test_oracle_format_by_hand():
    """The e4m3 table's landmarks, ties to the even code, saturation, the least
    scale and the byte order, from hand-computed rows."""
    assert co.E4M3[0] == 0 and co.E4M3[1] == 2.0 ** -9 and co.E4M3[8] == 2.0 ** -6
    assert co.E4M3[0x38] == 1.0 and co.E4M3[0x7E] == 448.0 and len(co.E4M3) == 0x7F
    assert np.array_equal(co.E4M3, np.unique(co.E4M3))
    t = torch.arange(0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(co.E4M3, t)  # the type as torch reads it
    x = np.zeros(16)
    x[:9] = [6, -0.25, 0.75, -1.25, 1.75, 2.5, -3.5, 5, 0.2500001]
    code, byte = co.quantise(x)  # amax 6: scale 1
    assert byte.tolist() == [0x38]
    assert code[:9].tolist() == [7, 0, 2, 8 + 2, 4, 4, 8 + 6, 6, 1]
    assert co.pack(code)[:2].tolist() == [0x07, 0xA2]
    back = co.values(co.pack(code), byte)
    assert back[:9].tolist() == [6, 0, 1, -1, 2, 2, -4, 4, 0.5]
    code, byte = co.quantise(np.full(16, 1e5))
    assert byte.tolist() == [0x7E] and (code == 7).all()  # 448 * 6
    code, byte = co.quantise(np.full(16, 3 * 2.0 ** -9))
    assert byte.tolist() == [1] and (code == 5).all()  # the least scale, 2^-9
    code, byte = co.quantise(np.full(16, 3 * 2.0 ** -9 * 8), exp=3)
    assert byte.tolist() == [1] and co.values(co.pack(code), byte, 3)[0] == 3 * 2.0 ** -6
    x[3] = np.nan
    code, byte = co.quantise(x)
    assert byte.tolist() == [0x7F] and np.isnan(co.values(co.pack(code), byte)).all()


def test_oracle_attention_by_hand():
    """Two keys, one of them hidden from the first query by the causal window."""
    k = np.zeros((1, 2, 16))
    k[0, 0, 0], k[0, 1, 0] = 1.0, 2.0
    v = np.zeros((1, 2, 16))
    v[0, 0, 1], v[0, 1, 1] = 10.0, 20.0
    q = np.zeros((1, 2, 16))
    q[0, :, 0] = np.log(3.0)
    out, lse, _, _, _ = co.attend(q, k, v, sigma=1.0)
    assert np.allclose(out[0, :, 1], [10.0, (3 * 10 + 9 * 20) / 12])
    assert np.allclose(lse[0], [np.log(3.0), np.log(12.0)])
    out, lse, _, _, _ = co.attend(q, k[:, :1], v[:, :1], sigma=1.0)  # 1 key, 2 queries
    assert out[0, 0, 1] == 0 and np.isneginf(lse[0, 0]) and np.isclose(out[0, 1, 1], 10.0)
    out, _, _, _, _ = co.attend(q, k, v, sigma=1.0, causal=False)
    assert np.allclose(out[0, :, 1], (3 * 10 + 9 * 20) / 12)


def test_the_window_of_scales_that_the_header_states():
    """Within it a group's scale is amax / 6 to 3 mantissa bits and its largest
    element is kept to the half step of a scale; above it that element is cut."""
    with open(os.path.join(ROOT, "include", "bsfa.h")) as f:
        text = re.sub(r"\s*\n \*\s*", " ", f.read())
    lo, hi = map(float, re.search(r"3 mantissa bits for a in \[([\d.]+), ([\d.]+)\]", text).groups())

    def back(a):
        code, byte = co.quantise(np.full(16, a))
        return co.values(co.pack(code), byte)[0]

    for a in np.geomspace(lo, hi, 2000):
        assert abs(back(a) - a) <= a / 16
    assert back(hi) == hi == back(hi * 1.001) == back(hi * 2)
    assert 6 * 2.0 ** -6 <= lo <= 6 * 2.0 ** -6 * 1.01  # e4m3's least normal number
