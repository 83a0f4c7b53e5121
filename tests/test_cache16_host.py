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
    n = _native()
    C, P, R = n.Cache16, n.Rope, n.Rows16
    assert got == (ctypes.sizeof(C), C.num_pages.offset, C.block_table.offset, C.dtype.offset,
                   ctypes.sizeof(P), P.position_stride.offset, P.num_axes.offset, P.axis.offset,
                   ctypes.sizeof(R), R.k_out_stride.offset, R.cu_seqlens.offset, R.dtype.offset,
                   4)


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
                                    "inst_decode16_d128_bf16", "inst_decode16_d128_f16",
                                    "inst_decode16_wide_d64", "inst_decode16_wide_d128"])
def test_kernels_do_not_spill(lib, source):
    """The compiler warns of registers that it spills to local memory."""
    from block_sparse_gated_gb300 import build
    log = os.path.join(build.OBJDIR, source + ".o.log")
    if not os.path.exists(log):
        pytest.skip("the library was built without a log")
    with open(log) as f:
        assert "are spilled" not in f.read()


@pytest.fixture(scope="module")
def b(lib):
    import block_sparse_gated_gb300 as b
    return b


# The binding looks at shapes, types and strides first and at the device last: a call on host
# tensors that is right in all else is refused for that, and nothing is launched.
HOST = "CUDA"


def _args():
    """A right call's tensors, on the host."""
    b = _bsfa()
    z = torch.zeros
    return dict(cache=b.cache16_empty(4, 2, 32, 128, device="cpu"), rope=b.Rope(cu.inv_freq(64)),
                table=z(3, 2, dtype=torch.int32), q=z(3, 8, 10, 128, dtype=BF),
                k=z(3, 2, 10, 128, dtype=BF), q1=z(3, 8, 1, 128, dtype=BF),
                lens=z(3, dtype=torch.int32))


def test_right_calls_reach_the_device_check(b):
    x = _args()
    cache, rope, table, q, k, lens = (x[n] for n in ("cache", "rope", "table", "q", "k", "lens"))
    t = torch.zeros(10, 12, 128, dtype=BF)  # queries, keys and values of packed tokens
    off, p = torch.zeros(4, dtype=torch.int32), torch.zeros(3, 3, 10, dtype=torch.int32)
    axes = (0,) * 20 + (1,) * 20 + (2,) * 24
    q0 = q[:, :, :0]
    for call in (
            lambda: b.rotary(rope, q), lambda: b.rotary(rope, q, k, start=lens),
            lambda: b.rotary(rope, q[0], k[0]), lambda: b.rotary(rope, q, k, out=(q, k)),
            lambda: b.rotary(rope, q, out=(q, None), inverse=True),
            lambda: b.rotary(rope, t[:, :8], t[:, 8:10], layout="thd", cu_seqlens=off, start=lens),
            lambda: b.rotary(rope, t[:8], t[8:10], cu_seqlens=off),
            lambda: b.rotary(rope._replace(axes=axes), q, positions=p),
            lambda: b.rotary(rope._replace(axes=list(axes)), q, positions=p[:, :1].expand(3, 3, 10)),
            lambda: b.rotary(rope, q, positions=p[0]), lambda: b.rotary(rope, q, positions=p),
            lambda: b.rotary(rope, q0, positions=p[0, :, :0]),
            lambda: b.rotary(rope._replace(axes=axes), t[:, :8], layout="thd", cu_seqlens=off,
                             positions=p[:, 0]),
            lambda: b.cache16_write(cache, k, k, table),
            lambda: b.cache16_write(cache, k, k, table, rope=rope, q=q, q_out=q, start=lens),
            lambda: b.cache16_write(cache, k.transpose(1, 2), k.transpose(1, 2), table,
                                    layout="blhd", rope=rope),
            lambda: b.decode16(x["q1"], cache, table, lens, return_lse=True),
            lambda: b.decode16(q, cache, table, lens, max_seqlen=64, softmax_scale=0.5,
                               causal=False, out=q),
            lambda: b.decode16(q[0], cache, table, lens[:1])):
        with pytest.raises(ValueError, match=HOST):
            call()
    cache = b.cache16_empty(4, 2, 32, 128, layout="pthd", dtype=HF, device="cpu")
    with pytest.raises(ValueError, match=HOST):
        b.cache16_write(cache, k.half(), k.half(), table, rope=rope, q=q.half())
    # the workspace's size is a matter of shapes alone
    assert b.decode16_workspace_bytes(x["q1"], x["cache"], table, lens) == 0
    wide = torch.zeros(3, 4000, dtype=torch.int32)
    assert b.decode16_workspace_bytes(x["q1"], x["cache"], wide, lens) > 0
    assert b.decode16_workspace_bytes(x["q1"], x["cache"], wide, lens, max_seqlen=64) == 0


def test_caches_that_the_binding_refuses(b):
    x = _args()
    cache, table, k, q1, lens = (x[n] for n in ("cache", "table", "k", "q1", "lens"))

    def both(cache, table, kind, what):
        with pytest.raises(kind, match=what):
            b.cache16_write(cache, k, k, table)
        with pytest.raises(kind, match=what):
            b.decode16(q1, cache, table, lens)

    turned = cache.k.transpose(2, 3).contiguous().transpose(2, 3)
    for bad in (cache._replace(v=cache.v[:2]), cache._replace(k=turned), cache._replace(v=turned)):
        both(bad, table, ValueError, "one shape, with the head dimension contiguous")
    both(cache._replace(k=cache.k[0]), table, ValueError, "4-D")
    both(cache._replace(layout="thpd"), table, ValueError, "thpd")
    both(cache._replace(layout="bhld"), table, ValueError, "pthd")
    for bad in (cache._replace(k=cache.k.half()), cache._replace(v=cache.v.float())):
        both(bad, table, TypeError, "one type")
    both(b.KVCache16(cache.k.float(), cache.v.float()), table, TypeError, "float16")
    both(cache._replace(k=None), table, TypeError, "cache.k must be a tensor")
    for bad in (table.long(), table[0], torch.zeros(2, 3, dtype=torch.int32).t()):
        both(cache, bad, ValueError, "block_table must be")
    both(cache, table[:2], ValueError, "fewer rows")
    both(cache, 3, TypeError, "block_table must be a tensor")


def test_rows_that_the_binding_refuses(b):
    x = _args()
    cache, rope, table, q, k, lens = (x[n] for n in ("cache", "rope", "table", "q", "k", "lens"))
    t, off = torch.zeros(10, 8, 128, dtype=HF), torch.zeros(4, dtype=torch.int32)
    shapes = "disagree|one shape|contiguous"
    for args in ((q, k[:, :, :9]), (q, k[:2]), (q, k[..., :64]), (q, k[0]),
                 (q, k.transpose(2, 3).contiguous().transpose(2, 3))):
        with pytest.raises(ValueError, match=shapes):
            b.rotary(rope, *args)
        with pytest.raises(ValueError, match=shapes):
            b.cache16_write(cache, args[1], args[1], table, rope=rope, q=q)
    for out in ((q[:, :4], k), (q, k[:, :, :3]), (q[:2], k)):
        with pytest.raises(ValueError, match=shapes):
            b.rotary(rope, q, k, out=out)
    with pytest.raises(ValueError, match=shapes):
        b.cache16_write(cache, k, k[:, :1], table)
    with pytest.raises(ValueError, match=shapes):
        b.cache16_write(cache, k, k, table, rope=rope, q=q, q_out=q[:, :4])
    for args in ((q, k.half()), (q.float(), None), (q, k.float())):
        with pytest.raises(TypeError):
            b.rotary(rope, *args)
    with pytest.raises(TypeError, match="element type"):
        b.rotary(rope, q, out=(q.half(), None))
    with pytest.raises(TypeError, match="element type"):
        b.cache16_write(cache, k, k.half(), table)
    with pytest.raises(TypeError, match="q must be a tensor"):
        b.rotary(rope, None)
    for bad in (lens[:2], lens.long(), lens[None], torch.zeros(6, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError, match="start"):
            b.rotary(rope, q, start=bad)
    for bad in (off.long(), off[None], off[:0]):
        with pytest.raises(ValueError, match="cu_seqlens"):
            b.rotary(rope, t, layout="thd", cu_seqlens=bad)
    for layout, kw in (("bhdl", {}), ("thd", {}), ("phtd", {}), ("bhld", dict(cu_seqlens=off))):
        y = t if kw else q
        with pytest.raises(ValueError, match="bhdl|batched rows|packed rows"):
            b.rotary(rope, y, layout=layout, **kw)
    with pytest.raises(ValueError, match="3-D"):
        b.rotary(rope, q, cu_seqlens=off)
    with pytest.raises(ValueError, match="4-D"):
        b.rotary(rope, q[0, 0])
    with pytest.raises(ValueError, match="pair"):
        b.rotary(rope, q, out=(q, k))
    with pytest.raises(ValueError, match="pair"):
        b.rotary(rope, q, k, out=(q, None))
    with pytest.raises(ValueError, match="two tensors"):
        b.rotary(rope, k, k, out=(k, k))
    with pytest.raises(ValueError, match="rope"):
        b.cache16_write(cache, k, k, table, q=q)
    with pytest.raises(ValueError, match="rope"):
        b.cache16_write(cache, k, k, table, positions=torch.zeros(3, 10, dtype=torch.int32))
    with pytest.raises(ValueError, match="q_out"):
        b.cache16_write(cache, k, k, table, rope=rope, q_out=q)
    for bad in (q, k[..., :64], k.half()):
        with pytest.raises(ValueError, match="cache's"):
            b.cache16_write(cache, bad, bad, table)


def test_ropes_that_the_binding_refuses(b):
    x = _args()
    f, q = x["rope"].inv_freq, x["q"]
    axes = (0,) * 20 + (1,) * 20 + (2,) * 24
    p = torch.zeros(3, 3, 10, dtype=torch.int32)
    for bad in (f[::2], f.double(), f[:0], torch.zeros(65), f[None]):
        with pytest.raises(ValueError, match="inv_freq"):
            b.rotary(b.Rope(bad), q)
    for bad in (axes[:63], (4,) * 64, (-1,) * 64, (1 << 40,) * 64):
        with pytest.raises(ValueError, match="axes"):
            b.rotary(b.Rope(f, bad), q)
    for bad in (3, (0.5,) * 64):
        with pytest.raises(TypeError):
            b.rotary(b.Rope(f, bad), q)
    for rope, bad in ((b.Rope(f, axes), p[:2]), (b.Rope(f, axes), p[0]), (b.Rope(f), p[0].long()),
                      (b.Rope(f), p[0, :2]), (b.Rope(f), p[0, 0]), (b.Rope(f), p[:, :, :9]),
                      (b.Rope(f), torch.zeros(10, 3, dtype=torch.int32).t()),
                      (b.Rope(f), torch.zeros(5, 3, 10, dtype=torch.int32))):
        with pytest.raises(ValueError, match="positions"):
            b.rotary(rope, q, positions=bad)
    with pytest.raises(ValueError, match="positions"):
        b.rotary(b.Rope(f), q[0], cu_seqlens=torch.zeros(2, dtype=torch.int32), positions=p)


def test_decode_calls_that_the_binding_refuses(b):
    x = _args()
    cache, table, q1, lens = (x[n] for n in ("cache", "table", "q1", "lens"))
    for bad, what in (((q1[:, :7], lens), "heads"), ((q1.half(), lens), "type"),
                      ((q1[..., :64], lens), "head dimension"), ((q1, lens.long()), "seqlens"),
                      ((q1, lens[:2]), "seqlens"), ((q1[0, 0], lens), "4-D")):
        with pytest.raises(ValueError, match=what):
            b.decode16(bad[0], cache, table, bad[1])
    for bad in (q1.half(), q1[:2], x["q"]):
        with pytest.raises(ValueError, match="shape and type"):
            b.decode16(q1, cache, table, lens, out=bad)
    with pytest.raises(ValueError, match="pages"):
        b.decode16(q1, cache, table, lens, max_seqlen=65)
    with pytest.raises(TypeError):
        b.decode16(q1, cache, table, lens, max_seqlen="64")
    with pytest.raises(ValueError, match="contiguous"):
        b.decode16(q1, cache, table, lens, workspace=torch.zeros(8, 8)[:, 1])
    with pytest.raises(ValueError, match="batched rows"):
        b.decode16(q1, cache, table, lens, layout="thd")


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
