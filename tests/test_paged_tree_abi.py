"""Tree attention, commit, reading back and scales per token without a GPU: what is refused on the host."""

from __future__ import annotations

import ctypes

import pytest

from quantized_cross_loop_gb300 import build as kbuild
from quantized_cross_loop_gb300 import kvq

BAD, UNSUP, MISALIGNED, WORKSPACE, CUDA = -1, -2, -3, -4, -5
P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4100)
TOKEN = 4


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return kvq.lib()


def _cache(L, dtype=0, **over):
    c = kvq.kvq_paged_cache()
    assert L.kvq_paged_cache_init(ctypes.byref(c), dtype, 10, 64, 8, 128) == 0
    c.k, c.v = 4096, 8192
    if dtype == TOKEN:
        c.k_scale = c.v_scale = 4096
    for name, value in over.items():
        setattr(c, name, value)
    return c


def _tree(L, c, B=2, W=4, table=P, lens=P, off=P, n=9, mask=P, words=1, q=P, q_dtype=0, q_stride=4096, Hq=32, scale=0.1,
          out=P, ws=P, size=8):
    return L.kvq_paged_tree_attn(ctypes.byref(c), table, W, B, lens, off, n, mask, words, q, q_dtype, q_stride, Hq, scale,
                                 out, None, ws, size, None)


def test_tree_attention_refusals(L):
    c = _cache(L)
    assert L.kvq_paged_tree_attn(None, P, 4, 2, P, P, 9, P, 1, P, 0, 4096, 32, 0.1, P, None, P, 8, None) == BAD
    assert _tree(L, _cache(L, version=2)) == UNSUP
    assert _tree(L, _cache(L, v=None)) == BAD
    assert _tree(L, c, B=-1) == BAD
    assert _tree(L, c, W=1 << 26) == BAD
    assert _tree(L, c, table=None) == BAD
    assert _tree(L, c, n=-1) == BAD
    assert _tree(L, c, off=None) == BAD  # nine rows of two requests
    assert _tree(L, c, lens=None) == BAD
    assert _tree(L, c, q=None) == BAD
    assert _tree(L, c, q=ODD) == MISALIGNED
    assert _tree(L, c, q_stride=4100) == MISALIGNED
    assert _tree(L, c, q_stride=-4096) == BAD
    assert _tree(L, c, q_stride=1 << 44) == BAD
    assert _tree(L, c, q_dtype=2) == BAD
    assert _tree(L, c, q_dtype=1) == UNSUP
    assert _tree(L, _cache(L, TOKEN), q_dtype=TOKEN) == BAD
    assert _tree(L, c, Hq=30) == BAD
    assert _tree(L, c, Hq=8 * 17) == UNSUP
    assert _tree(L, c, scale=float("nan")) == BAD and _tree(L, c, scale=0.0) == BAD
    assert _tree(L, c, mask=None) == BAD  # words of no mask
    assert _tree(L, c, words=0) == BAD
    assert _tree(L, c, words=33) == BAD and _tree(L, c, words=-1) == BAD
    assert _tree(L, c, out=None) == BAD
    assert _tree(L, c, out=ODD) == MISALIGNED
    assert _tree(L, c, B=0, n=0, off=None, table=None, lens=None, q=None, mask=None, words=0, out=None, ws=None) == 0
    assert _tree(L, c, n=0, q=None, out=None, ws=None) == 0
    assert _tree(L, c) in (WORKSPACE, CUDA) and _tree(L, c, ws=None) in (WORKSPACE, CUDA)
    for dtype, q_dtype in ((0, 0), (1, 1), (2, 0), (2, 1), (TOKEN, 0), (TOKEN, 1)):
        assert _tree(L, _cache(L, dtype), q_dtype=q_dtype) in (WORKSPACE, CUDA)
    for bad in ((-1, 8, 32, 4), (2, 0, 32, 4), (2, 8, 30, 4), (2, 8, 4, 4), (2, 8, 32, -1), (2, 8, 8 * 17, 4)):
        assert L.kvq_paged_tree_workspace_bytes(*bad) == 0


def test_caches_with_scales_per_token(L):
    """Their scales have to be there, bounds not; the calls that read a scale per head refuse them."""
    assert _tree(L, _cache(L, TOKEN, k_scale=None)) == BAD
    assert _tree(L, _cache(L, TOKEN, v_scale=None)) == BAD
    assert _tree(L, _cache(L, TOKEN, key_bounds=4096)) == BAD
    c = _cache(L)
    c.dtype = 3
    assert _tree(L, c) == BAD
    c = _cache(L, TOKEN)
    ref = ctypes.byref(c)
    assert L.kvq_paged_decode_attn(ref, P, 4, 2, P, P, 0, 4096, 32, 0.1, P, None, P, 1 << 30, None) == UNSUP
    assert b"kvq_paged_tree_attn" in L.kvq_last_error()
    assert L.kvq_paged_sparse_attn(ref, P, 4, 2, P, P, 0, 4096, 32, P, 4, 0.1, P, None, P, 1 << 30, None) == UNSUP
    assert L.kvq_paged_select(ref, P, 4, 2, P, P, 0, 4096, 32, 4, 1, 1, P, P, 1 << 30, None) == UNSUP
    r = kvq.kvq_paged_rows()
    r.start, r.n_rows, r.k, r.v, r.k_stride, r.v_stride = 4096, 2, 4096, 4096, 1024, 1024
    r.dtype = TOKEN
    assert L.kvq_paged_append(ref, P, 4, 2, ctypes.byref(r), None) == BAD
    r.dtype, r.k_stride = 1, 1028
    assert L.kvq_paged_append(ref, P, 4, 2, ctypes.byref(r), None) == MISALIGNED  # (FP16 rows pass)


def test_read_refusals(L):
    c = _cache(L, TOKEN)

    def read(c=c, B=2, start=P, off=P, n=9, dtype=0, k=P, v=P, ks=1024, vs=1024, W=4):
        return L.kvq_paged_read(ctypes.byref(c), P, W, B, start, off, n, dtype, k, v, ks, vs, None)

    assert read(_cache(L, k=None)) == BAD
    assert read(W=-1) == BAD
    assert read(n=-1) == BAD
    assert read(off=None) == BAD
    assert read(dtype=2) == BAD
    assert read(start=None) == BAD
    assert read(k=None) == BAD and read(v=None) == BAD
    assert read(k=ODD) == MISALIGNED and read(vs=1028) == MISALIGNED
    assert read(ks=512) == BAD  # rows overlap
    assert read(ks=-1024) == BAD and read(vs=1 << 43) == BAD
    assert read(B=0, off=None, n=0) == 0 and read(n=0, start=None, k=None) == 0


def test_commit_refusals(L):
    c = _cache(L)

    def commit(c=c, B=2, lens=P, acc=P, off=P, n=4, table=P):
        return L.kvq_paged_tree_commit(ctypes.byref(c), table, 4, B, lens, acc, off, n, None)

    assert commit(_cache(L, k=None)) == BAD
    assert commit(B=-1) == BAD
    assert commit(table=None) == BAD
    assert commit(n=-1) == BAD
    assert commit(lens=None) == BAD
    assert commit(acc=None) == BAD
    assert commit(off=None) == BAD
    assert commit(B=0, lens=None, acc=None, off=None, n=0) == 0
