"""The paged cache's C ABI without a GPU: struct layouts and what is refused on the host before any launch."""

from __future__ import annotations

import ctypes
import os
import subprocess

import pytest
import torch

from quantized_cross_loop_gb300 import build as kbuild
from quantized_cross_loop_gb300 import kvq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD, UNSUP, MISALIGNED, WORKSPACE, CUDA = -1, -2, -3, -4, -5
P = ctypes.c_void_p(4096)


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return kvq.lib()


def _cache(L, dtype=0, n_pages=10, page_size=64, n_heads=8, head_dim=128, **over):
    c = kvq.kvq_paged_cache()
    assert L.kvq_paged_cache_init(ctypes.byref(c), dtype, n_pages, page_size, n_heads, head_dim) == 0
    c.k, c.v, c.key_bounds = 4096, 8192, 4096
    for name, value in over.items():
        setattr(c, name, value)
    return c


def _rows(**over):
    r = kvq.kvq_paged_rows()
    r.start, r.offsets, r.n_rows, r.k, r.v, r.k_stride, r.v_stride = 4096, None, 2, 4096, 4096, 1024, 1024
    for name, value in over.items():
        setattr(r, name, value)
    return r


def test_struct_layouts_match_header(tmp_path):
    src = tmp_path / "layout.c"
    fields = {"kvq_paged_cache": kvq.kvq_paged_cache, "kvq_paged_rows": kvq.kvq_paged_rows}
    lines = [f'printf("%zu\\n", sizeof({n}));' + "".join(f'printf("%zu\\n", offsetof({n}, {f[0]}));' for f in t._fields_)
             for n, t in fields.items()]
    src.write_text('#include <stdio.h>\n#include "kvq.h"\nint main(void){' + "".join(lines) + "return 0;}")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I" + os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for t in fields.values():
        want += [ctypes.sizeof(t)] + [getattr(t, f[0]).offset for f in t._fields_]
    assert got == want


def test_cache_init(L):
    c = kvq.kvq_paged_cache()
    ref = ctypes.byref(c)
    assert L.kvq_paged_cache_init(ref, 0, 10, 16, 8, 128) == 0
    assert (c.head_stride, c.token_stride, c.page_stride) == (128, 1024, 16384) and c.version == 1
    assert L.kvq_paged_cache_init(None, 0, 10, 16, 8, 128) == BAD
    for bad in ((3, 10, 16, 8, 128), (-1, 10, 16, 8, 128), (0, 0, 16, 8, 128), (0, 10, 0, 8, 128),
                (0, 10, 1025, 8, 128), (0, 10, 16, 0, 128), (0, 10, 16, 8, 0)):
        assert L.kvq_paged_cache_init(ref, *bad) == BAD, bad


def _attn(L, c, n=2, width=4, q=P, q_dtype=0, q_stride=4096, Hq=32, scale=0.1, out=P, ws=P, ws_bytes=1 << 30, lens=P,
          table=P):
    return L.kvq_paged_decode_attn(ctypes.byref(c), table, width, n, lens, q, q_dtype, q_stride, Hq, scale, out, None, ws,
                                   ws_bytes, None)


def test_attention_refusals(L):
    assert L.kvq_paged_decode_attn(None, P, 4, 2, P, P, 0, 4096, 32, 0.1, P, None, P, 1 << 30, None) == BAD
    assert _attn(L, _cache(L, version=2)) == UNSUP
    assert _attn(L, _cache(L, head_dim=64)) == UNSUP
    c = _cache(L)
    c.dtype = 7
    assert _attn(L, c) == BAD
    c.dtype, c.page_size = 0, 2048
    assert _attn(L, c) == BAD
    assert _attn(L, _cache(L, k=None)) == BAD
    assert _attn(L, _cache(L, v=4104)) == MISALIGNED
    assert _attn(L, _cache(L, token_stride=1028)) == MISALIGNED  # 8-byte steps
    assert _attn(L, _cache(L, token_stride=512)) == BAD  # places overlap
    assert _attn(L, _cache(L, page_stride=64 * 1024 - 8)) == BAD
    assert _attn(L, _cache(L, head_stride=-128)) == BAD
    assert _attn(L, _cache(L, k_scale=4096)) == BAD  # scales on a 16-bit cache
    c = _cache(L)
    assert _attn(L, c, n=-1) == BAD
    assert _attn(L, c, width=-1) == BAD
    assert _attn(L, c, width=1 << 26) == BAD  # 2^32 tokens
    assert _attn(L, c, n=1 << 28) == BAD
    assert _attn(L, c, table=None) == BAD
    assert _attn(L, c, lens=None) == BAD
    assert _attn(L, c, q=None) == BAD
    assert _attn(L, c, q=ctypes.c_void_p(4100)) == MISALIGNED
    assert _attn(L, c, q_stride=4100) == MISALIGNED
    assert _attn(L, c, q_stride=-4096) == BAD
    assert _attn(L, c, q_dtype=2) == BAD
    assert _attn(L, c, q_dtype=1) == UNSUP  # FP16 queries of a BF16 cache
    assert _attn(L, c, Hq=30) == BAD
    assert _attn(L, c, Hq=4) == BAD
    assert _attn(L, c, Hq=8 * 17) == UNSUP
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert _attn(L, c, scale=scale) == BAD
    assert _attn(L, c, out=None) == BAD
    assert _attn(L, c, out=ctypes.c_void_p(4100)) == MISALIGNED
    assert _attn(L, c, n=0, table=None, lens=None, q=None, out=None, ws=None) == 0  # nothing to do
    assert _attn(L, c, ws=None) in (WORKSPACE, CUDA)  # (no device here)
    assert _attn(L, c, ws_bytes=8) in (WORKSPACE, CUDA)


def test_head_major_and_interleaved_strides_are_accepted(L):
    """The stride check passes what does not overlap: the refusal that follows is another one (out NULL)."""
    for strides in ((8 * 64 * 128, 128, 64 * 128), (2 * 64 * 1024, 2 * 1024, 128), (64 * 1024, 1024, 128)):
        c = _cache(L)
        c.page_stride, c.token_stride, c.head_stride = strides
        assert _attn(L, c, out=None) == BAD and b"out" in L.kvq_last_error()
    one = _cache(L, n_pages=1, page_size=1, n_heads=1)
    one.page_stride = one.token_stride = one.head_stride = 3  # strides of dimensions of one entry mean nothing
    assert _attn(L, one, Hq=4, out=None) == BAD and b"out" in L.kvq_last_error()


def test_pools_beyond_any_memory_are_refused(L):
    """A span whose product would wrap around 64 bits, or that no address reaches, is no layout."""
    for pages, stride in ((1 << 20, 1 << 39), (2**31 - 1, 1 << 40), (2**31 - 1, 1 << 33), (10, 1 << 62)):
        assert _attn(L, _cache(L, n_pages=pages, page_stride=stride), out=None) == BAD
        assert b"strides" in L.kvq_last_error()
    assert _attn(L, _cache(L, n_pages=1 << 20, page_stride=1 << 26), out=None) == BAD and b"out is" in L.kvq_last_error()


def test_sparse_and_selection_refusals(L):
    c = _cache(L)

    def sparse(sel=P, n_select=4):
        return L.kvq_paged_sparse_attn(ctypes.byref(c), P, 4, 2, P, P, 0, 4096, 32, sel, n_select, 0.1, P, None, P, 8, None)

    assert sparse(sel=None) == BAD
    assert sparse(n_select=0) == BAD
    assert sparse() in (WORKSPACE, CUDA)

    def select(c, n=4, first=1, last=1, sel=P):
        return L.kvq_paged_select(ctypes.byref(c), P, 4, 2, P, P, 0, 4096, 32, n, first, last, sel, P, 8, None)

    assert select(_cache(L, key_bounds=None)) == BAD
    assert select(_cache(L, key_bounds=4104)) == MISALIGNED
    assert select(c, n=0) == BAD
    assert select(c, first=-1) == BAD
    assert select(c, first=3, last=2) == BAD
    assert select(c, first=0x7FFFFFFF, last=0x7FFFFFFF) == BAD
    assert select(c, sel=None) == BAD
    assert select(_cache(L, k=None, v=None)) in (WORKSPACE, CUDA)  # the bounds alone are enough


def test_append_refusals(L):
    def append(c, r, n=2):
        return L.kvq_paged_append(ctypes.byref(c), P, 4, n, None if r is None else ctypes.byref(r), None)

    c = _cache(L)
    assert append(c, None) == BAD
    assert append(c, _rows(n_rows=3)) == BAD  # one row per request
    assert append(c, _rows(n_rows=-1, offsets=4096)) == BAD
    assert append(c, _rows(dtype=2)) == BAD
    assert append(c, _rows(dtype=1)) == UNSUP
    assert append(c, _rows(rotary_dim=12, rope=4096, rope_positions=9)) == BAD
    assert append(c, _rows(rotary_dim=136, rope=4096, rope_positions=9)) == BAD
    assert append(c, _rows(rotary_dim=64)) == BAD  # no table
    assert append(c, _rows(rotary_dim=64, rope=4096)) == BAD  # no positions in it
    assert append(c, _rows(rotary_dim=64, rope=4100, rope_positions=9)) == MISALIGNED
    assert append(c, _rows(start=None)) == BAD
    assert append(c, _rows(k=None)) == BAD
    assert append(c, _rows(v=4100)) == MISALIGNED
    assert append(c, _rows(k_stride=1028)) == MISALIGNED
    assert append(c, _rows(v_stride=-1024)) == BAD
    q = dict(q=4096, q_out=4096, n_q_heads=32, q_stride=4096, q_out_stride=4096)
    assert append(c, _rows(**{**q, "q_out": None})) == BAD
    assert append(c, _rows(**{**q, "n_q_heads": 12})) == BAD
    assert append(c, _rows(**{**q, "n_q_heads": 8 * 17})) == UNSUP
    assert append(c, _rows(**{**q, "q_out_stride": 2048})) == BAD
    assert append(c, _rows(**{**q, "q_stride": 4100})) == MISALIGNED
    assert append(c, _rows(n_rows=0), n=0) == 0
    assert append(c, _rows(n_rows=0, offsets=4096)) == 0
    if not torch.cuda.is_available():  # (with a device these made-up pointers would be launched)
        assert append(c, _rows()) == CUDA


def test_workspace_of_invalid_sizes_is_zero(L):
    for bad in ((-1, 8, 32, 4), (2, 0, 32, 4), (2, 8, 30, 4), (2, 8, 4, 4), (2, 8, 32, -1)):
        assert L.kvq_paged_workspace_bytes(*bad) == 0


def test_fast_division_by_every_page_size():
    """The kernels divide token numbers by multiplication: the formula against // at the numbers where it could fail."""
    for d in range(1, 1025):
        s = (d - 1).bit_length()
        mul = ((1 << 32) * ((1 << s) - d)) // d + 1
        assert mul < 1 << 32
        n = set(range(0, 3 * d + 2)) | {(1 << 31) - 1 - i for i in range(3 * d)}
        n |= {k * d + e for k in (1 << 10, (1 << 31) // d - 1) for e in (-1, 0, 1)}
        for x in n:
            if 0 <= x < 1 << 31:
                assert (((mul * x >> 32) + x) & 0xFFFFFFFF) >> s == x // d and (mul * x >> 32) + x < 1 << 32
