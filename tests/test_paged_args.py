"""What the paged cache's host code hands to its kernels, without a GPU."""

from __future__ import annotations

import ctypes
import subprocess

from quantized_cross_loop_gb300 import build as kbuild
from quantized_cross_loop_gb300 import kvq

SRC = r"""
#include <cstdio>
#include "kvq_paged.cuh"

int main() {
  kvq_paged_rows r = {};
  r.positions = reinterpret_cast<const int32_t*>(4096);
  r.n_rows = 7;
  kvq::paged::View c = {};
  for (int dim : {0, 8, 128}) {
    r.rotary_dim = dim;
    const kvq::paged::AppendArgs a = kvq::paged::append_args(c, KVQ_DT_BF16, nullptr, 0, 0, r);
    printf("%d %d %d\n", a.R, a.n_rows, a.positions != nullptr);
  }
}
"""


def test_positions_reach_no_kernel_without_a_rotation(tmp_path):
    """`positions` is not read when rotary_dim is 0: no kernel gets the pointer."""
    src, exe = tmp_path / "args.cu", tmp_path / "args"
    src.write_text(SRC)
    subprocess.run([kbuild.nvcc()] + kbuild.ARCH + kbuild.NVCC_FLAGS + [str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert out.split("\n")[:3] == ["0 7 0", "8 7 1", "128 7 1"]


def test_sizes_at_which_32_bit_positions_end_are_refused():
    """Tables of nearly 2^31 tokens, lists of nearly 2^31 pages: a kernel's step beyond the last position would wrap."""
    kbuild.build()
    L = kvq.lib()
    c = kvq.kvq_paged_cache()
    assert L.kvq_paged_cache_init(ctypes.byref(c), 0, 10, 1, 1, 128) == 0
    c.k = c.v = c.key_bounds = 4096
    P = ctypes.c_void_p(4096)

    def select(width, n_select):
        return L.kvq_paged_select(ctypes.byref(c), P, width, 1, P, P, 0, 128, 1, n_select, 0, 0, None, P, 8, None)

    def sparse(width, n_select):
        return L.kvq_paged_sparse_attn(ctypes.byref(c), P, width, 1, P, P, 0, 128, 1, P, n_select, 0.1, None, None, P, 8,
                                       None)

    most = 2**31 - 65536
    for call, missing in ((select, b"sel is"), (sparse, b"out is")):
        assert call(most + 1, 4) == -1 and b"tokens" in L.kvq_last_error()
        assert call(100, 2**30 + 1) == -1 and b"n_select" in L.kvq_last_error()
        assert call(100, 2**31 - 1) == -1 and b"n_select" in L.kvq_last_error()
        assert call(most, 2**30) == -1 and missing in L.kvq_last_error()  # these sizes pass: refused for the NULL behind
