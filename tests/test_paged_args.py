"""What the paged cache's host code hands to its kernels, without a GPU."""

from __future__ import annotations

import subprocess

from quantized_cross_loop_gb300 import build as kbuild

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
