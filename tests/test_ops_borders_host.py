"""The restated rule of which 4-bit calls stream (ops_borders) is the library's (no GPU needed)."""
import os
import shutil
import subprocess

import pytest

from tests import ops_borders as ob

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_moe_decode_gemv_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "moe_stream.cuh"
using namespace moe_op;
int main() {
  const int fmts[5][3] = {{W_AFFINE, 2, 32}, {W_AFFINE, 4, 64}, {W_AFFINE, 4, 128}, {W_NVFP4, 4, 16}, {W_MXFP4, 4, 32}};
  for (int f = 0; f < 5; ++f)
    for (int mats = 1; mats <= 2; ++mats)
      for (int K : {64, 640, 1920, 4096, 6144, 8192, 14336, 28672, 65536}) {
        int most = 0;
        for (int T = 1; T <= 16; ++T) {
          StreamPlan P;
          if (st_plan(fmts[f][0], mats == 2, fmts[f][1], (K + 63) / 64, T, 4096, 152, &P)) most = T;
        }
        std::printf("%d %d %d %d\n", f, mats, K, most);
      }
}
"""
FMTS = [("affine", 32), ("affine", 64), ("affine", 128), ("nvfp4", 16), ("mxfp4", 32)]


def test_streamed_rows(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    src, exe = tmp_path / "border.cu", tmp_path / "border"
    src.write_text(PROGRAM)
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "--expt-relaxed-constexpr", "-I",
                    os.path.join(ROOT, "include"), "-I", CSRC, str(src), "-o", str(exe)], check=True, timeout=600)
    lines = subprocess.run([str(exe)], capture_output=True, text=True, check=True, timeout=60).stdout.split("\n")
    rows = [tuple(map(int, l.split())) for l in lines if l]
    assert len(rows) == 90
    for f, mats, K, most in rows:
        assert ob.most_streamed_rows(*FMTS[f], mats, K) == most, (FMTS[f], mats, K)
    # the border lies below 16 rows where x is wide, and nothing is streamed at some widths
    assert ob.most_streamed_rows("affine", 64, 1, 4096) == 16 and 0 < ob.most_streamed_rows("affine", 64, 1, 14336) < 8
