"""Workspace of the operators' K splits, computed on the host (no GPU): no more
than the plans of a handle's calls use, and enough for the plans they would take
with more."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_moe_decode_gemv_gb300", "csrc")

PROGRAM = r"""
#include <chrono>
#include <cstdio>
#include "moe_qgemm.cuh"
using namespace moe_op;
int main() {
  int bad = 0, cases = 0;
  size_t largest = 0;
  double slowest = 0;
  for (int N : {1, 6, 96, 333, 1026, 4096, 8191, 16384, 46552})
    for (int chunks : {1, 15, 16, 29, 64, 96, 256, 1024})
      for (int M = 1; M <= 2; ++M)
        for (int top : {16, 64, 300, 2048}) {
          const auto t0 = std::chrono::steady_clock::now();
          const size_t part = qg_part_bytes(W_AFFINE, 4, M, chunks, top, N, 152);
          slowest = std::max(slowest, std::chrono::duration<double>(std::chrono::steady_clock::now() - t0).count());
          largest = std::max(largest, part);
          size_t used = 0;
          for (int T = 1; T <= top; ++T, ++cases) {
            const QGemmPlan a = qg_plan(W_AFFINE, 4, M, chunks, T, N, 152, part);
            const QGemmPlan b = qg_plan(W_AFFINE, 4, M, chunks, T, N, 152, 64u << 20);
            if (a.ksplit > 1) used = std::max(used, static_cast<size_t>(a.ksplit) * T * ((N + 3) / 4 * 4) * M * 4);
            bad += a.ksplit != b.ksplit || a.ntok != b.ntok || a.units != b.units || a.slots != b.slots;
          }
          bad += used > part || part > used + used / 64 + 4096 * 64;
        }
  // a projection as models have them, for up to 4096 rows: it used to hold 64 MB
  const size_t square = qg_part_bytes(W_AFFINE, 4, 1, 64, 4096, 4096, 152);
  std::printf("%d plans, %d bad, largest %zu, 4096 x 4096: %zu, slowest %.3f s\n", cases, bad, largest, square, slowest);
  return bad || square > (24u << 20) || slowest > 2;
}
"""


def test_split_workspace_is_what_the_plans_use(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    src = tmp_path / "part_check.cu"
    src.write_text(PROGRAM)
    exe = tmp_path / "part_check"
    r = subprocess.run([nvcc, "-O2", "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "--expt-relaxed-constexpr",
                        "-I", os.path.join(ROOT, "include"), "-I", CSRC, str(src), "-o", str(exe)],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    print(r.stdout)
