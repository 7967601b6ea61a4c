"""Workspace of the orthogonalised update, computed on the host (no GPU)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_moe_decode_gemv_gb300", "csrc")

NORMS = r"""
#include <cstdio>
#include "moe_ortho.cuh"
using namespace moe_op;
// The norms' partial sums of every call fit, and are no more than the header says.
int main() {
  int bad = 0, cases = 0;
  for (int sms : {1, 148, 152})
    for (int R : {1, 16, 64, 200, 1000, 8192, 32768})
      for (int C : {1, 16, 100, 513, 4096, 32768})
        for (int64_t top : {1, 2, 7, 152, 153, 1216, 1217, 65536}) {
          const int64_t room = or_norm_parts(R, C, top, sms);
          const int64_t eights = (R * ((C + 7) / 8) + 1023) / 1024;
          bad += room > 8 * sms + top || room > eights * top;
          for (int64_t n = 1; n <= top; n += n < 300 || n > top - 5 ? 1 : 37, ++cases) {
            const int c = or_start_ctas(R, C, n, sms);
            bad += c < 1 || c > OR_NORM_CTAS || (c > 1 && n * c > room);
          }
        }
  std::printf("%d cases, %d bad\n", cases, bad);
  return bad;
}
"""


def run(tmp_path, program):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    src = tmp_path / "check.cu"
    src.write_text(program)
    exe = tmp_path / "check"
    r = subprocess.run([nvcc, "-O2", "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "--expt-relaxed-constexpr",
                        "-I", os.path.join(ROOT, "include"), "-I", CSRC, str(src), "-o", str(exe)],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    print(r.stdout)
    assert r.returncode == 0, r.stdout + r.stderr


def test_partial_sums_of_norms(tmp_path):
    run(tmp_path, NORMS)
