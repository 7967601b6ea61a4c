"""The slot ring of the 4-bit tensor-core GEMM on the host (no GPU): every wait of
a decode warp has to know which release it waits for.

A barrier tells the parity of its releases only.  A warp that waits at block n (for
the release of block n - S, S slots) is let through at once when block n - 2 S has
not been released either, so before it waits it must have seen that one released;
releases come in order, so its last wait has to lie at block n - S or later.  The
walk that the kernel takes through its units' K blocks is compiled for the host and
held to that for every ring size, both decode groups and sequences of units of
every length, and so is the walk that passes over the other group's blocks without
waiting, which breaks it where units meet."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_moe_decode_gemv_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "moe_qgemm.cuh"
using namespace moe_op;

struct Result {
  int early = 0;       // waits that one release further behind would satisfy
  int wrong = 0;       // waits at another slot or parity than their block's, fills without a wait
  std::vector<int> filled;
};

// One decode group over units of the given K blocks; the pair's body as in the kernel.
template <bool GATED>
Result run(int S, int half, const std::vector<int>& units, bool blind) {
  Result R;
  QGemmRing Q;
  Q.S = S;
  int seen = -1;       // block of the last wait
  auto wait = [&](int n, int slot, uint32_t parity) {
    if (slot != n % S || parity != static_cast<uint32_t>((n / S - 1) & 1) || n < S) ++R.wrong;
    if (n >= 2 * S && seen < n - S) ++R.early;
    seen = n;
    return true;
  };
  auto fill = [&](int n) {   // the slot's former block has been released: some wait at n or later, or none needed
    if (n >= S && seen < n) ++R.wrong;
    R.filled.push_back(n);
  };
  const bool pairs = S >= 4;
  for (int L : units) {
    auto pair = [&](int c) {
      const bool two = c + 1 < L;
      if (pairs && two) {
        const int n = Q.block;
        Q.skip(1);
        Q.free_slot(wait);
        fill(n);
        fill(n + 1);
        Q.skip(1);
      } else {
        for (int i = 0; i < (two ? 2 : 1); ++i) {
          Q.free_slot(wait);
          fill(Q.block);
          Q.skip(1);
        }
      }
      return true;
    };
    if (!blind) {
      qg_walk<GATED>(Q, 0, L, half, pair, wait);
    } else {   // the other group's blocks are skipped, not waited for
      const int first = GATED ? 0 : 2 * half, step = GATED ? 2 : 4;
      Q.skip(first < L ? first : L);
      for (int c = first; c < L; c += step) {
        pair(c);
        if (!GATED) {
          const int end = c + step < L ? c + step : L;
          Q.skip(end > c + 2 ? end - (c + 2) : 0);
        }
      }
    }
  }
  return R;
}

template <bool GATED>
void check(int S, const std::vector<int>& units, bool blind, int* early, int* wrong, int* missing) {
  int total = 0;
  for (int L : units) total += L;
  std::vector<int> times(total, 0);
  for (int half = 0; half < 2; ++half) {
    const Result r = run<GATED>(S, half, units, blind);
    *early += r.early;
    *wrong += r.wrong;
    for (int n : r.filled) ++times[n];
  }
  for (int t : times) *missing += t != (GATED ? 2 : 1);
}

int main() {
  int early = 0, wrong = 0, missing = 0, cases = 0, blind_bad = 0;
  std::vector<std::vector<int>> seqs;
  for (int a = 1; a <= 41; ++a) {
    seqs.push_back(std::vector<int>(9, a));
    for (int b = 1; b <= 41; b += 3) {
      std::vector<int> v;
      for (int i = 0; i < 6; ++i) v.insert(v.end(), {a, b, a});
      seqs.push_back(v);
    }
  }
  for (const auto& q : seqs) {
    for (int S = 3; S <= QG_MAX_SLOTS; ++S, ++cases) check<false>(S, q, false, &early, &wrong, &missing);
    for (int S = 2; S <= QG_MAX_SLOTS; ++S, ++cases) check<true>(S, q, false, &early, &wrong, &missing);
  }
  for (int L : {30, 42}) {   // 1920 and 2688 columns, three slots
    int e = 0, w = 0, m = 0;
    check<false>(3, std::vector<int>(7, L), true, &e, &w, &m);
    blind_bad += e > 0;
  }
  // a plan with one matrix has three slots or more, with two at least two
  int few = 0, plans = 0;
  const int fmts[4][2] = {{W_AFFINE, 2}, {W_AFFINE, 4}, {W_NVFP4, 4}, {W_MXFP4, 4}};
  for (const auto& f : fmts)
    for (int T = 1; T <= 2100; T += T < 600 ? 1 : 37)
      for (int N : {1, 300, 4096, 16384, 70000})
        for (int chunks : {1, 30, 64, 1024})
          for (int M = 1; M <= 2; ++M, ++plans) {
            const QGemmPlan P = qg_plan(f[0], f[1], M, chunks, T, N, 152, 64u << 20);
            few += P.slots < (M == 1 ? 3 : 2) || P.slots > QG_MAX_SLOTS || P.depth < 2 || P.depth > 3 || P.ntok < 16 ||
                   P.ntok > 256 || qg_smem_bytes(f[0], f[1], M, P.ntok, P.slots, P.depth) > QG_SMEM_MAX;
          }
  std::printf("%d cases: early %d wrong %d missing %d; blind %d of 2; %d plans, %d with too few slots\n", cases, early,
              wrong, missing, blind_bad, plans, few);
  return early || wrong || missing || blind_bad != 2 || few;
}
"""


def test_every_wait_knows_its_release(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    src = tmp_path / "ring_check.cu"
    src.write_text(PROGRAM)
    exe = tmp_path / "ring_check"
    r = subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "--expt-relaxed-constexpr",
                        "-I", os.path.join(ROOT, "include"), "-I", CSRC, str(src), "-o", str(exe)],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
