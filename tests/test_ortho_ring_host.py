"""The ring between the orthogonalised update's epilogue warps and the warp that counts their
units, on the host (no GPU): every unit is counted once, after all of its warps have stored it,
in whatever order the warps run.

Barriers are modelled as the hardware has them: a wait for a parity is let through while the
phase under way has the other one, which says nothing of how many phases lie between.  The
slots, parities and waits are the kernel's own (or_slot, compiled for the host), and the
same walk without the wait for `taken` goes wrong, so the model sees what it is for."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_moe_decode_gemv_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "moe_ortho.cuh"
using namespace moe_op;

struct Barrier {
  int count, pending, phase = 0;
  explicit Barrier(int n) : count(n), pending(n) {}
  void arrive() {
    if (--pending == 0) {
      ++phase;
      pending = count;
    }
  }
  bool done(uint32_t parity) const { return (static_cast<uint32_t>(phase) & 1u) != parity; }
};

// One CTA with `units` units.  Order: 0 at random, 1 the counting warp only when nobody else can go on,
// 2 one epilogue warp as far behind as it can be, 3 one as far ahead.
// Wrong: units counted before their eighth arrival, or not at all.
int run(int units, int order, bool ring, unsigned seed) {
  std::vector<Barrier> stored(OR_STORED, Barrier(OR_EPI_WARPS)), taken(OR_STORED, Barrier(1));
  std::vector<int> arrivals(units, 0);
  uint32_t at[OR_EPI_WARPS] = {}, counted = 0;
  int wrong = 0;
  auto store = [&](int w) {
    const uint32_t n = at[w];
    if (n >= static_cast<uint32_t>(units)) return false;
    // (what else holds them together: accumulators of two units, released by all eight warps)
    for (uint32_t v : at)
      if (n >= v + 2) return false;
    const OrthoSlot q = or_slot(n);
    if (ring && q.again && !taken[q.slot].done(q.parity ^ 1u)) return false;
    stored[q.slot].arrive();
    ++arrivals[n];
    ++at[w];
    return true;
  };
  auto take = [&] {
    if (counted >= static_cast<uint32_t>(units)) return false;
    const OrthoSlot q = or_slot(counted);
    if (!stored[q.slot].done(q.parity)) return false;
    wrong += arrivals[counted] != OR_EPI_WARPS;
    if (ring) taken[q.slot].arrive();
    ++counted;
    return true;
  };
  unsigned x = seed * 2654435761u + 1u;
  auto any = [&](int n) {
    x = x * 1664525u + 1013904223u;
    return static_cast<int>((x >> 8) % static_cast<unsigned>(n));
  };
  for (;;) {
    bool moved = false;
    if (order == 0) {
      for (int tries = 0; tries < 200 && !moved; ++tries) {
        const int w = any(OR_EPI_WARPS + 1);
        moved = w == OR_EPI_WARPS ? take() : store(w);
      }
    }
    if (order == 1)
      for (int w = 0; w < OR_EPI_WARPS && !moved; ++w) moved = store((w + any(OR_EPI_WARPS)) % OR_EPI_WARPS);
    if (order == 2)
      for (int w = OR_EPI_WARPS - 1; w >= 0 && !moved; --w) moved = store(w);
    if (order == 3)
      for (int w = 0; w < OR_EPI_WARPS && !moved; ++w) moved = store(w);
    for (int w = 0; w < OR_EPI_WARPS && !moved; ++w) moved = store(w);
    if (!moved) moved = take();
    if (!moved) break;
  }
  return wrong + units - static_cast<int>(counted);
}

int main() {
  int bad = 0, cases = 0, blind = 0;
  for (int order = 0; order < 4; ++order)
    for (int units : {1, 2, 3, 4, 5, 7, 8, 9, 16, 33, 400})
      for (unsigned seed = 0; seed < 20; ++seed, ++cases) {
        bad += run(units, order, true, seed) != 0;
        blind += order == 1 && units > 8 && run(units, order, false, seed) == 0;
      }
  const bool fits = or_smem_bytes(5) <= OR_SMEM_MAX;   // as many slots of operands as without `taken`
  std::printf("%d cases: %d wrong; without the wait %d right that should not be\n", cases, bad, blind);
  return bad || blind || !fits;
}
"""


def test_every_unit_is_counted_once(tmp_path):
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
