// How the orthogonalised update's products are cut into units (host side, no CUDA calls).
#pragma once

#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "moe_ortho.cuh"

namespace moe_op {

inline int64_t or_parts(int64_t n, int side) { return (n + side - 1) / side; }

// Counters of split tiles: K is split where all splits run at once.
inline int ortho_counters(int sms) { return 3 * sms * OR_EPI_WARPS; }

constexpr int OR_MAX_SPLIT = 16;

// How n matrices are taken: CTAs of a tile (1: 128 x 128, 2: 256 x 256), matrices that go
// through the steps together, and the K splits of the three products.
struct OrthoPlan {
  int cg = 1;
  int group = 1;
  int ks[3] = {1, 1, 1};
  double clocks = 1e30;
  int tiles[3], kb[3];
  size_t part_bytes(int n) const {
    size_t t = 0;
    for (int p = 0; p < 3; ++p)
      if (ks[p] > 1) t += static_cast<size_t>(n) * tiles[p] * ks[p] * cg * or_part_floats(cg) * 4;
    return t;
  }
};

// What a matrix keeps in the L2 while it goes through its steps.
inline int64_t or_resident_bytes(int rows, int cols) {
  const int64_t m = std::min(rows, cols);
  return 6ll * rows * cols + 4 * m * m;
}
constexpr int64_t OR_RESIDENT = 100ll << 20;   // of 129 MB

// The least estimated time in SM clocks.  A product takes its tiles over the workers (whole
// rounds of them for one matrix; several matrices' products fill each other's last
// rounds) times a tile's K blocks, then the way of its last tile to whoever waits for it;
// a K split adds its partial sums' way through memory.  Measured on 1024 x 4096: a K block
// of a 128 x 128 tile 440 clocks with all CTAs at work (its bytes; its MMAs take 256), a
// pair's of 256 x 256 550 (512); joining 4 splits 3.5 us.
inline OrthoPlan ortho_plan(int rows, int cols, int n, const int (&workers)[3]) {
  OrthoPlan best;
  const int m = std::min(rows, cols);
  for (int cg = 1; cg <= 2; ++cg) {
    OrthoPlan p;
    p.cg = cg;
    p.clocks = 0.0;
    const int W = workers[cg];
    for (int mode = 0; mode < 3; ++mode) {
      p.tiles[mode] = mode == OR_APPLY ? or_tiles(mode, cg, rows, cols) : or_tiles(mode, cg, m, m);
      p.kb[mode] = ((mode == OR_GRAM ? std::max(rows, cols) : m) + 63) / 64;
    }
    // groups: of the matrices that the L2 holds, or of two rounds of tiles of the smaller products, so
    // that a matrix's products finish while others' run.  Up to three groups' worth go as one: no last
    // round of tiles is paid for between groups.  As groups / as one, us: 16 of 1856 x 1024 (1.0 groups)
    // 669 / 558, 24 of 1024 x 1024 (1.5) 583 / 541, 40 (2.5) 931 / 895, 12 of 1536 x 1536 (1.5) 734 / 710, 3 of 4096 x
    // 4096 (1.5) 3100 / 2709; 60 of 1856 x 1024 (3.8) 2189 / 2334, 300 of 640 x 640 (11.5) 2386 / 2892, 2000 of
    // 256 x 256 (13) 2506 / 2687, 200 of 1024 x 1024 (12.5) 4508 / 4733.
    const int64_t fit = std::max<int64_t>(OR_RESIDENT / or_resident_bytes(rows, cols), or_parts(2 * W, p.tiles[OR_GRAM]));
    const int64_t groups = n <= 3 * fit ? 1 : or_parts(n, static_cast<int>(fit));
    p.group = static_cast<int>(or_parts(n, static_cast<int>(groups)));
    for (int mode = 0; mode < 3; ++mode) {
      const double T = static_cast<double>(p.tiles[mode]) * p.group;
      double least = 1e30;
      for (int ks = 1; ks <= OR_MAX_SPLIT; ++ks) {
        if (ks > 1 && (groups > 1 || T * ks > W || p.kb[mode] / ks < 2)) break;
        const double rounds = n > 1 ? std::max(1.0, T * ks / W) : std::ceil(T * ks / W);
        const double kb = cg == 2 ? 550.0 : 260.0 + 180.0 * std::min(1.0, T * ks / W);
        const double t = rounds * ((p.kb[mode] + ks - 1) / ks) * kb + (cg == 2 ? 9000.0 : 6000.0) +
                         (ks > 1 ? (cg == 2 ? 9000.0 : 5000.0) + ks * 300.0 : 0.0);
        if (t < least) {
          least = t;
          p.ks[mode] = ks;
        }
      }
      p.clocks += least * groups;
    }
    if (p.clocks < best.clocks) best = p;
  }
  return best;
}

// The products of a plan for the kernel, their partial sums at `part` and counters at `arrived`;
// workers: resident CTAs or pairs.  Returns how many workers have something to do.
inline int ortho_phases(const OrthoPlan& p, int rows, int cols, int n, const int (&workers)[3], float* part, unsigned* arrived, OrthoArgs* a) {
  const int m = std::min(rows, cols);
  int64_t units = 0;
  for (int mode = 0; mode < 3; ++mode) {
    OrthoPhase& f = a->ph[mode];
    f.M = mode == OR_APPLY ? rows : m;
    f.N = mode == OR_APPLY ? cols : m;
    f.tiles = p.tiles[mode];
    f.kb = p.kb[mode];
    f.ks = p.ks[mode];
    const int64_t all = static_cast<int64_t>(p.group) * f.tiles * f.ks;
    units = std::max(units, all);
    f.part = part;
    f.arrived = arrived;
    if (f.ks > 1) {
      part += all * p.cg * or_part_floats(p.cg);
      arrived += n * f.tiles * p.cg * OR_EPI_WARPS;
    }
  }
  a->matrices = n;
  a->group = p.group;
  return static_cast<int>(std::min<int64_t>(units, workers[p.cg]));
}

}  // namespace moe_op
