"""How the orthogonalised update's products are cut, on the host (no GPU): the plans, the list of
units that the kernel's CTAs take, workspace and counters, by the functions that the kernel and its launch
use, compiled for the host.

For every plan over sizes, stacks and GPUs of several SM counts:
  - every tile and K split of every product of every step is one unit of the list, and the K splits
    of a tile cover its K blocks, none empty;
  - a unit waits for products whose units all lie before it in the list, until as many of their
    warps as there are have finished; splits of a tile, which wait for each other, are on
    different CTAs, as are all units of a split product;
  - partial sums and counters of a split lie apart from all others and inside what a handle has.
And the shapes of the GPU tests take every kind of plan that there is."""
import json

import pytest

from tests.test_ortho_workspace_host import run

# rows, cols, matrices: what the GPU tests run on 152 SMs, one or more for each kind of plan
SHAPES = [
    (300, 260, 1), (260, 300, 1), (520, 1030, 1), (1030, 520, 1), (1500, 4100, 1), (4100, 1500, 1), (2050, 4100, 1), (4100, 2050, 1),
    (1024, 4096, 1), (4100, 1000, 1), (2048, 7168, 1), (7168, 2048, 1), (1281, 9000, 1), (9000, 1281, 1), (2600, 2600, 2), (2700, 2500, 2),
    (760, 9000, 2), (9001, 755, 2), (1270, 6000, 2),
    (300, 4000, 4), (4000, 300, 4), (130, 1100, 3), (1100, 130, 3), (1030, 520, 2), (520, 1030, 2),
    (1856, 1024, 16), (1024, 1856, 16), (1100, 2100, 19), (2100, 1100, 19), (640, 640, 100), (640, 600, 100),
    (1100, 1300, 50), (1300, 1100, 50),
]

PROGRAM = r"""
#include <cstdio>
#include <cstring>
#include <map>
#include <random>
#include <set>
#include <string>
#include <vector>
#include "moe_ortho_plan.h"
using namespace moe_op;

int bad = 0;
void expect(bool ok, const char* what, int R, int C, int n) {
  if (!ok && ++bad < 20) std::printf("%s: %d x %d, %d matrices\n", what, R, C, n);
}

std::string kind(const OrthoPlan& p, int R, int C, int n) {
  char s[64];
  std::snprintf(s, sizeof s, "%s %s %s%s%s%s%s", p.cg == 2 ? "pairs" : "single", R > C ? "tall" : "wide",
                n == 1 ? "one" : p.group < n ? "groups" : "stack", p.ks[0] + p.ks[1] + p.ks[2] > 3 ? " split" : "",
                p.ks[0] > 1 ? "G" : "", p.ks[1] > 1 ? "P" : "", p.ks[2] > 1 ? "A" : "");
  return s;
}

template <int CG>
void check_units(const OrthoPlan& p, int R, int C, int n, const int (&workers)[3], int sms, size_t room) {
  OrthoArgs a{};
  std::vector<unsigned> done(3 * static_cast<size_t>(n));
  float* const part = reinterpret_cast<float*>(1 << 20);
  unsigned* const arrived = reinterpret_cast<unsigned*>(1 << 20);
  a.steps = 2;
  a.done = done.data();
  const int busy = ortho_phases(p, R, C, n, workers, part, arrived, &a);
  expect(busy >= 1 && busy <= workers[CG], "workers", R, C, n);
  const int groups = (n + p.group - 1) / p.group;
  int64_t units = 0;
  for (int i = 0; i < 3; ++i) units += static_cast<int64_t>(a.ph[i].tiles) * a.ph[i].ks;
  units *= static_cast<int64_t>(n) * a.steps;
  std::map<std::vector<int>, int64_t> first, last;          // (z, step, mode): where its units lie
  std::map<std::vector<int>, std::set<std::vector<int>>> tiles;
  std::map<std::vector<int>, int> blocks;                   // of a tile, by all of its splits
  std::map<std::vector<int>, std::set<int64_t>> on;         // workers of a split product
  std::set<int64_t> sums, counters;
  for (int64_t g = 0; g < units; ++g) {
    const OrthoUnit U = or_unit<CG>(a, g);
    const OrthoPhase& f = a.ph[U.mode];
    expect(U.z >= 0 && U.z < n && U.step >= 0 && U.step < a.steps && U.m0 >= 0 && U.m0 < f.M && U.n0 >= 0 && U.n0 < f.N &&
               U.m0 % (CG * 128) == 0 && U.n0 % (CG * 128) == 0 && (U.mode == OR_APPLY || U.n0 <= U.m0),
           "unit out of range", R, C, n);
    expect(U.nkb >= 1 && U.kb0 >= 0 && U.kb0 + U.nkb <= f.kb && U.ks == f.ks, "K blocks", R, C, n);
    const std::vector<int> product{U.z, U.step, U.mode}, tile{U.z, U.step, U.mode, U.m0, U.n0};
    if (!first.count(product)) first[product] = g;
    last[product] = g;
    tiles[product].insert({U.m0, U.n0});
    blocks[tile] += U.nkb;
    if (U.step == 0 && f.ks > 1) {
      expect(sums.insert((f.part - part) + static_cast<int64_t>(U.unit) * CG * or_part_floats(CG)).second, "partial sums shared", R, C, n);
      if (U.split == 0)
        for (int i = 0; i < CG * OR_EPI_WARPS; ++i)
          expect(counters.insert((f.arrived - arrived) + U.tile * CG * OR_EPI_WARPS + i).second, "counters shared", R, C, n);
      expect(on[{U.mode}].insert(g % busy).second, "a split product's units on one worker", R, C, n);
    }
  }
  for (const auto& b : blocks) expect(b.second == a.ph[b.first[2]].kb, "a tile's K blocks", R, C, n);
  for (const auto& t : tiles) expect(static_cast<int>(t.second.size()) == a.ph[t.first[2]].tiles, "a product's tiles", R, C, n);
  expect(first.size() == static_cast<size_t>(n) * a.steps * 3, "products", R, C, n);
  for (int64_t g = 0; g < units; ++g) {
    const OrthoUnit U = or_unit<CG>(a, g);
    unsigned count = 0;
    const unsigned* d = or_needs<CG>(a, U, &count);
    const int from = U.mode == OR_GRAM ? OR_APPLY : U.mode - 1;
    const int rounds = U.mode == OR_GRAM ? U.step : U.step + 1;
    expect(d == a.done + U.z * 3 + from, "the counter of another product", R, C, n);
    expect(count == static_cast<unsigned>(rounds * a.ph[from].tiles * a.ph[from].ks * OR_EPI_WARPS * CG), "the count", R, C, n);
    for (int s = 0; s < rounds; ++s) expect(last[{U.z, s, from}] < first[{U.z, U.step, U.mode}], "waits for a later unit", R, C, n);
  }
  for (int64_t at : sums) expect(at >= 0 && static_cast<size_t>(at + CG * or_part_floats(CG)) * 4 <= room, "partial sums outside", R, C, n);
  for (int64_t at : counters) expect(at >= 0 && at < ortho_counters(sms), "counters outside", R, C, n);
  expect(groups == 1 || sums.empty(), "splits in several groups", R, C, n);
}

void check(int R, int C, int n, int sms, size_t room, bool walk) {
  const int workers[3] = {0, sms, sms / 2};
  const OrthoPlan p = ortho_plan(R, C, n, workers);
  expect(p.part_bytes(n) <= room, "workspace", R, C, n);
  expect(p.group >= 1 && p.group <= n, "group", R, C, n);
  if (walk) p.cg == 2 ? check_units<2>(p, R, C, n, workers, sms, room) : check_units<1>(p, R, C, n, workers, sms, room);
}

// As a handle's create sizes it.
size_t room_of(int R, int C, int top, int sms) {
  const int workers[3] = {0, sms, sms / 2};
  size_t room = 0;
  for (int i = 1; i <= std::min(top, sms); ++i) room = std::max(room, ortho_plan(R, C, i, workers).part_bytes(i));
  return room;
}

int main() {
  std::mt19937 rng(7);
  auto size = [&](int most) { return static_cast<int>(std::exp(std::uniform_real_distribution<>(0.0, std::log(most + 0.99))(rng))); };
  int cases = 0;
  std::map<std::string, int> kinds;
  for (int i = 0; i < 1500; ++i) {
    const int sms = i % 4 == 0 ? 20 : i % 4 == 1 ? 132 : 152, R = size(9000), C = size(9000), top = i % 2 ? 1 : size(400);
    const size_t room = room_of(R, C, top, sms);
    for (int j = 0; j < 3; ++j, ++cases) {
      const int n = j == 0 ? top : std::min(top, size(top));
      const int64_t tiles = or_parts(R, 128) * or_parts(C, 128) * n;
      check(R, C, n, sms, room, tiles < 3000);
    }
  }
  const int workers[3] = {0, 152, 76};
  for (int i = 0; i < 60000; ++i) {   // what kinds there are
    const int R = size(32768), C = size(32768), n = i % 2 ? 1 : size(300);
    ++kinds[kind(ortho_plan(R, C, n, workers), R, C, n)];
  }
  std::map<std::string, int> taken;
  const int shapes[][3] = {SHAPES};
  for (const auto& s : shapes) {
    ++taken[kind(ortho_plan(s[0], s[1], s[2], workers), s[0], s[1], s[2])];
    check(s[0], s[1], s[2], 152, room_of(s[0], s[1], s[2], 152), true);
  }
  int missing = 0;
  for (const auto& k : kinds) {
    if (!taken.count(k.first)) ++missing;
    std::printf("%-28s %6d  %s\n", k.first.c_str(), k.second, taken.count(k.first) ? "" : "MISSING");
  }
  std::printf("%d plans, %d bad, %d kinds without a GPU test\n", cases, bad, missing);
  return bad || missing;
}
"""


def test_plans(tmp_path):
    shapes = json.dumps(SHAPES).replace("[", "{").replace("]", "}")[1:-1]
    run(tmp_path, PROGRAM.replace("{SHAPES}", "{" + shapes + "}"))
