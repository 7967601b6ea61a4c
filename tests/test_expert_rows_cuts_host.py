"""Rows that begin anywhere in a 16-byte word: the kernels' own arithmetic of words (which word a lane
reads and writes, how two lanes' elements make one, the ends of a piece), compiled for the host and
run for a warp's lanes in turn (no GPU needed)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_moe_decode_gemv_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <cstring>
#include <vector>
#include "moe_rows.cuh"
using namespace moe_op;
using u16 = unsigned short;

// As rw_put does: lanes that have no word of their own, and those without an end element, write nothing.
void put(u16* row, int piece, int H, const u16 (&values)[256], std::vector<int>& times, const u16* base) {
  const int shift = rw_shift(row);
  RowPiece lanes[32];
  std::memcpy(lanes, values, sizeof values);
  const RowEnds ends = rw_ends(piece, H, shift);
  for (int lane = 0; lane < 32; ++lane) {
    const int c = (piece * 32 + lane) * 8;
    const RowPiece g = rw_join(lanes[lane ? lane - 1 : 0], lanes[lane], shift);
    if (rw_whole(ends, c, shift)) {
      u16* p = row + c - shift;
      if (reinterpret_cast<uintptr_t>(p) % 16) times[0] += 1000;   // not a whole word
      std::memcpy(p, &g, 16);
      for (int i = 0; i < 8; ++i) ++times[p + i - base];
    }
    int e;
    if (rw_end(ends, lane, &e)) {
      row[ends.c0 + e] = values[e];
      ++times[row + ends.c0 + e - base];
    }
  }
}

int main() {
  int bad = 0, cases = 0;
  alignas(16) static u16 memory[4096];
  std::vector<int> widths;
  for (int H = 1; H <= 40; ++H) widths.push_back(H);
  for (int H = 240; H <= 280; ++H) widths.push_back(H);
  for (int H : {500, 511, 512, 513, 521, 767, 768, 769, 1001}) widths.push_back(H);
  for (int shift = 0; shift < 8; ++shift)
    for (int H : widths) {
      ++cases;
      // written: each element of the row once, with its value, and no other
      std::memset(memory, 0xEE, sizeof memory);
      std::vector<int> times(4096, 0);
      u16* row = memory + 800 + shift;
      for (int piece = 0; piece * 256 < H; ++piece) {
        u16 values[256];
        for (int i = 0; i < 256; ++i) values[i] = static_cast<u16>(piece * 256 + i < H ? 7 + piece * 256 + i : 0xABCD);
        put(row, piece, H, values, times, memory);
      }
      for (int i = 0; i < 4096; ++i) {
        const int c = i - 800 - shift;
        const bool in = c >= 0 && c < H;
        bad += times[i] != (in ? 1 : 0) || memory[i] != (in ? static_cast<u16>(7 + c) : 0xEEEE);
      }
      // read by way of a slot: the row's elements, zeros behind it; nothing that lies behind the row is touched,
      // and before it only what shares its first word
      for (int i = 0; i < 4096; ++i) memory[i] = static_cast<u16>(i);
      for (int piece = 0; piece * 256 < H; ++piece) {
        u16 slot[264] = {};
        auto part = [&](int to, const u16* from, int bytes) {
          if (reinterpret_cast<uintptr_t>(from) % 16 || bytes % 2 || bytes < 0 || bytes > 16) ++bad;
          if (bytes && (from + bytes / 2 > row + H || from < row - shift)) ++bad;
          std::memset(slot + to, 0, 16);
          std::memcpy(slot + to, from, bytes);
        };
        for (int lane = 0; lane < 32; ++lane) {
          const int c = (piece * 32 + lane) * 8;
          const int left = rw_left(c, shift, H), own = rw_own_bytes(left), next = rw_next_bytes(left, shift);
          part(lane * 8, own ? row + c - shift : row - shift, own);
          if (lane == 31) part(256, next ? row + c - shift + 8 : row - shift, next);
        }
        for (int lane = 0; lane < 32; ++lane) {
          uint32_t x[5];
          const int at = rw_slot_at(lane, shift);
          if (at % 4 || at + 20 > rw_slot_row(false)) ++bad;
          std::memcpy(x, reinterpret_cast<const char*>(slot) + at, 20);
          const RowPiece v = rw_cut(x, shift & 1);
          u16 got[8];
          std::memcpy(got, &v, 16);
          for (int i = 0; i < 8; ++i) {
            const int c = (piece * 32 + lane) * 8 + i;
            if (c < H) bad += got[i] != static_cast<u16>(800 + shift + c);
            else if (c < (piece + 1) * 256) bad += got[i] != 0;
          }
        }
      }
    }
  std::printf("%d cases, %d bad\n", cases, bad);
  return bad != 0;
}
"""


def test_words_of_a_piece(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    src = tmp_path / "cuts.cu"
    src.write_text(PROGRAM)
    exe = tmp_path / "cuts"
    r = subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "--expt-relaxed-constexpr",
                        "-I", os.path.join(ROOT, "include"), "-I", CSRC, str(src), "-o", str(exe)],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
