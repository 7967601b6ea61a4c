// Products of a streamed 16-bit weight matrix with a few token rows (k_stream16):
// the gated block at decode sizes.
//
//   y[t, n] = sum_k x[t, k] W[n, k],  t < 8 NT (at most 16), W row-major
//
// The time is that of reading W once.  Persistent CTAs take 16-row tiles of W in
// turn; a CTA's 8 warps split a tile's 64-column chunks among them.  Every lane
// keeps its own ring of the next chunks in shared memory, filled by 16-byte
// asynchronous copies that run on over tile boundaries: its pieces of the weights
// and of the token rows (those through L1, where the next tile finds them again).
// A lane reads only what it copied itself, so the ring needs no barrier; one
// barrier a tile joins the warps' partial sums, while the copies of the next
// tiles are under way.  (Bulk copies, one a row and stage, took 12.2 us where
// this takes 5.9 to 6.6 (5.2 to 4.6 TB/s): 30.4 MB at one token; they are 256 bytes each.)
//
// The arithmetic is warp-level mma.sync m16n8k16 with the weights as A and the
// token rows as B (columns of absent tokens are zero).  The MMA's k index runs
// through a chunk's columns in the order in which a lane's 16-byte pieces hold
// them -- lane (g, t): columns 8 t and 32 + 8 t on, of rows g and g + 8 of W and
// of token row g -- so that both come as they lie in memory.
#pragma once

#include "moe_stream.cuh"   // mma_16816, lds16

namespace moe_op {

constexpr int S16_WARPS = 8;
constexpr int S16_THREADS = S16_WARPS * 32;

struct Stream16Args {
  const void *w_gate, *w_up;   // row-major [N, K]
  const void* x;
  int64_t ldx;
  void* out;
  int64_t ldo;
  float *save_gate, *save_up;
  int K, N, T;
  int chunks;               // ceil(K / 64)
  int act;
  int depth;                // stages of a lane's ring, 2..8
};

// One warp's stage: 2 KB of weights a matrix and the token rows' 128 bytes each.
__host__ __device__ inline int s16_stage_bytes(bool gated, int T) { return 2048 * (gated ? 2 : 1) + T * 128; }
__host__ __device__ constexpr int s16_red_floats(bool gated, int nt) { return S16_WARPS * (gated ? 2 : 1) * nt * 128; }
__host__ __device__ inline int s16_smem_bytes(bool gated, int T, int depth) {
  return S16_WARPS * depth * s16_stage_bytes(gated, T) + 2 * 4 * s16_red_floats(gated, T > 8 ? 2 : 1);
}

template <bool FP16, bool GATED, int NT>
__global__ void __launch_bounds__(S16_THREADS, 2) k_stream16(const Stream16Args A) {
  constexpr int M = GATED ? 2 : 1;
  constexpr int DT = FP16 ? DT_FP16 : DT_BF16;
  constexpr int WB = 2048;
  extern __shared__ __align__(128) char st_smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int tiles = (A.N + 15) / 16, D = A.depth;
  const int stage = s16_stage_bytes(GATED, A.T);
  float* red = reinterpret_cast<float*>(st_smem + S16_WARPS * D * stage);
  const uint32_t ring = smem_u32(st_smem) + warp * D * stage;
  // this lane's places in a stage
  const uint32_t o_w = lane * 16, o_x = M * WB;
  // its two 16-byte pieces of token rows g (and g + 8): the slots of odd rows are
  // exchanged so that eight lanes read eight different ones
  const int p0 = t, p1 = t + 4, odd = (g & 1) * 4;
  const uint32_t o_x0 = o_x + g * 128 + (p0 ^ odd) * 16, o_x1 = o_x + g * 128 + (p1 ^ odd) * 16;
  const char* xrow = static_cast<const char*>(A.x) + static_cast<int64_t>(g) * A.ldx * 2;

  auto copy_weights = [&](uint32_t st, int tile, int c) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const char* w = static_cast<const char*>(GATED && m == 0 ? A.w_gate : A.w_up);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = tile * 16 + g + 8 * h;
        const char* wr = w + static_cast<int64_t>(min(row, A.N - 1)) * A.K * 2;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int col = c * 64 + 32 * k + 8 * t;
          const bool in = row < A.N && col < A.K;
          copy16(st + m * WB + (2 * k + h) * 512 + o_w, in ? wr + col * 2 : w, in);
        }
      }
    }
  };
  auto copy_rows = [&](uint32_t st, int c) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (n * 8 + g < A.T) {
        const char* q = xrow + (static_cast<int64_t>(n) * 8 * A.ldx + c * 64) * 2;
        const bool in0 = c * 64 + p0 * 8 < A.K, in1 = c * 64 + p1 * 8 < A.K;
        copy16_l1(st + n * 1024 + o_x0, in0 ? q + p0 * 16 : q, in0);
        copy16_l1(st + n * 1024 + o_x1, in1 ? q + p1 * 16 : q, in1);
      }
    }
  };

  // the next stage to copy: tile and chunk of this warp, and its slot
  const bool some = warp < A.chunks;
  int ct = some ? static_cast<int>(blockIdx.x) : tiles, cc = warp, cs = 0;
  auto advance = [&] {
    cc += S16_WARPS;
    if (cc >= A.chunks) {
      cc = warp;
      ct += gridDim.x;
    }
    if (++cs == D) cs = 0;
  };
  // The first stages.  (The caller's weights and rows may come from the kernel
  // before this one in the stream: nothing is read ahead of it.)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  for (int i = 0; i < D - 1; ++i) {
    if (ct < tiles) {
      copy_weights(ring + cs * stage, ct, cc);
      copy_rows(ring + cs * stage, cc);
    }
    copies_commit();
    advance();
  }

  int slot = 0, buf = 0;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    float acc[M][NT][4];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.0f;
    for (int c = warp; c < A.chunks; c += S16_WARPS) {
      if (ct < tiles) {
        copy_weights(ring + cs * stage, ct, cc);
        copy_rows(ring + cs * stage, cc);
      }
      copies_commit();
      advance();
      copies_wait(D - 1);
      const uint32_t st = ring + slot * stage;
      if (++slot == D) slot = 0;
      // B fragments: 16-column steps j = 0..3, two registers each
      uint32_t bf[NT][8];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
        if (n * 8 + g < A.T) {
          v0 = lds16(st + n * 1024 + o_x0);
          v1 = lds16(st + n * 1024 + o_x1);
        }
        bf[n][0] = v0.x; bf[n][1] = v0.y; bf[n][2] = v0.z; bf[n][3] = v0.w;
        bf[n][4] = v1.x; bf[n][5] = v1.y; bf[n][6] = v1.z; bf[n][7] = v1.w;
      }
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint4 lo = lds16(st + m * WB + 2 * k * 512 + o_w), hi = lds16(st + m * WB + (2 * k + 1) * 512 + o_w);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_16816(acc[m][n], lo.x, hi.x, lo.y, hi.y, bf[n][4 * k], bf[n][4 * k + 1], FP16);
            mma_16816(acc[m][n], lo.z, hi.z, lo.w, hi.w, bf[n][4 * k + 2], bf[n][4 * k + 3], FP16);
          }
        }
    }
    // the warps' partial sums; then one thread per output adds them in warp order
    // (two buffers: the next tile's sums do not wait for these to be read)
    float* rb = red + buf * s16_red_floats(GATED, NT);
    buf ^= 1;
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) rb[((warp * M + m) * NT + n) * 128 + i * 32 + lane] = acc[m][n][i];
    __syncthreads();
    if (tid < NT * 128) {
      const int ei = (tid >> 5) & 3, n = tid >> 7;
      const int row = tile * 16 + g + (ei >> 1) * 8, tok = n * 8 + t * 2 + (ei & 1);
      if (row < A.N && tok < A.T) {
        float v[M];
#pragma unroll
        for (int m = 0; m < M; ++m) {
          v[m] = 0.0f;
#pragma unroll
          for (int w = 0; w < S16_WARPS; ++w) v[m] += rb[((w * M + m) * NT + n) * 128 + (tid & 127)];
        }
        if (A.save_up) {
          const int64_t o = static_cast<int64_t>(tok) * A.N + row;
          if (GATED) A.save_gate[o] = v[0];
          A.save_up[o] = v[M - 1];
        }
        float y = GATED ? act_value(ACT_SWIGLU, v[0], v[M - 1]) : act_value(A.act, 0.0f, v[0]);
        static_cast<unsigned short*>(A.out)[static_cast<int64_t>(tok) * A.ldo + row] = pack1(y, DT);
      }
    }
  }
  copies_wait(0);
}

// Host: depth of the ring and grid of a launch.  Two CTAs an SM where at least
// four stages fit beside each other, else one (the most a stage needs is 6 KB a
// warp: four stages and the sums fit).
constexpr int S16_SMEM_MAX = 226 * 1024;
struct Stream16Plan {
  int depth, grid, smem;
};
inline Stream16Plan s16_plan(bool gated, int T, int N, int sms) {
  const int tiles = (N + 15) / 16;
  Stream16Plan P{8, 0, 0};
  int per_sm = 2;
  while (P.depth > 4 && s16_smem_bytes(gated, T, P.depth) > S16_SMEM_MAX / 2 - 1024) --P.depth;
  if (s16_smem_bytes(gated, T, P.depth) > S16_SMEM_MAX / 2 - 1024) {
    per_sm = 1;
    P.depth = 8;
    while (P.depth > 2 && s16_smem_bytes(gated, T, P.depth) > S16_SMEM_MAX) --P.depth;
  }
  const int slots = sms * per_sm, rounds = (tiles + slots - 1) / slots;
  P.grid = (tiles + rounds - 1) / rounds;
  P.smem = s16_smem_bytes(gated, T, P.depth);
  return P;
}

}  // namespace moe_op
