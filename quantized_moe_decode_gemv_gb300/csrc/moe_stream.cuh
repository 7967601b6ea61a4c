// Products of a streamed weight matrix with a few token rows (k_stream): the
// 4-bit linear operators and the 16-bit gated block at decode sizes.
//
//   y[t, n] = sum_k x[t, k] W[n, k],  t < 8 NT (at most 16)
//
// The time is that of reading W once, so the kernel is built around that
// stream.  Persistent CTAs take 16-row tiles of W in turn; a CTA's 8 warps split
// a tile's 64-column chunks among them.  Every lane keeps its own ring of the
// next chunks in shared memory, filled by 16-byte asynchronous copies that run
// on over tile boundaries: its codes or weights, its scales and its pieces of
// the token rows (those through L1, where the next tile finds them again).  A
// lane reads only what it copied itself, so the ring needs no barrier; one
// barrier a tile joins the warps' partial sums, while the copies of the next
// tiles are under way.  About 100 KB an SM are in flight, twice what the memory
// latency asks for.
//
// The arithmetic is warp-level mma.sync m16n8k16 with the weights as A and the
// token rows as B (columns of absent tokens are zero): at up to 16 rows that is
// far from the tensor cores' rate, and it costs no instruction per token.  The
// warps' partial sums meet in shared memory and are added in a fixed order.
//
// The MMA's k index may run through a chunk's 64 columns in any order that A
// and B share; each format takes the one that makes its loads wide and its
// scales few (lane (g, t) of a warp: rows g and g + 8, four lanes t a row):
//   16-bit   the row-major matrix as it lies: 16 bytes of a row at columns 8 t
//            and 32 + 8 t
//   affine   the same columns; codes re-laid at create time (ql_tile) so that a
//            16-byte load holds the lane's codes of the chunk, and a shift and a
//            mask-and-or make M + q (M = 128 in bf16, 64 in fp16: the code in
//            the low mantissa bits of M).  The MMAs of a group accumulate apart
//            and fold in fp32:  y += s d + (b - M s) X,  X the group's sum of x,
//            which one more MMA with ones for A delivers in the same lanes.
//            (M is small so that the cancellation costs at most 7 bits of the
//            fp32 accumulator.)
//   fp4      columns 16 t .. 16 t + 15, one scale block (or half of one): a lane
//            needs two scales a chunk.  Codes are re-laid so that sign, exponent
//            and mantissa bits land in a 16-bit float's fields by shifts and
//            masks: the E2M1 value times 2^-126 (bf16) or 2^-14 (fp16),
//            subnormals included.  One packed multiply applies the block scale;
//            the product of an E2M1 value (2 significant bits) and an E4M3 (4
//            bits) or E8M0 scale is exact in both types, so the accumulators run
//            through all of K and a per-row fp32 factor closes the sum (ql_rows).
#pragma once

#include <cuda_runtime.h>

#include "moe_sm103.cuh"

namespace moe_op {

enum : int { W_AFFINE = 0, W_NVFP4 = 1, W_MXFP4 = 2, W_DENSE = 3 };

constexpr int ST_WARPS = 8;
constexpr int ST_THREADS = ST_WARPS * 32;
constexpr int ST_MAX_T = 16;

struct StreamArgs {
  const uint4* codes;       // 4-bit: [N/16][chunks][matrices][32 lanes]
  const void* scales;       // 4-bit: see ql_tile
  const void *w_gate, *w_up;   // 16-bit: row-major [N, K]
  const float *nscale_gate, *nscale;   // fp4: per-row factors
  const void* bias;
  const void* x;
  int64_t ldx;
  void* out;
  int64_t ldo;
  float *save_gate, *save_up;
  int K, N, T;
  int chunks;               // ceil(K / 64)
  int group;                // affine: group size
  int act, sdt;             // activation; affine: type of the scales
  int depth;                // stages of a lane's ring, 2..8
};

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1, bool fp16) {
  if (fp16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ---- decoding of a re-laid code word: a[i] holds codes i and i + 4 ----

template <bool FP16>
__device__ __forceinline__ void affine_word(uint32_t w, uint32_t (&a)[4]) {
  if (FP16) {
    a[0] = ((w << 4) & 0x00F000F0u) | 0x54005400u;
    a[1] = (w & 0x00F000F0u) | 0x54005400u;
    a[2] = ((w >> 4) & 0x00F000F0u) | 0x54005400u;
    a[3] = ((w >> 8) & 0x00F000F0u) | 0x54005400u;
  } else {
    a[0] = (w & 0x000F000Fu) | 0x43004300u;
    a[1] = ((w >> 4) & 0x000F000Fu) | 0x43004300u;
    a[2] = ((w >> 8) & 0x000F000Fu) | 0x43004300u;
    a[3] = ((w >> 12) & 0x000F000Fu) | 0x43004300u;
  }
}
template <bool FP16>
__device__ __host__ constexpr float affine_offset() { return FP16 ? 64.0f : 128.0f; }

// Where the four E2M1 codes of a half word keep their bits (fp4_place) and how
// they come out (fp4_word).
//   fp16 (field: sign 15, eem 11..9)  code 0: 15, 11..9   1: 12, 8..6   2: 14, 5..3   3: 13, 2..0
//   bf16 (field: sign 15, eem 8..6)   code 0: 15, 8..6    1: 12, 5..3   2: 14, 2..0   3: 13, 11..9
__host__ __device__ inline uint32_t fp4_place(uint32_t code, int i, bool fp16) {
  const uint32_t s = (code >> 3) & 1u, eem = code & 7u;
  if (fp16) {
    const int sp = i == 0 ? 15 : i == 1 ? 12 : i == 2 ? 14 : 13;
    return (s << sp) | (eem << (9 - 3 * i));
  }
  const int sp = i == 0 ? 15 : i == 1 ? 12 : i == 2 ? 14 : 13;
  return (s << sp) | (eem << (i == 3 ? 9 : 6 - 3 * i));
}
template <bool FP16>
__device__ __forceinline__ void fp4_word(uint32_t w, uint32_t (&a)[4]) {
  if (FP16) {
    a[0] = w & 0x8E008E00u;
    a[1] = (w << 3) & 0x8E008E00u;
    a[2] = ((w << 6) & 0x0E000E00u) | ((w << 1) & 0x80008000u);
    a[3] = ((w << 9) & 0x0E000E00u) | ((w << 2) & 0x80008000u);
  } else {
    a[0] = w & 0x81C081C0u;
    a[1] = (w << 3) & 0x81C081C0u;
    a[2] = ((w << 6) & 0x01C001C0u) | ((w << 1) & 0x80008000u);
    a[3] = ((w >> 3) & 0x01C001C0u) | ((w << 2) & 0x80008000u);
  }
}
// A stored scale byte as a pair of 16-bit floats (the byte's value, made by
// ql_scale_byte, sits in the exponent and mantissa fields).
template <int FMT, bool FP16>
__device__ __forceinline__ uint32_t fp4_scale(uint32_t bytes, int sel) {
  const uint32_t bb = __byte_perm(bytes, 0u, 0x4040u | static_cast<uint32_t>(sel) | (static_cast<uint32_t>(sel) << 8));
  // bb = the byte in the low 8 bits of both halves
  if (FMT == W_NVFP4) return FP16 ? bb << 7 : (bb << 4) | 0x70007000u;
  return FP16 ? bb << 10 : bb << 7;
}
template <bool FP16>
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t s) {
  if (FP16) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&s));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  const __nv_bfloat162 r =
      __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&s));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// One warp's stage of the ring: the chunk's weights, scales, and the token
// rows' 128 bytes each.
__host__ __device__ constexpr int st_weight_bytes(int fmt, bool gated) { return (fmt == W_DENSE ? 2048 : 512) * (gated ? 2 : 1); }
// (bytes a lane: affine 8 a group, fp4 4 -- two are used -- a matrix)
__host__ __device__ constexpr int st_scale_lane(int fmt, int gb) {
  return fmt == W_DENSE ? 0 : fmt == W_AFFINE ? (gb == 2 ? 16 : 8) : 4;
}
__host__ __device__ inline int st_stage_bytes(int fmt, bool gated, int gb, int T) {
  return st_weight_bytes(fmt, gated) + 32 * st_scale_lane(fmt, gb) * (gated ? 2 : 1) + T * 128;
}
__host__ __device__ constexpr int st_red_floats(bool gated, int nt) { return ST_WARPS * (gated ? 2 : 1) * nt * 128; }
__host__ __device__ inline int st_smem_bytes(int fmt, bool gated, int gb, int T, int nt, int depth) {
  return ST_WARPS * depth * st_stage_bytes(fmt, gated, gb, T) + 2 * 4 * st_red_floats(gated, nt);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {   // past the matrix: zeros
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy16_l1(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void copy_small(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// until at most n of this thread's groups are under way
__device__ __forceinline__ void copies_wait(int n) {
  switch (n) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
    case 6: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 7;" ::: "memory"); break;
  }
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds4(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// GB: 16-column blocks per fold (affine: 2 for groups of 32, else 4)
template <int FMT, bool FP16, bool GATED, int NT, int GB>
__global__ void __launch_bounds__(ST_THREADS, 2) k_stream(const StreamArgs A) {
  constexpr int M = GATED ? 2 : 1;
  constexpr int DT = FP16 ? DT_FP16 : DT_BF16;
  constexpr bool FP4 = FMT == W_NVFP4 || FMT == W_MXFP4;
  constexpr int WB = st_weight_bytes(FMT, false), SB = st_scale_lane(FMT, GB);
  extern __shared__ __align__(16) char st_smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int tiles = (A.N + 15) / 16, D = A.depth;
  const int stage = st_stage_bytes(FMT, GATED, GB, A.T);
  float* red = reinterpret_cast<float*>(st_smem + ST_WARPS * D * stage);
  const uint32_t ring = smem_u32(st_smem) + warp * D * stage;
  // this lane's places in a stage
  const uint32_t o_w = lane * 16, o_s = M * WB + lane * SB, o_x = M * (WB + 32 * SB);
  // its two 16-byte pieces of token rows g (and g + 8): the slots of odd rows are
  // exchanged so that eight lanes read eight different ones
  const int p0 = FP4 ? 2 * t : t, p1 = FP4 ? 2 * t + 1 : t + 4, odd = (g & 1) * (FP4 ? 1 : 4);
  const uint32_t o_x0 = o_x + g * 128 + (p0 ^ odd) * 16, o_x1 = o_x + g * 128 + (p1 ^ odd) * 16;
  const char* xrow = static_cast<const char*>(A.x) + static_cast<int64_t>(g) * A.ldx * 2;

  auto copy_weights = [&](uint32_t st, int tile, int c) {
    if constexpr (FMT == W_DENSE) {
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
    } else {
      const int64_t tc = (static_cast<int64_t>(tile) * A.chunks + c) * M;
#pragma unroll
      for (int m = 0; m < M; ++m) {
        copy16(st + m * WB + o_w, A.codes + (tc + m) * 32 + lane, true);
        const uint32_t ds = st + o_s + m * 32 * SB;
        const char* sp = static_cast<const char*>(A.scales);
        if constexpr (FMT == W_AFFINE) {
          if constexpr (GB == 2) {
            const char* q = sp + ((tc + m) * 16 + g) * 8;
            copy_small<8>(ds, q);
            copy_small<8>(ds + 8, q + 64);
          } else {
            const int gpc = A.group / 64;   // chunks of a group (1 or 2)
            const int64_t ng = (A.chunks + gpc - 1) / gpc;
            copy_small<8>(ds, sp + (((static_cast<int64_t>(tile) * ng + c / gpc) * M + m) * 8 + g) * 8);
          }
        } else {
          // two bytes a lane (two lanes): the aligned word that holds them
          const int64_t o = FMT == W_NVFP4 ? (tc + m) * 64 + (lane & ~1) * 2 : (tc + m) * 32 + g * 4;
          copy_small<4>(ds, sp + o);
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
    cc += ST_WARPS;
    if (cc >= A.chunks) {
      cc = warp;
      ct += gridDim.x;
    }
    if (++cs == D) cs = 0;
  };
  // The first stages.  The weights of a handle do not depend on the kernel
  // before this one in the stream; the token rows (and the caller's 16-bit
  // weights) may, and the outputs may be read by it.
  if (FMT == W_DENSE) asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int i = 0; i < D - 1; ++i) {
    if (ct < tiles) copy_weights(ring + cs * stage, ct, cc);
    advance();
  }
  asm volatile("griddepcontrol.launch_dependents;");
  if (FMT != W_DENSE) asm volatile("griddepcontrol.wait;" ::: "memory");
  ct = some ? static_cast<int>(blockIdx.x) : tiles, cc = warp, cs = 0;
  for (int i = 0; i < D - 1; ++i) {
    if (ct < tiles) copy_rows(ring + cs * stage, cc);
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
    for (int c = warp; c < A.chunks; c += ST_WARPS) {
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
      if constexpr (FMT == W_DENSE) {
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
      } else if constexpr (FMT == W_AFFINE) {
        constexpr uint32_t one = FP16 ? 0x3C003C00u : 0x3F803F80u;
#pragma unroll
        for (int f = 0; f < 4 / GB; ++f) {
          float X[NT][4];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            X[n][0] = X[n][1] = X[n][2] = X[n][3] = 0.0f;
#pragma unroll
            for (int j = f * GB; j < f * GB + GB; ++j)
              mma_16816(X[n], one, one, one, one, bf[n][2 * j], bf[n][2 * j + 1], FP16);
          }
#pragma unroll
          for (int m = 0; m < M; ++m) {
            const uint4 w = lds16(st + m * WB + o_w);
            const uint2 v = lds8(st + o_s + m * 32 * SB + f * 8);
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
            float d[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) d[n][0] = d[n][1] = d[n][2] = d[n][3] = 0.0f;
#pragma unroll
            for (int j = f * GB; j < f * GB + GB; ++j) {
              uint32_t a[4];
              affine_word<FP16>(ws[j], a);
#pragma unroll
              for (int n = 0; n < NT; ++n) mma_16816(d[n], a[0], a[1], a[2], a[3], bf[n][2 * j], bf[n][2 * j + 1], FP16);
            }
            const float s0 = lo16(v.x, A.sdt), s1 = lo16(v.y, A.sdt);
            const float o0 = hi16(v.x, A.sdt) - affine_offset<FP16>() * s0;
            const float o1 = hi16(v.y, A.sdt) - affine_offset<FP16>() * s1;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              float(&y)[4] = acc[m][n];
              y[0] = fmaf(s0, d[n][0], fmaf(o0, X[n][0], y[0]));
              y[1] = fmaf(s0, d[n][1], fmaf(o0, X[n][1], y[1]));
              y[2] = fmaf(s1, d[n][2], fmaf(o1, X[n][0], y[2]));
              y[3] = fmaf(s1, d[n][3], fmaf(o1, X[n][1], y[3]));
            }
          }
        }
      } else {
#pragma unroll
        for (int m = 0; m < M; ++m) {
          const uint4 w = lds16(st + m * WB + o_w);
          const uint32_t sv = lds4(st + o_s + m * 32 * SB);
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
          const int b0 = FMT == W_NVFP4 ? 2 * (lane & 1) : t & 2;
          const uint32_t s0 = fp4_scale<FMT, FP16>(sv, b0), s1 = fp4_scale<FMT, FP16>(sv, b0 + 1);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t a[4];
            fp4_word<FP16>(ws[j], a);
            a[0] = mul2<FP16>(a[0], s0);
            a[1] = mul2<FP16>(a[1], s1);
            a[2] = mul2<FP16>(a[2], s0);
            a[3] = mul2<FP16>(a[3], s1);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma_16816(acc[m][n], a[0], a[1], a[2], a[3], bf[n][2 * j], bf[n][2 * j + 1], FP16);
          }
        }
      }
    }
    // the warps' partial sums; then one thread per output adds them in warp order
    // (two buffers: the next tile's sums do not wait for these to be read)
    float* rb = red + buf * st_red_floats(GATED, NT);
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
          for (int w = 0; w < ST_WARPS; ++w) v[m] += rb[((w * M + m) * NT + n) * 128 + (tid & 127)];
        }
        if constexpr (FP4) {
          if (GATED) v[0] *= __ldg(A.nscale_gate + row);
          v[M - 1] *= __ldg(A.nscale + row);
        }
        if (A.save_up) {
          const int64_t o = static_cast<int64_t>(tok) * A.N + row;
          if (GATED) A.save_gate[o] = v[0];
          A.save_up[o] = v[M - 1];
        }
        float y = GATED ? act_value(ACT_SWIGLU, v[0], v[M - 1]) : act_value(A.act, 0.0f, v[0]);
        if (A.bias) y += ld16(A.bias, row, DT);
        static_cast<unsigned short*>(A.out)[static_cast<int64_t>(tok) * A.ldo + row] = pack1(y, DT);
      }
    }
  }
  copies_wait(0);
}

// Host: depth of the ring and grid of a launch.  Two CTAs an SM where at least
// four stages fit beside each other, else one.
struct StreamPlan {
  int depth, grid, smem;
};
inline StreamPlan st_plan(int fmt, bool gated, int gb, int T, int N, int sms) {
  const int nt = T > 8 ? 2 : 1, tiles = (N + 15) / 16;
  StreamPlan P{8, 0, 0};
  int per_sm = 2;
  while (P.depth > 4 && st_smem_bytes(fmt, gated, gb, T, nt, P.depth) > 112 * 1024) --P.depth;
  if (st_smem_bytes(fmt, gated, gb, T, nt, P.depth) > 112 * 1024) {
    per_sm = 1;
    P.depth = 8;
    while (P.depth > 2 && st_smem_bytes(fmt, gated, gb, T, nt, P.depth) > 226 * 1024) --P.depth;
  }
  const int slots = sms * per_sm, rounds = (tiles + slots - 1) / slots;
  P.grid = (tiles + rounds - 1) / rounds;
  P.smem = st_smem_bytes(fmt, gated, gb, T, nt, P.depth);
  return P;
}

using StreamKernel = void (*)(const StreamArgs);

inline cudaError_t st_launch(StreamKernel k, const StreamArgs& a, const StreamPlan& P, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(P.grid));
  cfg.blockDim = dim3(ST_THREADS);
  cfg.dynamicSmemBytes = static_cast<size_t>(P.smem);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, a);
}

}  // namespace moe_op
