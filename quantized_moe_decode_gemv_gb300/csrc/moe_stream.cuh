// Products of a streamed weight matrix with a few token rows (k_stream): the
// 4-bit linear operators and the 16-bit gated block at decode sizes.
//
//   y[t, n] = sum_k x[t, k] W[n, k],  t < 8 NT (at most 16)
//
// The time is that of reading W once, so the kernel is built around that
// stream: a CTA takes 16-row tiles of W, its 8 warps split a tile's 64-column
// chunks among them, and a lane's loads are 16 bytes from consecutive
// addresses across the warp, issued one batch ahead of the arithmetic and over
// tile boundaries.  The arithmetic is warp-level mma.sync m16n8k16 with the
// weights as A and the token rows as B (columns of absent tokens are zero):
// at up to 16 rows that is far from the tensor cores' rate, and it costs no
// instruction per token.  The warps' partial sums meet in shared memory and
// are added in a fixed order.
//
// A's registers, per weight format:
//   16-bit   the row-major matrix as it lies: lane (g, t) loads 16 bytes of
//            rows g and g + 8 at columns 8 t and 32 + 8 t of the chunk; the
//            MMA's k index runs through the columns in the order those
//            registers hold them, and x is staged in the same order.
//   affine   codes re-laid at create time (ql_tile) so that a lane's word holds
//            its eight codes of a 16-column block; a shift and a mask-and-or
//            make M + q (M = 128 in bf16, 64 in fp16: the code in the low
//            mantissa bits of M).  The MMAs of a group accumulate apart and
//            fold in fp32:  y += s (d - M X) + b X,  X the group's sum of x.
//            (M stays small so that the cancellation costs at most 7 bits of
//            the fp32 accumulator.)
//   fp4      codes re-laid so that sign, exponent and mantissa bits land in a
//            16-bit float's fields by shifts and masks: the E2M1 value times
//            2^-126 (bf16) or 2^-14 (fp16), subnormals included.  One packed
//            multiply applies the block scale; the product of an E2M1 value
//            (2 significant bits) and an E4M3 (4 bits) or E8M0 scale is exact
//            in both types, so the accumulators run through all of K and a
//            per-row fp32 factor closes the sum (ql_rows).
#pragma once

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
};

// Shared memory of a launch: x rows (permuted, 16 bytes of padding so that the
// fragment reads of eight lanes cover all banks), the group sums of x (affine),
// the warps' partial sums (double-buffered).
struct StreamPlan {
  int x_stride, sum_off, sums, red_off, red_floats, total;
};
__host__ __device__ inline StreamPlan st_plan(int chunks, int T, int nt, int mats, int gx) {
  StreamPlan P;
  P.x_stride = chunks * 128 + 16;
  P.sum_off = T * P.x_stride;
  P.sums = gx > 0 ? chunks * 64 / gx : 0;
  P.red_off = P.sum_off + P.sums * nt * 8 * 4;
  P.red_floats = ST_WARPS * mats * nt * 128;
  P.total = P.red_off + 2 * P.red_floats * 4;
  return P;
}

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

__device__ __forceinline__ uint4 ldg_weights(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
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
//   bf16 (field: sign 15, eem 8..6)   code 0: 15, 8..6    1: 12, 5..3   2: 9, 2..0    3: 14, 11 10 (ee), 13 (m)
__host__ __device__ inline uint32_t fp4_place(uint32_t code, int i, bool fp16) {
  const uint32_t s = (code >> 3) & 1u, eem = code & 7u;
  if (fp16) {
    const int sp = i == 0 ? 15 : i == 1 ? 12 : i == 2 ? 14 : 13;
    return (s << sp) | (eem << (9 - 3 * i));
  }
  if (i < 3) return (s << (15 - 3 * i)) | (eem << (6 - 3 * i));
  return (s << 14) | ((eem >> 1) << 10) | ((eem & 1u) << 13);
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
    a[2] = (w << 6) & 0x81C081C0u;
    a[3] = ((w >> 3) & 0x01800180u) | ((w >> 7) & 0x00400040u) | ((w << 1) & 0x80008000u);
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

// What a lane holds of one chunk of one matrix.
template <int FMT, int GB>
struct StreamRegs {
  uint4 w[FMT == W_DENSE ? 4 : 1];
  uint32_t s[FMT == W_AFFINE ? (GB == 2 ? 4 : 2) : FMT == W_NVFP4 ? 2 : 1];
};

// GB: 16-column blocks per fold (affine: 2 for groups of 32, else 4)
template <int FMT, bool FP16, bool GATED, int NT, int GB>
__global__ void __launch_bounds__(ST_THREADS, 2) k_stream(const StreamArgs A) {
  constexpr int M = GATED ? 2 : 1;
  // chunks of a load batch: 2 KB (4-bit) or 4 KB (16-bit) a warp in flight
  // beside the batch being multiplied
  constexpr int CB = FMT == W_DENSE ? (GATED ? 1 : 2) : (GATED ? 2 : 4);
  constexpr int DT = FP16 ? DT_FP16 : DT_BF16;
  extern __shared__ __align__(16) char st_smem[];
  const int gx = FMT == W_AFFINE ? 16 * GB : 0;
  const StreamPlan P = st_plan(A.chunks, A.T, NT, M, gx);
  float* sums = reinterpret_cast<float*>(st_smem + P.sum_off);
  float* red = reinterpret_cast<float*>(st_smem + P.red_off);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int tiles = (A.N + 15) / 16;
  const int nb = (A.chunks + ST_WARPS * CB - 1) / (ST_WARPS * CB);   // batches of a tile

  auto load = [&](int tile, int b, StreamRegs<FMT, GB> (&r)[CB][M]) {
#pragma unroll
    for (int i = 0; i < CB; ++i) {
      const int c = warp + ST_WARPS * (b * CB + i);
      const bool in = c < A.chunks && tile < tiles;
#pragma unroll
      for (int m = 0; m < M; ++m) {
        if (FMT == W_DENSE) {
          const char* w = static_cast<const char*>(GATED && m == 0 ? A.w_gate : A.w_up);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = tile * 16 + g + 8 * h;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int col = c * 64 + 32 * k + 8 * t;
              r[i][m].w[2 * k + h] = (in && row < A.N && col < A.K)
                                         ? ldg_weights(w + (static_cast<int64_t>(row) * A.K + col) * 2)
                                         : make_uint4(0, 0, 0, 0);
            }
          }
        } else {
          const int64_t tc = (static_cast<int64_t>(tile) * A.chunks + c) * M + m;
          r[i][m].w[0] = in ? ldg_weights(A.codes + tc * 32 + lane) : make_uint4(0, 0, 0, 0);
          if (FMT == W_AFFINE) {
            const uint2* sp = static_cast<const uint2*>(A.scales);
            if (GB == 2) {
              const int64_t o = tc * 16 + g;
              const uint2 v0 = in ? __ldg(sp + o) : make_uint2(0, 0), v1 = in ? __ldg(sp + o + 8) : make_uint2(0, 0);
              r[i][m].s[0] = v0.x; r[i][m].s[1] = v0.y;
              r[i][m].s[FMT == W_AFFINE && GB == 2 ? 2 : 0] = v1.x; r[i][m].s[FMT == W_AFFINE && GB == 2 ? 3 : 1] = v1.y;
            } else {
              const int gpc = A.group / 64;   // chunks of a group (1 or 2)
              const int64_t ng = (A.chunks + gpc - 1) / gpc;
              const int64_t o = ((static_cast<int64_t>(tile) * ng + c / gpc) * M + m) * 8 + g;
              const uint2 v = in ? __ldg(sp + o) : make_uint2(0, 0);
              r[i][m].s[0] = v.x; r[i][m].s[1] = v.y;
            }
          } else if (FMT == W_NVFP4) {
            const uint2 v = in ? __ldg(static_cast<const uint2*>(A.scales) + tc * 8 + g) : make_uint2(0, 0);
            r[i][m].s[0] = v.x; r[i][m].s[FMT == W_NVFP4 ? 1 : 0] = v.y;
          } else {
            r[i][m].s[0] = in ? __ldg(static_cast<const uint32_t*>(A.scales) + tc * 8 + g) : 0u;
          }
        }
      }
    }
  };

  StreamRegs<FMT, GB> cur[CB][M], nxt[CB][M];
  load(blockIdx.x, 0, cur);

  // stage x: 8-byte pieces (four columns) in the order the fragments read them
  {
    const int pieces = A.chunks * 16;
    for (int i = tid; i < A.T * pieces; i += ST_THREADS) {
      const int row = i / pieces, p = i - row * pieces, col = p * 4;
      const int c = p >> 4, q = p & 15;
      const int dst = FMT == W_DENSE ? ((q >> 1) & 3) * 32 + (((q >> 3) << 1) | (q & 1)) * 8 : (q & 3) * 32 + (q >> 2) * 8;
      uint2 v = make_uint2(0, 0);
      if (col < A.K)
        v = __ldg(reinterpret_cast<const uint2*>(static_cast<const unsigned short*>(A.x) + static_cast<int64_t>(row) * A.ldx +
                                                 col));
      *reinterpret_cast<uint2*>(st_smem + row * P.x_stride + c * 128 + dst) = v;
    }
  }
  __syncthreads();
  if (FMT == W_AFFINE) {
    // group sums in fp32, [group][token]; absent tokens zero
    for (int i = tid; i < P.sums * NT * 8; i += ST_THREADS) {
      const int grp = i / (NT * 8), tok = i - grp * (NT * 8);
      float s = 0.0f;
      if (tok < A.T) {
        const int c = grp * gx / 64, j0 = GB == 2 ? (grp & 1) * 2 : 0;
        for (int tt = 0; tt < 4; ++tt)
#pragma unroll
          for (int j = 0; j < GB; ++j) {
            const uint2 v = *reinterpret_cast<const uint2*>(st_smem + tok * P.x_stride + c * 128 + tt * 32 + (j0 + j) * 8);
            s += (lo16(v.x, DT) + hi16(v.x, DT)) + (lo16(v.y, DT) + hi16(v.y, DT));
          }
      }
      sums[i] = s;
    }
    __syncthreads();
  }

  float acc[M][NT][4];
  int buf = 0;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;
    for (int b = 0; b < nb; ++b) {
      const bool last = b + 1 == nb;
      load(last ? tile + static_cast<int>(gridDim.x) : tile, last ? 0 : b + 1, nxt);
#pragma unroll
      for (int i = 0; i < CB; ++i) {
        const int c = warp + ST_WARPS * (b * CB + i);
        if (c < A.chunks) {
          // B fragments of the chunk: blocks j = 0..3, two registers each
          uint32_t bf[NT][8];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const int tok = n * 8 + g;
            if (tok < A.T) {
              const uint4* px = reinterpret_cast<const uint4*>(st_smem + tok * P.x_stride + c * 128 + t * 32);
              const uint4 v0 = px[0], v1 = px[1];
              bf[n][0] = v0.x; bf[n][1] = v0.y; bf[n][2] = v0.z; bf[n][3] = v0.w;
              bf[n][4] = v1.x; bf[n][5] = v1.y; bf[n][6] = v1.z; bf[n][7] = v1.w;
            } else {
#pragma unroll
              for (int k = 0; k < 8; ++k) bf[n][k] = 0u;
            }
          }
#pragma unroll
          for (int m = 0; m < M; ++m) {
            const StreamRegs<FMT, GB>& R = cur[i][m];
            if (FMT == W_DENSE) {
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint4 lo = R.w[2 * k], hi = R.w[FMT == W_DENSE ? 2 * k + 1 : 0];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  mma_16816(acc[m][n], lo.x, hi.x, lo.y, hi.y, bf[n][4 * k], bf[n][4 * k + 1], FP16);
                  mma_16816(acc[m][n], lo.z, hi.z, lo.w, hi.w, bf[n][4 * k + 2], bf[n][4 * k + 3], FP16);
                }
              }
            } else {
              const uint32_t ws[4] = {R.w[0].x, R.w[0].y, R.w[0].z, R.w[0].w};
              if (FMT == W_AFFINE) {
#pragma unroll
                for (int f = 0; f < 4 / GB; ++f) {
                  float d[NT][4];
#pragma unroll
                  for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < 4; ++k) d[n][k] = 0.0f;
#pragma unroll
                  for (int j = 0; j < GB; ++j) {
                    uint32_t a[4];
                    affine_word<FP16>(ws[f * GB + j], a);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                      mma_16816(d[n], a[0], a[1], a[2], a[3], bf[n][2 * (f * GB + j)], bf[n][2 * (f * GB + j) + 1], FP16);
                  }
                  const uint32_t v0 = R.s[FMT == W_AFFINE ? 2 * f : 0], v1 = R.s[FMT == W_AFFINE ? 2 * f + 1 : 0];
                  const float s0 = lo16(v0, A.sdt), s1 = lo16(v1, A.sdt);
                  const float o0 = hi16(v0, A.sdt) - affine_offset<FP16>() * s0;
                  const float o1 = hi16(v1, A.sdt) - affine_offset<FP16>() * s1;
#pragma unroll
                  for (int n = 0; n < NT; ++n) {
                    const float2 X =
                        *reinterpret_cast<const float2*>(sums + (c * (4 / GB) + f) * (NT * 8) + n * 8 + 2 * t);
                    acc[m][n][0] = fmaf(s0, d[n][0], fmaf(o0, X.x, acc[m][n][0]));
                    acc[m][n][1] = fmaf(s0, d[n][1], fmaf(o0, X.y, acc[m][n][1]));
                    acc[m][n][2] = fmaf(s1, d[n][2], fmaf(o1, X.x, acc[m][n][2]));
                    acc[m][n][3] = fmaf(s1, d[n][3], fmaf(o1, X.y, acc[m][n][3]));
                  }
                }
              } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  uint32_t a[4];
                  fp4_word<FP16>(ws[j], a);
                  // bytes (row g, row g + 8) of block j (nvfp4) or of its pair of blocks (mxfp4)
                  const uint32_t sb = FMT == W_NVFP4 ? R.s[FMT == W_NVFP4 ? j >> 1 : 0] : R.s[0];
                  const int b0 = FMT == W_NVFP4 ? 2 * (j & 1) : 2 * (j >> 1);
                  const uint32_t s0 = fp4_scale<FMT, FP16>(sb, b0), s1 = fp4_scale<FMT, FP16>(sb, b0 + 1);
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
        }
      }
#pragma unroll
      for (int i = 0; i < CB; ++i)
#pragma unroll
        for (int m = 0; m < M; ++m) cur[i][m] = nxt[i][m];
    }
    // the warps' partial sums, then one thread per output adds them in warp order
    float* rb = red + buf * P.red_floats;
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) rb[((warp * M + m) * NT + n) * 128 + i * 32 + lane] = acc[m][n][i];
    __syncthreads();
    for (int e = tid; e < NT * 128; e += ST_THREADS) {
      const int el = e & 31, ei = (e >> 5) & 3, n = e >> 7;
      const int row = tile * 16 + (el >> 2) + (ei >> 1) * 8, tok = n * 8 + (el & 3) * 2 + (ei & 1);
      if (row < A.N && tok < A.T) {
        float v[M];
#pragma unroll
        for (int m = 0; m < M; ++m) {
          v[m] = 0.0f;
#pragma unroll
          for (int w = 0; w < ST_WARPS; ++w) v[m] += rb[((w * M + m) * NT + n) * 128 + (e & 127)];
        }
        if (FMT == W_NVFP4 || FMT == W_MXFP4) {
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
    buf ^= 1;
  }
}

}  // namespace moe_op
