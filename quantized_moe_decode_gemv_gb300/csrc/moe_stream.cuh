// Products of a streamed 4-bit weight matrix with a few token rows (k_stream):
// the 4-bit linear operators at decode sizes.
//
//   y[t, n] = sum_k x[t, k] W[n, k],  t < 8 NT (at most 16)
//
// The time is that of reading W once, so the kernel is built around that
// stream and around the instructions a weight costs.  One CTA of 16 warps an SM
// takes 16-row tiles of W in turn; its warps split a tile's 64-column chunks
// among them, each a consecutive range.  A warp has a ring of stages in shared
// memory, a stage's codes and scales consecutive in the handle's layout, filled
// by 16-byte asynchronous copies of its lanes, over tile boundaries and a few
// stages ahead of the arithmetic, 45 KB or more an SM under way.  (Bulk copies,
// one for a stage's codes and one for its scales, took 22.1 us where these take
// 19.9: 75.6 MB of NVFP4 weights at one token; now 18.8 to 19.3, 4.0 TB/s.)
// The token rows lie in shared memory as they are.  The warps' partial sums meet
// in shared memory one tile late: a warp leaves its sums of a tile, goes on to
// the next one, and adds its share of the former when it is through, so that no
// warp waits for the slowest.
//
// The arithmetic is warp-level mma.sync m16n8k16 with the weights as A and the
// token rows as B (columns of absent tokens are zero): at up to 16 rows that is
// far from the tensor cores' rate, and it costs no instruction per token.  The
// warps' partial sums are added in a fixed order.
//
// The MMA's k index may run through a chunk's 64 columns in any order that A
// and B share; each format takes the one that makes its loads wide and its
// scales few (lane (g, t) of a warp: rows g and g + 8, four lanes t a row):
//   all but groups of 32: columns 16 t .. 16 t + 15 of the chunk, a scale group
//            or part of one, so that a lane needs two scales a chunk
//   affine in groups of 32: columns 8 t and 32 + 8 t on, eight of each group
// Affine codes are re-laid at create time (ql_tile) so that a 16-byte load holds
// the lane's codes of the chunk, and a shift and a mask-and-or make M + q (M = 128
// in bf16, 64 in fp16: the code in the low mantissa bits of M).  The MMAs of a
// group accumulate apart and fold in fp32:  y += s d + (b - M s) X,  X the group's
// sum of x, which one more MMA with ones for A delivers in the same lanes.  (M is
// small so that the cancellation costs at most 7 bits of the fp32 accumulator.)
// fp4 codes are re-laid so that sign, exponent and mantissa bits land in a 16-bit
// float's fields by shifts and masks: the E2M1 value times 2^-126 (bf16) or 2^-14
// (fp16), subnormals included.  One packed multiply applies the block scale; the
// product of an E2M1 value (2 significant bits) and an E4M3 (4 bits) or E8M0 scale
// is exact in both types, so the accumulators run through all of K and a per-row
// fp32 factor closes the sum (ql_rows).
#pragma once

#include "moe_sm103.cuh"

namespace moe_op {

enum : int { W_AFFINE = 0, W_NVFP4 = 1, W_MXFP4 = 2 };

constexpr int ST_WARPS = 16;
constexpr int ST_THREADS = ST_WARPS * 32;
constexpr int ST_MAX_T = 16;

struct StreamArgs {
  const uint4* codes;       // 4-bit: [N/16][chunks][matrices][32 lanes]
  const void* scales;       // 4-bit: see ql_tile
  const float *nscale_gate, *nscale;   // fp4: per-row factors
  const void* bias;
  const void* x;
  int64_t ldx;
  void* out;
  int64_t ldo;
  int K, N, T;
  int chunks;               // ceil(K / 64)
  int group;                // affine: group size
  int act, sdt;             // activation; affine: type of the scales
  int depth;                // stages of a warp's ring, 2..4
  int* status;
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

// s q + b rounded once, two codes a register: a holds M + q, so q is exact
template <bool FP16>
__device__ __forceinline__ uint32_t affine16(uint32_t a, uint32_t s, uint32_t b) {
  if (FP16) {
    const uint32_t m = 0x54005400u;
    const __half2 r = __hfma2(__hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&m)),
                              *reinterpret_cast<const __half2*>(&s), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  const uint32_t m = 0x43004300u;
  const __nv_bfloat162 r =
      __hfma2(__hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&m)),
              *reinterpret_cast<const __nv_bfloat162*>(&s), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

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
// scale_byte at create time, sits in the exponent and mantissa fields).
template <int FMT, bool FP16>
__device__ __forceinline__ uint32_t fp4_scale(uint32_t bytes, int sel) {
  const uint32_t bb = __byte_perm(bytes, 0u, 0x4040u | static_cast<uint32_t>(sel) | (static_cast<uint32_t>(sel) << 8));
  // bb = the byte in the low 8 bits of both halves
  // (multiplications: they run beside the shifts and masks of the codes)
  if (FMT == W_NVFP4) return FP16 ? bb * 128u : bb * 16u + 0x70007000u;
  return FP16 ? bb * 1024u : bb * 128u;
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

// Shared memory of a launch:
//   [ST_WARPS rings of `depth` stages][token rows][a stage's width of zeros][partial
//   sums, two tiles][barriers]
// A stage holds st_chunks() chunks: their matrices x 512 bytes of codes, then the
// scales.  Token rows are 16 bytes longer than K (64 with groups of 32), so that
// the fragment reads of eight lanes (two rows of four lanes) touch all banks once.
__host__ __device__ constexpr int st_scale_bytes(int fmt, int gb) {   // a chunk and matrix (affine: a group)
  return fmt == W_AFFINE ? (gb == 2 ? 128 : 64) : fmt == W_NVFP4 ? 64 : 32;
}
// Whether a lane's columns of a chunk are consecutive (else eight of each half).
__host__ __device__ constexpr bool st_wide(int fmt, int gb) { return fmt != W_AFFINE || gb == 4; }
// Chunks of a stage: 2 KB of codes, or 1 KB with two token tiles, whose rows and
// sums need the room (affine: at least the two chunks of a group of 128).
__host__ __device__ constexpr int st_chunks(int fmt, int mats, int nt, int gb) {
  return nt == 1 ? 4 / mats : (fmt == W_AFFINE && gb == 4) ? 2 : 2 / mats;
}
__host__ __device__ constexpr int st_stage_bytes(int fmt, int mats, int nt, int gb) {
  return mats * st_chunks(fmt, mats, nt, gb) * (512 + st_scale_bytes(fmt, gb));
}
__host__ __device__ inline int st_row_bytes(int fmt, int gb, int chunks) { return chunks * 128 + (st_wide(fmt, gb) ? 16 : 64); }
__host__ __device__ constexpr int st_red_floats(int mats, int nt) { return ST_WARPS * mats * nt * 128; }
__host__ __device__ inline int st_smem_bytes(int fmt, int mats, int gb, int chunks, int T, int depth) {
  const int nt = T > 8 ? 2 : 1;
  return ST_WARPS * depth * st_stage_bytes(fmt, mats, nt, gb) + T * st_row_bytes(fmt, gb, chunks) +
         st_chunks(fmt, mats, nt, gb) * 128 +
         8 * st_red_floats(mats, nt) + 16;
}

__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds2(uint32_t a) {
  uint32_t v;
  asm volatile("{\n\t.reg .u16 h;\n\tld.shared.u16 h, [%1];\n\tcvt.u32.u16 %0, h;\n\t}" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// GB: 16-column blocks per fold (affine: 2 for groups of 32, else 4)
template <int FMT, bool FP16, bool GATED, int NT, int GB>
__global__ void __launch_bounds__(ST_THREADS, 1) k_stream(const StreamArgs A) {
  constexpr int M = GATED ? 2 : 1;
  constexpr int DT = FP16 ? DT_FP16 : DT_BF16;
  constexpr bool FP4 = FMT == W_NVFP4 || FMT == W_MXFP4, WIDE = st_wide(FMT, GB);
  constexpr int SCB = st_scale_bytes(FMT, GB);
  extern __shared__ __align__(128) char st_smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  constexpr int CB = st_chunks(FMT, M, NT, GB), stage = st_stage_bytes(FMT, M, NT, GB);
  const int tiles = (A.N + 15) / 16, D = A.depth;
  const int xrow = st_row_bytes(FMT, GB, A.chunks);
  char* const xs = st_smem + ST_WARPS * D * stage;
  char* const zeros = xs + A.T * xrow;   // what lanes of absent tokens read
  float* const red = reinterpret_cast<float*>(zeros + CB * 128);
  uint64_t* const bars = reinterpret_cast<uint64_t*>(red + 2 * st_red_floats(M, NT));
  const uint32_t ring = smem_u32(st_smem) + warp * D * stage;
  const uint32_t rbar = smem_u32(bars);   // two: the sums of even and odd tiles

  // this warp's chunks (whole groups of 128)
  const int qs = FMT == W_AFFINE && A.group == 128 ? 1 : 0, q = 1 << qs, nu = A.chunks >> qs;
  const int c_lo = q * (warp * nu / ST_WARPS), c_hi = q * ((warp + 1) * nu / ST_WARPS);

  // the next stage to fill: tile, chunk, their codes and scales, the slot
  int ft = c_lo < c_hi ? static_cast<int>(blockIdx.x) : tiles, fc = c_lo;
  const char *fsrc = nullptr, *fsc = nullptr;
  uint32_t fst = ring + lane * 16;
  const uint32_t ring_end = fst + D * stage;
  auto settle = [&] {   // to the start of this warp's chunks of tile ft
    fc = c_lo;
    fsrc = reinterpret_cast<const char*>(A.codes) + (static_cast<int64_t>(ft) * A.chunks + c_lo) * (M * 512) + lane * 16;
    fsc = static_cast<const char*>(A.scales) + (static_cast<int64_t>(ft) * nu + (c_lo >> qs)) * (M * SCB) + lane * 16;
  };
  auto fill_next = [&] {
    if (ft < tiles) {
      const int n = min(CB, c_hi - fc);
#pragma unroll
      for (int i = 0; i < CB; ++i)
        if (i < n) {
#pragma unroll
          for (int m = 0; m < M; ++m) copy16(fst + (i * M + m) * 512, fsrc + (i * M + m) * 512, true);
        }
      const int sbytes = (n >> qs) * (M * SCB);
#pragma unroll
      for (int i = 0; i < (CB * M * SCB + 511) / 512; ++i)
        if (lane * 16 + i * 512 < sbytes) copy16(fst + CB * M * 512 + i * 512, fsc + i * 512, true);
      fsrc += CB * M * 512;
      fsc += (CB >> qs) * (M * SCB);
      fc += CB;
      if (fc >= c_hi) {
        ft += gridDim.x;
        settle();
      }
    }
    fst += stage;
    if (fst == ring_end) fst = ring + lane * 16;
    copies_commit();
  };
  auto stage_here = [&] {   // until the oldest stage has landed
    if (D == 2) copies_wait_n<1>();
    else if (D == 3) copies_wait_n<2>();
    else copies_wait_n<3>();
  };

  if (tid == 0) {
    bar_init(rbar, ST_WARPS);
    bar_init(rbar + 8, ST_WARPS);
  }
  bar_fence_init();

  // The first stages.  A handle's weights do not depend on the kernel before
  // this one in the stream; the token rows may, and the outputs may be read by it.
  settle();
  for (int i = 0; i < D - 1; ++i) fill_next();
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  {
    const int w = A.chunks * 8;   // 16-byte pieces of a row; past K zeros
    for (int i = tid; i < A.T * w; i += ST_THREADS) {
      const int r = i / w, p = i - r * w;
      const char* src = static_cast<const char*>(A.x) + static_cast<int64_t>(r) * A.ldx * 2;
      copy16(smem_u32(xs) + r * xrow + p * 16, p * 8 < A.K ? src + p * 16 : src, p * 8 < A.K);
    }
    copies_commit();
    for (int i = tid; i < CB * 8; i += ST_THREADS) *reinterpret_cast<uint4*>(zeros + i * 16) = make_uint4(0, 0, 0, 0);
    copies_wait(0);
  }
  __syncthreads();
  bool ok = true;

  // this lane's 16-byte pieces of a chunk's 128 bytes of token rows g (and g + 8)
  uint32_t xat[NT];
  int xstep[NT];   // bytes from a chunk to the next
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const bool in = n * 8 + g < A.T;
    xat[n] = smem_u32(in ? xs + (n * 8 + g) * xrow : zeros) + (WIDE ? 32 * t : 16 * t);
    xstep[n] = in ? 128 : 0;
  }

  // adds the warps' sums of a tile: one thread an output, a quarter (or half) of the CTA
  auto join = [&](int tile, int n_done) {
    const int part = NT == 1 ? (tid >> 7) - (n_done & 3) : (tid >> 8) - (n_done & 1);
    if (part != 0) return;
    const int e = tid & (NT * 128 - 1), ei = (e >> 5) & 3, n = e >> 7;
    const int row = tile * 16 + g + (ei >> 1) * 8, tok = n * 8 + t * 2 + (ei & 1);
    if (row >= A.N || tok >= A.T) return;
    const float* rb = red + (n_done & 1) * st_red_floats(M, NT);
    float v[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
      v[m] = 0.0f;
#pragma unroll
      for (int w = 0; w < ST_WARPS; ++w) v[m] += rb[((w * M + m) * NT + n) * 128 + (e & 127)];
    }
    if constexpr (FP4) {
      if (GATED) v[0] *= __ldg(A.nscale_gate + row);
      v[M - 1] *= __ldg(A.nscale + row);
    }
    float y = GATED ? act_value(ACT_SWIGLU, v[0], v[M - 1]) : act_value(A.act, 0.0f, v[0]);
    if (A.bias) y += ld16(A.bias, row, DT);
    static_cast<unsigned short*>(A.out)[static_cast<int64_t>(tok) * A.ldo + row] = pack1(y, DT);
  };

  uint32_t cst = ring;
  int n_done = 0, prev = 0;
  for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x, ++n_done) {
    float acc[M][NT][4];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.0f;
    for (int cs = c_lo; cs < c_hi; cs += CB) {
      __syncwarp();   // every lane has read the slot that is filled now
      fill_next();
      stage_here();
      __syncwarp();   // every lane's copies have landed
      const uint32_t st = cst;
      cst += stage;
      if (cst == ring + D * stage) cst = ring;
      const int n_c = min(CB, c_hi - cs);
#pragma unroll
      for (int i = 0; i < CB; ++i) {
        if (i >= n_c) break;
        // B fragments: 16-column steps j = 0..3, two registers each
        uint32_t bf[NT][8];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint32_t at = xat[n] + cs * xstep[n] + i * 128;
          const uint4 v0 = lds16(at), v1 = lds16(at + (WIDE ? 16 : 64));
          bf[n][0] = v0.x; bf[n][1] = v0.y; bf[n][2] = v0.z; bf[n][3] = v0.w;
          bf[n][4] = v1.x; bf[n][5] = v1.y; bf[n][6] = v1.z; bf[n][7] = v1.w;
        }
        if constexpr (FMT == W_AFFINE) {
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
              const uint4 w = lds16(st + (i * M + m) * 512 + lane * 16);
              const uint2 v = lds8(st + CB * M * 512 + ((i >> qs) * M + m) * SCB + f * 64 + g * 8);
              const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
              float d[NT][4];
#pragma unroll
              for (int n = 0; n < NT; ++n) d[n][0] = d[n][1] = d[n][2] = d[n][3] = 0.0f;
#pragma unroll
              for (int j = f * GB; j < f * GB + GB; ++j) {
                uint32_t a[4];
                affine_word<FP16>(ws[j], a);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                  mma_16816(d[n], a[0], a[1], a[2], a[3], bf[n][2 * j], bf[n][2 * j + 1], FP16);
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
            const uint4 w = lds16(st + (i * M + m) * 512 + lane * 16);
            const uint32_t sv = lds2(st + CB * M * 512 + (i * M + m) * SCB +
                                     (FMT == W_NVFP4 ? lane * 2 : g * 4 + (t & 2)));
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
            const uint32_t s0 = fp4_scale<FMT, FP16>(sv, 0), s1 = fp4_scale<FMT, FP16>(sv, 1);
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
    }
    // The tile before this one: its sums are complete once every warp has left
    // its own.  (A warp arrives for a tile after it has added its share of the
    // one before; so when the wait is over, the buffer of the tile two back,
    // which this tile's sums overwrite, has been read.)
    if (n_done > 0) {
      if (!(ok = bar_wait(rbar + ((n_done - 1) & 1) * 8, ((n_done - 1) >> 1) & 1))) break;
      join(prev, n_done - 1);
    }
    float* rb = red + (n_done & 1) * st_red_floats(M, NT);
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) rb[((warp * M + m) * NT + n) * 128 + i * 32 + lane] = acc[m][n][i];
    __syncwarp();
    if (lane == 0) bar_arrive(rbar + (n_done & 1) * 8);
    prev = tile;
  }
  if (ok && n_done > 0) {
    ok = bar_wait(rbar + ((n_done - 1) & 1) * 8, ((n_done - 1) >> 1) & 1);
    if (ok) join(prev, n_done - 1);
  }
  copies_wait(0);
  if (!ok) atomicOr(A.status, STATUS_TIMEOUT);   // a wait ran out
}

// Host: the ring of a launch, two to four stages.  False when the token rows leave
// no room for it.
struct StreamPlan {
  int depth = 0, grid = 0, smem = 0;
};
constexpr int ST_SMEM_MAX = 226 * 1024;
inline bool st_plan(int fmt, bool gated, int gb, int chunks, int T, int N, int sms, StreamPlan* P) {
  const int mats = gated ? 2 : 1;
  int d = 4;
  while (d >= 2 && st_smem_bytes(fmt, mats, gb, chunks, T, d) > ST_SMEM_MAX) --d;
  if (d < 2) return false;
  const int tiles = (N + 15) / 16, rounds = (tiles + sms - 1) / sms;
  P->depth = d;
  P->grid = (tiles + rounds - 1) / rounds;
  P->smem = st_smem_bytes(fmt, mats, gb, chunks, T, d);
  return true;
}

}  // namespace moe_op
