// Newton-Schulz products (moe_ortho_* in include/moe_layer.h) on tcgen05: a matrix X
// with small side m becomes p(X) = a X + b (X X^T) X + c (X X^T)^2 X, step by step.
//
//   GRAM   A = X X^T                     [m, m], symmetric
//   POLY   B = b A + c A A               [m, m], symmetric
//   APPLY  X <- a X + B X                (tall matrices: X^T X, and X B)
//
// What is held in which precision.  Operands are fp16: at the rate of bf16 with three
// more bits.  X is scaled by s = 2^q and A, B by s^2, 4^q about m, so that neither the
// entries of X (about 1 / sqrt(m n) of its norm at the start) nor the largest value of
// A and B (2.8 s^2) leave fp16's range; powers of two, so exact.  Two things keep the
// result's error below the rounding of its bf16 output (1.66e-3 of its norm; with it
// measured 1.8e-3 on 1024 x 4096 and 8192 x 4096, 1.9e-3 on 64 x 256):
//   - The diagonals d of A and e of B are kept apart in fp32 and the fp16 matrices have
//     zeros there: A = O + diag(d), and
//       (A A)_ij = (O O)_ij + O_ij (d_i + d_j) + [i = j] d_i^2
//     in the epilogue.  Near the fixed point A is close to a multiple of 1, so the
//     diagonal is most of A's norm, and of its rounding: with it in fp16 the error of a
//     full-rank matrix was 1.5 to 1.7e-3, without 1.0 to 1.2e-3.
//   - X is kept as two fp16 terms, hi + 2^-11 lo.  Products take hi, the linear term a X both:
//     what rounding leaves of X lies in directions that X itself may not have, where p
//     multiplies by a = 3.4 a step; without lo a gradient of 9 tokens was off by 4e-2.  lo is
//     stored 2^11 times larger, as large as hi: at its own size it would be among fp16's
//     subnormal numbers and end at 2^-24 (9 tokens, 64 x 8192, eight steps: off by 1.1e-2, this
//     way 1.4e-3).
//
// All steps are one launch (k_ortho).  The tiles of all products, (group of matrices, step,
// product, matrix, tile), are one list that CTAs (pairs, for 256 x 256 tiles) take in turn; a tile waits
// until the products that it reads are done, by counters of finished epilogues for each
// matrix and product.  Tiles only wait for tiles before them in the list and all CTAs are
// resident (a cooperative launch), so somebody always can go on.  As launches of their
// own, products were 2.1 waves taken as 3 (16 matrices of 1856 x 1024, tiles of 256 x
// 256 on 76 pairs), and each paid for its launch, its pipeline's filling and its
// epilogues' end.  (A group is a stack's matrices that the L2 holds, if they are enough.)
//
// Roles of a CTA's 12 warps, as in k_gemm16: tensor copies, MMAs, tensor memory, and
// eight epilogue warps; accumulators double-buffered.  Tiles are square, CG * 128 on a
// side; of a symmetric matrix those on and below the diagonal are computed and stored, and
// who reads one above it reads its transpose, an MN-major operand instead of a K-major one
// (both are what a tensor copy makes of rows; the majors are part of each MMA's descriptor).
// Where tiles are fewer than CTAs, K is split; each split then adds the partial sums, in
// order, of a share of the tile's pieces.
//
// An epilogue warp's piece is 32 x 32 values, a row a lane.  What paced the epilogues was
// what they wrote (all CTAs at once: 6 KB a piece, X twice and symmetric tiles twice, took 8 us
// for 256 x 256 values, 6 with the 4 KB of X and 3.5 with the 2 KB of O; MMAs take 4.3 at
// K = 1024).
// So X's hi is its operand's rows and nothing else, its lo lies as lanes read it, and
// symmetric tiles are stored once.  What a piece reads comes two pieces ahead by the lanes'
// own asynchronous copies; tensor copies would queue behind those of the ring.
//
// Measured, five steps, passes back to back: 8192 x 4096 1.63 to 1.73 ms (1.39 to 1.48 PFLOP/s, the symmetric
// products counted by halves; power and the tensor pipe), 16 x 1856 x 1024 0.55 to 0.63 ms (the L2: 250
// MB), 1024 x 4096 186 us and 64 x 256 60 us (fifteen products one after the other).
//
// Every wait is bounded; a role whose wait runs out sets the timeout bit of the status
// word and winds down.
#pragma once

#include "moe_sm103.cuh"

namespace moe_op {

constexpr int OR_THREADS = 384;
constexpr int OR_EPI_WARPS = 8;
constexpr int OR_MAX_STAGES = 8;
constexpr int OR_EPI_BYTES = OR_EPI_WARPS * 8192;   // hi and lo of a warp's next two pieces
constexpr int OR_STORED = 4;         // units between the epilogue and the warp that counts them, at most
constexpr int OR_BARS = 2 * OR_MAX_STAGES + 5 + 2 * OR_STORED;
constexpr int OR_SMEM_MAX = 227 * 1024;
constexpr float OR_LO = 2048.0f;     // X = hi + lo / OR_LO: fp16 has 11 bits
enum : int { OR_GRAM = 0, OR_POLY = 1, OR_APPLY = 2 };

// A product of every step: output rows and columns, tiles of a matrix, K blocks and their
// splits.  (Partial sums have a place for each product: one matrix may be a product ahead
// of another.)
struct OrthoPhase {
  int M, N, tiles, kb, ks;
  float* part;              // [unit][CG][4][BN / 32][32 x 32]: partial sums of a split K
  unsigned* arrived;        // [tile][CG][8]: splits that have left theirs, in all steps so far
};

struct OrthoArgs {
  CUtensorMap tx[2], ta, tb;         // boxes of 64 x 64: X of even and odd steps, O, P
  OrthoPhase ph[3];
  int steps, matrices, group;   // matrices that go through the steps together
  int stages;               // slots of the ring, a K block each
  unsigned short* lo;       // X's second term (times OR_LO) in pieces of 32 x 32, a lane's 16-byte words side by side
  int64_t step_lo;
  int cols_lo;              // pieces in a row of them
  float *d, *e;             // the diagonals
  int64_t step_diag;
  unsigned short *x[2], *a, *b;   // the same as rows
  int64_t ld_x, ld_a, step_x, step_a;
  unsigned short* out;      // the caller's bf16 matrices
  int64_t ld_out, step_out;
  int vec_out;              // their rows take 32-byte stores
  float ka, kb, kc, inv_s2;   // a, b, c / s^2, 1 / s^2
  float ka_lo;                // a / OR_LO
  float inv_s;
  unsigned* done;           // [matrix][3]: epilogue warps that are through with a unit of each product
  int* status;
};

__host__ __device__ inline int or_stage_bytes() { return 2 * 128 * 128; }   // 128 rows of A and of B (CG 2: a half of it)
__host__ __device__ inline int or_smem_bytes(int stages) { return stages * or_stage_bytes() + OR_EPI_BYTES + 8 * (OR_BARS + 1) + 1024; }
// Partial sums of a CTA's part of a tile: 128 rows, CG * 128 columns.
__host__ __device__ constexpr int or_part_floats(int cg) { return 128 * 128 * cg; }
__host__ __device__ inline int or_tiles(int mode, int cg, int M, int N) {
  const int tm = (M + cg * 128 - 1) / (cg * 128), tn = (N + cg * 128 - 1) / (cg * 128);
  return mode == OR_APPLY ? tm * tn : tm * (tm + 1) / 2;
}

struct OrthoUnit {
  int mode, step, z, m0, n0, kb0, nkb, ks, split;
  int tile;     // of the product, over the group's matrices
  int unit;     // the same with its split
};

// Unit g of the list: groups, steps, products, matrices, tiles, K splits.  Symmetric: tile
// rows one after the other, each up to the diagonal; else in groups of 8 tile rows, rows fastest.
template <int CG>
__host__ __device__ __forceinline__ OrthoUnit or_unit(const OrthoArgs& A, int64_t g) {
  constexpr int TS = CG * 128;
  OrthoUnit U;
  const int u0 = A.ph[0].tiles * A.ph[0].ks, u1 = A.ph[1].tiles * A.ph[1].ks, u2 = A.ph[2].tiles * A.ph[2].ks;   // of a matrix
  const int64_t whole = static_cast<int64_t>(u0 + u1 + u2) * A.group * A.steps;
  const int z0 = static_cast<int>(g / whole) * A.group, nz = A.group < A.matrices - z0 ? A.group : A.matrices - z0;
  g -= g / whole * whole;
  const int per = (u0 + u1 + u2) * nz;
  U.step = static_cast<int>(g / per);
  int r = static_cast<int>(g - static_cast<int64_t>(U.step) * per);
  U.mode = OR_GRAM;
  if (r >= u0 * nz) {
    r -= u0 * nz;
    U.mode = OR_POLY;
    if (r >= u1 * nz) {
      r -= u1 * nz;
      U.mode = OR_APPLY;
    }
  }
  const OrthoPhase& P = A.ph[U.mode];
  U.ks = P.ks;
  U.unit = r;
  U.tile = r / P.ks;
  U.split = r - U.tile * P.ks;
  U.z = U.tile / P.tiles;
  int t = U.tile - U.z * P.tiles;
  U.z += z0;
  if (U.mode != OR_APPLY) {
    int i = static_cast<int>((sqrtf(8.0f * t + 1.0f) - 1.0f) * 0.5f);
    while (i * (i + 1) / 2 > t) --i;
    while ((i + 1) * (i + 2) / 2 <= t) ++i;
    const int j = t - i * (i + 1) / 2;
    U.m0 = i * TS;
    U.n0 = j * TS;
  } else {
    const int tm = (P.M + TS - 1) / TS, tn = (P.N + TS - 1) / TS;
    const int gr = t / (8 * tn), rows = tm - 8 * gr < 8 ? tm - 8 * gr : 8;
    t -= gr * 8 * tn;
    U.m0 = (8 * gr + t % rows) * TS;
    U.n0 = (t / rows) * TS;
  }
  U.kb0 = U.split * P.kb / P.ks;
  U.nkb = (U.split + 1) * P.kb / P.ks - U.kb0;
  return U;
}

// Where a CTA's unit n stands in the ring of stored units.  Epilogue warps arrive at
// stored[slot], which completes its phase of `parity`; the warp that counts waits for that
// and then arrives at taken[slot].  A barrier tells the parity of its phases only, so an
// epilogue warp that comes to the slot again waits for taken[slot]'s phase before this one:
// else the counting warp, four units behind, would take a completed phase for one to come.
struct OrthoSlot {
  int slot;
  uint32_t parity;
  bool again;        // the slot has been used: first wait for taken's phase of parity ^ 1
};
__host__ __device__ __forceinline__ OrthoSlot or_slot(uint32_t n) {
  return OrthoSlot{static_cast<int>(n % OR_STORED), (n / OR_STORED) & 1u, n >= OR_STORED};
}

// Whether K block k0 of the unit's A or B (TALL: of tall matrices) is an MN-major operand: X where
// its rows are K, and the tiles of a symmetric matrix that are stored as their transposes.
template <int CG, bool TALL>
__device__ __forceinline__ bool or_a_mn(const OrthoUnit& U, int k0) {
  return U.mode == OR_GRAM ? TALL : (U.mode == OR_POLY || !TALL) && k0 >= U.m0 + CG * 128;
}
template <int CG, bool TALL>
__device__ __forceinline__ bool or_b_mn(const OrthoUnit& U, int k0) {
  return U.mode == OR_GRAM ? TALL : U.mode == OR_APPLY && !TALL ? true : k0 >= U.n0 + CG * 128;
}

// The counter that a unit's inputs are done by, and the value it has to reach.
template <int CG>
__host__ __device__ __forceinline__ const unsigned* or_needs(const OrthoArgs& A, const OrthoUnit& U, unsigned* count) {
  const int from = U.mode == OR_GRAM ? OR_APPLY : U.mode - 1;
  const int rounds = U.mode == OR_GRAM ? U.step : U.step + 1;
  *count = static_cast<unsigned>(rounds) * static_cast<unsigned>(A.ph[from].tiles * A.ph[from].ks) * (OR_EPI_WARPS * CG);
  return A.done + U.z * 3 + from;
}
// Bounded wait of a warp until other CTAs have counted so far; what they wrote before is
// seen by this warp's loads and by tensor copies that it issues.
__device__ __forceinline__ bool or_wait_count(const unsigned* p, unsigned count) {
  const long long t0 = clock64();
  do {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    if (__all_sync(0xFFFFFFFFu, v >= count)) {
      asm volatile("fence.proxy.async.global;" ::: "memory");
      return true;
    }
  } while (clock64() - t0 < WAIT_CLOCKS);
  return false;
}

__device__ __forceinline__ void or_pack(const float (&v)[32], int dt, uint4 (&w)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = make_uint4(pack2(v[8 * j], v[8 * j + 1], dt), pack2(v[8 * j + 2], v[8 * j + 3], dt),
                      pack2(v[8 * j + 4], v[8 * j + 5], dt), pack2(v[8 * j + 6], v[8 * j + 7], dt));
}
// A lane's row of a piece to global memory: 64 bytes, 32-byte aligned.
__device__ __forceinline__ void or_store(unsigned short* p, const uint4 (&w)[4]) {
  stg32(p, w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w);
  stg32(p + 16, w[2].x, w[2].y, w[2].z, w[2].w, w[3].x, w[3].y, w[3].z, w[3].w);
}
// A piece of rows ld apart into shared memory, 16-byte words of a row exchanged by the
// row so that lanes read their rows without bank conflicts.  Rows from `rows` on are zero.
__device__ __forceinline__ void or_copy_rows(uint32_t to, const unsigned short* p, int64_t ld, int rows, int lane) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = j * 8 + (lane >> 2), w = lane & 3;
    copy16(to + static_cast<uint32_t>(r * 64 + ((w ^ (r >> 1 & 3)) << 4)), p + (r < rows ? r * ld : 0) + w * 8, r < rows);
  }
}
__device__ __forceinline__ void or_load_rows(uint32_t p, uint4 (&w)[4], int lane) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[j].x), "=r"(w[j].y), "=r"(w[j].z), "=r"(w[j].w)
                 : "r"(p + static_cast<uint32_t>(lane * 64 + ((j ^ (lane >> 1 & 3)) << 4)))
                 : "memory");
}
// A piece that lies as lanes read it: each copies, reads and writes its own words.
__device__ __forceinline__ void or_copy(uint32_t to, const unsigned short* p, int lane) {
#pragma unroll
  for (int j = 0; j < 4; ++j) copy16(to + static_cast<uint32_t>(j * 512 + lane * 16), p + j * 256 + lane * 8, true);
}
__device__ __forceinline__ void or_load(uint32_t p, uint4 (&w)[4], int lane) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[j].x), "=r"(w[j].y), "=r"(w[j].z), "=r"(w[j].w)
                 : "r"(p + static_cast<uint32_t>(j * 512 + lane * 16))
                 : "memory");
}
__device__ __forceinline__ void or_save(unsigned short* p, const uint4 (&w)[4], int lane) {
#pragma unroll
  for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(p + j * 256 + lane * 8) = w[j];
}
__device__ __forceinline__ float or_value(const uint4 (&w)[4], int j) {
  const uint4& u = w[j / 8];
  const uint32_t x = j % 8 < 2 ? u.x : j % 8 < 4 ? u.y : j % 8 < 6 ? u.z : u.w;
  return j & 1 ? hi16(x, DT_FP16) : lo16(x, DT_FP16);
}

template <int CG, bool TALL>
__global__ void __launch_bounds__(OR_THREADS, 1) k_ortho(const __grid_constant__ OrthoArgs A) {
  constexpr int BN = CG * 128;
  extern __shared__ __align__(1024) char or_smem[];
  char* base = or_smem + ((1024u - (smem_u32(or_smem) & 1023u)) & 1023u);
  const int S = A.stages;
  const int stage_bytes = or_stage_bytes();
  char* epi = base + S * stage_bytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(epi + OR_EPI_BYTES);
  uint64_t *full = bars, *empty = bars + OR_MAX_STAGES, *accf = bars + 2 * OR_MAX_STAGES, *acce = accf + 2, *drain = acce + 2, *stored = drain + 1, *taken = stored + OR_STORED;
  uint32_t* holder = reinterpret_cast<uint32_t*>(bars + OR_BARS);
  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  const int worker = blockIdx.x / CG, nworkers = gridDim.x / CG;
  const int64_t units = static_cast<int64_t>(A.ph[0].tiles * A.ph[0].ks + A.ph[1].tiles * A.ph[1].ks + A.ph[2].tiles * A.ph[2].ks) *
                        A.matrices * A.steps;
  constexpr uint32_t tm_cols = 2 * BN;

  if (warp == 2) tm_alloc<CG>(smem_u32(holder), tm_cols);
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      bar_init(smem_u32(&full[s]), 1);
      bar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      bar_init(smem_u32(&accf[b]), 1);
      bar_init(smem_u32(&acce[b]), OR_EPI_WARPS * CG);
    }
    bar_init(smem_u32(drain), 1);
    for (int i = 0; i < OR_STORED; ++i) {
      bar_init(smem_u32(&stored[i]), OR_EPI_WARPS);
      bar_init(smem_u32(&taken[i]), 1);
    }
    bar_fence_init();
  }
  tm_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();
  tm_fence_after();
  const uint32_t tmem = *holder;
  bool ok = true;
  auto gave_up = [&] {
    atomicOr(A.status, STATUS_TIMEOUT);
    ok = false;
    return false;
  };
  auto wait = [&](uint64_t* b, uint32_t parity) { return bar_wait(smem_u32(b), parity) || gave_up(); };
  // (a CTA may have to wait for others between its units: two limits, so that the one that waits for them gives up first)
  auto wait_long = [&](uint64_t* b, uint32_t parity) { return bar_wait(smem_u32(b), parity) || wait(b, parity); };
  auto wait_inputs = [&](const OrthoUnit& U) {
    unsigned count;
    const unsigned* p = or_needs<CG>(A, U, &count);
    return count == 0 || or_wait_count(p, count) || gave_up();
  };

  if (warp == 0) {
    // ---------------- tensor copies ----------------
    RingPos R;
    bool again = false;   // slots have been used before
    uint32_t q = 0;
    for (int64_t g = worker; ok && g < units; g += nworkers) {
      const OrthoUnit U = or_unit<CG>(A, g);
      const int am = U.m0 + static_cast<int>(rank) * 128, bn = U.n0 + static_cast<int>(rank) * 128;
      // boxes of 64 x 64: K-major, k across and 64 rows each; MN-major, 64 rows across and k down
      const CUtensorMap* x = &A.tx[U.step & 1];
      const CUtensorMap* ma = U.mode == OR_GRAM ? x : U.mode == OR_POLY ? &A.ta : TALL ? x : &A.tb;
      const CUtensorMap* mb = U.mode == OR_GRAM ? x : U.mode == OR_POLY ? &A.ta : TALL ? &A.tb : x;
      if (!wait_inputs(U)) break;
      for (int i = 0; i < U.nkb; ++i, ++q) {
        const int s = R.slot;
        if (again && !wait(&empty[s], R.parity ^ 1u)) break;
        R.next(S);
        again = again || R.slot == 0;
        // both CTAs' copies complete on the even CTA's barrier
        const uint32_t own = smem_u32(&full[s]), fb = CG == 2 ? cluster_addr(own, 0) : own;
        if (elect_lane()) {
          if (rank == 0) bar_expect_tx(own, static_cast<uint32_t>(CG * stage_bytes));
          const int k0 = (U.kb0 + i) * 64;
          const bool amn = or_a_mn<CG, TALL>(U, k0), bmn = or_b_mn<CG, TALL>(U, k0);
          const uint32_t da = smem_u32(base + s * stage_bytes), db = da + 128 * 128;
          tma_3d<CG>(da, ma, amn ? am : k0, amn ? k0 : am, U.z, fb);
          tma_3d<CG>(da + 8192, ma, amn ? am + 64 : k0, amn ? k0 : am + 64, U.z, fb);
          tma_3d<CG>(db, mb, bmn ? bn : k0, bmn ? k0 : bn, U.z, fb);
          tma_3d<CG>(db + 8192, mb, bmn ? bn + 64 : k0, bmn ? k0 : bn + 64, U.z, fb);
        }
        __syncwarp();
      }
    }
    // the last use of every slot is released (so the MMAs' arrivals at this
    // CTA's barriers have landed) before the CTA ends; after a wait that ran
    // out, at least the copies already issued land first
    const uint32_t used = q < static_cast<uint32_t>(S) ? q : static_cast<uint32_t>(S);
    for (uint32_t j = q - used; j < q; ++j) {
      if (ok) {
        wait(&empty[j % S], (j / S) & 1);
      } else if (rank == 0) {
        bar_wait(smem_u32(&full[j % S]), (j / S) & 1);
      }
    }
  } else if (warp == 1) {
    // ---------------- MMAs (the pair's even CTA) ----------------
    if (rank == 0) {
      RingPos R;
      uint32_t n = 0;
      for (int64_t g = worker; ok && g < units; g += nworkers, ++n) {
        const OrthoUnit U = or_unit<CG>(A, g);
        const int buf = n & 1;
        if (n >= 2 && !wait(&acce[buf], ((n >> 1) - 1) & 1)) break;
        tm_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(buf * BN);
        for (int i = 0; i < U.nkb; ++i) {
          const int s = R.slot, k0 = (U.kb0 + i) * 64;
          const bool amn = or_a_mn<CG, TALL>(U, k0), bmn = or_b_mn<CG, TALL>(U, k0);
          const uint32_t idesc = f16_idesc(CG * 128, BN, DT_FP16, amn, bmn);
          const uint32_t la = amn ? 8192 : 16, lb = bmn ? 8192 : 16, ka = amn ? 2048 : 32, kb = bmn ? 2048 : 32;
          if (!wait_long(&full[s], R.parity)) break;
          R.next(S);
          tm_fence_after();
          if (elect_lane()) {
            const uint32_t sa = smem_u32(base + s * stage_bytes), sb = sa + 128 * 128;
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k)
              tm_mma<CG>(d, sw128_desc(sa + k * ka, la), sw128_desc(sb + k * kb, lb), idesc, (i | k) != 0);
            tm_commit<CG>(smem_u32(&empty[s]));
          }
          __syncwarp();
        }
        if (ok && elect_lane()) tm_commit<CG>(smem_u32(&accf[buf]));
        __syncwarp();
      }
      if (!ok) {   // MMAs already issued end before their tensor memory is freed
        if (elect_lane()) tm_commit<CG>(smem_u32(drain));
        __syncwarp();
        bar_wait(smem_u32(drain), 0);
      }
    }
  } else if (warp == 3) {
    // ---------------- counts of finished units, for other CTAs ----------------
    uint32_t n = 0;
    for (int64_t g = worker; ok && g < units; g += nworkers, ++n) {
      const OrthoUnit U = or_unit<CG>(A, g);
      const OrthoSlot q = or_slot(n);
      if (!wait_long(&stored[q.slot], q.parity)) break;
      __syncwarp();   // (all lanes have seen it)
      if (lane == 0) {
        bar_arrive(smem_u32(&taken[q.slot]));
        asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(A.done + U.z * 3 + U.mode), "n"(OR_EPI_WARPS) : "memory");
      }
      __syncwarp();
    }
  } else if (warp >= 4) {
    // ---------------- epilogue ----------------
    constexpr int NP = BN / 64;   // pieces of a warp
    const int w8 = warp - 4, ew = warp & 3, half = w8 >> 2;
    const uint32_t st = smem_u32(epi + w8 * 8192);
    uint32_t n = 0;
    for (int64_t g = worker; ok && g < units; g += nworkers, ++n) {
      const OrthoUnit U = or_unit<CG>(A, g);
      const OrthoPhase& P = A.ph[U.mode];
      const int buf = n & 1;
      const bool apply = U.mode == OR_APPLY, poly = U.mode == OR_POLY, final = apply && U.step + 1 == A.steps;
      const uint32_t tcol = tmem + (static_cast<uint32_t>(ew * 32) << 16) + static_cast<uint32_t>(buf * BN);
      const int row0 = U.m0 + static_cast<int>(rank) * 128 + ew * 32, row = row0 + lane;
      const bool in = row < P.M, rows_live = row0 < P.M;
      const float* diag = (apply ? A.e : A.d) + U.z * A.step_diag;
      // the piece's own rows of X (apply: read, and written for the next step), of O (read by poly, written by gram) and of P
      const int64_t at_x = U.z * A.step_x + row0 * A.ld_x, at_a = U.z * A.step_a + row0 * A.ld_a;
      const unsigned short* from = apply ? A.x[U.step & 1] + at_x : A.a + at_a;
      unsigned short* lo_pieces = A.lo + U.z * A.step_lo + (static_cast<int64_t>(row0 >> 5) * A.cols_lo + (U.n0 >> 5)) * 1024;
      // pieces that this warp finishes: all of its own, or its split's share
      auto live = [&](int i) { return rows_live && U.n0 + 32 * half + 64 * i < P.N; };
      auto takes = [&](int i) { return live(i) && (U.ks == 1 || (w8 * NP + i) % U.ks == U.split); };
      // what a piece needs of its own elements, into the buffer of its number's parity
      auto fetch = [&](int i) {
        if (i < NP && U.mode != OR_GRAM && takes(i)) {
          or_copy_rows(st + (i & 1) * 4096, from + U.n0 + 32 * half + 64 * i, apply ? A.ld_x : A.ld_a, P.M - row0, lane);
          if (apply) or_copy(st + (i & 1) * 4096 + 2048, lo_pieces + half * 1024 + i * 2048, lane);
        }
        copies_commit();
      };
      if (!wait_inputs(U)) break;
      fetch(0);
      fetch(1);
      const float d_row = (poly || (apply && !TALL)) && in ? diag[row] : 0.0f;
      auto col_diag = [&](int i) { return (poly || (apply && TALL)) && i < NP && live(i) ? diag[U.n0 + 32 * half + 64 * i + lane] : 0.0f; };
      float d_next = col_diag(0);
      if (!wait_long(&accf[buf], (n >> 1) & 1)) break;
      tm_fence_after();
      // the accumulators are in registers: the buffer may be rewritten
      auto release = [&] {
        tm_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (CG == 2) bar_arrive_cluster(smem_u32(&acce[buf]), 0);
          else bar_arrive(smem_u32(&acce[buf]));
        }
      };
      // K split: this unit's partial sums to memory, and a wait for the tile's other splits
      float* part = P.part + (static_cast<int64_t>(U.unit) * CG + rank) * or_part_floats(CG) + (ew * (BN / 32) + half) * 1024 + lane * 4;
      if (U.ks > 1) {
#pragma unroll 1
        for (int i = 0; i < NP; ++i) {
          uint32_t a[32];
          tm_ld32(tcol + 32 * half + 64 * i, a);
          tm_wait_ld();
          if (i == NP - 1) release();
          if (live(i))
#pragma unroll
            for (int j = 0; j < 32; j += 4) *reinterpret_cast<uint4*>(part + i * 2048 + j * 32) = make_uint4(a[j], a[j + 1], a[j + 2], a[j + 3]);
        }
        unsigned* count = P.arrived + (U.tile * CG + static_cast<int>(rank)) * OR_EPI_WARPS + w8;
        __syncwarp();
        if (lane == 0) asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(count) : "memory");
        __syncwarp();
        if (!or_wait_count(count, static_cast<unsigned>(U.ks) * static_cast<unsigned>(U.step + 1))) {
          gave_up();
          break;
        }
        part -= static_cast<int64_t>(U.split) * CG * or_part_floats(CG);   // the first split's
      }
      // (not unrolled: the code of every piece and product once is what fits the instruction cache)
#pragma unroll 1
      for (int i = 0; i < NP; ++i) {
        const int c = 32 * half + 64 * i, col0 = U.n0 + c;
        const float d_col = d_next;
        d_next = col_diag(i + 1);
        float r[32];
        if (U.ks == 1) {
          uint32_t a[32];
          tm_ld32(tcol + c, a);
          tm_wait_ld();
          if (i == NP - 1) release();
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = __uint_as_float(a[j]);
        }
        if (!takes(i)) {
          fetch(i + 2);
          continue;
        }
        if (U.ks > 1) {
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = 0.0f;
          const float* p = part + i * 2048;
#pragma unroll 2
          for (int s = 0; s < U.ks; ++s, p += CG * or_part_floats(CG)) {
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 f = __ldcg(reinterpret_cast<const float4*>(p + j * 32));
              r[j] += f.x, r[j + 1] += f.y, r[j + 2] += f.z, r[j + 3] += f.w;
            }
          }
        }
        float v[32];
        if (U.mode == OR_GRAM) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = r[j];
        } else {
          copies_wait_n<1>();
          __syncwarp();
          const uint32_t mine = st + (i & 1) * 4096;
          uint4 hi[4];
          or_load_rows(mine, hi, lane);
          if (poly) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float o = or_value(hi, j);
              v[j] = fmaf(A.kb, o, A.kc * fmaf(o, d_row + __shfl_sync(0xFFFFFFFFu, d_col, j), r[j]));
            }
          } else {
            uint4 lo[4];
            or_load(mine + 2048, lo, lane);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float e = TALL ? __shfl_sync(0xFFFFFFFFu, d_col, j) : d_row;
              v[j] = fmaf(A.ka + e, or_value(hi, j), fmaf(A.ka_lo, or_value(lo, j), A.inv_s2 * r[j]));
            }
          }
        }
        if (!apply && row0 == col0) {   // the diagonal: kept apart, in fp32
          float x = 0.0f;
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j == lane) {
              x = r[j];
              v[j] = 0.0f;
            }
          if (in) {
            if (poly) x = (A.kb * d_row + A.kc * fmaf(d_row, d_row, x)) * A.inv_s2;
            (poly ? A.e : A.d)[U.z * A.step_diag + row] = x;
          }
        }
        if (final) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] *= A.inv_s;
        }
        // (the caller's rows that 32-byte stores do not fit go by way of this piece's buffer)
        const bool staged = final && !(A.vec_out && col0 + 32 <= P.N);
        if (!staged) {
          __syncwarp();   // this piece's buffer has been read
          fetch(i + 2);
        }
        uint4 w[4];
        or_pack(v, final ? DT_BF16 : DT_FP16, w);
        if (!apply) {
          if (in) or_store((poly ? A.b : A.a) + at_a + lane * A.ld_a + col0, w);
        } else if (!final) {
          if (in) or_store(A.x[(U.step + 1) & 1] + at_x + lane * A.ld_x + col0, w);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = OR_LO * (v[j] - or_value(w, j));
          or_pack(v, DT_FP16, w);
          or_save(lo_pieces + half * 1024 + i * 2048, w, lane);
        } else if (!staged) {
          if (in) or_store(A.out + U.z * A.step_out + row * A.ld_out + col0, w);
        } else {
          const uint32_t mine = st + (i & 1) * 4096;
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 4; ++j)
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(mine + static_cast<uint32_t>(lane * 80 + j * 16)), "r"(w[j].x),
                         "r"(w[j].y), "r"(w[j].z), "r"(w[j].w)
                         : "memory");
          __syncwarp();
          if (col0 + lane < P.N) {
            unsigned short* out = A.out + U.z * A.step_out + row0 * A.ld_out + col0 + lane;
            const int rows = min(32, P.M - row0);
#pragma unroll 8
            for (int k = 0; k < rows; ++k) {
              unsigned short x;
              asm volatile("ld.shared.b16 %0, [%1];" : "=h"(x) : "r"(mine + static_cast<uint32_t>(k * 80 + lane * 2)) : "memory");
              out[k * A.ld_out] = x;
            }
          }
          __syncwarp();
          fetch(i + 2);
        }
      }
      // this warp's part is on its way to memory: tensor copies of other CTAs may read it
      // once warp 3 has said so
      asm volatile("fence.proxy.async.global;" ::: "memory");
      __syncwarp();
      const OrthoSlot q = or_slot(n);
      if (q.again && !wait(&taken[q.slot], q.parity ^ 1u)) break;
      __syncwarp();
      if (lane == 0) bar_arrive(smem_u32(&stored[q.slot]));
    }
  }
  tm_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();
  if (warp == 2) {
    tm_fence_after();
    tm_free<CG>(tmem, tm_cols);
  }
}

// ---------------------------------------------------------------------------
// the start: X = s G / (|G| + eps)
// ---------------------------------------------------------------------------

constexpr int OR_NORM_CTAS = 608;   // partial sums of a matrix at most

// CTAs of each of n matrices of R x C for the norm and the start: one for up to 32 K elements, in one
// launch, else one for 8 K, up to eight an SM in all.  One launch / two, one step, us: 64 x 64 15.6 / 15.7, 64 x
// 256 20.6 / 19.2, 128 x 256 28.4 / 21.8, 64 of 64 x 256 23.9 / 22.3, 256 x 512 69.6 / 23.9: equal
// at 4 K elements; what one launch costs at 32 K is more than the 2.5 us of the host that it saves.  A CTA for 4 K / 8 K / 16 K elements: 256 x 512
// 22.5 / 23.9 / 27.1, 1024 x 1024 32.7 / 32.3 / 35.4, 1024 x 4096 51.0 / 50.0 / 50.9.
__host__ __device__ inline int or_start_ctas(int64_t R, int64_t C, int64_t n, int sms) {
  const int64_t pieces = R * ((C + 7) / 8);
  if (pieces <= 4096) return 1;
  int64_t c = (pieces + 1023) / 1024;
  if (c > (8ll * sms + n - 1) / n) c = (8ll * sms + n - 1) / n;
  return static_cast<int>(c < OR_NORM_CTAS ? c : OR_NORM_CTAS);
}
// Partial sums that calls of up to n matrices need room for: n of them take n times ceil(8 SMs / n) at most.
__host__ __device__ inline int64_t or_norm_parts(int64_t R, int64_t C, int64_t n, int sms) {
  const int64_t most = or_start_ctas(R, C, 1, sms);
  if (most == 1) return 1;   // the start makes its own
  return n * most < 8ll * sms + n ? n * most : 8ll * sms + n;
}

struct OrthoStart {
  const void* g;
  int dt;                   // moe_dtype of g
  int64_t ldg, step_g;
  int M, N, ctas;           // CTAs a matrix
  float* part;              // [matrix][ctas][3]
  unsigned short* hi;       // X as the tensor copies read it
  int64_t ld_x, step_x;
  unsigned short* lo;       // and its second term, in pieces
  int64_t step_lo;
  int cols_lo;
  int vec;                  // elements of a row come eight at a time
  double s, eps;
  unsigned* done;           // [matrix][3], cleared
  unsigned* arrived;        // cleared by the first matrix
  int n_arrived;
};

// Up to eight elements from column c of a row (zeros past the last one).
__device__ __forceinline__ void or_read(const OrthoStart& A, int64_t at, int left, float (&v)[8]) {
  if (A.vec && left >= 8) {
    if (A.dt == 2) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(A.g) + at);
      *reinterpret_cast<float4*>(v) = p[0];
      *reinterpret_cast<float4*>(v + 4) = p[1];
    } else {
      const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const unsigned short*>(A.g) + at);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = lo16(u[j], A.dt);
        v[2 * j + 1] = hi16(u[j], A.dt);
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    v[j] = j >= left ? 0.0f : A.dt == 2 ? static_cast<const float*>(A.g)[at + j] : ld16(A.g, at + j, A.dt);
}

// A warp's unit: 4 rows of 64 columns, a lane has 8 of them (row lane / 8).  f(row, column,
// values) for the units of this CTA in turn, four of them under way at a time.
template <typename F>
__device__ __forceinline__ void or_elements(const OrthoStart& A, int z, F&& f) {
  const int lane = threadIdx.x & 31, r = lane >> 3, c = (lane & 7) * 8;
  const int cols = (A.N + 63) / 64;
  const int n = (A.M + 3) / 4 * cols;   // (at most 8192 * 512)
  const int step = static_cast<int>(gridDim.x) * 8;
  for (int u = static_cast<int>(blockIdx.x) * 8 + (threadIdx.x >> 5); u < n; u += 4 * step) {
    float v[4][8];
    int row[4], col[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = u + k * step, b = i / cols;
      row[k] = b * 4 + r;
      col[k] = (i - b * cols) * 64 + c;
      if (i >= n || row[k] >= A.M || col[k] >= A.N) row[k] = -1;
      if (row[k] >= 0) or_read(A, z * A.step_g + row[k] * A.ldg + col[k], A.N - col[k], v[k]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (row[k] >= 0) f(row[k], col[k], v[k]);
  }
}

// A CTA's share of a matrix's squares, summed in fp32: eight at a time where their sum is far
// from fp32's ends, else each in one of three ranges (of 2^-40 and 2^40) that is scaled
// so that no square, from 2^-149 to 2^128, vanishes and no sum of 2^30 of them overflows.
// sums[0..2]: the ranges.
__device__ __forceinline__ void or_squares(const OrthoStart& A, int z, float (*warps)[3], float* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float s[3] = {0.0f, 0.0f, 0.0f};
  or_elements(A, z, [&](int, int, const float (&v)[8]) {
    float t = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) t = fmaf(v[j], v[j], t);
    if (t > 0x1p-80f && t < 0x1p80f) {
      s[1] += t;
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = fabsf(v[j]);
      if (x > 0x1p40f) {
        s[2] = fmaf(x * 0x1p-90f, x * 0x1p-90f, s[2]);
      } else if (x < 0x1p-40f) {
        s[0] = fmaf(x * 0x1p85f, x * 0x1p85f, s[0]);
      } else {
        s[1] = fmaf(x, x, s[1]);   // (NaN too)
      }
    }
  });
#pragma unroll
  for (int k = 0; k < 3; ++k) {
#pragma unroll
    for (int d = 16; d > 0; d /= 2) s[k] += __shfl_xor_sync(0xFFFFFFFFu, s[k], d);
    if (lane == 0) warps[warp][k] = s[k];
  }
  __syncthreads();
  if (threadIdx.x < 3) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += warps[w][threadIdx.x];
    sums[threadIdx.x] = t;
  }
}

__global__ void __launch_bounds__(256) k_ortho_norm(const OrthoStart A) {
  __shared__ float warps[8][3];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  or_squares(A, blockIdx.y, warps, A.part + (static_cast<int64_t>(blockIdx.y) * A.ctas + blockIdx.x) * 3);
}

// X = hi + lo / OR_LO in fp16.  Every CTA adds the matrix's partial sums in order (one that has the
// matrix alone makes them); the factor s / (|G| + eps) is applied as two, so that it has
// 64-bit numbers' range.
__global__ void __launch_bounds__(256) k_ortho_start(const OrthoStart A) {
  __shared__ float factor[2], warps[8][3], alone[3];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int z = blockIdx.y;
  if (A.ctas == 1) {
    or_squares(A, z, warps, alone);
    __syncthreads();
  }
  if (threadIdx.x < 32) {
    const float* part = A.ctas == 1 ? alone : A.part + static_cast<int64_t>(z) * A.ctas * 3;
    double t[3] = {0.0, 0.0, 0.0};
    for (int i = threadIdx.x; i < A.ctas; i += 32)
#pragma unroll
      for (int k = 0; k < 3; ++k) t[k] += part[i * 3 + k];
    double sum = t[0] * 0x1p-170 + t[1] + t[2] * 0x1p180;
#pragma unroll
    for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    if (threadIdx.x == 0) {
      const double r = A.s / (sqrt(sum) + A.eps);
      int ex = 0;
      if (r > 0.0 && r < 1e300) {
        frexp(r, &ex);
        factor[0] = static_cast<float>(ldexp(1.0, ex / 2));
        factor[1] = static_cast<float>(ldexp(r, -(ex / 2)));
      } else {
        factor[0] = 1.0f;
        factor[1] = static_cast<float>(r);
      }
    }
  }
  if (blockIdx.x == 0) {
    if (threadIdx.x < 3) A.done[z * 3 + threadIdx.x] = 0;
    if (z == 0)
      for (int i = threadIdx.x; i < A.n_arrived; i += 256) A.arrived[i] = 0;
  }
  __syncthreads();
  const float f0 = factor[0], f1 = factor[1];
  or_elements(A, z, [&](int row, int col, const float (&v)[8]) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = v[2 * j] * f0 * f1, b = v[2 * j + 1] * f0 * f1;
      h[j] = pack2(a, b, DT_FP16);
      l[j] = pack2(OR_LO * (a - lo16(h[j], DT_FP16)), OR_LO * (b - hi16(h[j], DT_FP16)), DT_FP16);
    }
    *reinterpret_cast<uint4*>(A.hi + z * A.step_x + row * A.ld_x + col) = make_uint4(h[0], h[1], h[2], h[3]);   // (rows are padded to 32 elements)
    unsigned short* p = A.lo + z * A.step_lo + (static_cast<int64_t>(row >> 5) * A.cols_lo + (col >> 5)) * 1024 +
                        ((col >> 3) & 3) * 256 + (row & 31) * 8;
    *reinterpret_cast<uint4*>(p) = make_uint4(l[0], l[1], l[2], l[3]);
  });
}

}  // namespace moe_op
