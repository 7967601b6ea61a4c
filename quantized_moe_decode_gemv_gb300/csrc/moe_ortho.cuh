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
//   - X is kept as two fp16 terms, hi + lo.  Products take hi, the linear term a X both:
//     what rounding leaves of X lies in directions that X itself may not have, where p
//     multiplies by a = 3.4 a step; without lo a gradient of 9 tokens was off by 4e-2.
//
// All steps are one launch (k_ortho).  The tiles of all products, (step, product, matrix,
// tile), are one list that CTAs (pairs, for 256 x 256 tiles) take in turn; a tile waits
// until the products that it reads are done, by counters of finished epilogues for each
// matrix and product.  Tiles only wait for tiles before them in the list and all CTAs are
// resident (a cooperative launch), so somebody always can go on.  As launches of their
// own, products were 2.1 waves taken as 3 (16 matrices of 1856 x 1024, tiles of 256 x
// 256 on 76 pairs), and each paid for its launch, its pipeline's filling and its
// epilogues' end.
//
// Roles of a CTA's 12 warps, as in k_gemm16: tensor copies, MMAs, tensor memory, and
// eight epilogue warps; accumulators double-buffered.  Tiles are square, CG * 128 on a
// side; a symmetric product computes those on and below the diagonal and stores the
// others as their transposes.  Where tiles are fewer than CTAs, K is split; the last of a
// tile's splits to arrive, warp by warp, adds the partial sums in order.
//
// An epilogue warp's piece is 32 x 32 values, a row a lane.  Memory that lanes address by
// their rows is 32 lines an instruction, and that paced the epilogues (17 thousand clocks
// for a 256 x 256 tile, more than the MMAs of K = 1024).  So what an epilogue reads of its
// own element, X for the linear term and O for b A, lies a second time in pieces as lanes
// read them (16 bytes of 32 lanes side by side), and rows are written by tensor copies
// from shared memory.
//
// Every wait is bounded; a role whose wait runs out sets the timeout bit of the status
// word and winds down.
#pragma once

#include "moe_sm103.cuh"

namespace moe_op {

constexpr int OR_THREADS = 384;
constexpr int OR_EPI_WARPS = 8;
constexpr int OR_MAX_STAGES = 8;
constexpr int OR_EPI_BYTES = OR_EPI_WARPS * 8192;   // a warp's 32 x 32 values and their transpose; hi and lo of its next piece
constexpr int OR_BARS = 2 * OR_MAX_STAGES + 9 + OR_EPI_WARPS;
constexpr int OR_SMEM_MAX = 227 * 1024;
enum : int { OR_GRAM = 0, OR_POLY = 1, OR_APPLY = 2 };

// A product of every step: output rows and columns, tiles of a matrix, K blocks and their
// splits.  (Partial sums have a place for each product: one matrix may be a product ahead
// of another.)
struct OrthoPhase {
  int M, N, tiles, kb, ks, units;   // units: of all matrices
  float* part;              // [unit][CG][4][BN / 32][32 x 32]: partial sums of a split K
  unsigned* arrived;        // [tile][CG][8]: splits that have left theirs, in all steps so far
};

struct OrthoArgs {
  CUtensorMap lx[2], la, lb;         // loads (64 x 64): X of even and odd steps, O, P
  CUtensorMap sx[2], sa, sb, out;    // stores (32 x 32): the same, and the caller's matrices
  OrthoPhase ph[3];
  int steps;
  int stages;               // slots of the ring, a K block each
  // pieces of 32 x 32 values as epilogues read them: O (written by GRAM, read by POLY), X as hi and lo (APPLY)
  unsigned short *own_a, *own_x;
  int64_t step_own_a, step_own_x;
  int cols_a, cols_x;       // pieces in a row of them
  float *d, *e;             // the diagonals
  int64_t step_diag;
  unsigned short* last;     // the caller's bf16 matrices where tensor copies cannot write them, else null
  int64_t ld_last, step_last;
  float ka, kb, kc, inv_s2;   // a, b, c / s^2, 1 / s^2
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
  int tile;     // of the product, over all matrices
  int unit;     // the same with its split
  bool mirror;
};

// Unit g of the list: steps, products, matrices, tiles, K splits.  Symmetric: tile rows
// one after the other, each up to the diagonal; else in groups of 8 tile rows, rows fastest.
template <int CG>
__device__ __forceinline__ OrthoUnit or_unit(const OrthoArgs& A, int64_t g) {
  constexpr int TS = CG * 128;
  OrthoUnit U;
  const int per = A.ph[0].units + A.ph[1].units + A.ph[2].units;
  U.step = static_cast<int>(g / per);
  int r = static_cast<int>(g - static_cast<int64_t>(U.step) * per);
  U.mode = OR_GRAM;
  if (r >= A.ph[0].units) {
    r -= A.ph[0].units;
    U.mode = OR_POLY;
    if (r >= A.ph[1].units) {
      r -= A.ph[1].units;
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
  if (U.mode != OR_APPLY) {
    int i = static_cast<int>((sqrtf(8.0f * t + 1.0f) - 1.0f) * 0.5f);
    while (i * (i + 1) / 2 > t) --i;
    while ((i + 1) * (i + 2) / 2 <= t) ++i;
    const int j = t - i * (i + 1) / 2;
    U.m0 = i * TS;
    U.n0 = j * TS;
    U.mirror = i != j;
  } else {
    const int tm = (P.M + TS - 1) / TS, tn = (P.N + TS - 1) / TS;
    const int gr = t / (8 * tn), rows = min(8, tm - 8 * gr);
    t -= gr * 8 * tn;
    U.m0 = (8 * gr + t % rows) * TS;
    U.n0 = (t / rows) * TS;
    U.mirror = false;
  }
  U.kb0 = U.split * P.kb / P.ks;
  U.nkb = (U.split + 1) * P.kb / P.ks - U.kb0;
  return U;
}

// The counter that a unit's inputs are done by, and the value it has to reach.
template <int CG>
__device__ __forceinline__ const unsigned* or_needs(const OrthoArgs& A, const OrthoUnit& U, unsigned* count) {
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

// A warp's piece in shared memory as a tensor copy of 32 columns reads it: rows of 64
// bytes, their 16-byte words exchanged by the row (64-byte swizzle).
__device__ __forceinline__ uint32_t or_at(uint32_t st, int row, int word) {
  return st + static_cast<uint32_t>(row * 64 + ((word ^ (row >> 1 & 3)) << 4));
}
__device__ __forceinline__ void or_stage(uint32_t st, const uint4 (&w)[4], int lane) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(or_at(st, lane, j)), "r"(w[j].x), "r"(w[j].y), "r"(w[j].z), "r"(w[j].w)
                 : "memory");
}
// Its transpose.  Neighbouring lanes trade one of two columns, so that a lane writes two
// rows' values of a column at once.
__device__ __forceinline__ void or_stage_mirror(uint32_t st, const float (&v)[32], int lane) {
  const int odd = lane & 1;
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    const float give = odd ? v[j] : v[j + 1];
    const float got = __shfl_xor_sync(0xFFFFFFFFu, give, 1);
    const uint32_t w = odd ? pack2(got, v[j + 1], DT_FP16) : pack2(v[j], got, DT_FP16);
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(or_at(st, j + odd, lane >> 3) + static_cast<uint32_t>(lane & 6) * 2), "r"(w) : "memory");
  }
}

__device__ __forceinline__ void or_pack(const float (&v)[32], int dt, uint4 (&w)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = make_uint4(pack2(v[8 * j], v[8 * j + 1], dt), pack2(v[8 * j + 2], v[8 * j + 3], dt),
                      pack2(v[8 * j + 4], v[8 * j + 5], dt), pack2(v[8 * j + 6], v[8 * j + 7], dt));
}
// Half of a piece (hi or lo): a lane's row as four words, those of the lanes side by side.
__device__ __forceinline__ void or_load(uint32_t p, uint4 (&w)[4], int lane) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[j].x), "=r"(w[j].y), "=r"(w[j].z), "=r"(w[j].w)
                 : "r"(p + static_cast<uint32_t>(j * 512 + lane * 16)));
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
  uint64_t *full = bars, *empty = bars + OR_MAX_STAGES, *accf = bars + 2 * OR_MAX_STAGES, *acce = accf + 2, *drain = acce + 2,
           *stored = drain + 1, *piece_in = stored + 4;
  uint32_t* holder = reinterpret_cast<uint32_t*>(bars + OR_BARS);
  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  const int worker = blockIdx.x / CG, nworkers = gridDim.x / CG;
  const int64_t units = static_cast<int64_t>(A.ph[0].units + A.ph[1].units + A.ph[2].units) * A.steps;
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
    for (int i = 0; i < 4; ++i) bar_init(smem_u32(&stored[i]), OR_EPI_WARPS);
    for (int i = 0; i < OR_EPI_WARPS; ++i) bar_init(smem_u32(&piece_in[i]), 1);
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
      const CUtensorMap* x = &A.lx[U.step & 1];
      const CUtensorMap* ma = U.mode == OR_GRAM ? x : U.mode == OR_POLY ? &A.la : TALL ? x : &A.lb;
      const CUtensorMap* mb = U.mode == OR_GRAM ? x : U.mode == OR_POLY ? &A.la : TALL ? &A.lb : x;
      const bool amn = TALL && U.mode == OR_GRAM, bmn = TALL ? U.mode == OR_GRAM : U.mode == OR_APPLY;
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
        const bool amn = TALL && U.mode == OR_GRAM, bmn = TALL ? U.mode == OR_GRAM : U.mode == OR_APPLY;
        const uint32_t idesc = f16_idesc(CG * 128, BN, DT_FP16, amn, bmn);
        const uint32_t la = amn ? 8192 : 16, lb = bmn ? 8192 : 16, ka = amn ? 2048 : 32, kb = bmn ? 2048 : 32;
        const int buf = n & 1;
        if (n >= 2 && !wait(&acce[buf], ((n >> 1) - 1) & 1)) break;
        tm_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(buf * BN);
        for (int i = 0; i < U.nkb; ++i) {
          const int s = R.slot;
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
      if (!wait_long(&stored[n & 3], (n >> 2) & 1)) break;
      if (lane == 0)
        asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(A.done + U.z * 3 + U.mode), "n"(OR_EPI_WARPS) : "memory");
      __syncwarp();
    }
  } else if (warp >= 4) {
    // ---------------- epilogue ----------------
    constexpr int NP = BN / 64;   // pieces of a warp
    const int w8 = warp - 4, ew = warp & 3, half = w8 >> 2;
    const uint32_t st = smem_u32(epi + w8 * 8192), st_in = st + 4096, in_bar = smem_u32(&piece_in[w8]);
    uint32_t n = 0, in_parity = 0;
    // A unit counts as done when its stores are: with the next unit's first piece, unless the
    // next unit is not there yet.
    int pending = -1;
    auto flush = [&](bool all) {
      if (pending < 0) return;
      __syncwarp();
      if (lane == 0) {
        if (all) tma_store_done<0>();
        else tma_store_done<1>();
        bar_arrive(smem_u32(&stored[pending]));
      }
      pending = -1;
    };
    for (int64_t g = worker; ok && g < units; g += nworkers, ++n) {
      const OrthoUnit U = or_unit<CG>(A, g);
      const OrthoPhase& P = A.ph[U.mode];
      const int buf = n & 1;
      const bool apply = U.mode == OR_APPLY, poly = U.mode == OR_POLY, final = apply && U.step + 1 == A.steps;
      const uint32_t tcol = tmem + (static_cast<uint32_t>(ew * 32) << 16) + static_cast<uint32_t>(buf * BN);
      const int row0 = U.m0 + static_cast<int>(rank) * 128 + ew * 32, row = row0 + lane;
      const bool in = row < P.M, rows_live = row0 < P.M;
      const float* diag = (apply ? A.e : A.d) + U.z * A.step_diag;
      const int64_t at = static_cast<int64_t>(row0 >> 5) * (apply ? A.cols_x : A.cols_a) + (U.n0 >> 5);
      unsigned short* own = apply ? A.own_x + U.z * A.step_own_x + at * 2048 : A.own_a + U.z * A.step_own_a + at * 1024;
      // pieces that this warp finishes: all of its own, or its split's share
      auto live = [&](int i) { return rows_live && U.n0 + 32 * half + 64 * i < P.N; };
      auto takes = [&](int i) { return live(i) && (U.ks == 1 || (w8 * NP + i) % U.ks == U.split); };
      // what a piece needs of its own elements is on its way before its accumulators are there
      auto fetch = [&](int i) {
        if (U.mode == OR_GRAM) return;
        while (i < NP && !takes(i)) ++i;
        __syncwarp();   // the piece before has been read
        if (i < NP && lane == 0) {
          const uint32_t bytes = apply ? 4096u : 2048u;
          bar_expect_tx(in_bar, bytes);
          bulk_load(st_in, own + ((32 * half + 64 * i) >> 5) * (apply ? 2048 : 1024), bytes, in_bar);
        }
      };
      if (!__all_sync(0xFFFFFFFFu, bar_over(smem_u32(&accf[buf]), (n >> 1) & 1))) flush(true);
      if (!wait_inputs(U)) break;
      fetch(0);
      const float d_row = (poly || (apply && !TALL)) && in ? diag[row] : 0.0f;
      float d_col[NP];
#pragma unroll
      for (int i = 0; i < NP; ++i) d_col[i] = (poly || (apply && TALL)) && live(i) ? diag[U.n0 + 32 * half + 64 * i + lane] : 0.0f;
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
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          uint32_t a[32];
          tm_ld32(tcol + 32 * half + 64 * i, a);
          tm_wait_ld();
          if (i == NP - 1) release();
          if (live(i))
#pragma unroll
            for (int j = 0; j < 32; j += 4) *reinterpret_cast<uint4*>(part + i * 2048 + j * 32) = make_uint4(a[j], a[j + 1], a[j + 2], a[j + 3]);
        }
        flush(true);
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
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int c = 32 * half + 64 * i, col0 = U.n0 + c;
        float r[32];
        if (U.ks == 1) {
          uint32_t a[32];
          tm_ld32(tcol + c, a);
          tm_wait_ld();
          if (i == NP - 1) release();
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = __uint_as_float(a[j]);
        }
        if (!takes(i)) continue;
        if (U.ks > 1) {
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = 0.0f;
          const float* p = part + i * 2048;
#pragma unroll 2
          for (int s = 0; s < U.ks; ++s, p += CG * or_part_floats(CG)) {
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 f = *reinterpret_cast<const float4*>(p + j * 32);
              r[j] += f.x, r[j + 1] += f.y, r[j + 2] += f.z, r[j + 3] += f.w;
            }
          }
        }
        float v[32];
        if (U.mode == OR_GRAM) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = r[j];
        } else {
          if (!bar_wait(in_bar, in_parity)) {
            gave_up();
            break;
          }
          in_parity ^= 1u;
          uint4 hi[4];
          or_load(st_in, hi, lane);
          if (poly) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float o = or_value(hi, j);
              v[j] = fmaf(A.kb, o, A.kc * fmaf(o, d_row + __shfl_sync(0xFFFFFFFFu, d_col[i], j), r[j]));
            }
          } else {
            uint4 lo[4];
            or_load(st_in + 2048, lo, lane);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float e = TALL ? __shfl_sync(0xFFFFFFFFu, d_col[i], j) : d_row;
              v[j] = fmaf(A.ka + e, or_value(hi, j), fmaf(A.ka, or_value(lo, j), A.inv_s2 * r[j]));
            }
          }
          fetch(i + 1);
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
        uint4 w[4];
        or_pack(v, final ? DT_BF16 : DT_FP16, w);
        unsigned short* piece = own + (c >> 5) * (apply ? 2048 : 1024);
        if (U.mode == OR_GRAM) or_save(piece, w, lane);
        if (lane == 0) tma_store_read();   // the piece before has left shared memory
        __syncwarp();
        or_stage(st, w, lane);
        if (U.mirror) or_stage_mirror(st + 2048, v, lane);
        if (apply && !final) {
          or_save(piece, w, lane);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] -= or_value(w, j);
          uint4 l[4];
          or_pack(v, DT_FP16, l);
          or_save(piece + 1024, l, lane);
        }
        if (final && A.last) {
          // rows that tensor copies cannot write: a lane a column
          __syncwarp();
          if (col0 + lane < P.N) {
            unsigned short* out = A.last + U.z * A.step_last + row0 * A.ld_last + col0 + lane;
            const int rows = min(32, P.M - row0);
#pragma unroll 8
            for (int k = 0; k < rows; ++k) {
              unsigned short x;
              asm volatile("ld.shared.b16 %0, [%1];" : "=h"(x) : "r"(or_at(st, k, lane >> 3) + static_cast<uint32_t>(lane & 7) * 2));
              out[k * A.ld_last] = x;
            }
          }
          __syncwarp();
          continue;
        }
        tma_store_fence();
        __syncwarp();
        if (lane == 0) {
          const CUtensorMap* to = final ? &A.out : apply ? &A.sx[(U.step + 1) & 1] : poly ? &A.sb : &A.sa;
          tma_store_3d(to, st, col0, row0, U.z);
          if (U.mirror) tma_store_3d(to, st + 2048, row0, col0, U.z);
          tma_store_commit();
        }
        flush(false);   // (the unit before)
      }
      if (!ok) break;
      flush(true);
      pending = static_cast<int>(n & 3);
    }
    flush(true);
    if (lane == 0) tma_store_done<0>();
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

struct OrthoStart {
  const void* g;
  int dt;                   // moe_dtype of g
  int64_t ldg, step_g;
  int M, N, ctas;           // CTAs a matrix
  float* part;              // [matrix][OR_NORM_CTAS][3]
  unsigned short* hi;       // X as the tensor copies read it
  int64_t ld_x, step_x;
  unsigned short* own;      // X as the epilogues do
  int64_t step_own;
  int own_cols;
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

// A warp's unit: 8 rows of 32 columns, a lane has 8 of them (row lane / 4).  f(row, column,
// values) for the units of this CTA in turn, four of them under way at a time.
template <typename F>
__device__ __forceinline__ void or_elements(const OrthoStart& A, int z, F&& f) {
  const int lane = threadIdx.x & 31, r = lane >> 2, c = (lane & 3) * 8;
  const int cols = (A.N + 31) / 32;
  const int n = (A.M + 7) / 8 * cols;   // (at most 4096 * 1024)
  const int step = static_cast<int>(gridDim.x) * 8;
  for (int u = static_cast<int>(blockIdx.x) * 8 + (threadIdx.x >> 5); u < n; u += 4 * step) {
    float v[4][8];
    int row[4], col[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = u + k * step, b = i / cols;
      row[k] = b * 8 + r;
      col[k] = (i - b * cols) * 32 + c;
      if (i >= n || row[k] >= A.M || col[k] >= A.N) row[k] = -1;
      if (row[k] >= 0) or_read(A, z * A.step_g + row[k] * A.ldg + col[k], A.N - col[k], v[k]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (row[k] >= 0) f(row[k], col[k], v[k]);
  }
}

// Squares summed in fp32 in three ranges (of 2^-40 and 2^40), each scaled into the
// middle: a square of any fp32 value neither overflows nor vanishes.
__global__ void __launch_bounds__(256) k_ortho_norm(const OrthoStart A) {
  __shared__ float sums[8][3];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int z = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float s[3] = {0.0f, 0.0f, 0.0f};
  or_elements(A, z, [&](int, int, const float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = fabsf(v[j]);
      if (x > 0x1p40f) {
        s[2] = fmaf(x * 0x1p-60f, x * 0x1p-60f, s[2]);
      } else if (x < 0x1p-40f) {
        s[0] = fmaf(x * 0x1p60f, x * 0x1p60f, s[0]);
      } else {
        s[1] = fmaf(x, x, s[1]);   // (NaN too)
      }
    }
  });
#pragma unroll
  for (int k = 0; k < 3; ++k) {
#pragma unroll
    for (int d = 16; d > 0; d /= 2) s[k] += __shfl_xor_sync(0xFFFFFFFFu, s[k], d);
    if (lane == 0) sums[warp][k] = s[k];
  }
  __syncthreads();
  if (threadIdx.x < 3) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += sums[w][threadIdx.x];
    A.part[(static_cast<int64_t>(z) * OR_NORM_CTAS + blockIdx.x) * 3 + threadIdx.x] = t;
  }
}

// X = hi + lo in fp16.  Every CTA adds the matrix's partial sums in order; the factor
// s / (|G| + eps) is applied as two, so that it has 64-bit numbers' range.
__global__ void __launch_bounds__(256) k_ortho_start(const OrthoStart A) {
  __shared__ float factor[2];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int z = blockIdx.y;
  if (threadIdx.x < 32) {
    double t[3] = {0.0, 0.0, 0.0};
    for (int i = threadIdx.x; i < A.ctas; i += 32)
#pragma unroll
      for (int k = 0; k < 3; ++k) t[k] += A.part[(static_cast<int64_t>(z) * OR_NORM_CTAS + i) * 3 + k];
    double sum = t[0] * 0x1p-120 + t[1] + t[2] * 0x1p120;
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
      l[j] = pack2(a - lo16(h[j], DT_FP16), b - hi16(h[j], DT_FP16), DT_FP16);
    }
    const uint4 hw = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(A.hi + z * A.step_x + row * A.ld_x + col) = hw;   // (rows are padded to 32 elements)
    unsigned short* p = A.own + z * A.step_own + (static_cast<int64_t>(row >> 5) * A.own_cols + (col >> 5)) * 2048 +
                        ((col >> 3) & 3) * 256 + (row & 31) * 8;
    *reinterpret_cast<uint4*>(p) = hw;
    *reinterpret_cast<uint4*>(p + 1024) = make_uint4(l[0], l[1], l[2], l[3]);
  });
}

}  // namespace moe_op
