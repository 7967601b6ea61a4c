// 16-bit GEMM on tcgen05 with warp-specialised roles (k_gemm16): the products
// of the gated block's forward and backward pass.
//
//   D[m, n] = sum_k A[m, k] B[n, k]        fp32 accumulators in tensor memory
//
// A and B come by tensor copies from K-major memory (rows of consecutive k) or
// MN-major memory (rows of consecutive m or n), so that the three products of
// a training step read the tensors as they lie:
//
//   forward    x[T, K]      gate/up[N, K]      both K-major
//   d_x        dg|du[T, N]  gate|up[N, K]      A K-major, B MN-major, two K parts
//   d_weights  dg, du[T, N] x[T, K]            both MN-major, two batches
//
// A tile is CG * 128 rows by BN columns.  With CG = 2 a pair of CTAs shares
// it: each holds 128 rows of A and half of B's rows, one tcgen05.mma reads both
// CTAs' shared memory, and B's tile is read from L2 once for 256 rows instead
// of once per 128.  (At 256 x 256 a 64-wide K step moves 64 KB into the pair for
// 4.2 million multiply-adds: 64 bytes a clock and SM beside a saturated tensor
// pipe; with CG = 1, 96.)
// Measured on 4096 rows of 4096 against 2 x 8192, passes back to back: 280 to 288 us,
// 1.97 to 1.91 PFLOP/s; with the pre-activations saved 306 to 320 us.
//
// Roles of a CTA's 12 warps: warp 0 issues the tensor copies into a ring of
// shared-memory slots, warp 1 (of the pair's even CTA) issues the MMAs, warp 2
// owns the tensor-memory allocation, warps 4-11 read finished accumulators and
// write the epilogue (two warps a quarter of the lanes, taking turns at the
// columns: with one, a product of few K blocks and many outputs waited for its
// epilogues).  Accumulators are double-buffered (2 x BN <= 512
// columns), so an epilogue overlaps the next tile's MMAs.  CTAs (pairs) are
// persistent and walk the tiles in groups of 8 tile rows, whose operands stay
// in L2 while the columns pass.
//
// A slot of the ring holds one 64-wide K block, or two where a block's MMAs are
// short: a wait and a commit cost the issuing warp some 400 clocks.
//
// Every wait is bounded; a role whose wait runs out sets the timeout bit of
// the status word and winds down.
#pragma once

#include "moe_sm103.cuh"

namespace moe_op {

constexpr int GM_THREADS = 384;
constexpr int GM_EPI_WARPS = 8;
constexpr int GM_MAX_STAGES = 12;
constexpr int GM_EPI_BYTES = GM_EPI_WARPS * 32 * 80;   // epilogue staging: a warp's 32 rows x 64 (+16) bytes
constexpr int GM_SMEM_MAX = 227 * 1024;

struct GemmArgs {
  CUtensorMap ta[2], tb[2];
  int M, N;             // rows and columns of the output (dual: columns of the block's output)
  int BN;               // accumulator columns of a tile: 64, 128 or 256
  int dual;             // SwiGLU: columns [0, BN/2) from tb[0] (gate), [BN/2, BN) from tb[1] (up)
  int batches;          // batch z: ta[z], tb[0], out[z]
  int parts, kb[2];     // K parts (part p: ta[p], tb[p]) and their 64-wide K blocks
  int ksplit;           // K blocks divided over this many units; partial sums to `part`
  int stages, sub;      // slots of the ring and K blocks a slot
  int dt;               // 16-bit type of A, B and the output
  int act;
  void* out[2];
  int64_t ldo;
  int out_vec;          // out and ldo allow 16-byte (1) or 32-byte (2) stores
  float *save_gate, *save_up;   // pre-activations [M, N] fp32, or null
  float* part;          // [ksplit][batch][M][ld_part] fp32
  int64_t ld_part;      // columns of a partial row (dual: gate at 0, up at ld_part / 2)
  int* status;
};

__host__ __device__ inline int gm_stage_bytes(int BN, int CG) { return 128 * 128 + BN / CG * 128; }
__host__ __device__ inline int gm_smem_bytes(int BN, int CG, int stages, int sub) {
  return stages * sub * gm_stage_bytes(BN, CG) + GM_EPI_BYTES + 8 * (2 * GM_MAX_STAGES + 6) + 1024;
}

struct GemmUnit {
  int z, split, m0, n0, kb0, nkb;
};

// Unit u: batches, then K splits, then tiles; tiles in groups of 8 tile rows,
// rows fastest.
template <int CG>
__device__ __forceinline__ GemmUnit gm_unit(const GemmArgs& A, int u) {
  const int bn_out = A.dual ? A.BN / 2 : A.BN;
  const int tm = (A.M + CG * 128 - 1) / (CG * 128), tn = (A.N + bn_out - 1) / bn_out;
  const int tiles = tm * tn;
  GemmUnit U;
  int t = u % tiles;
  const int zs = u / tiles;
  U.split = zs % A.ksplit;
  U.z = zs / A.ksplit;
  const int g = t / (8 * tn);
  const int rows = min(8, tm - 8 * g);
  t -= g * 8 * tn;
  U.m0 = (8 * g + t % rows) * CG * 128;
  U.n0 = (t / rows) * bn_out;
  const int nkb = A.kb[0] + (A.parts > 1 ? A.kb[1] : 0);
  U.kb0 = static_cast<int>(static_cast<int64_t>(U.split) * nkb / A.ksplit);
  U.nkb = static_cast<int>(static_cast<int64_t>(U.split + 1) * nkb / A.ksplit) - U.kb0;
  return U;
}

// A warp's 32 rows x 32 columns of 16-bit values (lane = row) to global memory: a
// lane writes its row's 64 bytes as two whole sectors.  Rows that are not 32-byte
// aligned, or end inside the piece, go through the warp's staging rows instead,
// four lanes to 64 bytes of a row, or a lane to a column.
__device__ __forceinline__ void gm_store16(char* st, const float (&v)[32], int dt, unsigned short* out, int64_t ld,
                                           int row0, int col0, int M, int N, int vec, int lane) {
  if (vec == 2 && col0 + 32 <= N) {
    if (row0 + lane < M) {
      unsigned short* p = out + static_cast<int64_t>(row0 + lane) * ld + col0;
#pragma unroll
      for (int j = 0; j < 32; j += 16)
        stg32(p + j, pack2(v[j], v[j + 1], dt), pack2(v[j + 2], v[j + 3], dt), pack2(v[j + 4], v[j + 5], dt),
              pack2(v[j + 6], v[j + 7], dt), pack2(v[j + 8], v[j + 9], dt), pack2(v[j + 10], v[j + 11], dt),
              pack2(v[j + 12], v[j + 13], dt), pack2(v[j + 14], v[j + 15], dt));
    }
    return;
  }
  uint4* w = reinterpret_cast<uint4*>(st + lane * 80);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = make_uint4(pack2(v[8 * j], v[8 * j + 1], dt), pack2(v[8 * j + 2], v[8 * j + 3], dt),
                      pack2(v[8 * j + 4], v[8 * j + 5], dt), pack2(v[8 * j + 6], v[8 * j + 7], dt));
  __syncwarp();
  if (vec && col0 + 32 <= N) {
    unsigned short* p = out + static_cast<int64_t>(row0 + (lane >> 2)) * ld + col0 + (lane & 3) * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = (lane >> 2) + 8 * i;
      const uint4 x = *reinterpret_cast<const uint4*>(st + r * 80 + (lane & 3) * 16);
      if (row0 + r < M) *reinterpret_cast<uint4*>(p + static_cast<int64_t>(8 * i) * ld) = x;
    }
  } else if (col0 + lane < N) {
    // rows that 16-byte stores do not fit: a lane a column
    unsigned short* p = out + static_cast<int64_t>(row0) * ld + col0 + lane;
    const int rows = min(32, M - row0);
#pragma unroll 8
    for (int r = 0; r < rows; ++r)
      p[static_cast<int64_t>(r) * ld] = *reinterpret_cast<const unsigned short*>(st + r * 80 + lane * 2);
  }
  __syncwarp();
}

// The same for fp32 values, staged 16 columns at a time; `ld` and `out` keep
// 16-byte alignment (host-checked) and N is a multiple of 4.
__device__ __forceinline__ void gm_store32(char* st, const uint32_t (&v)[32], float* out, int64_t ld, int row0, int col0,
                                           int M, int N, int lane) {
  if (ld % 8 == 0 && (reinterpret_cast<uintptr_t>(out) & 31) == 0 && col0 + 32 <= N) {
    if (row0 + lane < M) {
      float* p = out + static_cast<int64_t>(row0 + lane) * ld + col0;
#pragma unroll
      for (int j = 0; j < 32; j += 8) stg32(p + j, v[j], v[j + 1], v[j + 2], v[j + 3], v[j + 4], v[j + 5], v[j + 6], v[j + 7]);
    }
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint4* w = reinterpret_cast<uint4*>(st + lane * 80);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = make_uint4(v[16 * h + 4 * j], v[16 * h + 4 * j + 1], v[16 * h + 4 * j + 2], v[16 * h + 4 * j + 3]);
    __syncwarp();
    const int c = col0 + 16 * h + (lane & 3) * 4;
    float* p = out + static_cast<int64_t>(row0 + (lane >> 2)) * ld + c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = (lane >> 2) + 8 * i;
      const uint4 x = *reinterpret_cast<const uint4*>(st + r * 80 + (lane & 3) * 16);
      if (row0 + r < M && c + 4 <= N) *reinterpret_cast<uint4*>(p + static_cast<int64_t>(8 * i) * ld) = x;
    }
    __syncwarp();
  }
}

template <int CG, bool AMN, bool BMN>
__global__ void __launch_bounds__(GM_THREADS, 1) k_gemm16(const __grid_constant__ GemmArgs A) {
  extern __shared__ __align__(1024) char gm_smem[];
  char* base = gm_smem + ((1024u - (smem_u32(gm_smem) & 1023u)) & 1023u);
  const int S = A.stages, BN = A.BN;
  const int b_rows = BN / CG;                       // B rows this CTA holds
  const int stage_bytes = gm_stage_bytes(BN, CG);
  const int slot_bytes = A.sub * stage_bytes;
  char* epi = base + S * slot_bytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(epi + GM_EPI_BYTES);
  uint64_t *full = bars, *empty = bars + GM_MAX_STAGES, *accf = bars + 2 * GM_MAX_STAGES, *acce = accf + 2,
           *drain = acce + 2;
  uint32_t* holder = reinterpret_cast<uint32_t*>(drain + 1);
  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  const int worker = blockIdx.x / CG, nworkers = gridDim.x / CG;

  const int bn_out = A.dual ? BN / 2 : BN;
  const int tm = (A.M + CG * 128 - 1) / (CG * 128), tn = (A.N + bn_out - 1) / bn_out;
  const int units = tm * tn * A.ksplit * A.batches;
  const uint32_t tm_cols = static_cast<uint32_t>(2 * BN);

  if (warp == 2) tm_alloc<CG>(smem_u32(holder), tm_cols);
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      bar_init(smem_u32(&full[s]), 1);
      bar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      bar_init(smem_u32(&accf[b]), 1);
      bar_init(smem_u32(&acce[b]), GM_EPI_WARPS * CG);
    }
    bar_init(smem_u32(drain), 1);
    bar_fence_init();
  }
  tm_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();
  tm_fence_after();
  const uint32_t tmem = *holder;
  // everything above may run while the kernel before this one in the stream ends
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  bool ok = true;
  auto wait = [&](uint64_t* b, uint32_t parity) {
    if (bar_wait(smem_u32(b), parity)) return true;
    atomicOr(A.status, STATUS_TIMEOUT);
    ok = false;
    return false;
  };

  if (warp == 0) {
    // ---------------- tensor copies ----------------
    RingPos R;
    bool again = false;   // slots have been used before
    uint32_t q = 0;
    for (int u = worker; ok && u < units; u += nworkers) {
      const GemmUnit U = gm_unit<CG>(A, u);
      const int am = U.m0 + static_cast<int>(rank) * 128, bn = U.n0 + (A.dual ? 0 : static_cast<int>(rank) * b_rows);
      for (int i = 0; i < U.nkb; i += A.sub, ++q) {
        const int s = R.slot, nk = min(A.sub, U.nkb - i);
        if (again && !wait(&empty[s], R.parity ^ 1u)) break;
        R.next(S);
        again = again || R.slot == 0;
        // both CTAs' copies complete on the even CTA's barrier
        const uint32_t own = smem_u32(&full[s]), fb = CG == 2 ? cluster_addr(own, 0) : own;
        if (elect_lane()) {
          if (rank == 0) bar_expect_tx(own, static_cast<uint32_t>(CG * stage_bytes * nk));
          for (int j = 0; j < nk; ++j) {
            int kb = U.kb0 + i + j, p = 0;
            if (A.parts > 1 && kb >= A.kb[0]) {
              kb -= A.kb[0];
              p = 1;
            }
            const uint32_t da = smem_u32(base + s * slot_bytes + j * stage_bytes), db = da + 128 * 128;
            const CUtensorMap* ma = &A.ta[A.batches > 1 ? U.z : p];
            if (AMN) {
              tma_2d<CG>(da, ma, am, kb * 64, fb);
              tma_2d<CG>(da + 8192, ma, am + 64, kb * 64, fb);
            } else {
              tma_2d<CG>(da, ma, kb * 64, am, fb);
            }
            if (A.dual) {
              if (CG == 2) {
                tma_2d<CG>(db, &A.tb[rank], kb * 64, bn, fb);
              } else {
                tma_2d<CG>(db, &A.tb[0], kb * 64, bn, fb);
                tma_2d<CG>(db + static_cast<uint32_t>(BN / 2 * 128), &A.tb[1], kb * 64, bn, fb);
              }
            } else if (BMN) {
              for (int r = 0; r < b_rows; r += 64)
                tma_2d<CG>(db + static_cast<uint32_t>(r * 128), &A.tb[p], bn + r, kb * 64, fb);
            } else {
              tma_2d<CG>(db, &A.tb[p], kb * 64, bn, fb);
            }
          }
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
      const uint32_t idesc = f16_idesc(CG * 128, BN, A.dt, AMN, BMN);
      RingPos R;
      uint32_t n = 0;
      for (int u = worker; ok && u < units; u += nworkers, ++n) {
        const GemmUnit U = gm_unit<CG>(A, u);
        const int buf = n & 1;
        if (n >= 2 && !wait(&acce[buf], ((n >> 1) - 1) & 1)) break;
        tm_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(buf * BN);
        for (int i = 0; i < U.nkb; i += A.sub) {
          const int s = R.slot, nk = min(A.sub, U.nkb - i);
          if (!wait(&full[s], R.parity)) break;
          R.next(S);
          tm_fence_after();
          if (elect_lane()) {
            for (int j = 0; j < nk; ++j) {
              const uint32_t sa = smem_u32(base + s * slot_bytes + j * stage_bytes), sb = sa + 128 * 128;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint64_t da = AMN ? sw128_desc(sa + k * 2048, 8192) : sw128_desc(sa + k * 32, 16);
                const uint64_t db = BMN ? sw128_desc(sb + k * 2048, 8192) : sw128_desc(sb + k * 32, 16);
                tm_mma<CG>(d, da, db, idesc, (i | j | k) != 0);
              }
            }
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
  } else if (warp >= 4) {
    // ---------------- epilogue ----------------
    const int ew = warp & 3, half = (warp - 4) >> 2;
    char* st = epi + (warp - 4) * 32 * 80;
    uint32_t n = 0;
    for (int u = worker; ok && u < units; u += nworkers, ++n) {
      const GemmUnit U = gm_unit<CG>(A, u);
      const int buf = n & 1;
      if (!wait(&accf[buf], (n >> 1) & 1)) break;
      tm_fence_after();
      const uint32_t tcol = tmem + (static_cast<uint32_t>(ew * 32) << 16) + static_cast<uint32_t>(buf * BN);
      const int row0 = U.m0 + static_cast<int>(rank) * 128 + ew * 32;
      const int c_last = bn_out >= 64 ? bn_out - 64 + 32 * half : 0;   // this warp's last columns
      if (bn_out < 64 && half == 1) {   // a single piece of columns: the other warp's
        if (lane == 0) {
          if (CG == 2) bar_arrive_cluster(smem_u32(&acce[buf]), 0);
          else bar_arrive(smem_u32(&acce[buf]));
        }
        continue;
      }
      for (int c = 32 * half; c < bn_out; c += 64) {
        uint32_t r0[32], r1[32];
        tm_ld32(tcol + c, r0);
        if (A.dual) tm_ld32(tcol + BN / 2 + c, r1);
        tm_wait_ld();
        if (c == c_last) {
          // the accumulators are in registers: the buffer may be rewritten
          tm_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (CG == 2) bar_arrive_cluster(smem_u32(&acce[buf]), 0);
            else bar_arrive(smem_u32(&acce[buf]));
          }
        }
        const int col0 = U.n0 + c;
        if (row0 >= A.M || col0 >= A.N) continue;
        float v[32];
        if (A.ksplit > 1) {
          float* p = A.part + static_cast<int64_t>(U.split * A.batches + U.z) * A.M * A.ld_part;
          const int nh = static_cast<int>(A.dual ? A.ld_part / 2 : A.ld_part);
          gm_store32(st, r0, p, A.ld_part, row0, col0, A.M, nh, lane);
          if (A.dual) gm_store32(st, r1, p + nh, A.ld_part, row0, col0, A.M, nh, lane);
          continue;
        }
        if (A.save_up) {
          if (A.dual) {
            gm_store32(st, r0, A.save_gate, A.N, row0, col0, A.M, A.N, lane);
            gm_store32(st, r1, A.save_up, A.N, row0, col0, A.M, A.N, lane);
          } else {
            gm_store32(st, r0, A.save_up, A.N, row0, col0, A.M, A.N, lane);
          }
        }
        // (each choice outside its loop: a warp is alone on its scheduler here, and 32
        // independent elements are what hides the latency of the arithmetic)
        if (A.dual) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = act_value(ACT_SWIGLU, __uint_as_float(r0[j]), __uint_as_float(r1[j]));
        } else if (A.act == ACT_RELU2) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = act_value(ACT_RELU2, 0.0f, __uint_as_float(r0[j]));
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r0[j]);
        }
        gm_store16(st, v, A.dt, static_cast<unsigned short*>(U.z ? A.out[1] : A.out[0]), A.ldo, row0, col0, A.M, A.N, A.out_vec,
                   lane);
      }
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

// Sums the K splits' partials in order and applies the epilogue (k_qgemm's too,
// with its per-column factors and bias): one thread per output row and four
// columns.
struct GemmFinishArgs {
  const float* part;
  int64_t ld_part;
  int ksplit, batches, M, N, dual, act, dt, out_vec;
  void* out[2];
  int64_t ldo;
  float *save_gate, *save_up;
  const float *nscale_gate, *nscale;
  const void* bias;
};

__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

__global__ void __launch_bounds__(128) k_gemm16_finish(const GemmFinishArgs A) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int q = (A.N + 3) / 4;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
  if (i >= static_cast<int64_t>(A.batches) * A.M * q) return;
  const int c = static_cast<int>(i % q) * 4;
  const int64_t zr = i / q;
  const int r = static_cast<int>(zr % A.M), z = static_cast<int>(zr / A.M);
  const int64_t half = A.dual ? A.ld_part / 2 : A.ld_part;
  const int64_t step = static_cast<int64_t>(A.batches) * A.M * A.ld_part;
  const float* p = A.part + (static_cast<int64_t>(z) * A.M + r) * A.ld_part + c;
  float4 s0 = make_float4(0, 0, 0, 0), s1 = s0;
#pragma unroll 4
  for (int s = 0; s < A.ksplit; ++s) {
    s0 = add4(s0, *reinterpret_cast<const float4*>(p + s * step));
    if (A.dual) s1 = add4(s1, *reinterpret_cast<const float4*>(p + s * step + half));
  }
  float g[4] = {s0.x, s0.y, s0.z, s0.w}, u[4] = {s1.x, s1.y, s1.z, s1.w};
  if (A.save_up) {   // (N is a multiple of 8 wherever pre-activations are saved)
    const int64_t o = static_cast<int64_t>(r) * A.N + c;
    if (A.dual) *reinterpret_cast<float4*>(A.save_gate + o) = s0;
    *reinterpret_cast<float4*>(A.save_up + o) = A.dual ? s1 : s0;
  }
  float y[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int cc = min(c + j, A.N - 1);
    if (A.nscale) {
      g[j] *= A.dual ? A.nscale_gate[cc] : A.nscale[cc];
      if (A.dual) u[j] *= A.nscale[cc];
    }
    y[j] = A.dual ? act_value(ACT_SWIGLU, g[j], u[j]) : act_value(A.act, 0.0f, g[j]);
    if (A.bias) y[j] += ld16(A.bias, cc, A.dt);
  }
  unsigned short* o = static_cast<unsigned short*>(z ? A.out[1] : A.out[0]) + static_cast<int64_t>(r) * A.ldo + c;
  if (A.out_vec && c + 4 <= A.N) {
    *reinterpret_cast<uint2*>(o) = make_uint2(pack2(y[0], y[1], A.dt), pack2(y[2], y[3], A.dt));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j < A.N) o[j] = pack1(y[j], A.dt);
  }
}

}  // namespace moe_op
