// 4-bit weights times many token rows on tcgen05 (k_qgemm): the 4-bit linear
// operators above the few rows that k_stream takes.
//
//   D[n, t] = sum_k W[n, k] x[t, k]      weights as M, tokens as N
//
// A CTA's tile is 128 weight rows (SwiGLU: two blocks, the gate's and the up
// matrix's rows of the same 128 outputs) by up to 256 tokens, with fp32
// accumulators in tensor memory.  (Two blocks of one matrix a CTA, which read the
// token rows once for both, were slower at every size: 41 us against 28 at 160
// rows, 206 against 188 at 2048, because two tiles' accumulators no longer fit.)  Tokens are N because N goes in steps of 16: a
// ragged batch pays for at most 15 rows that are not there, where as M it would
// pay for up to 127.  Weights are never written out: each 16-bit A tile is made
// from the codes in shared memory, once per token tile, beside the MMAs:
//
// A slot of the ring holds a 64-wide K block: the tile's A blocks and its token
// rows.  One barrier says that both are there and one that the MMAs are done with
// them -- a wait or a commit is some 250 clocks in the warp that issues the MMAs,
// and with barriers for each A block and for the token rows it could not keep the
// tensor pipe fed.
//
//   warp 0     tensor copies of the token rows
//   warps 8-23 decode, a 16-row tile of a block each: with two blocks eight warps a
//              block, with one two groups of eight that take turns at pairs of K
//              blocks.  Codes and scales come by 16-byte asynchronous copies
//              into a private ring, are decoded as k_stream does (an affine weight
//              is rounded once to the 16-bit type, a relative error of at most
//              2^-8 or 2^-11 beside the output's own, in fp16 more below 2^-14,
//              where its steps stay 2^-24; an fp4 weight times its block scale is
//              exact) and stored in the 128-byte swizzle
//   warp 1     issues the MMAs of a slot and commits them to its release
//   warp 2     owns the tensor memory
//   warps 4-7  the epilogue: a lane a weight row; four lanes exchange four tokens'
//              values so that each stores four consecutive outputs of one.  It
//              overlaps the next tile's MMAs where two tiles' accumulators fit
//              the 512 columns
//
// Per K block of two matrices and 256 tokens: 1024 clocks of MMA beside 32 KB of
// token rows, 9 KB of codes (41 bytes a clock) and 16 x 100 decode instructions
// (40% of the issue slots).  Measured, passes back to back in a graph: 2048 rows of
// 4096 against 16384, affine, 191 us (1.44 PFLOP/s; 203 in a run of seconds, where
// power bounds the clock), NVFP4 180 us; 300 rows against 2 x 8192, MXFP4, 39.5 us
// (1.02).  With few rows a K block takes what its decode takes: 0.30 us with one
// affine matrix, 0.26 NVFP4, 0.49 with an affine pair (32 rows of 8192 less 32 of 4096).
//
// Every wait is bounded; a role whose wait runs out sets the timeout bit of the
// status word and winds down.
#pragma once

#include <algorithm>

#include "moe_stream.cuh"

namespace moe_op {

constexpr int QG_THREADS = 768;
constexpr int QG_DEC_WARPS = 16;
constexpr int QG_MAX_SLOTS = 8;
constexpr int QG_SMEM_MAX = 227 * 1024;

struct QGemmArgs {
  CUtensorMap tx;           // token rows [T, K], boxes of 64 columns x ntok rows
  const uint4* codes;
  const void* scales;
  const float *nscale_gate, *nscale;
  const void* bias;
  void* out;
  int64_t ldo;
  int out_vec;              // out and ldo allow 8-byte stores
  float* part;              // [ksplit][T][ld_part] fp32 (ksplit > 1; SwiGLU: gate at 0, up at ld_part / 2)
  int64_t ld_part;
  int* status;
  int T, N, chunks, group, sdt, act;
  int ntok, ksplit;
  int slots, depth;         // of the ring, and stages of a warp's code ring (2 or 3)
};

__host__ __device__ inline int qg_region(int ntok) {   // accumulator columns of a block
  return ntok <= 32 ? 32 : ntok <= 64 ? 64 : ntok <= 128 ? 128 : 256;
}
// A stage of a warp's code ring: two chunks of its tile.
__host__ __device__ constexpr int qg_code_bytes(int fmt, int gb) { return 2 * (512 + st_scale_bytes(fmt, gb)); }
__host__ __device__ inline int qg_slot_bytes(int mt, int ntok) { return mt * 16384 + (ntok * 128 + 1023) / 1024 * 1024; }
__host__ __device__ inline int qg_smem_bytes(int fmt, int gb, int mt, int ntok, int slots, int depth) {
  return slots * qg_slot_bytes(mt, ntok) + QG_DEC_WARPS * depth * qg_code_bytes(fmt, gb) + 8 * (2 * QG_MAX_SLOTS + 8) + 1024;
}

struct QGemmUnit {
  int split, row, t0, c0, c1;   // 128-row block, first token, chunks [c0, c1)
};
__host__ __device__ __forceinline__ QGemmUnit qg_unit(const QGemmArgs& A, int row_tiles, int tok_tiles, int u) {
  QGemmUnit U;
  U.t0 = (u % tok_tiles) * A.ntok;
  u /= tok_tiles;
  U.row = u % row_tiles;
  U.split = u / row_tiles;
  // splits at even chunks (groups of 128 and code stages stay whole)
  const int ns = (A.chunks + 1) / 2;
  U.c0 = static_cast<int>(static_cast<int64_t>(U.split) * ns / A.ksplit) * 2;
  U.c1 = static_cast<int>(static_cast<int64_t>(U.split + 1) * ns / A.ksplit) * 2;
  if (U.c1 > A.chunks) U.c1 = A.chunks;
  return U;
}

// A decode warp's place in the ring.  Before it fills a block's slot it waits for
// the release of the block S before it, and a barrier tells only the parity of its
// releases: a slot one release further behind looks the same.  So the wait at block
// n is right only if the warp knows that block n - 2 S was released, that is, if
// its last wait (releases come in order) was at block n - S or later.
struct QGemmRing {
  int S = 0;            // slots
  RingPos R;
  bool again = false;   // slots have been used before
  int block = 0;        // blocks of this CTA so far
  __host__ __device__ __forceinline__ void skip(int n) {
    for (int i = 0; i < n; ++i) {
      R.next(S);
      again = again || R.slot == 0;
      ++block;
    }
  }
  // wait(block, slot, parity): until the slot of the next block is free
  template <typename W>
  __host__ __device__ __forceinline__ bool free_slot(W&& wait) const {
    return !again || wait(block, R.slot, R.parity ^ 1u);
  }
  // n blocks of the other group go by; their slots' releases are seen
  template <typename W>
  __host__ __device__ __forceinline__ bool pass(int n, W&& wait) {
    if (n < 1) return true;
    skip(n - 1);
    if (!free_slot(wait)) return false;
    skip(1);
    return true;
  }
};

// The K blocks [c0, c1) of a unit as a decode group takes them: pair(c) for blocks c
// and c + 1, all pairs of a gated product, every other one where two groups take
// turns.  Inside a unit three blocks lie between a group's waits (four where it
// waits at the later block of a pair, with S >= 4), which the ring's three or more
// slots allow (qg_plan).  Where units meet there may be more, so the blocks passed
// over there are waited for like the group's own.
template <bool GATED, typename P, typename W>
__host__ __device__ __forceinline__ bool qg_walk(QGemmRing& Q, int c0, int c1, int half, P&& pair, W&& wait) {
  constexpr int step = GATED ? 2 : 4;
  const int first = GATED ? 0 : 2 * half;
  if (!GATED && half && !Q.pass(first < c1 - c0 ? first : c1 - c0, wait)) return false;
  for (int c = c0 + first; c < c1; c += step) {
    if (!pair(c)) return false;
    if (!GATED) {
      const int end = c + step < c1 ? c + step : c1, n = end > c + 2 ? end - (c + 2) : 0;
      if (c + step < c1) Q.skip(n);
      else if (!Q.pass(n, wait)) return false;
    }
  }
  return true;
}

template <int FMT, bool FP16, bool GATED, int GB>
__global__ void __launch_bounds__(QG_THREADS, 1) k_qgemm(const __grid_constant__ QGemmArgs A) {
  constexpr int M = GATED ? 2 : 1;
  constexpr int DT = FP16 ? DT_FP16 : DT_BF16;
  constexpr int SCB = st_scale_bytes(FMT, GB);
  extern __shared__ __align__(1024) char gm_smem[];
  char* base = gm_smem + ((1024u - (smem_u32(gm_smem) & 1023u)) & 1023u);
  constexpr int mt = M;   // A blocks of a tile
  const int S = A.slots, D = A.depth, ntok = A.ntok;
  constexpr int code_bytes = qg_code_bytes(FMT, GB);
  const int slot_bytes = qg_slot_bytes(mt, ntok);
  char* rings = base + S * slot_bytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(rings + QG_DEC_WARPS * D * code_bytes);
  uint64_t *full = bars, *empty = full + QG_MAX_SLOTS, *accf = empty + QG_MAX_SLOTS, *acce = accf + 2, *drain = acce + 2;
  uint32_t* holder = reinterpret_cast<uint32_t*>(drain + 1);
  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;

  const int q = FMT == W_AFFINE && A.group == 128 ? 2 : 1, nu = A.chunks / q;   // chunks of a scale group
  const int row_tiles = (A.N + 127) / 128, tok_tiles = (A.T + ntok - 1) / ntok;
  const int units = row_tiles * tok_tiles * A.ksplit;
  const int region = qg_region(ntok), nbuf = 2 * mt * region <= 512 ? 2 : 1;
  const uint32_t tm_cols = static_cast<uint32_t>(nbuf * mt * region);

  if (warp == 2) tm_alloc<1>(smem_u32(holder), tm_cols);
  if (tid == 0) {
    tma_prefetch(&A.tx);
    for (int i = 0; i < S; ++i) {
      bar_init(smem_u32(&full[i]), 8 * mt + 1);   // eight decode warps a block, and the token rows' copy
      bar_init(smem_u32(&empty[i]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      bar_init(smem_u32(&accf[b]), 1);
      bar_init(smem_u32(&acce[b]), 4);
    }
    bar_init(smem_u32(drain), 1);
    bar_fence_init();
  }
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tmem = *holder;
  bool ok = true;
  auto wait = [&](uint32_t b, uint32_t parity) {
    if (bar_wait(b, parity)) return true;
    atomicOr(A.status, STATUS_TIMEOUT);
    ok = false;
    return false;
  };
  asm volatile("griddepcontrol.launch_dependents;");

  if (warp == 0) {
    // ---------------- token rows ----------------
    asm volatile("griddepcontrol.wait;" ::: "memory");
    RingPos R;
    bool again = false;   // slots have been used before
    uint32_t n = 0;
    for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
      const QGemmUnit U = qg_unit(A, row_tiles, tok_tiles, u);
      for (int c = U.c0; c < U.c1; ++c, ++n) {
        const int sl = R.slot;
        if (again && !wait(smem_u32(&empty[sl]), R.parity ^ 1u)) break;
        R.next(S);
        again = again || R.slot == 0;
        const uint32_t bar = smem_u32(&full[sl]);
        if (elect_lane()) {
          bar_expect_tx(bar, static_cast<uint32_t>(ntok * 128));
          tma_2d<1>(smem_u32(base + sl * slot_bytes + mt * 16384), &A.tx, c * 64, U.t0, bar);
        }
        __syncwarp();
      }
    }
    if (!ok) {   // copies already issued land before the CTA ends
      const uint32_t used = n < static_cast<uint32_t>(S) ? n : static_cast<uint32_t>(S);
      for (uint32_t j = n - used; j < n; ++j) bar_wait(smem_u32(&full[j % S]), (j / S) & 1);
    }
  } else if (warp == 1) {
    // ---------------- MMAs ----------------
    const uint32_t idesc = f16_idesc(128, ntok, DT, 0, 0);
    asm volatile("griddepcontrol.wait;" ::: "memory");   // no token rows come before: the waits are bounded
    RingPos R;
    uint32_t done = 0;
    for (int u = blockIdx.x; ok && u < units; u += gridDim.x, ++done) {
      const QGemmUnit U = qg_unit(A, row_tiles, tok_tiles, u);
      const uint32_t buf = nbuf == 2 ? done & 1 : 0, use = nbuf == 2 ? done >> 1 : done;
      if (use > 0 && !wait(smem_u32(&acce[buf]), (use - 1) & 1)) break;
      tm_fence_after();
      const uint32_t d = tmem + buf * static_cast<uint32_t>(mt * region);
      for (int c = U.c0; c < U.c1; ++c) {
        const int sl = R.slot;
        if (!wait(smem_u32(&full[sl]), R.parity)) break;
        R.next(S);
        tm_fence_after();
        const uint32_t sa = smem_u32(base + sl * slot_bytes), sx = sa + static_cast<uint32_t>(mt) * 16384;
        if (elect_lane()) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tm_mma<1>(d, sw128_desc(sa + k * 32, 16), sw128_desc(sx + k * 32, 16), idesc, (c > U.c0) | (k != 0));
          if (mt == 2) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tm_mma<1>(d + static_cast<uint32_t>(region), sw128_desc(sa + 16384 + k * 32, 16),
                        sw128_desc(sx + k * 32, 16), idesc, (c > U.c0) | (k != 0));
          }
          tm_commit<1>(smem_u32(&empty[sl]));
        }
        __syncwarp();
      }
      if (ok && elect_lane()) tm_commit<1>(smem_u32(&accf[buf]));
      __syncwarp();
    }
    // all MMAs end before the shared and tensor memory go
    if (elect_lane()) tm_commit<1>(smem_u32(drain));
    __syncwarp();
    bar_wait(smem_u32(drain), 0);
  } else if (warp >= 8) {
    // ---------------- decode ----------------
    const int dw = (warp - 8) & 7, half = (warp - 8) >> 3, g = lane >> 2, t = lane & 3;
    const int m = GATED ? half : 0;         // matrix, and its A block
    const int step = GATED ? 2 : 4;         // chunks from one of this warp's pairs to the next
    const int first = GATED ? 0 : 2 * half;
    const uint32_t ring = smem_u32(rings) + (warp - 8) * D * code_bytes;
    const int tiles16 = (A.N + 15) / 16;
    auto tile_of = [&](const QGemmUnit& U) { return U.row * 8 + dw; };
    // the next stage to fill: unit, chunks fc and fc + 1, their codes and scales, the slot
    int fu = static_cast<int>(blockIdx.x) - static_cast<int>(gridDim.x), fc = 0, fend = 0;
    bool fin = false;   // the unit's tile is inside the matrix
    const char *fsrc = nullptr, *fsc = nullptr;
    uint32_t fst = ring + lane * 16;
    const uint32_t ring_end = fst + D * code_bytes;
    // this lane's piece of the scales: chunk and bytes (a group of 128 has one set for both chunks)
    const int sk = lane / (SCB / 16);
    const int s_off = sk * (M - 1) * SCB + lane * 16;
    auto settle = [&] {   // to a unit that has a pair for this warp
      while (fu < units && fc >= fend) {
        fu += gridDim.x;
        if (fu >= units) break;
        const QGemmUnit FU = qg_unit(A, row_tiles, tok_tiles, fu);
        fc = FU.c0 + first;
        fend = FU.c1;
        const int64_t tile = tile_of(FU);
        fin = tile < tiles16;
        fsrc = reinterpret_cast<const char*>(A.codes + ((tile * A.chunks + fc) * M + m) * 32 + lane);
        fsc = static_cast<const char*>(A.scales) + ((tile * nu + fc / q) * M + m) * SCB + s_off;
      }
    };
    settle();
    auto fill_next = [&] {
      if (fu < units) {
        if (fin) {
          const bool two = fc + 1 < fend;
          copy16(fst, fsrc, true);
          if (two) copy16(fst + 512, fsrc + M * 512, true);
          if (sk < (two && q == 1 ? 2 : 1)) copy16(fst + 1024, fsc, true);
          fsrc += step * (M * 512);
          fsc += (q == 1 ? step : step / 2) * (M * SCB);
        }
        fc += step;
        if (fc >= fend) settle();
      }
      fst += code_bytes;
      if (fst == ring_end) fst = ring + lane * 16;
      copies_commit();
    };
    for (int i = 0; i < D - 1; ++i) fill_next();
    uint32_t cst = ring;
    QGemmRing Q;
    Q.S = S;
    // The first slots are filled while the kernel before this one in the stream
    // ends; a bounded wait begins after it, or its time would count.
    bool after = false;
    auto slot_free = [&](int, int sl, uint32_t parity) {
      if (!after) asm volatile("griddepcontrol.wait;" ::: "memory");
      after = true;
      return wait(smem_u32(&empty[sl]), parity);
    };
    // With four slots or more a pair of K blocks is taken at once: the slots are
    // released in order, so the later one's release is both's.
    const bool pairs = S >= 4;
    const uint32_t row_off = static_cast<uint32_t>((dw * 16 + g) * 128);
    for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
      const QGemmUnit U = qg_unit(A, row_tiles, tok_tiles, u);
      // rows past the matrix: their A rows stay what they were, their outputs are not written
      const bool in = tile_of(U) < tiles16;
      qg_walk<GATED>(Q, U.c0, U.c1, half, [&](int c) {
        __syncwarp();   // every lane has read the stage that is filled now
        fill_next();
        if (D == 3) copies_wait_n<2>();
        else copies_wait_n<1>();
        __syncwarp();   // every lane's copies have landed
        const uint32_t st = cst;
        cst += code_bytes;
        if (cst == ring + D * code_bytes) cst = ring;
        uint4 w[2];
        uint2 sv[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          w[i] = lds16(st + i * 512 + lane * 16);
          const uint32_t sst = st + 1024 + (q == 1 ? i * SCB : 0);
          if constexpr (FMT == W_AFFINE) {
            sv[i][0] = lds8(sst + g * 8);
            sv[i][1] = GB == 2 ? lds8(sst + 64 + g * 8) : sv[i][0];
          } else {
            sv[i][0].x = lds2(sst + (FMT == W_NVFP4 ? lane * 2 : g * 4 + (t & 2)));
          }
        }
        const bool two = c + 1 < U.c1;
        const int sl0 = Q.R.slot;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i == 1 && !two) break;
          if (pairs && i == 0 && two) Q.skip(1);
          const int sl = pairs && i == 0 ? sl0 : Q.R.slot;
          if (!(pairs && i == 1) && !Q.free_slot(slot_free)) break;
          if (in) {
            // (groups of 32: odd rows store their halves in the other order, so that eight lanes' stores touch all banks)
            if (!st_wide(FMT, GB) && (g & 1)) {
              w[i] = make_uint4(w[i].z, w[i].w, w[i].x, w[i].y);
              const uint2 x = sv[i][0];
              sv[i][0] = sv[i][1];
              sv[i][1] = x;
            }
            const uint32_t ws[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            const uint32_t row = smem_u32(base + sl * slot_bytes + m * 16384) + row_off;
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
              uint32_t v[2][4];
              if constexpr (FMT == W_AFFINE) {
                const uint2 x = sv[i][jj];
                if (A.sdt == DT) {
                  const uint32_t s0 = __byte_perm(x.x, 0, 0x1010), b0 = __byte_perm(x.x, 0, 0x3232);
                  const uint32_t s1 = __byte_perm(x.y, 0, 0x1010), b1 = __byte_perm(x.y, 0, 0x3232);
#pragma unroll
                  for (int j = 0; j < 2; ++j) {
                    affine_word<FP16>(ws[2 * jj + j], v[j]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) v[j][r] = affine16<FP16>(v[j][r], (r & 1) ? s1 : s0, (r & 1) ? b1 : b0);
                  }
                } else {
#pragma unroll
                  for (int j = 0; j < 2; ++j) {
                    affine_word<FP16>(ws[2 * jj + j], v[j]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                      const uint32_t y = (r & 1) ? x.y : x.x;
                      const float sc = lo16(y, A.sdt), bb = hi16(y, A.sdt), off = affine_offset<FP16>();
                      v[j][r] = pack2(fmaf(lo16(v[j][r], DT) - off, sc, bb), fmaf(hi16(v[j][r], DT) - off, sc, bb), DT);
                    }
                  }
                }
              } else {
                const uint32_t s0 = fp4_scale<FMT, FP16>(sv[i][0].x, 0), s1 = fp4_scale<FMT, FP16>(sv[i][0].x, 1);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  fp4_word<FP16>(ws[2 * jj + j], v[j]);
#pragma unroll
                  for (int r = 0; r < 4; ++r) v[j][r] = mul2<FP16>(v[j][r], (r & 1) ? s1 : s0);
                }
              }
              // eight consecutive columns of rows g and g + 8, in the 128-byte swizzle
              const int p = st_wide(FMT, GB) ? 2 * t + jj : 4 * (jj ^ (g & 1)) + t;
              sts16(row + ((p ^ g) * 16), v[0][0], v[0][2], v[1][0], v[1][2]);
              sts16(row + 1024 + ((p ^ g) * 16), v[0][1], v[0][3], v[1][1], v[1][3]);
            }
          }
          if (!pairs || i == 1 || !two) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
              if (pairs && i == 1) bar_arrive(smem_u32(&full[sl0]));
              bar_arrive(smem_u32(&full[sl]));
            }
            Q.skip(1);
          }
        }
        return ok;
      }, slot_free);
    }
    copies_wait(0);
  } else if (warp >= 4) {
    // ---------------- epilogue ----------------
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int ew = warp - 4;
    uint32_t done = 0;
    for (int u = blockIdx.x; ok && u < units; u += gridDim.x, ++done) {
      const QGemmUnit U = qg_unit(A, row_tiles, tok_tiles, u);
      const uint32_t buf = nbuf == 2 ? done & 1 : 0, use = nbuf == 2 ? done >> 1 : done;
      if (!wait(smem_u32(&accf[buf]), use & 1)) break;
      tm_fence_after();
      const uint32_t tcol = tmem + (static_cast<uint32_t>(ew * 32) << 16) + buf * static_cast<uint32_t>(mt * region);
      const int nt = min(ntok, A.T - U.t0);
      {
        const int row = U.row * 128 + ew * 32 + lane;
        const bool in = row < A.N;
        const int rc = min(row, A.N - 1);
        float f0 = 1.0f, f1 = 1.0f, bias = 0.0f;
        if constexpr (FMT != W_AFFINE) {
          f0 = __ldg((GATED ? A.nscale_gate : A.nscale) + rc);
          if (GATED) f1 = __ldg(A.nscale + rc);
        }
        if (A.bias) bias = ld16(A.bias, rc, DT);
        for (int j0 = 0; j0 < nt; j0 += 16) {
          uint32_t r0[16], r1[16];
          tm_ld16(tcol + j0, r0);
          if (GATED) tm_ld16(tcol + region + j0, r1);
          tm_wait_ld();
          if (j0 + 16 >= nt) {
            // the accumulators are in registers: the buffer may be rewritten
            tm_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(smem_u32(&acce[buf]));
          }
          if (A.ksplit > 1) {
            float* p = A.part + (static_cast<int64_t>(U.split) * A.T + U.t0 + j0) * A.ld_part + row;
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (in && j0 + j < nt) {
                p[static_cast<int64_t>(j) * A.ld_part] = __uint_as_float(r0[j]);
                if (GATED) p[static_cast<int64_t>(j) * A.ld_part + A.ld_part / 2] = __uint_as_float(r1[j]);
              }
            continue;
          }
          if (GATED) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              r0[j] = __float_as_uint(act_value(ACT_SWIGLU, __uint_as_float(r0[j]) * f0, __uint_as_float(r1[j]) * f1));
          } else if (A.act == ACT_RELU2) {
#pragma unroll
            for (int j = 0; j < 16; ++j) r0[j] = __float_as_uint(act_value(ACT_RELU2, 0.0f, __uint_as_float(r0[j]) * f0));
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) r0[j] = __float_as_uint(fmaf(__uint_as_float(r0[j]), f0, bias));
          }
          unsigned short* p = static_cast<unsigned short*>(A.out) + static_cast<int64_t>(U.t0 + j0) * A.ldo;
          if (A.out_vec && row - lane + 32 <= A.N) {
            // tokens j..j+3: after two exchanges lane l has token j + l % 4 of rows l / 4 * 4 on
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              uint32_t v0 = pack2(__uint_as_float(r0[j]), __uint_as_float(r0[j + 1]), DT);
              uint32_t v1 = pack2(__uint_as_float(r0[j + 2]), __uint_as_float(r0[j + 3]), DT);
              const uint32_t x0 = __shfl_xor_sync(0xFFFFFFFFu, v0, 1), x1 = __shfl_xor_sync(0xFFFFFFFFu, v1, 1);
              const uint32_t sel = lane & 1 ? 0x3276u : 0x5410u;
              v0 = __byte_perm(v0, x0, sel);
              v1 = __byte_perm(v1, x1, sel);
              const uint32_t y = __shfl_xor_sync(0xFFFFFFFFu, lane & 2 ? v0 : v1, 2);
              const uint2 w = lane & 2 ? make_uint2(y, v1) : make_uint2(v0, y);
              const int tk = j + (lane & 3);
              if (j0 + tk < nt)
                *reinterpret_cast<uint2*>(p + static_cast<int64_t>(tk) * A.ldo + (row - (lane & 3))) = w;
            }
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (in && j0 + j < nt) p[static_cast<int64_t>(j) * A.ldo + row] = pack1(__uint_as_float(r0[j]), DT);
          }
        }
      }
    }
  }
  tm_fence_before();
  __syncthreads();
  if (warp == 2) {
    tm_fence_after();
    tm_free<1>(tmem, tm_cols);
  }
}

// Host: token tile and K split of a call: the least estimated time in SM clocks.  A
// tile's 64-wide block takes the longest of its MMAs (2 ntok clocks a matrix), its
// decode (taken as 700 clocks for a pair, half of that for one matrix, whose two
// groups of warps take turns; measured: about 950 and 600) and its bytes at 40 a
// clock; a tile that does not overlap the next one adds its epilogue.
struct QGemmPlan {
  int ntok = 0, ksplit = 1, slots = 0, depth = 0, units = 0;
};
// Bytes of partial sums of a K split (rounded up from [ks][T][M] rows of (N + 3) / 4 * 4).
inline size_t qg_split_bytes(int M, int N, int T, int ks) {
  return static_cast<size_t>(ks) * T * (N + 3) / 4 * 4 * M * 4;
}
inline QGemmPlan qg_plan(int fmt, int gb, int M, int chunks, int T, int N, int sms, size_t part_bytes) {
  QGemmPlan best;
  double best_t = 1e30;
  const int rt = (N + 127) / 128;
  for (int tt = (T + 255) / 256, last = tt + 3; tt <= last; ++tt) {
    const int ntok = std::max(16, ((T + tt - 1) / tt + 15) / 16 * 16);
    if ((T + ntok - 1) / ntok < tt) continue;
    for (int ks = 1; ks <= 8; ++ks) {
      if (ks > 1) {
        if (chunks / ks < 8) break;
        if (qg_split_bytes(M, N, T, ks) > part_bytes) break;
      }
      const int units = rt * tt * ks;
      const double waves = (units + sms - 1) / sms;
      const double kb = std::max({2.0 * M * ntok, M == 2 ? 700.0 : 350.0,
                                  (ntok * 128.0 + 8.0 * M * (512 + st_scale_bytes(fmt, gb))) / 40.0});
      const bool two = 2 * M * qg_region(ntok) <= 512;
      const double epi = 6.0 * M * ntok;
      const double t = waves * (static_cast<double>(chunks) / ks * kb + (two ? 0.0 : epi)) + epi + 4000.0 +
                       (ks > 1 ? 7000.0 + 0.25 * ks * T * M * N / sms : 0.0);
      if (t < best_t) {
        best_t = t;
        best.ntok = ntok;
        best.ksplit = ks;
        best.units = units;
      }
    }
  }
  // shared memory: slots first, then a third code stage.  Two slots of a pair of
  // matrices and two stages fit at 256 tokens; with one matrix three do, which its
  // decode groups need (qg_walk).
  best.depth = 2;
  best.slots = 2;
  auto fits = [&](int n, int d) { return qg_smem_bytes(fmt, gb, M, best.ntok, n, d) <= QG_SMEM_MAX; };
  while (best.slots < 4 && fits(best.slots + 1, 2)) ++best.slots;
  if (fits(best.slots, 3)) best.depth = 3;
  while (best.slots < QG_MAX_SLOTS && fits(best.slots + 1, best.depth)) ++best.slots;
  return best;
}

// Host: bytes of partial sums that the plans of 1 to max_tokens rows use, of 64 MB
// that they may ask for.  (4096 x 4096, 4096 rows: 9 MB.)
inline size_t qg_part_bytes(int fmt, int gb, int M, int chunks, int max_tokens, int N, int sms) {
  constexpr size_t cap = 64ull << 20;
  size_t most = 0;
  for (int T = 1; T <= max_tokens && chunks >= 16 && qg_split_bytes(M, N, T, 2) <= cap; ++T) {
    const QGemmPlan P = qg_plan(fmt, gb, M, chunks, T, N, sms, cap);
    if (P.ksplit > 1) most = std::max(most, qg_split_bytes(M, N, T, P.ksplit));
  }
  return most;
}

}  // namespace moe_op
