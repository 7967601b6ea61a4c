// Tokens sorted by expert and back (moe_rows_* in include/moe_layer.h): the plan
// (a stable counting sort of the picks), rows taken in its order, rows summed back
// with weights, and the gradients of both.
//
// A pick i = t k + j is token t's j-th expert.  All of it is memory traffic: a token's
// row is read once and written k times, or k rows are read and one is written, with
// one multiply-add an element.  So a CTA has one token: its row's pieces of 32 lanes
// times VEC elements go to the warps in turn, and what a token's k rows have in
// common (places, weights) is read once a warp and passed by shuffles.
#pragma once

#include "moe_sm103.cuh"

namespace moe_op {

constexpr int RW_MAX_K = 16;
constexpr int RW_MAX_E = 1024;
constexpr int RW_PLAN_THREADS = 1024;
constexpr int RW_ROUNDS = 4;             // picks a thread of the plan
constexpr int RW_CHUNK = RW_PLAN_THREADS * RW_ROUNDS;   // picks a CTA

struct PlanArgs {
  const void* ids;
  int id64;              // ids of 64 bits
  int P, E;
  int chunks;
  int* totals;           // [chunks][E + 1] picks of every expert (several chunks only)
  int *offsets, *order, *place;
  int* status;
};

__host__ __device__ inline int rw_plan_smem(int E) { return 32 * (E + 1) * 2 + (E + 1) * 4 + 32 * 4 + 16; }

// What a CTA of the plan finds out about its picks first + 32 r: their bins (-1: past the
// last pick) and how many of their bins the warp had before them; counters in shared memory.
struct PlanPicks {
  int first;
  int bin[RW_ROUNDS], before[RW_ROUNDS];
};

// Exclusive sum over the bins: a thread has all of a bin's picks and those of the CTAs
// before this one; base[bin] becomes this CTA's first row of it.
__device__ __forceinline__ void rw_starts(const PlanArgs& A, bool write, char* smem, int all, int low) {
  int* base = reinterpret_cast<int*>(smem);
  int* sums = base + A.E + 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int incl = all;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int s = sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, s, d);
      if (lane >= d) s += v;
    }
    sums[lane] = s;
  }
  __syncthreads();
  const int start = incl - all + (warp ? sums[warp - 1] : 0);
  if (tid < A.E) {
    base[tid] = start + low;
    if (write) A.offsets[tid] = start;
  }
  if (tid == A.E - 1) {   // (E <= 1024 threads)
    base[A.E] += start + all;
    if (write) A.offsets[A.E] = start + all;
  }
  __syncthreads();
}

// Stable sort of the picks by expert, E + 1 bins (the last one: no expert).  A warp has
// 128 consecutive picks and counts them bin by bin, 32 at a time, in its own row of
// counters: lanes of equal bin find each other (match), so a pick knows how many of its
// bin came before it in the warp.  Sums over the warps before, the CTAs before and the
// bins below give its row.  COUNT: totals of every CTA alone, for picks of several CTAs.
// WRITE: this CTA writes offsets.
template <bool COUNT>
__device__ __forceinline__ void rw_plan(const PlanArgs& A, int chunk, bool write, char* smem, PlanPicks& K) {
  const int nb = A.E + 1;
  int* base = reinterpret_cast<int*>(smem);
  unsigned short* count = reinterpret_cast<unsigned short*>(base + nb + 32);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  K.first = chunk * RW_CHUNK + warp * 32 * RW_ROUNDS + lane;
  bool bad = false;
#pragma unroll
  for (int r = 0; r < RW_ROUNDS; ++r) {
    const int i = K.first + 32 * r;
    K.bin[r] = -1;
    if (i < A.P) {
      const long long e = A.id64 ? static_cast<const long long*>(A.ids)[i] : static_cast<const int*>(A.ids)[i];
      bad = bad || e < -1 || e >= A.E;
      K.bin[r] = e < 0 || e >= A.E ? A.E : static_cast<int>(e);
    }
  }
  if (bad && !COUNT) atomicOr(A.status, STATUS_INDEX);
  __syncthreads();   // the counters are zero
  unsigned short* mine = count + warp * nb;
#pragma unroll
  for (int r = 0; r < RW_ROUNDS; ++r) {
    K.before[r] = 0;
    if (chunk * RW_CHUNK + warp * 32 * RW_ROUNDS + 32 * r >= A.P) continue;   // (the whole warp)
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, K.bin[r]);
    const int rank = __popc(same & ((1u << lane) - 1u));
    const int old = K.bin[r] >= 0 ? mine[K.bin[r]] : 0;
    __syncwarp();
    if (K.bin[r] >= 0 && rank == 0) mine[K.bin[r]] = static_cast<unsigned short>(old + __popc(same));
    __syncwarp();
    K.before[r] = old + rank;
  }
  __syncthreads();
  const int warps = min(32, (A.P - chunk * RW_CHUNK + 32 * RW_ROUNDS - 1) / (32 * RW_ROUNDS));   // those with picks
  int all = 0, low = 0;
  for (int b = tid; b < nb; b += RW_PLAN_THREADS) {
    int run = 0;
#pragma unroll 8
    for (int w = 0; w < warps; ++w) {
      const int v = count[w * nb + b];
      count[w * nb + b] = static_cast<unsigned short>(run);
      run += v;
    }
    if (COUNT) {
      A.totals[static_cast<int64_t>(chunk) * nb + b] = run;
      continue;
    }
    int sum = run, ahead = 0;
    if (A.chunks > 1) {
      sum = 0;
#pragma unroll 8
      for (int c = 0; c < A.chunks; ++c) {
        const int v = A.totals[static_cast<int64_t>(c) * nb + b];
        sum += v;
        ahead += c < chunk ? v : 0;
      }
    }
    if (b < A.E) {
      all = sum;
      low = ahead;
    } else {
      base[b] = ahead;
    }
  }
  if constexpr (!COUNT) rw_starts(A, write, smem, all, low);
}

// The row of a pick (those without an expert: behind all others).
__device__ __forceinline__ int rw_row(const PlanPicks& K, int r, int nb, const char* smem) {
  const int* base = reinterpret_cast<const int*>(smem);
  const unsigned short* count = reinterpret_cast<const unsigned short*>(base + nb + 32);
  const int b = K.bin[r];
  return base[b] + count[(threadIdx.x >> 5) * nb + b] + K.before[r];
}

__device__ __forceinline__ void rw_clear_counts(char* smem, int nb) {
  uint32_t* count = reinterpret_cast<uint32_t*>(smem + nb * 4 + 32 * 4);
  for (int i = threadIdx.x; i < 16 * nb; i += RW_PLAN_THREADS) count[i] = 0;
}

template <bool COUNT>
__global__ void __launch_bounds__(RW_PLAN_THREADS) k_rows_plan(const PlanArgs A) {
  extern __shared__ __align__(16) char rw_smem[];
  rw_clear_counts(rw_smem, A.E + 1);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  PlanPicks K;
  rw_plan<COUNT>(A, blockIdx.x, !COUNT && blockIdx.x == 0, rw_smem, K);
  if constexpr (!COUNT) {
#pragma unroll
    for (int r = 0; r < RW_ROUNDS; ++r) {
      if (K.bin[r] < 0) continue;
      const int i = K.first + 32 * r, row = rw_row(K, r, A.E + 1, rw_smem);
      A.order[row] = K.bin[r] < A.E ? i : -1;
      A.place[i] = K.bin[r] < A.E ? row : -1;
    }
  }
}

// VEC 16-bit elements of a lane, as words (VEC 1: the low half).
template <int VEC>
struct RowPiece {
  uint32_t w[VEC > 1 ? VEC / 2 : 1];
};
template <int VEC>
__device__ __forceinline__ RowPiece<VEC> rw_load(const unsigned short* p) {
  RowPiece<VEC> v;
  if constexpr (VEC == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    v.w[0] = u.x, v.w[1] = u.y, v.w[2] = u.z, v.w[3] = u.w;
  } else if constexpr (VEC == 2) {
    v.w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    v.w[0] = *p;
  }
  return v;
}
template <int VEC>
__device__ __forceinline__ void rw_store(unsigned short* p, const RowPiece<VEC>& v) {
  if constexpr (VEC == 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
  } else if constexpr (VEC == 2) {
    *reinterpret_cast<uint32_t*>(p) = v.w[0];
  } else {
    *p = static_cast<unsigned short>(v.w[0]);
  }
}
template <int VEC>
__device__ __forceinline__ RowPiece<VEC> rw_zero() {
  RowPiece<VEC> v;
#pragma unroll
  for (uint32_t& w : v.w) w = 0;
  return v;
}
template <int VEC>
__device__ __forceinline__ void rw_float(const RowPiece<VEC>& v, int dt, float (&f)[VEC]) {
#pragma unroll
  for (int j = 0; j < VEC; ++j) f[j] = j & 1 ? hi16(v.w[j / 2], dt) : lo16(v.w[j / 2], dt);
}
template <int VEC>
__device__ __forceinline__ RowPiece<VEC> rw_pack(const float (&f)[VEC], int dt) {
  RowPiece<VEC> v;
  if constexpr (VEC == 1) {
    v.w[0] = pack1(f[0], dt);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; j += 2) v.w[j / 2] = pack2(f[j], f[j + 1], dt);
  }
  return v;
}

struct RowArgs {
  const unsigned short* tok;   // dispatch: x; gradient of the combine: d_out; [T, H]
  int64_t ld_tok;
  unsigned short* tok_out;     // combine: out [T, H]
  const unsigned short* row;   // combine and its gradient: y [P, H]
  int64_t ld_row;
  unsigned short* row_out;     // dispatch: the sorted rows; gradient of the combine: d_y
  int64_t ld_row_out;
  const void* w;               // [T, k] or null (ones)
  void* d_w;
  int w_dt;                    // moe_dtype of w and d_w
  const int *offsets, *place;
  int T, k, H, E, dt;
  int* status;
};

__device__ __forceinline__ float rw_weight(const void* w, int64_t i, int w_dt) {
  return w_dt == 2 ? static_cast<const float*>(w)[i] : ld16(w, i, w_dt);
}

// Lane j < k: the row of the token's pick j, or -1 (one past the rows is reported).
__device__ __forceinline__ int rw_place(const RowArgs& A, int t, int lane) {
  int r = -1;
  if (lane < A.k) {
    r = A.place[static_cast<int64_t>(t) * A.k + lane];
    if (r >= A.T * A.k) {
      atomicOr(A.status, STATUS_INDEX);
      r = -1;
    }
  }
  return r;
}

// Rows from offsets[E] on belong to no pick: zero, so that what is summed over all rows
// later (a weight gradient) needs to know no length.
template <int VEC>
__device__ __forceinline__ void rw_clear_tail(const RowArgs& A) {
  const int P = A.T * A.k;
  for (int64_t r = max(A.offsets[A.E], 0) + static_cast<int64_t>(blockIdx.x); r < P; r += gridDim.x)
    for (int c = threadIdx.x * VEC; c < A.H; c += blockDim.x * VEC) rw_store<VEC>(A.row_out + r * A.ld_row_out + c, rw_zero<VEC>());
}

// rows[place[t, j]] = x[t].
template <int VEC>
__global__ void __launch_bounds__(512) k_rows_take(const RowArgs A) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int t = blockIdx.x, lane = threadIdx.x & 31;
  const int place = rw_place(A, t, lane);
  for (int c = threadIdx.x * VEC; c - lane * VEC < A.H; c += blockDim.x * VEC) {
    const bool in = c < A.H;
    const RowPiece<VEC> v = in ? rw_load<VEC>(A.tok + t * A.ld_tok + c) : rw_zero<VEC>();
    for (int j = 0; j < A.k; ++j) {
      const int r = __shfl_sync(0xFFFFFFFFu, place, j);
      if (in && r >= 0) rw_store<VEC>(A.row_out + r * A.ld_row_out + c, v);
    }
  }
  rw_clear_tail<VEC>(A);
}

// The plan and the rows of up to RW_CHUNK picks in one launch: every CTA makes the plan
// for itself (some 3 us, as long as a second launch and its wait take), the first one
// writes it, and each takes some of the tokens' pieces.
template <int VEC>
__global__ void __launch_bounds__(RW_PLAN_THREADS) k_rows_small(const PlanArgs P, const RowArgs A) {
  extern __shared__ __align__(16) char rw_smem[];
  const int nb = P.E + 1;
  int* place = reinterpret_cast<int*>(rw_smem + (rw_plan_smem(P.E) + 15) / 16 * 16);
  rw_clear_counts(rw_smem, nb);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  PlanPicks K;
  rw_plan<false>(P, 0, blockIdx.x == 0, rw_smem, K);
  const int present = reinterpret_cast<const int*>(rw_smem)[P.E];
#pragma unroll
  for (int r = 0; r < RW_ROUNDS; ++r) {
    if (K.bin[r] < 0) continue;
    const int i = K.first + 32 * r, row = rw_row(K, r, nb, rw_smem);
    place[i] = K.bin[r] < P.E ? row : -1;
    if (blockIdx.x == 0) {
      P.order[row] = K.bin[r] < P.E ? i : -1;
      P.place[i] = K.bin[r] < P.E ? row : -1;
    }
  }
  __syncthreads();
  // a warp takes a piece of a token's row
  const int lane = threadIdx.x & 31, pieces = (A.H + 32 * VEC - 1) / (32 * VEC), warps = gridDim.x * (RW_PLAN_THREADS / 32);
  for (int u = blockIdx.x * (RW_PLAN_THREADS / 32) + (threadIdx.x >> 5); u < A.T * pieces; u += warps) {
    const int t = u / pieces, c = (u - t * pieces) * 32 * VEC + lane * VEC;
    if (c >= A.H) continue;
    const RowPiece<VEC> v = rw_load<VEC>(A.tok + t * A.ld_tok + c);
    for (int j = 0; j < A.k; ++j) {
      const int r = place[t * A.k + j];
      if (r >= 0) rw_store<VEC>(A.row_out + r * A.ld_row_out + c, v);
    }
  }
  for (int64_t r = present + blockIdx.x; r < P.P; r += gridDim.x)
    for (int c = threadIdx.x * VEC; c < A.H; c += RW_PLAN_THREADS * VEC) rw_store<VEC>(A.row_out + r * A.ld_row_out + c, rw_zero<VEC>());
}

// out[t] = sum over j, in order, of w[t, j] y[place[t, j]] in fp32, rounded once.  CTAs
// go through tokens; the rows of NB picks are under way at a time, and the next
// token's places and weights with them.
template <int VEC, int NB>
__global__ void __launch_bounds__(512) k_rows_combine(const RowArgs A) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int lane = threadIdx.x & 31;
  auto place_of = [&](int t) { return t < A.T ? rw_place(A, t, lane) : -1; };
  auto weight_of = [&](int t) {
    return t < A.T && lane < A.k && A.w ? rw_weight(A.w, static_cast<int64_t>(t) * A.k + lane, A.w_dt) : 1.0f;
  };
  int next_place = place_of(blockIdx.x);
  float next_weight = weight_of(blockIdx.x);
  for (int t = blockIdx.x; t < A.T; t += gridDim.x) {
    const int place = next_place;
    const float weight = place >= 0 ? next_weight : 0.0f;   // (a pick without an expert: 0 times 0)
    next_place = place_of(t + gridDim.x);
    next_weight = weight_of(t + gridDim.x);
    for (int c = threadIdx.x * VEC; c - lane * VEC < A.H; c += blockDim.x * VEC) {
      const bool in = c < A.H;
      float sum[VEC];
#pragma unroll
      for (float& s : sum) s = 0.0f;
      for (int j0 = 0; j0 < A.k; j0 += NB) {
        RowPiece<VEC> v[NB];
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const int r = __shfl_sync(0xFFFFFFFFu, place, j0 + j);   // (lanes from k on: -1)
          v[j] = in && r >= 0 ? rw_load<VEC>(A.row + r * A.ld_row + c) : rw_zero<VEC>();
        }
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const float f = __shfl_sync(0xFFFFFFFFu, weight, j0 + j);
          float y[VEC];
          rw_float<VEC>(v[j], A.dt, y);
#pragma unroll
          for (int i = 0; i < VEC; ++i) sum[i] = fmaf(f, y[i], sum[i]);
        }
      }
      if (in) rw_store<VEC>(A.tok_out + t * A.ld_tok + c, rw_pack<VEC>(sum, A.dt));
    }
  }
}

// d_y[place[t, j]] = w[t, j] d_out[t];  d_w[t, j] = <d_out[t], y[place[t, j]]>: a lane's
// part of all k sums stays in registers over the row; lanes and warps are added in a
// fixed order.  (W: d_w is wanted; Y: d_y is.)  CTAs go through tokens as above.
template <int VEC, bool Y, bool W>
__global__ void __launch_bounds__(512) k_rows_grad(const RowArgs A) {
  constexpr int NB = VEC == 8 ? 8 : 4;   // rows under way at a time
  __shared__ float part[2][16][RW_MAX_K];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto place_of = [&](int t) { return t < A.T ? rw_place(A, t, lane) : -1; };
  auto weight_of = [&](int t) {
    return Y && t < A.T && lane < A.k ? rw_weight(A.w, static_cast<int64_t>(t) * A.k + lane, A.w_dt) : 0.0f;
  };
  int next_place = place_of(blockIdx.x), turn = 0;
  float next_weight = weight_of(blockIdx.x);
  for (int t = blockIdx.x; t < A.T; t += gridDim.x, turn ^= 1) {
    const int place = next_place;
    const float weight = next_weight;
    next_place = place_of(t + gridDim.x);
    next_weight = weight_of(t + gridDim.x);
    float dot[RW_MAX_K];
#pragma unroll
    for (float& d : dot) d = 0.0f;
    for (int c = threadIdx.x * VEC; c - lane * VEC < A.H; c += blockDim.x * VEC) {
      const bool in = c < A.H;
      float e[VEC];
      rw_float<VEC>(in ? rw_load<VEC>(A.tok + t * A.ld_tok + c) : rw_zero<VEC>(), A.dt, e);
#pragma unroll
      for (int j0 = 0; j0 < RW_MAX_K; j0 += NB) {
        if (j0 >= A.k) break;
        RowPiece<VEC> v[NB];
        int r[NB];
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          r[j] = __shfl_sync(0xFFFFFFFFu, place, j0 + j);
          if (W && in && r[j] >= 0) v[j] = rw_load<VEC>(A.row + r[j] * A.ld_row + c);
        }
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const float f = Y ? __shfl_sync(0xFFFFFFFFu, weight, j0 + j) : 0.0f;
          if (!in || r[j] < 0) continue;
          if (Y) {
            float g[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) g[i] = f * e[i];
            rw_store<VEC>(A.row_out + r[j] * A.ld_row_out + c, rw_pack<VEC>(g, A.dt));
          }
          if (W) {
            float y[VEC];
            rw_float<VEC>(v[j], A.dt, y);
#pragma unroll
            for (int i = 0; i < VEC; ++i) dot[j0 + j] = fmaf(e[i], y[i], dot[j0 + j]);
          }
        }
      }
    }
    if constexpr (W) {
#pragma unroll
      for (int j = 0; j < RW_MAX_K; ++j) {
        if (j >= A.k) break;
        float d = dot[j];
#pragma unroll
        for (int s = 16; s > 0; s /= 2) d += __shfl_xor_sync(0xFFFFFFFFu, d, s);
        if (lane == 0) part[turn][warp][j] = d;
      }
      __syncthreads();   // (the other turn's sums have been read: their reader has come here since)
      if (warp == 0 && lane < A.k) {
        float d = 0.0f;
        for (int v = 0; v < static_cast<int>(blockDim.x) / 32; ++v) d += part[turn][v][lane];
        const int64_t i = static_cast<int64_t>(t) * A.k + lane;
        if (A.w_dt == 2) static_cast<float*>(A.d_w)[i] = d;
        else static_cast<unsigned short*>(A.d_w)[i] = pack1(d, A.w_dt);
      }
    }
  }
  if constexpr (Y) rw_clear_tail<VEC>(A);
}

}  // namespace moe_op
