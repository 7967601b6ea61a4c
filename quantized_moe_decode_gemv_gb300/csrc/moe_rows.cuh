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
constexpr int RW_CHUNK = 1024;           // picks of a CTA of the plan, one a thread
constexpr int RW_DIRECT_CHUNKS = 128;    // up to so many, every CTA adds the chunks before it by itself

struct PlanArgs {
  const void* ids;
  int id64;              // ids of 64 bits
  int P, E;
  int chunks;
  int* totals;           // [chunks + 1][E + 1]: picks of every bin in a chunk; after k_rows_scan before it, and in all
  int *offsets, *order, *place;
  int* status;
};

// Counters of a CTA: [E + 1] first rows, [32] sums of warps, [32][E + 1] 16-bit counts of warps.
__host__ __device__ inline int rw_plan_smem(int E) { return (E + 1) * 4 + 32 * 4 + 32 * (E + 1) * 2 + 16; }

// A pick's bin, and whether its id is neither -1 nor an expert.
__device__ __forceinline__ int rw_bin(const PlanArgs& A, int i, bool* bad) {
  const long long e = A.id64 ? static_cast<const long long*>(A.ids)[i] : static_cast<const int*>(A.ids)[i];
  *bad = e < -1 || e >= A.E;
  return e < 0 || e >= A.E ? A.E : static_cast<int>(e);
}

__device__ __forceinline__ void rw_clear_counts(char* smem, int nb) {
  uint32_t* count = reinterpret_cast<uint32_t*>(smem + nb * 4 + 32 * 4);
  for (int i = threadIdx.x; i < 16 * nb; i += RW_CHUNK) count[i] = 0;
}

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

// Stable sort of the picks by expert, E + 1 bins (the last one: no expert); a thread has
// pick i = chunk * 1024 + tid, and is told its bin and row (-1: no such pick).  Lanes of
// equal bin find each other (match), and a warp's counts of its bins go to its row of
// counters; sums over the lanes and warps before, the chunks before and the bins below
// give the row.  `write`: this CTA writes offsets.  Picks of several chunks have been
// counted by the kernels before; what comes ahead of the totals needs nothing of those
// and begins while they run (they have waited for whoever wrote the ids).
// (Four picks a thread and a quarter of the CTAs took 12.4 us for 8192 x 9 picks, this 11.6;
// 10.7 and 7.4 for 4096 x 8.)
__device__ __forceinline__ void rw_plan(const PlanArgs& A, int chunk, bool write, char* smem, int* bin, int* row) {
  const int nb = A.E + 1;
  int* base = reinterpret_cast<int*>(smem);
  unsigned short* count = reinterpret_cast<unsigned short*>(base + nb + 32);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, i = chunk * RW_CHUNK + tid;
  bool bad = false;
  *bin = i < A.P ? rw_bin(A, i, &bad) : -1;
  if (bad) atomicOr(A.status, STATUS_INDEX);
  const uint32_t same = __match_any_sync(0xFFFFFFFFu, *bin);
  const int rank = __popc(same & ((1u << lane) - 1u));
  __syncthreads();   // the counters are zero
  if (*bin >= 0 && rank == 0) count[warp * nb + *bin] = static_cast<unsigned short>(__popc(same));
  __syncthreads();
  if (A.chunks > 1) asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warps = min(32, (A.P - chunk * RW_CHUNK + 31) / 32);   // those with picks
  int all = 0, low = 0;
  for (int b = tid; b < nb; b += RW_CHUNK) {
    int sum = 0, ahead = 0;
#pragma unroll 8
    for (int w = 0; w < warps; ++w) {
      const int v = count[w * nb + b];
      count[w * nb + b] = static_cast<unsigned short>(sum);
      sum += v;
    }
    if (A.chunks > RW_DIRECT_CHUNKS) {
      ahead = A.totals[static_cast<int64_t>(chunk) * nb + b];
      sum = A.totals[static_cast<int64_t>(A.chunks) * nb + b];
    } else if (A.chunks > 1) {
      sum = 0;
#pragma unroll 8
      for (int c = 0; c < A.chunks; ++c) {
        const int v = A.totals[c * nb + b];
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
  rw_starts(A, write, smem, all, low);
  *row = *bin >= 0 ? base[*bin] + count[warp * nb + *bin] + rank : -1;
}

// totals[chunk]: how many picks of every bin a chunk has.
__global__ void __launch_bounds__(RW_CHUNK, 1) k_rows_count(const PlanArgs A) {
  __shared__ int count[RW_MAX_E + 1];
  const int nb = A.E + 1;
  for (int b = threadIdx.x; b < nb; b += RW_CHUNK) count[b] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  __syncthreads();
  const int i = blockIdx.x * RW_CHUNK + threadIdx.x;
  bool bad;
  if (i < A.P) atomicAdd(&count[rw_bin(A, i, &bad)], 1);
  __syncthreads();
  for (int b = threadIdx.x; b < nb; b += RW_CHUNK) A.totals[static_cast<int64_t>(blockIdx.x) * nb + b] = count[b];
}

// Many chunks: totals of the chunks before each, and of all, in their place.  A lane has a
// bin, a warp a 32nd of the chunks.
__global__ void __launch_bounds__(RW_CHUNK, 1) k_rows_scan(const PlanArgs A) {
  __shared__ int sums[32][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nb = A.E + 1, b = blockIdx.x * 32 + lane;
  const int per = (A.chunks + 31) / 32, c0 = min(warp * per, A.chunks), c1 = min(c0 + per, A.chunks);
  int* t = A.totals + b;
  int sum = 0;
  if (b < nb)
#pragma unroll 8
    for (int c = c0; c < c1; ++c) sum += t[static_cast<int64_t>(c) * nb];
  sums[warp][lane] = sum;
  __syncthreads();
  int run = 0;
  for (int w = 0; w < warp; ++w) run += sums[w][lane];
  if (b < nb) {
#pragma unroll 8
    for (int c = c0; c < c1; ++c) {
      const int v = t[static_cast<int64_t>(c) * nb];
      t[static_cast<int64_t>(c) * nb] = run;
      run += v;
    }
    if (warp == 31) t[static_cast<int64_t>(A.chunks) * nb] = run;
  }
}

__global__ void __launch_bounds__(RW_CHUNK, 1) k_rows_plan(const PlanArgs A) {
  extern __shared__ __align__(16) char rw_smem[];
  rw_clear_counts(rw_smem, A.E + 1);
  if (A.chunks == 1) asm volatile("griddepcontrol.wait;" ::: "memory");   // (else in rw_plan)
  int bin, row;
  rw_plan(A, blockIdx.x, blockIdx.x == 0, rw_smem, &bin, &row);
  asm volatile("griddepcontrol.launch_dependents;");
  if (bin < 0) return;
  const int i = blockIdx.x * RW_CHUNK + threadIdx.x;
  A.order[row] = bin < A.E ? i : -1;
  A.place[i] = bin < A.E ? row : -1;
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
// for itself, the first one writes it, and each takes some of the tokens' pieces.  One
// token 3.3 us and a launch's 2 us of the host less; as two launches 4.2.
template <int VEC>
__global__ void __launch_bounds__(RW_CHUNK, 1) k_rows_small(const PlanArgs P, const RowArgs A) {
  extern __shared__ __align__(16) char rw_smem[];
  const int nb = P.E + 1;
  int* place = reinterpret_cast<int*>(rw_smem + (rw_plan_smem(P.E) + 15) / 16 * 16);
  rw_clear_counts(rw_smem, nb);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  // a warp takes a piece of a token's row: the first one is under way while the plan is made
  const int lane = threadIdx.x & 31, pieces = (A.H + 32 * VEC - 1) / (32 * VEC), warps = gridDim.x * (RW_CHUNK / 32);
  int u = blockIdx.x * (RW_CHUNK / 32) + (threadIdx.x >> 5);
  auto column = [&](int unit) { return unit % pieces * 32 * VEC + lane * VEC; };
  auto load = [&](int unit) {
    const int c = column(unit);
    return unit < A.T * pieces && c < A.H ? rw_load<VEC>(A.tok + unit / pieces * A.ld_tok + c) : rw_zero<VEC>();
  };
  RowPiece<VEC> v = load(u);
  int bin, row;
  rw_plan(P, 0, blockIdx.x == 0, rw_smem, &bin, &row);
  const int present = reinterpret_cast<const int*>(rw_smem)[P.E];   // (the only CTA of the plan: no pick lies before it)
  if (bin >= 0) {
    place[threadIdx.x] = bin < P.E ? row : -1;
    if (blockIdx.x == 0) {
      P.order[row] = bin < P.E ? static_cast<int>(threadIdx.x) : -1;
      P.place[threadIdx.x] = bin < P.E ? row : -1;
    }
  }
  __syncthreads();
  for (; u < A.T * pieces; u += warps, v = load(u)) {
    const int t = u / pieces, c = column(u);
    const int mine = lane < A.k ? place[t * A.k + lane] : -1;
    for (int j = 0; j < A.k; ++j) {
      const int r = __shfl_sync(0xFFFFFFFFu, mine, j);
      if (r >= 0 && c < A.H) rw_store<VEC>(A.row_out + r * A.ld_row_out + c, v);
    }
  }
  for (int64_t r = present + blockIdx.x; r < P.P; r += gridDim.x)
    for (int c = threadIdx.x * VEC; c < A.H; c += RW_CHUNK * VEC) rw_store<VEC>(A.row_out + r * A.ld_row_out + c, rw_zero<VEC>());
}

// out[t] = sum over j, in order, of w[t, j] y[place[t, j]] in fp32, rounded once.  CTAs
// go through tokens; the rows of NB picks are under way at a time, and the next
// token's places and weights with them.
template <int VEC>
__global__ void __launch_bounds__(512) k_rows_combine(const RowArgs A) {
  constexpr int NB = 8;   // rows under way at a time
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

// ---------------------------------------------------------------------------
// the same for many tokens: rows by way of shared memory
// ---------------------------------------------------------------------------
//
// With rows in registers a warp has one batch of them under way, and the next only when
// that has come: 8192 tokens of 9 rows of 1024 came at 2.9 TB/s with 20 warps an SM. Here
// a warp has a ring of S slots of its own, each a piece (256 columns) of all k rows (and
// of the token's, for the gradient), filled by the lanes' asynchronous copies (zeros where a
// pick has no expert) S - 1 pieces ahead; every lane reads what it copied itself.
// A CTA goes through tokens, its warps through a row's pieces.

struct RowStream {
  const RowArgs& A;
  uint32_t smem;                    // this warp's ring
  int slots, rows;                  // pieces ahead + 1, rows of a slot
  int warps, warp, lane;
  int t, piece, slot = 0;           // next piece to be fetched
  int place, next_place;            // of token t and of the one after

  __device__ __forceinline__ RowStream(const RowArgs& a, char* base, int slots_, int rows_)
      : A(a), slots(slots_), rows(rows_), warps(blockDim.x >> 5), warp(threadIdx.x >> 5), lane(threadIdx.x & 31) {
    smem = smem_u32(base) + static_cast<uint32_t>(warp * slots * rows * 512);
    t = blockIdx.x;
    piece = warp;
    place = place_of(t);
    next_place = place_of(t + gridDim.x);
  }
  __device__ __forceinline__ int place_of(int u) const { return u < A.T ? rw_place(A, u, lane) : -1; }
  // Row `row` of a slot, this lane's 16 bytes.
  __device__ __forceinline__ uint32_t at(int s, int row) const { return smem + static_cast<uint32_t>((s * rows + row) * 512 + lane * 16); }
  // The next piece into the next slot: the k rows, and for TOK the token's own behind them.
  template <bool TOK>
  __device__ __forceinline__ void fetch() {
    if (t < A.T) {
      const int c = (piece * 32 + lane) * 8;
      const bool in = c < A.H;
      for (int j = 0; j < A.k; ++j) {
        const int r = __shfl_sync(0xFFFFFFFFu, place, j);
        copy16(at(slot, j), A.row + max(r, 0) * A.ld_row + (in ? c : 0), in && r >= 0);
      }
      if (TOK) copy16(at(slot, A.k), A.tok + t * A.ld_tok + (in ? c : 0), in);
      piece += warps;
      if (piece * 256 >= A.H) {
        piece = warp;
        t += gridDim.x;
        place = next_place;
        next_place = place_of(t + gridDim.x);
      }
    }
    copies_commit();
    slot = slot + 1 == slots ? 0 : slot + 1;
  }
};

__device__ __forceinline__ RowPiece<8> rw_shared(uint32_t p) {
  RowPiece<8> v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]) : "r"(p) : "memory");
  return v;
}

// As k_rows_combine.  Rows and widths of whole 16-byte words.
__global__ void __launch_bounds__(512) k_rows_combine_stream(const RowArgs A, int slots) {
  extern __shared__ __align__(16) char rw_smem[];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  RowStream S(A, rw_smem, slots, A.k);
  for (int i = 0; i < slots - 1; ++i) S.fetch<false>();
  const int lane = S.lane;
  auto weight_of = [&](int t) {
    return t < A.T && lane < A.k && A.w ? rw_weight(A.w, static_cast<int64_t>(t) * A.k + lane, A.w_dt) : 1.0f;
  };
  float next_weight = weight_of(blockIdx.x);
  int next_place = S.place_of(blockIdx.x), slot = 0;
  for (int t = blockIdx.x; t < A.T; t += gridDim.x) {
    const float weight = next_place >= 0 ? next_weight : 0.0f;   // (a pick without an expert: 0 times 0)
    next_weight = weight_of(t + gridDim.x);
    next_place = S.place_of(t + gridDim.x);
    for (int piece = S.warp; piece * 256 < A.H; piece += S.warps) {
      S.fetch<false>();
      copies_wait(slots - 1);
      float sum[8];
#pragma unroll
      for (float& s : sum) s = 0.0f;
#pragma unroll 4
      for (int j = 0; j < A.k; ++j) {
        const float f = __shfl_sync(0xFFFFFFFFu, weight, j);
        float y[8];
        rw_float<8>(rw_shared(S.at(slot, j)), A.dt, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = fmaf(f, y[i], sum[i]);
      }
      slot = slot + 1 == slots ? 0 : slot + 1;
      const int c = (piece * 32 + lane) * 8;
      if (c < A.H) rw_store<8>(A.tok_out + t * A.ld_tok + c, rw_pack<8>(sum, A.dt));
    }
  }
}

// As k_rows_grad with W.
template <bool Y>
__global__ void __launch_bounds__(512) k_rows_grad_stream(const RowArgs A, int slots) {
  extern __shared__ __align__(16) char rw_smem[];
  __shared__ float part[2][16][RW_MAX_K];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  RowStream S(A, rw_smem, slots, A.k + 1);
  for (int i = 0; i < slots - 1; ++i) S.fetch<true>();
  const int lane = S.lane;
  auto weight_of = [&](int t) {
    return Y && t < A.T && lane < A.k ? rw_weight(A.w, static_cast<int64_t>(t) * A.k + lane, A.w_dt) : 0.0f;
  };
  float next_weight = weight_of(blockIdx.x);
  int next_place = S.place_of(blockIdx.x), slot = 0, turn = 0;
  for (int t = blockIdx.x; t < A.T; t += gridDim.x, turn ^= 1) {
    const float weight = next_weight;
    const int place = next_place;
    next_weight = weight_of(t + gridDim.x);
    next_place = S.place_of(t + gridDim.x);
    float dot[RW_MAX_K];
#pragma unroll
    for (float& d : dot) d = 0.0f;
    for (int piece = S.warp; piece * 256 < A.H; piece += S.warps) {
      S.fetch<true>();
      copies_wait(slots - 1);
      const int c = (piece * 32 + lane) * 8;
      float e[8];
      rw_float<8>(rw_shared(S.at(slot, A.k)), A.dt, e);
#pragma unroll
      for (int j = 0; j < RW_MAX_K; ++j) {
        if (j >= A.k) break;
        float y[8];
        rw_float<8>(rw_shared(S.at(slot, j)), A.dt, y);
        const int r = __shfl_sync(0xFFFFFFFFu, place, j);
        if (Y) {
          const float f = __shfl_sync(0xFFFFFFFFu, weight, j);
          float g[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] = f * e[i];
          if (c < A.H && r >= 0) rw_store<8>(A.row_out + r * A.ld_row_out + c, rw_pack<8>(g, A.dt));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) dot[j] = fmaf(e[i], y[i], dot[j]);
      }
      slot = slot + 1 == slots ? 0 : slot + 1;
    }
#pragma unroll
    for (int j = 0; j < RW_MAX_K; ++j) {
      if (j >= A.k) break;
      float d = dot[j];
#pragma unroll
      for (int s = 16; s > 0; s /= 2) d += __shfl_xor_sync(0xFFFFFFFFu, d, s);
      if (lane == 0) part[turn][S.warp][j] = d;
    }
    __syncthreads();   // (the other turn's sums have been read: their reader has come here since)
    if (S.warp == 0 && lane < A.k) {
      float d = 0.0f;
      for (int v = 0; v < S.warps; ++v) d += part[turn][v][lane];
      if (place < 0) d = 0.0f;   // (an infinite d_out times no row's zeros)
      const int64_t i = static_cast<int64_t>(t) * A.k + lane;
      if (A.w_dt == 2) static_cast<float*>(A.d_w)[i] = d;
      else static_cast<unsigned short*>(A.d_w)[i] = pack1(d, A.w_dt);
    }
  }
  if constexpr (Y) rw_clear_tail<8>(A);
}

}  // namespace moe_op
