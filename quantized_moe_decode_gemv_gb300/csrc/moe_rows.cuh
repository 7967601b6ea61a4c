// Tokens sorted by expert and back (moe_rows_* in include/moe_layer.h): the plan
// (a stable counting sort of the picks), rows taken in its order, rows summed back
// with weights, and the gradients of both.
//
// A pick i = t k + j is token t's j-th expert.  All of it is memory traffic: a token's
// row is read once and written k times, or k rows are read and one is written, with
// one multiply-add an element.  So a CTA has one token at a time: its row's pieces of 256
// columns go to the warps in turn, and what a token's k rows have in common (places,
// weights) is read once a warp and passed by shuffles.
#pragma once

#include "moe_sm103.cuh"

namespace moe_op {

constexpr int RW_MAX_K = 16;
constexpr int RW_MAX_E = 1024;
constexpr int RW_CHUNK = 1024;           // picks of a CTA of the plan, one a thread
// Up to so many chunks every CTA of the plan adds those before it by itself; more are added by a kernel of
// their own.  The kernels alone, by itself / with the kernel, us: 256 experts, 32 chunks 6.4 / 6.6, 64 8.1 / 7.0, 128
// 11.5 / 8.4; 1024 experts, 32 chunks 8.0 / 8.5, 64 10.8 / 8.9, 128 16.6 / 9.7.  But one launch more takes the
// host 2.5 us: calls one after the other, plan of 128 chunks 15.0 / 17.4, dispatch to rows of 64
// columns 96 chunks 23.2 / 24.8, 128 28.9 / 26.2, to rows of 1024 64 30.3 / 30.4, 128 57.0 / 54.6 (496 experts).
constexpr int RW_DIRECT_CHUNKS = 128;

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
// (Four picks a thread and a quarter of the CTAs took 12.4 us for 8192 x 9 picks, this 8.8;
// 10.7 and 6.4 for 4096 x 8.)
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

// Eight 16-bit elements of a lane, as four words.
struct RowPiece {
  uint32_t w[4];
};
__device__ __forceinline__ RowPiece rw_load(const unsigned short* p) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  return RowPiece{{u.x, u.y, u.z, u.w}};
}
__device__ __forceinline__ void rw_store(unsigned short* p, const RowPiece& v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
}
__device__ __forceinline__ RowPiece rw_zero() { return RowPiece{{0, 0, 0, 0}}; }
__device__ __forceinline__ void rw_float(const RowPiece& v, int dt, float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = j & 1 ? hi16(v.w[j / 2], dt) : lo16(v.w[j / 2], dt);
}
__device__ __forceinline__ RowPiece rw_pack(const float (&f)[8], int dt) {
  RowPiece v;
#pragma unroll
  for (int j = 0; j < 8; j += 2) v.w[j / 2] = pack2(f[j], f[j + 1], dt);
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

// ---------------------------------------------------------------------------
// rows of any address and width, 256 columns a warp at a time
// ---------------------------------------------------------------------------
//
// A lane has 8 consecutive elements of a piece as four words.  Where all rows are whole
// 16-byte words (ALIGNED) it loads and stores just those.  Else rows begin anywhere in a
// word of 16 bytes.  Rows that are summed (RowStream: the combine, d_w) are read as the 33 whole
// words that hold a piece, and a lane cuts its elements out of two of them; a token's row
// that goes to its k places (rw_get: dispatch, take, d_y) is read element by element, once.  Both are
// stored as whole words, made of two lanes' elements, with the ends of a piece element by
// element.  (An element a lane at a time, 8192 tokens of 9 rows of 1001 came back in 117 us
// and went out in 51; 48 and 35 this way, 31 and 25 at 1024, where the traffic alone takes 25.)

// Eight elements from word 0..4 on, `odd`: from its second half.
__host__ __device__ __forceinline__ RowPiece rw_cut(const uint32_t (&x)[5], bool odd) {
  RowPiece v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#ifdef __CUDA_ARCH__
    v.w[i] = odd ? __funnelshift_r(x[i], x[i + 1], 16) : x[i];
#else
    v.w[i] = odd ? x[i] >> 16 | x[i + 1] << 16 : x[i];
#endif
  }
  return v;
}

// How many elements into its 16-byte word a row begins.
__host__ __device__ __forceinline__ int rw_shift(const unsigned short* p) { return static_cast<int>((reinterpret_cast<uintptr_t>(p) >> 1) & 7); }

// The 16-byte word that a lane writes: the last `shift` elements of the lane before, then its own.
__host__ __device__ __forceinline__ RowPiece rw_join(const RowPiece& before, const RowPiece& own, int shift) {
  uint32_t x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = before.w[i];
    x[4 + i] = own.w[i];
  }
  // from element 8 - shift of these 16 on: whole words by halves, then the odd element
  const int from = 8 - shift;
#pragma unroll
  for (int d = 4; d > 0; d /= 2)
    if (from / 2 & d)
#pragma unroll
      for (int i = 0; i < 8 - d; ++i) x[i] = x[i + d];
  const uint32_t y[5] = {x[0], x[1], x[2], x[3], x[4]};   // (the fifth counts for odd shifts only)
  return rw_cut(y, from & 1);
}

// Columns c0 .. c1 - 1 of a piece, and how many of them lie before its first whole word and behind the last.
struct RowEnds {
  int c0, c1, head, tail;
};
__host__ __device__ __forceinline__ RowEnds rw_ends(int piece, int H, int shift) {
  RowEnds e;
  e.c0 = piece * 256;
  e.c1 = min(H, e.c0 + 256);
  e.head = shift ? min(8 - shift, e.c1 - e.c0) : 0;
  e.tail = min((e.c1 + shift) & 7, e.c1 - e.c0 - e.head);
  return e;
}
// Whether the word that begins `shift` elements before column c is the piece's own.
__host__ __device__ __forceinline__ bool rw_whole(const RowEnds& e, int c, int shift) { return c - shift >= e.c0 && c - shift + 8 <= e.c1; }
// The end element of a lane (lanes 0 to 7: the head, 8 to 15: the tail), counted from c0; whether it has one.
__host__ __device__ __forceinline__ bool rw_end(const RowEnds& e, int lane, int* at) {
  *at = lane < 8 ? lane : e.c1 - e.c0 - e.tail + lane - 8;
  return lane < 8 ? lane < e.head : lane < 8 + e.tail;
}

// Bytes of the row from the word on that begins `shift` elements before column c (0 and less: none); of them in
// that word, and what lane 31 takes from the word behind it.
__host__ __device__ __forceinline__ int rw_left(int c, int shift, int H) { return (H - (c - shift)) * 2; }
__host__ __device__ __forceinline__ int rw_own_bytes(int left) { return max(0, min(16, left)); }
__host__ __device__ __forceinline__ int rw_next_bytes(int left, int shift) { return max(0, min(2 * shift, left - 16)); }
// Where the five words that hold a lane's elements begin in a slot, in bytes.
__host__ __device__ __forceinline__ int rw_slot_at(int lane, int shift) { return (shift >> 1) * 4 + lane * 16; }

// A piece's elements to `row` (its first column: piece * 256; H columns in all) by the
// whole warp.
template <bool ALIGNED>
__device__ __forceinline__ void rw_put(unsigned short* row, int piece, int H, const RowPiece& v, int lane) {
  const int c = (piece * 32 + lane) * 8;
  if (ALIGNED) {
    if (c < H) rw_store(row + c, v);
    return;
  }
  const int shift = rw_shift(row);
  RowPiece before;
#pragma unroll
  for (int i = 0; i < 4; ++i) before.w[i] = __shfl_up_sync(0xFFFFFFFFu, v.w[i], 1);
  const RowPiece g = rw_join(before, v, shift);
  const RowEnds ends = rw_ends(piece, H, shift);
  if (rw_whole(ends, c, shift)) rw_store(row + c - shift, g);
  int e;
  const bool has = rw_end(ends, lane, &e);
  uint32_t t = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t w = __shfl_sync(0xFFFFFFFFu, v.w[q], e >> 3 & 31);
    if ((e >> 1 & 3) == q) t = w;
  }
  if (has) row[ends.c0 + e] = static_cast<unsigned short>(e & 1 ? t >> 16 : t);
}

// A lane's elements of a token's row, zeros past the last (rows that are not whole words: element by element).
template <bool ALIGNED>
__device__ __forceinline__ RowPiece rw_get(const unsigned short* row, int piece, int H, int lane) {
  const int c = (piece * 32 + lane) * 8;
  RowPiece v = rw_zero();
  if (ALIGNED) {
    if (c < H) v = rw_load(row + c);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < H) v.w[i / 2] |= static_cast<uint32_t>(row[c + i]) << (i & 1 ? 16 : 0);
  }
  return v;
}

// Rows from `first` on belong to no pick: zero, so that what is summed over all rows later (a
// weight gradient) needs to know no length.
template <bool ALIGNED>
__device__ __forceinline__ void rw_clear_tail(const RowArgs& A, int first) {
  const int P = A.T * A.k;
  for (int64_t r = max(first, 0) + static_cast<int64_t>(blockIdx.x); r < P; r += gridDim.x)
    for (int piece = threadIdx.x >> 5; piece * 256 < A.H; piece += blockDim.x >> 5)
      rw_put<ALIGNED>(A.row_out + r * A.ld_row_out, piece, A.H, rw_zero(), threadIdx.x & 31);
}

// rows[place[t, j]] = x[t]: one read, k writes.  4096 tokens to 8 rows of 6144 each: 72 us, 6.3
// TB/s.
template <bool ALIGNED>
__global__ void __launch_bounds__(512, 1) k_rows_take(const RowArgs A) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int t = blockIdx.x, lane = threadIdx.x & 31;
  const int place = rw_place(A, t, lane);
  for (int piece = threadIdx.x >> 5; piece * 256 < A.H; piece += blockDim.x >> 5) {
    const RowPiece v = rw_get<ALIGNED>(A.tok + t * A.ld_tok, piece, A.H, lane);
    for (int j = 0; j < A.k; ++j) {
      const int r = __shfl_sync(0xFFFFFFFFu, place, j);
      if (r >= 0) rw_put<ALIGNED>(A.row_out + r * A.ld_row_out, piece, A.H, v, lane);
    }
  }
  rw_clear_tail<ALIGNED>(A, A.offsets[A.E]);
}

// The plan and the rows of up to RW_CHUNK picks in one launch: every CTA makes the plan
// for itself, the first one writes it, and each takes some of the tokens' pieces.  One
// token 3.3 us and a launch's 2 us of the host less; as two launches 4.2.
template <bool ALIGNED>
__global__ void __launch_bounds__(RW_CHUNK, 1) k_rows_small(const PlanArgs P, const RowArgs A) {
  extern __shared__ __align__(16) char rw_smem[];
  const int nb = P.E + 1;
  int* place = reinterpret_cast<int*>(rw_smem + (rw_plan_smem(P.E) + 15) / 16 * 16);
  rw_clear_counts(rw_smem, nb);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  // a warp takes a piece of a token's row: the first one is under way while the plan is made
  const int lane = threadIdx.x & 31, pieces = (A.H + 255) / 256, warps = gridDim.x * (RW_CHUNK / 32);
  int u = blockIdx.x * (RW_CHUNK / 32) + (threadIdx.x >> 5);
  auto load = [&](int unit) {
    return unit < A.T * pieces ? rw_get<ALIGNED>(A.tok + unit / pieces * A.ld_tok, unit % pieces, A.H, lane) : rw_zero();
  };
  RowPiece v = load(u);
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
    const int t = u / pieces;
    const int mine = lane < A.k ? place[t * A.k + lane] : -1;
    for (int j = 0; j < A.k; ++j) {
      const int r = __shfl_sync(0xFFFFFFFFu, mine, j);
      if (r >= 0) rw_put<ALIGNED>(A.row_out + r * A.ld_row_out, u % pieces, A.H, v, lane);
    }
  }
  rw_clear_tail<ALIGNED>(A, present);
}

// The sums over rows have a ring in shared memory for each warp.  With rows in registers
// a warp has one batch of them under way, and the next only when that has come: 8192
// tokens of 9 rows of 1024 came at 2.9 TB/s with 20 warps an SM, 5.3 with the ring.  A slot
// is a piece of all k rows (and of the token's, for the gradient), filled by the lanes'
// asynchronous copies, zeros where a pick has no expert, slots - 1 pieces ahead.  A
// CTA goes through tokens, its warps through a row's pieces.

__device__ __forceinline__ void rw_copy_part(uint32_t dst, const void* src, int bytes) {   // of 16; the others zero
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__host__ __device__ constexpr int rw_slot_row(bool aligned) { return aligned ? 512 : 528; }   // bytes of a piece in a slot

template <bool ALIGNED>
struct RowStream {
  static constexpr int ROW = rw_slot_row(ALIGNED);
  const RowArgs& A;
  uint32_t smem;                    // this warp's ring
  int slots, rows;                  // pieces ahead + 1, rows of a slot
  int warps, warp, lane;
  int t, piece, slot = 0;           // next piece to be fetched
  int place, next_place;            // of token t and of the one after

  __device__ __forceinline__ RowStream(const RowArgs& a, char* base, int slots_, int rows_)
      : A(a), slots(slots_), rows(rows_), warps(blockDim.x >> 5), warp(threadIdx.x >> 5), lane(threadIdx.x & 31) {
    smem = smem_u32(base) + static_cast<uint32_t>(warp * slots * rows * ROW);
    t = blockIdx.x;
    piece = warp;
    place = place_of(t);
    next_place = place_of(t + gridDim.x);
  }
  __device__ __forceinline__ int place_of(int u) const { return u < A.T ? rw_place(A, u, lane) : -1; }
  __device__ __forceinline__ uint32_t at(int s, int row) const { return smem + static_cast<uint32_t>((s * rows + row) * ROW); }

  // The piece of one row into a slot (here: there is such a row).
  __device__ __forceinline__ void copy(uint32_t to, const unsigned short* row, bool here) {
    const int c = (piece * 32 + lane) * 8;
    if (ALIGNED) {
      const bool in = here && c < A.H;
      copy16(to + static_cast<uint32_t>(lane * 16), row + (in ? c : 0), in);
    } else {
      // whole words from the one that the piece begins in: what is read before the row's first element
      // shares its word, and nothing behind its last one is read
      const int shift = rw_shift(row);
      const unsigned short* word = row + c - shift;
      const int left = here ? rw_left(c, shift, A.H) : 0;
      const int own = rw_own_bytes(left);
      rw_copy_part(to + static_cast<uint32_t>(lane * 16), own ? word : row - shift, own);
      if (lane == 31) {
        const int next = rw_next_bytes(left, shift);
        rw_copy_part(to + 512, next ? word + 8 : row - shift, next);
      }
    }
  }
  // The next piece into the next slot: the k rows, and for TOK the token's own behind them.
  template <bool TOK>
  __device__ __forceinline__ void fetch() {
    if (!ALIGNED) __syncwarp();   // the slot has been read
    if (t < A.T) {
      for (int j = 0; j < A.k; ++j) {
        const int r = __shfl_sync(0xFFFFFFFFu, place, j);
        copy(at(slot, j), A.row + max(r, 0) * A.ld_row, r >= 0);
      }
      if (TOK) copy(at(slot, A.k), A.tok + t * A.ld_tok, true);
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
  // until the oldest piece has come
  __device__ __forceinline__ void wait() const {
    copies_wait(slots - 1);
    if (!ALIGNED) __syncwarp();
  }
  // This lane's elements of a slot's row, which begins at `row` in memory.
  __device__ __forceinline__ RowPiece read(int s, int j, const unsigned short* row) const {
    if (ALIGNED) {
      RowPiece v;
      asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3])
                   : "r"(at(s, j) + static_cast<uint32_t>(lane * 16))
                   : "memory");
      return v;
    }
    const int shift = rw_shift(row);
    const uint32_t p = at(s, j) + static_cast<uint32_t>(rw_slot_at(lane, shift));
    uint32_t x[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x[i]) : "r"(p + static_cast<uint32_t>(i * 4)) : "memory");
    return rw_cut(x, shift & 1);
  }
};

// out[t] = sum over j, in order, of w[t, j] y[place[t, j]] in fp32, rounded once.  4096
// tokens of 8 rows of 6144: 71 us, 6.4 TB/s.
template <bool ALIGNED>
__global__ void __launch_bounds__(512, 1) k_rows_combine(const RowArgs A, int slots) {
  extern __shared__ __align__(16) char rw_smem[];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  RowStream<ALIGNED> S(A, rw_smem, slots, A.k);
  for (int i = 0; i < slots - 1; ++i) S.template fetch<false>();
  const int lane = S.lane;
  auto weight_of = [&](int t) {
    return t < A.T && lane < A.k && A.w ? rw_weight(A.w, static_cast<int64_t>(t) * A.k + lane, A.w_dt) : 1.0f;
  };
  float next_weight = weight_of(blockIdx.x);
  int next_place = S.place_of(blockIdx.x), slot = 0;
  for (int t = blockIdx.x; t < A.T; t += gridDim.x) {
    const int place = next_place;
    const float weight = place >= 0 ? next_weight : 0.0f;   // (a pick without an expert: 0 times 0)
    next_weight = weight_of(t + gridDim.x);
    next_place = S.place_of(t + gridDim.x);
    for (int piece = S.warp; piece * 256 < A.H; piece += S.warps) {
      S.template fetch<false>();
      S.wait();
      float sum[8];
#pragma unroll
      for (float& s : sum) s = 0.0f;
#pragma unroll 4
      for (int j = 0; j < A.k; ++j) {
        const float f = __shfl_sync(0xFFFFFFFFu, weight, j);
        const int r = ALIGNED ? 0 : __shfl_sync(0xFFFFFFFFu, place, j);
        float y[8];
        rw_float(S.read(slot, j, A.row + max(r, 0) * A.ld_row), A.dt, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = fmaf(f, y[i], sum[i]);
      }
      slot = slot + 1 == slots ? 0 : slot + 1;
      rw_put<ALIGNED>(A.tok_out + t * A.ld_tok, piece, A.H, rw_pack(sum, A.dt), lane);
    }
  }
}

// d_y[place[t, j]] = w[t, j] d_out[t];  d_w[t, j] = <d_out[t], y[place[t, j]]>: a lane's
// part of all k sums stays in registers over the row; lanes and warps are added in a
// fixed order.  (Y: d_y is wanted.)
template <bool ALIGNED, bool Y>
__global__ void __launch_bounds__(512, 1) k_rows_grad(const RowArgs A, int slots) {
  extern __shared__ __align__(16) char rw_smem[];
  __shared__ float part[2][16][RW_MAX_K];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  RowStream<ALIGNED> S(A, rw_smem, slots, A.k + 1);
  for (int i = 0; i < slots - 1; ++i) S.template fetch<true>();
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
      S.template fetch<true>();
      S.wait();
      float e[8];
      rw_float(S.read(slot, A.k, A.tok + t * A.ld_tok), A.dt, e);
#pragma unroll
      for (int j = 0; j < RW_MAX_K; ++j) {
        if (j >= A.k) break;
        const int r = __shfl_sync(0xFFFFFFFFu, place, j);
        float y[8];
        rw_float(S.read(slot, j, A.row + max(r, 0) * A.ld_row), A.dt, y);
        if (Y) {
          const float f = __shfl_sync(0xFFFFFFFFu, weight, j);
          float g[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] = f * e[i];
          if (r >= 0) rw_put<ALIGNED>(A.row_out + r * A.ld_row_out, piece, A.H, rw_pack(g, A.dt), lane);
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
  if (Y) rw_clear_tail<ALIGNED>(A, A.offsets[A.E]);
}

// d_y alone: no row is read.
template <bool ALIGNED>
__global__ void __launch_bounds__(512, 1) k_rows_scale(const RowArgs A) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int t = blockIdx.x, lane = threadIdx.x & 31;
  const int place = rw_place(A, t, lane);
  const float weight = lane < A.k ? rw_weight(A.w, static_cast<int64_t>(t) * A.k + lane, A.w_dt) : 0.0f;
  for (int piece = threadIdx.x >> 5; piece * 256 < A.H; piece += blockDim.x >> 5) {
    float e[8];
    rw_float(rw_get<ALIGNED>(A.tok + t * A.ld_tok, piece, A.H, lane), A.dt, e);
    for (int j = 0; j < A.k; ++j) {
      const int r = __shfl_sync(0xFFFFFFFFu, place, j);
      const float f = __shfl_sync(0xFFFFFFFFu, weight, j);
      float g[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = f * e[i];
      if (r >= 0) rw_put<ALIGNED>(A.row_out + r * A.ld_row_out, piece, A.H, rw_pack(g, A.dt), lane);
    }
  }
  rw_clear_tail<ALIGNED>(A, A.offsets[A.E]);
}

}  // namespace moe_op
