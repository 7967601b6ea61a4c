// Tokens sorted by expert and back (moe_rows_* in include/moe_layer.h): host side
// and C ABI.
#include <cuda_runtime.h>

#include <algorithm>
#include <new>

#include "moe_op_host.h"
#include "moe_rows.cuh"

using namespace moe_op;

struct moe_rows : OpHandle {
  moe_rows_config cfg{};
  int* totals = nullptr;   // picks of every expert in every chunk of the plan
};

namespace {

thread_local std::string g_error;

constexpr int64_t kMaxPicks = 1 << 24;

moe_status validate(const moe_rows_config* c, std::string* why) {
  auto fail = [&](moe_status s, const char* msg) {
    *why = msg;
    return s;
  };
  if (!c) return fail(MOE_ERR_INVALID_ARG, "config is NULL");
  if (c->n_experts < 1 || c->max_tokens < 1) return fail(MOE_ERR_INVALID_ARG, "n_experts and max_tokens must be positive");
  if (c->act_dtype < 0 || c->act_dtype > 2) return fail(MOE_ERR_INVALID_ARG, "unknown dtype");
  if (c->top_k < 1 || c->top_k > c->n_experts) return fail(MOE_ERR_TOPK_GT_E, "top_k must be in 1..n_experts");
  if (c->n_experts > RW_MAX_E) return fail(MOE_ERR_UNSUPPORTED, "n_experts above 1024");
  if (c->top_k > RW_MAX_K) return fail(MOE_ERR_UNSUPPORTED, "top_k above 16");
  if (c->act_dtype == MOE_DTYPE_FP32) return fail(MOE_ERR_UNSUPPORTED, "fp32 activations");
  if (static_cast<int64_t>(c->max_tokens) * c->top_k > kMaxPicks)
    return fail(MOE_ERR_UNSUPPORTED, "max_tokens * top_k above 2^24");
  return MOE_OK;
}

// Rows of 16-bit elements: n of them, `cols` wide, ld apart.  (p NULL: none)
struct Rows {
  const void* p;
  int64_t ld, n, cols;
  int64_t bytes() const { return n > 0 ? ((n - 1) * ld + cols) * 2 : 0; }
};

struct Range {
  const void* p;
  int64_t bytes;
  Range(const void* q, int64_t n) : p(q), bytes(n) {}
  Range(const Rows& r) : p(r.p), bytes(r.bytes()) {}
};

bool overlap(const Range& a, const Range& b) {
  const char *x = static_cast<const char*>(a.p), *y = static_cast<const char*>(b.p);
  return x && y && x < y + b.bytes && y < x + a.bytes;
}

// Whether an output meets an input or another output.
bool clash(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
  for (const Range* o = outs.begin(); o != outs.end(); ++o) {
    for (const Range& i : ins)
      if (overlap(*o, i)) return true;
    for (const Range* p = outs.begin(); p != o; ++p)
      if (overlap(*o, *p)) return true;
  }
  return false;
}

// Whether rows meet rows in memory.  Column ranges of one buffer may interleave; a single row
// has no stride of its own.
bool meet(const Rows& a, const Rows& b) {
  if (!overlap(a, b)) return false;
  const int64_t lda = a.n > 1 ? a.ld : b.ld, ldb = b.n > 1 ? b.ld : a.ld;
  return lda != ldb || rows_overlap(a.p, lda, a.cols, b.p, ldb, b.cols, std::max(a.n, b.n));
}

// Whether all rows are whole 16-byte words.
bool whole_words(std::initializer_list<Rows> all) {
  int64_t bits = all.begin()->cols * 2;
  for (const Rows& r : all)
    if (r.p) bits |= static_cast<int64_t>(reinterpret_cast<uintptr_t>(r.p)) | (r.n > 1 ? r.ld * 2 : 0);
  return bits % 16 == 0;
}

// A CTA's warps: one for each 256 columns, up to 8; up to 16 where tokens alone do not fill the SMs.  8 / 16
// warps, 8 rows of 6144, us: 152 tokens, out 3.8 / 3.5, back 4.8 / 4.0, d_y 4.4 / 3.9; 228, 5.1 / 5.0, 5.5 / 6.9, 5.5 /
// 5.4; 303, 5.4 / 5.3, 7.2 / 7.8, 5.8 / 7.0; 330, 6.9 / 8.4, 7.4 / 9.8, 7.2 / 7.0.  Rows of 2560: 16 up to a third faster
// until 303 (back 4.5 / 3.4), slower at 330 (4.5 / 4.8).
int row_warps(int T, int H, int sms) { return std::min((H + 255) / 256, T < 2 * sms ? 16 : 8); }

int small_smem(int E, int P) { return (rw_plan_smem(E) + 15) / 16 * 16 + 4 * P; }
using RowKernel = void (*)(const RowArgs);
using StreamKernel = void (*)(const RowArgs, int);

// A CTA's warps and slots of `rows` rows.  One piece under way a warp and many warps beat
// several and few: on 8192 tokens of 9 rows of 1024, 2 slots (20 warps an SM) 31.5 us, 3 (12
// warps) 41; few rows take more slots, 2 KB under way a warp.
constexpr int kStreamSmem = 8 * 2 * (RW_MAX_K + 1) * rw_slot_row(false);   // the most it may be
struct StreamShape {
  int threads, slots, smem, ctas;
};
StreamShape stream_shape(int T, int H, int rows, bool aligned, int sms) {
  StreamShape s;
  s.slots = std::max(2, 2048 / (rows * 512) + 1);   // (at most 5)
  const int slot = rows * rw_slot_row(aligned);
  int warps = row_warps(T, H, sms);
  if (warps * s.slots * slot > kStreamSmem) warps = 8;
  s.threads = 32 * warps;
  s.smem = warps * s.slots * slot;
  const int fit = std::max(1, std::min({2048 / s.threads, 220 * 1024 / (s.smem + 2048), 32}));
  s.ctas = std::min(T, sms * fit);
  return s;
}

bool misaligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

moe_status fail(moe_rows* h, moe_status st, const char* msg) {
  h->last_error = msg;
  return st;
}

moe_status launched(moe_rows* h, cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  h->last_error = std::string("launch: ") + cudaGetErrorString(e);
  return MOE_ERR_CUDA;
}

// What every call checks of its sizes; MOE_OK with nothing to do when T is 0.
moe_status check_sizes(moe_rows* h, int32_t T, int32_t width) {
  if (T < 0 || T > h->cfg.max_tokens) return fail(h, MOE_ERR_INVALID_ARG, "T must be in 0..max_tokens");
  if (width < 1 || width > 65536) return fail(h, MOE_ERR_INVALID_ARG, "width must be in 1..65536");
  return MOE_OK;
}

moe_status check_rows(moe_rows* h, const Rows& r, const char* what) {
  if (!r.p || misaligned(r.p, 2) || (r.n > 1 && r.ld < r.cols)) {
    h->last_error = std::string(what) + " must not be NULL, and its rows must be at least width elements apart";
    return MOE_ERR_INVALID_ARG;
  }
  return MOE_OK;
}

moe_status check_ids(moe_rows* h, const void* ids, int32_t id_bytes, const int32_t* offsets, const int32_t* order,
                     const int32_t* place, int32_t T) {
  if (id_bytes != 4 && id_bytes != 8) return fail(h, MOE_ERR_INVALID_ARG, "ids have 4 or 8 bytes");
  if (!offsets || misaligned(offsets, 4) || misaligned(order, 4) || misaligned(place, 4) ||
      misaligned(ids, static_cast<uintptr_t>(id_bytes)) || (T > 0 && (!ids || !order || !place)))
    return fail(h, MOE_ERR_INVALID_ARG, "ids, offsets, order and place must be aligned and not NULL");
  return MOE_OK;
}

PlanArgs plan_args(moe_rows* h, const void* ids, int32_t id_bytes, int32_t T, int32_t* offsets, int32_t* order, int32_t* place) {
  PlanArgs a{};
  a.ids = ids;
  a.id64 = id_bytes == 8;
  a.P = T * h->cfg.top_k;
  a.E = h->cfg.n_experts;
  a.chunks = (a.P + RW_CHUNK - 1) / RW_CHUNK;
  a.totals = h->totals;
  a.offsets = offsets;
  a.order = order;
  a.place = place;
  a.status = h->status;
  return a;
}

cudaError_t launch_plan(moe_rows* h, const PlanArgs& a, cudaStream_t s) {
  if (a.P == 0) return cudaMemsetAsync(a.offsets, 0, static_cast<size_t>(a.E + 1) * 4, s);
  const size_t smem = static_cast<size_t>(rw_plan_smem(a.E));
  cudaError_t e = cudaSuccess;
  if (a.chunks > 1) {
    e = launch_chained(k_rows_count, a.chunks, RW_CHUNK, 0, 1, s, a);
    ++h->last_launches;
    if (e == cudaSuccess && a.chunks > RW_DIRECT_CHUNKS) {
      e = launch_chained(k_rows_scan, (a.E + 32) / 32, RW_CHUNK, 0, 1, s, a);
      ++h->last_launches;
    }
  }
  if (e == cudaSuccess) {
    e = launch_chained(k_rows_plan, a.chunks, RW_CHUNK, smem, 1, s, a);
    ++h->last_launches;
  }
  return e;
}

RowArgs row_args(moe_rows* h, int32_t T, int32_t width, const int32_t* offsets, const int32_t* place) {
  RowArgs a{};
  a.offsets = offsets;
  a.place = place;
  a.T = T;
  a.k = h->cfg.top_k;
  a.H = width;
  a.E = h->cfg.n_experts;
  a.dt = h->cfg.act_dtype;
  a.status = h->status;
  return a;
}

moe_status plan(moe_rows* h, const void* ids, int32_t id_bytes, int32_t T, int32_t* offsets, int32_t* order, int32_t* place,
                void* stream) {
  if (!h) return MOE_ERR_INVALID_ARG;
  moe_status st = check_sizes(h, T, 1);
  if (st == MOE_OK) st = check_ids(h, ids, id_bytes, offsets, order, place, T);
  if (st != MOE_OK) return st;
  const int64_t P = static_cast<int64_t>(T) * h->cfg.top_k;
  if (clash({{offsets, 4ll * (h->cfg.n_experts + 1)}, {order, 4 * P}, {place, 4 * P}}, {{ids, id_bytes * P}}))
    return fail(h, MOE_ERR_INVALID_ARG, "the plan overlaps the ids or itself");
  DeviceScope dev(h->device);
  if (!dev.ok) return fail(h, MOE_ERR_DEVICE, "the handle's device cannot be made current");
  h->last_launches = 0;
  return launched(h, launch_plan(h, plan_args(h, ids, id_bytes, T, offsets, order, place), static_cast<cudaStream_t>(stream)));
}

// The rows alone (ids NULL), or the plan and the rows.
moe_status take(moe_rows* h, bool with_plan, const void* x, int64_t ldx, int32_t T, int32_t width, const void* ids,
                int32_t id_bytes, int32_t* offsets, int32_t* order, int32_t* place, void* rows, int64_t ld_rows,
                void* stream) {
  if (!h) return MOE_ERR_INVALID_ARG;
  moe_status st = check_sizes(h, T, width);
  if (st == MOE_OK && with_plan) st = check_ids(h, ids, id_bytes, offsets, order, place, T);
  if (st != MOE_OK) return st;
  h->last_launches = 0;
  if (T == 0 && !with_plan) return MOE_OK;
  const int64_t P = static_cast<int64_t>(T) * h->cfg.top_k, nb = 4ll * (h->cfg.n_experts + 1);
  const Rows in{x, ldx, T, width}, out{rows, ld_rows, P, width};
  if (T > 0) {
    if (st == MOE_OK) st = check_rows(h, in, "x");
    if (st == MOE_OK) st = check_rows(h, out, "rows");
    if (st != MOE_OK) return st;
    if (!offsets || !place || misaligned(offsets, 4) || misaligned(place, 4))
      return fail(h, MOE_ERR_INVALID_ARG, "offsets and place must be aligned and not NULL");
    if (meet(in, out)) return fail(h, MOE_ERR_INVALID_ARG, "rows overlaps x");
    if (with_plan ? clash({{offsets, nb}, {order, 4 * P}, {place, 4 * P}, out}, {{ids, id_bytes * P}}) ||
                        clash({{offsets, nb}, {order, 4 * P}, {place, 4 * P}}, {in})
                  : clash({out}, {{offsets, nb}, {place, 4 * P}}))
      return fail(h, MOE_ERR_INVALID_ARG, "the rows, the plan and the inputs overlap");
  }
  DeviceScope dev(h->device);
  if (!dev.ok) return fail(h, MOE_ERR_DEVICE, "the handle's device cannot be made current");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  RowArgs a = row_args(h, T, width, offsets, place);
  a.tok = static_cast<const unsigned short*>(x);
  a.ld_tok = ldx;
  a.row_out = static_cast<unsigned short*>(rows);
  a.ld_row_out = ld_rows;
  const bool aligned = whole_words({in, out});
  if (with_plan && T > 0 && P <= RW_CHUNK) {
    const int64_t pieces = static_cast<int64_t>(T) * ((width + 255) / 256);
    ++h->last_launches;
    return launched(h, launch_chained(aligned ? k_rows_small<true> : k_rows_small<false>, std::min<int64_t>(h->num_sms, (pieces + 7) / 8), RW_CHUNK,
                                      static_cast<size_t>(small_smem(a.E, static_cast<int>(P))), 1, s,
                                      plan_args(h, ids, id_bytes, T, offsets, order, place), a));
  }
  cudaError_t e = with_plan ? launch_plan(h, plan_args(h, ids, id_bytes, T, offsets, order, place), s) : cudaSuccess;
  if (e == cudaSuccess && T > 0) {
    ++h->last_launches;
    const RowKernel k = aligned ? k_rows_take<true> : k_rows_take<false>;
    e = launch_chained(k, T, 32 * row_warps(T, width, h->num_sms), 0, 1, s, a);
  }
  return launched(h, e);
}

moe_status combine(moe_rows* h, const void* y, int64_t ldy, int32_t T, int32_t width, const void* w, int32_t w_dtype,
                   const int32_t* place, void* out, int64_t ldo, void* stream) {
  if (!h) return MOE_ERR_INVALID_ARG;
  moe_status st = check_sizes(h, T, width);
  if (st != MOE_OK) return st;
  if (w && (w_dtype < 0 || w_dtype > 2)) return fail(h, MOE_ERR_INVALID_ARG, "unknown type of w");
  h->last_launches = 0;
  if (T == 0) return MOE_OK;
  const int64_t P = static_cast<int64_t>(T) * h->cfg.top_k;
  const Rows in{y, ldy, P, width}, to{out, ldo, T, width};
  st = check_rows(h, in, "y");
  if (st == MOE_OK) st = check_rows(h, to, "out");
  if (st != MOE_OK) return st;
  if (!place || misaligned(place, 4) || misaligned(w, w_dtype == 2 ? 4 : 2))
    return fail(h, MOE_ERR_INVALID_ARG, "place must be aligned and not NULL, w aligned");
  if (meet(in, to) || clash({to}, {{w, P * (w_dtype == 2 ? 4 : 2)}, {place, 4 * P}}))
    return fail(h, MOE_ERR_INVALID_ARG, "out overlaps an input");
  DeviceScope dev(h->device);
  if (!dev.ok) return fail(h, MOE_ERR_DEVICE, "the handle's device cannot be made current");
  RowArgs a = row_args(h, T, width, nullptr, place);
  a.row = static_cast<const unsigned short*>(y);
  a.ld_row = ldy;
  a.tok_out = static_cast<unsigned short*>(out);
  a.ld_tok = ldo;
  a.w = w;
  a.w_dt = w_dtype;
  const bool aligned = whole_words({in, to});
  const StreamShape f = stream_shape(T, width, a.k, aligned, h->num_sms);
  ++h->last_launches;
  return launched(h, launch_chained(aligned ? k_rows_combine<true> : k_rows_combine<false>, f.ctas, f.threads,
                                    static_cast<size_t>(f.smem), 1, static_cast<cudaStream_t>(stream), a, f.slots));
}

moe_status combine_backward(moe_rows* h, const void* d_out, int64_t ldd, int32_t T, int32_t width, const void* y, int64_t ldy,
                            const void* w, int32_t w_dtype, const int32_t* offsets, const int32_t* place, void* d_y,
                            int64_t lddy, void* d_w, void* stream) {
  if (!h) return MOE_ERR_INVALID_ARG;
  moe_status st = check_sizes(h, T, width);
  if (st != MOE_OK) return st;
  if (w_dtype < 0 || w_dtype > 2) return fail(h, MOE_ERR_INVALID_ARG, "unknown type of w");
  h->last_launches = 0;
  if (T == 0 || (!d_y && !d_w)) return MOE_OK;
  const int64_t P = static_cast<int64_t>(T) * h->cfg.top_k;
  const Rows e{d_out, ldd, T, width}, in{d_w ? y : nullptr, ldy, P, width}, to{d_y, lddy, P, width};
  st = check_rows(h, e, "d_out");
  if (st == MOE_OK && d_w) st = check_rows(h, in, "y");
  if (st == MOE_OK && d_y) st = check_rows(h, to, "d_y");
  if (st != MOE_OK) return st;
  const uintptr_t wb = w_dtype == 2 ? 4 : 2;
  if (!place || misaligned(place, 4) || (d_y && (!w || !offsets)) || misaligned(offsets, 4) || misaligned(w, wb) ||
      misaligned(d_w, wb))
    return fail(h, MOE_ERR_INVALID_ARG, "w, offsets and place must be aligned and not NULL");
  const int64_t nw = P * static_cast<int64_t>(wb), nb = 4ll * (h->cfg.n_experts + 1);
  if (meet(e, to) || meet(in, to) || clash({{d_w, nw}}, {e, in, {w, nw}, {offsets, nb}, {place, 4 * P}}) ||
      clash({to, {d_w, nw}}, {{w, nw}, {offsets, nb}, {place, 4 * P}}))
    return fail(h, MOE_ERR_INVALID_ARG, "a gradient overlaps an input or the other gradient");
  DeviceScope dev(h->device);
  if (!dev.ok) return fail(h, MOE_ERR_DEVICE, "the handle's device cannot be made current");
  RowArgs a = row_args(h, T, width, offsets, place);
  a.tok = static_cast<const unsigned short*>(d_out);
  a.ld_tok = ldd;
  a.row = static_cast<const unsigned short*>(in.p);
  a.ld_row = ldy;
  a.row_out = static_cast<unsigned short*>(d_y);
  a.ld_row_out = lddy;
  a.w = w;
  a.d_w = d_w;
  a.w_dt = w_dtype;
  // Both gradients in one kernel where rows are whole words.  Else cutting and joining words takes
  // the registers of too many warps: 8192 x 9 x 1001 in one kernel 131 us, in two 57 + 41 (100 one after the other).
  const bool aligned = whole_words({e, in, to}), both = aligned && d_y && d_w;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t err = cudaSuccess;
  if (d_w) {
    const StreamShape f = stream_shape(T, width, a.k + 1, aligned, h->num_sms);
    const StreamKernel k = both ? k_rows_grad<true, true> : aligned ? k_rows_grad<true, false> : k_rows_grad<false, false>;
    ++h->last_launches;
    err = launch_chained(k, f.ctas, f.threads, static_cast<size_t>(f.smem), 1, s, a, f.slots);
  }
  if (d_y && !both && err == cudaSuccess) {
    const RowKernel k = aligned ? k_rows_scale<true> : k_rows_scale<false>;
    ++h->last_launches;
    err = launch_chained(k, T, 32 * row_warps(T, width, h->num_sms), 0, 1, s, a);
  }
  return launched(h, err);
}

// (h: the handle while it is not the caller's, for the entry point to free when an exception ends this)
moe_status create(const moe_rows_config* cfg, moe_rows** out, moe_rows*& h) {
  if (out) *out = nullptr;
  std::string why;
  moe_status st = validate(cfg, &why);
  if (st == MOE_OK && !out) {
    st = MOE_ERR_INVALID_ARG;
    why = "out must not be NULL";
  }
  int device = 0, sms = 0;
  if (st == MOE_OK) st = op_device(&device, &sms, &why);
  if (st != MOE_OK) {
    g_error = why;
    return st;
  }
  h = new (std::nothrow) moe_rows();
  if (!h) {
    g_error = "host memory";
    return MOE_ERR_OOM;
  }
  h->device = device;
  h->num_sms = sms;
  h->cfg = *cfg;
  cudaError_t e = h->alloc(reinterpret_cast<void**>(&h->status), 64);
  if (e == cudaSuccess) e = cudaMemset(h->status, 0, 64);
  const int64_t chunks = (static_cast<int64_t>(cfg->max_tokens) * cfg->top_k + RW_CHUNK - 1) / RW_CHUNK;
  if (e == cudaSuccess && chunks > 1)
    e = h->alloc(reinterpret_cast<void**>(&h->totals), static_cast<size_t>(chunks + 1) * (cfg->n_experts + 1) * 4);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(k_rows_plan), cudaFuncAttributeMaxDynamicSharedMemorySize, rw_plan_smem(RW_MAX_E));
  for (auto k : {k_rows_small<true>, k_rows_small<false>})
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(reinterpret_cast<const void*>(k), cudaFuncAttributeMaxDynamicSharedMemorySize,
                               small_smem(RW_MAX_E, RW_CHUNK));
  for (StreamKernel k : {k_rows_combine<true>, k_rows_combine<false>, k_rows_grad<true, true>, k_rows_grad<true, false>,
                         k_rows_grad<false, false>})
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(reinterpret_cast<const void*>(k), cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamSmem);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();   // the status word's clear runs on the default stream
  if (e != cudaSuccess) {
    g_error = std::string("create: ") + cudaGetErrorString(e);
    h->free_all();
    delete h;
    h = nullptr;
    return e == cudaErrorMemoryAllocation ? MOE_ERR_OOM : MOE_ERR_CUDA;
  }
  *out = h;
  h = nullptr;
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_rows_validate(const moe_rows_config* cfg) {
  return op_entry([&] {
    std::string why;
    const moe_status st = validate(cfg, &why);
    if (st != MOE_OK) g_error = why;
    return st;
  });
}

moe_status moe_rows_create(const moe_rows_config* cfg, moe_rows** out) {
  moe_rows* h = nullptr;
  const moe_status st = op_entry([&] { return create(cfg, out, h); });
  if (h) {
    h->free_all();
    delete h;
  }
  return st;
}

moe_status moe_rows_plan(moe_rows* h, const void* ids, int32_t id_bytes, int32_t T, int32_t* offsets, int32_t* order,
                         int32_t* place, void* stream) {
  return op_entry([&] { return plan(h, ids, id_bytes, T, offsets, order, place, stream); });
}

moe_status moe_rows_dispatch(moe_rows* h, const void* x, int64_t ldx, int32_t T, int32_t width, const void* ids,
                             int32_t id_bytes, int32_t* offsets, int32_t* order, int32_t* place, void* rows, int64_t ld_rows,
                             void* stream) {
  return op_entry([&] { return take(h, true, x, ldx, T, width, ids, id_bytes, offsets, order, place, rows, ld_rows, stream); });
}

moe_status moe_rows_take(moe_rows* h, const void* x, int64_t ldx, int32_t T, int32_t width, const int32_t* offsets,
                         const int32_t* place, void* rows, int64_t ld_rows, void* stream) {
  return op_entry([&] {
    return take(h, false, x, ldx, T, width, nullptr, 4, const_cast<int32_t*>(offsets), nullptr, const_cast<int32_t*>(place),
                rows, ld_rows, stream);
  });
}

moe_status moe_rows_combine(moe_rows* h, const void* y, int64_t ldy, int32_t T, int32_t width, const void* w, int32_t w_dtype,
                            const int32_t* place, void* out, int64_t ldo, void* stream) {
  return op_entry([&] { return combine(h, y, ldy, T, width, w, w_dtype, place, out, ldo, stream); });
}

moe_status moe_rows_combine_backward(moe_rows* h, const void* d_out, int64_t ldd, int32_t T, int32_t width, const void* y,
                                     int64_t ldy, const void* w, int32_t w_dtype, const int32_t* offsets,
                                     const int32_t* place, void* d_y, int64_t lddy, void* d_w, void* stream) {
  return op_entry(
      [&] { return combine_backward(h, d_out, ldd, T, width, y, ldy, w, w_dtype, offsets, place, d_y, lddy, d_w, stream); });
}

moe_status moe_rows_device_status(moe_rows* h, void* stream) {
  return op_entry([&] { return h ? h->read_status(stream) : MOE_ERR_INVALID_ARG; });
}

int64_t moe_rows_device_bytes(const moe_rows* h) { return h ? h->bytes : 0; }

int32_t moe_rows_last_launch_count(const moe_rows* h) { return h ? h->last_launches : 0; }

moe_status moe_rows_destroy(moe_rows* h) {
  if (!h) return MOE_OK;
  {
    DeviceScope dev(h->device);
    cudaDeviceSynchronize();
    h->free_all();
  }
  delete h;
  return MOE_OK;
}

const char* moe_rows_last_error(const moe_rows* h) { return h ? h->last_error.c_str() : g_error.c_str(); }

}  // extern "C"
