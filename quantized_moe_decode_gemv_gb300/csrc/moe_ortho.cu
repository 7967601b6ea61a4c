// Orthogonalised updates (moe_ortho_* in include/moe_layer.h): host side and C ABI.
#include "moe_ortho.cuh"

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "moe_op_host.h"

using namespace moe_op;

struct moe_ortho : OpHandle {
  int64_t own_step_x() const { return (cfg.rows + 31) / 32 * (ld_x / 32) * 2048; }
  int64_t own_step_a() const { return (m + 31) / 32 * (ld_a / 32) * 1024; }
  moe_ortho_config cfg{};
  int m = 0;                        // the smaller side: A and B are [m, m]
  int64_t ld_x = 0, ld_a = 0;       // row strides of X and of A, B
  int q = 0;                        // scale of X: 2^q
  unsigned short *hi[2] = {nullptr, nullptr}, *a = nullptr, *b = nullptr;   // rows, as tensor copies read them
  unsigned short *own_x = nullptr, *own_a = nullptr;   // 32 x 32 pieces, as epilogues do
  float *d = nullptr, *e = nullptr, *sums = nullptr;
};

namespace {

thread_local std::string g_error;

constexpr int kMaxSide = 32768;
constexpr int kMaxSteps = 64;

// The largest |singular value| and |b l + c l^2| (l its square) that the steps can
// reach from singular values in [0, 1].  Each step maps [0, top] by p on a grid.
struct Reach {
  double x = 1.0, b = 0.0;
};
Reach reach(const moe_ortho_config& c) {
  Reach R;
  double top = 1.0;
  for (int i = 0; i < c.steps && top < 64.0; ++i) {
    double next = 0.0;
    for (int j = 0; j <= 2048; ++j) {
      const double s = top * j / 2048, l = s * s, b = c.b * l + c.c * l * l;
      next = std::max(next, std::fabs((c.a + b) * s));
      R.b = std::max(R.b, std::fabs(b));
    }
    R.x = std::max(R.x, next);
    top = next;
  }
  return R;
}

// X is scaled by 2^q: 4^q about the smaller side, so that A's entries are about 1 at
// the start, and 4^q times the largest value of A or B below 2^15 (fp16 ends at 2^16).
int scale_of(const moe_ortho_config& c, const Reach& R) {
  const double most = std::max(R.x * R.x, R.b);
  int q = 0;
  while (4ll << (2 * q) <= std::min(c.rows, c.cols) && static_cast<double>(4ll << (2 * q)) * most <= 32768.0) ++q;
  return q;
}

int64_t tiles(int64_t n, int side) { return (n + side - 1) / side; }

moe_status validate(const moe_ortho_config* c, std::string* why) {
  auto fail = [&](moe_status s, const char* msg) {
    *why = msg;
    return s;
  };
  if (!c) return fail(MOE_ERR_INVALID_ARG, "config is NULL");
  if (c->rows < 1 || c->cols < 1 || c->max_matrices < 1) return fail(MOE_ERR_INVALID_ARG, "rows, cols and max_matrices must be positive");
  if (c->dtype < 0 || c->dtype > 2) return fail(MOE_ERR_INVALID_ARG, "unknown dtype");
  if (c->steps < 1) return fail(MOE_ERR_INVALID_ARG, "steps must be positive");
  if (!std::isfinite(c->a) || !std::isfinite(c->b) || !std::isfinite(c->c) || !std::isfinite(c->eps) || c->eps < 0)
    return fail(MOE_ERR_INVALID_ARG, "the coefficients and eps must be finite, eps not negative");
  if (c->rows > kMaxSide || c->cols > kMaxSide) return fail(MOE_ERR_UNSUPPORTED, "rows or cols above 32768");
  if (c->steps > kMaxSteps) return fail(MOE_ERR_UNSUPPORTED, "steps above 64");
  if (tiles(c->rows, 128) * tiles(c->cols, 128) * c->max_matrices > (1 << 24))
    return fail(MOE_ERR_UNSUPPORTED, "more than 2^24 tiles of 128 x 128 in all matrices");
  const Reach R = reach(*c);
  if (R.x > 4.0 || R.b > 64.0) return fail(MOE_ERR_UNSUPPORTED, "the coefficients let singular values of 1 and less grow above 4");
  return MOE_OK;
}

using Kernel = void (*)(const OrthoArgs);

// of a mode and, for GRAM and APPLY, of tall matrices
Kernel kernel_of(int mode, bool tall, int cg) {
  if (mode == OR_POLY) return cg == 2 ? k_ortho<2, false, false, OR_POLY> : k_ortho<1, false, false, OR_POLY>;
  if (mode == OR_GRAM) {
    if (tall) return cg == 2 ? k_ortho<2, true, true, OR_GRAM> : k_ortho<1, true, true, OR_GRAM>;
    return cg == 2 ? k_ortho<2, false, false, OR_GRAM> : k_ortho<1, false, false, OR_GRAM>;
  }
  if (tall) return cg == 2 ? k_ortho<2, false, false, OR_APPLY> : k_ortho<1, false, false, OR_APPLY>;
  return cg == 2 ? k_ortho<2, false, true, OR_APPLY> : k_ortho<1, false, true, OR_APPLY>;
}

// Tiles of 256 x 256 on pairs, or 128 x 128: those with fewer waves.  A 64-wide K block of
// either takes a CTA as long (its bytes are the same), a wave of pairs does four times
// the work of a wave's half.
int group_of(bool sym, int M, int N, int n, int sms) {
  const int64_t u1 = sym ? or_units<1, true>(M, N, n) : or_units<1, false>(M, N, n);
  const int64_t u2 = sym ? or_units<2, true>(M, N, n) : or_units<2, false>(M, N, n);
  return tiles(u2, sms / 2) <= tiles(u1, sms) ? 2 : 1;
}

cudaError_t launch(moe_ortho* h, int mode, bool tall, OrthoArgs a, int k, const void* pa, int64_t lda, const void* pb, int64_t ldb,
                   cudaStream_t s, std::string* why) {
  const bool sym = mode != OR_APPLY;
  const int cg = group_of(sym, a.M, a.N, a.batches, h->num_sms);
  const bool amn = mode == OR_GRAM && tall, bmn = (mode == OR_GRAM && tall) || (mode == OR_APPLY && !tall);
  a.kb = (k + 63) / 64;
  a.sub = cg == 2 ? 1 : 2;
  a.stages = OR_MAX_STAGES;
  while (or_smem_bytes(a.stages, a.sub) > OR_SMEM_MAX) --a.stages;
  const int64_t xs = h->cfg.rows * h->ld_x, as = h->m * h->ld_a;
  const bool ok = (amn ? encode_stack16(&a.ta, pa, a.M, k, lda, a.batches, xs, 64, 64)
                       : encode_stack16(&a.ta, pa, k, a.M, lda, a.batches, mode == OR_GRAM || (mode == OR_APPLY && tall) ? xs : as, 64, 128)) &&
                  (bmn ? encode_stack16(&a.tb, pb, a.N, k, ldb, a.batches, xs, 64, 64)
                       : encode_stack16(&a.tb, pb, k, a.N, ldb, a.batches, mode == OR_GRAM ? xs : as, 64, 128));
  if (!ok) {
    *why = "tensor map refused";
    return cudaErrorInvalidValue;
  }
  const int64_t units = sym ? (cg == 2 ? or_units<2, true>(a.M, a.N, a.batches) : or_units<1, true>(a.M, a.N, a.batches))
                            : (cg == 2 ? or_units<2, false>(a.M, a.N, a.batches) : or_units<1, false>(a.M, a.N, a.batches));
  const int64_t workers = std::min<int64_t>(units, h->num_sms / cg);
  ++h->last_launches;
  return launch_chained(kernel_of(mode, tall, cg), workers * cg, OR_THREADS, static_cast<size_t>(or_smem_bytes(a.stages, a.sub)), cg, s, a);
}

int64_t span(int64_t n, int64_t step, int64_t rows, int64_t ld, int64_t cols) { return (n - 1) * step + (rows - 1) * ld + cols; }

moe_status forward(moe_ortho* h, const void* g, int64_t ldg, int64_t step_g, int32_t n, void* out, int64_t ldo, int64_t step_o,
                   void* stream) {
  if (!h) return MOE_ERR_INVALID_ARG;
  const moe_ortho_config& c = h->cfg;
  auto fail = [&](moe_status st, const char* msg) {
    h->last_error = msg;
    return st;
  };
  if (n < 0 || n > c.max_matrices) return fail(MOE_ERR_INVALID_ARG, "n must be in 0..max_matrices");
  h->last_launches = 0;
  if (n == 0) return MOE_OK;
  const int64_t R = c.rows, C = c.cols;
  const int gb = c.dtype == MOE_DTYPE_FP32 ? 4 : 2;
  if (!g || !out) return fail(MOE_ERR_INVALID_ARG, "g and out must not be NULL");
  if (reinterpret_cast<uintptr_t>(g) % gb || reinterpret_cast<uintptr_t>(out) % 2)
    return fail(MOE_ERR_INVALID_ARG, "g and out must be aligned to their elements");
  if ((R > 1 && (ldg < C || ldo < C)) || (n > 1 && (step_g < 0 || step_o < span(1, 0, R, R > 1 ? ldo : C, C))))
    return fail(MOE_ERR_INVALID_ARG, "rows must be at least cols elements apart, matrices of out apart from each other");
  if (R == 1) ldg = ldo = C;
  if (n == 1) step_g = step_o = 0;
  const int64_t ng = span(n, step_g, R, ldg, C) * gb, no = span(n, step_o, R, ldo, C) * 2;
  const char *gp = static_cast<const char*>(g), *op = static_cast<const char*>(out);
  if (gp < op + no && op < gp + ng) return fail(MOE_ERR_INVALID_ARG, "out overlaps g");
  DeviceScope dev(h->device);
  if (!dev.ok) return fail(MOE_ERR_DEVICE, "the handle's device cannot be made current");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool tall = R > C;
  const int m = h->m;
  const int64_t xs = R * h->ld_x, as = m * h->ld_a, ds = (m + 31) / 32 * 32;
  const double scale = std::ldexp(1.0, h->q);

  OrthoStart t{};
  t.g = g;
  t.dt = c.dtype;
  t.ldg = ldg;
  t.step_g = step_g;
  t.M = c.rows;
  t.N = c.cols;
  const int64_t pieces = R * ((C + 7) / 8);
  t.ctas = static_cast<int>(std::min<int64_t>({OR_NORM_CTAS, (pieces + 1023) / 1024, tiles(8ll * h->num_sms, n)}));
  t.part = h->sums;
  t.hi = h->hi[0];
  t.own = h->own_x;
  t.step_own = h->own_step_x();
  t.own_cols = static_cast<int>(h->ld_x / 32);
  t.ld_x = h->ld_x;
  t.step_x = xs;
  t.vec = reinterpret_cast<uintptr_t>(g) % 16 == 0 && (R == 1 || ldg * gb % 16 == 0) && step_g * gb % 16 == 0;
  t.s = scale;
  t.eps = c.eps;
  cudaError_t e = cudaSuccess;
  std::string why;
  for (int z = 0; z < n && e == cudaSuccess; z += 65535) {   // (a grid's second dimension)
    const int nz = std::min(n - z, 65535);
    OrthoStart p = t;
    p.g = gp + z * step_g * gb;
    p.part += static_cast<int64_t>(z) * OR_NORM_CTAS * 3;
    p.hi += z * xs;
    p.own += z * t.step_own;
    const dim3 grid(static_cast<unsigned>(t.ctas), static_cast<unsigned>(nz));
    e = launch_chained(k_ortho_norm, grid, 256, 0, 1, s, p);
    if (e == cudaSuccess) e = launch_chained(k_ortho_start, grid, 256, 0, 1, s, p);
    h->last_launches += 2;
  }

  OrthoArgs base{};
  base.batches = n;
  base.ka = c.a;
  base.kb_ = c.b;
  base.kc = static_cast<float>(c.c / (scale * scale));
  base.inv_s = static_cast<float>(1.0 / scale);
  base.inv_s2 = static_cast<float>(1.0 / (scale * scale));
  base.step_diag = ds;
  base.status = h->status;
  // where the epilogues' tensor copies write: pieces of 32 x 32
  auto rows_of = [&](CUtensorMap* map, const void* p, int64_t cols, int64_t rows, int64_t ld, int64_t step) {
    if (encode_stack16(map, p, cols, rows, ld, n, step, 32, 32)) return true;
    why = "tensor map refused";
    e = cudaErrorInvalidValue;
    return false;
  };
  for (int i = 0; i < c.steps && e == cudaSuccess; ++i) {
    const unsigned short* x = h->hi[i & 1];
    OrthoArgs a = base;      // O = X X^T without its diagonal
    a.M = a.N = m;
    a.own = h->own_a;
    a.step_own = h->own_step_a();
    a.own_cols = static_cast<int>(h->ld_a / 32);
    a.diag_out = h->d;
    if (!rows_of(&a.to, h->a, m, m, h->ld_a, as)) break;
    e = launch(h, OR_GRAM, tall, a, tall ? c.rows : c.cols, x, h->ld_x, x, h->ld_x, s, &why);
    if (e != cudaSuccess) break;
    a.diag = h->d;           // P = b A + c A A without its diagonal
    a.diag_out = h->e;
    if (!rows_of(&a.to, h->b, m, m, h->ld_a, as)) break;
    e = launch(h, OR_POLY, tall, a, m, h->a, h->ld_a, h->a, h->ld_a, s, &why);
    if (e != cudaSuccess) break;
    a = base;
    a.M = c.rows;
    a.N = c.cols;
    a.own = h->own_x;
    a.step_own = t.step_own;
    a.own_cols = t.own_cols;
    a.diag = h->e;
    a.e_by_row = !tall;
    a.final = i + 1 == c.steps;
    if (!a.final) {
      if (!rows_of(&a.to, h->hi[(i + 1) & 1], C, R, h->ld_x, xs)) break;
    } else if (reinterpret_cast<uintptr_t>(out) % 16 == 0 && ldo % 8 == 0 && step_o % 8 == 0) {
      if (!rows_of(&a.to, out, C, R, ldo, n > 1 ? step_o : (R * ldo + 7) / 8 * 8)) break;
    } else {
      a.last = static_cast<unsigned short*>(out);
      a.ld_last = ldo;
      a.step_last = step_o;
    }
    e = tall ? launch(h, OR_APPLY, true, a, m, x, h->ld_x, h->b, h->ld_a, s, &why)
             : launch(h, OR_APPLY, false, a, m, h->b, h->ld_a, x, h->ld_x, s, &why);
  }
  if (e != cudaSuccess) {
    h->last_error = why.empty() ? std::string("launch: ") + cudaGetErrorString(e) : why;
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

// (h: the handle while it is not the caller's, for the entry point to free when an exception ends this)
moe_status create(const moe_ortho_config* cfg, moe_ortho** out, moe_ortho*& h) {
  if (out) *out = nullptr;
  std::string why;
  moe_status st = validate(cfg, &why);
  if (st == MOE_OK && !out) {
    st = MOE_ERR_INVALID_ARG;
    why = "out must not be NULL";
  }
  int device = 0, sms = 0;
  if (st == MOE_OK) st = op_device(&device, &sms, &why);
  if (st == MOE_OK && !encoder_found(&why)) st = MOE_ERR_CUDA;
  if (st != MOE_OK) {
    g_error = why;
    return st;
  }
  h = new (std::nothrow) moe_ortho();
  if (!h) {
    g_error = "host memory";
    return MOE_ERR_OOM;
  }
  h->device = device;
  h->num_sms = sms;
  h->cfg = *cfg;
  const moe_ortho_config& c = h->cfg;
  h->m = std::min(c.rows, c.cols);
  h->ld_x = (c.cols + 31) / 32 * 32;
  h->ld_a = (h->m + 31) / 32 * 32;
  h->q = scale_of(c, reach(c));
  const size_t n = static_cast<size_t>(c.max_matrices), x = n * c.rows * h->ld_x * 2, a = n * h->m * h->ld_a * 2;
  cudaError_t e = h->alloc(reinterpret_cast<void**>(&h->status), 64);
  if (e == cudaSuccess) e = cudaMemset(h->status, 0, 64);
  for (unsigned short** p : {&h->hi[0], &h->hi[1]})
    if (e == cudaSuccess) e = h->alloc(reinterpret_cast<void**>(p), x);
  if (e == cudaSuccess) e = h->alloc(reinterpret_cast<void**>(&h->own_x), n * h->own_step_x() * 2);
  if (e == cudaSuccess) e = h->alloc(reinterpret_cast<void**>(&h->own_a), n * h->own_step_a() * 2);
  for (unsigned short** p : {&h->a, &h->b})
    if (e == cudaSuccess) e = h->alloc(reinterpret_cast<void**>(p), a);
  for (float** p : {&h->d, &h->e})
    if (e == cudaSuccess) e = h->alloc(reinterpret_cast<void**>(p), n * h->ld_a * 4);
  if (e == cudaSuccess) e = h->alloc(reinterpret_cast<void**>(&h->sums), n * OR_NORM_CTAS * 3 * 4);
  for (int mode = 0; mode < 3; ++mode)
    for (int cg = 1; cg <= 2; ++cg)
      for (int tall = 0; tall < 2; ++tall)
        if (e == cudaSuccess)
          e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel_of(mode, tall, cg)),
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, OR_SMEM_MAX);
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

moe_status moe_ortho_validate(const moe_ortho_config* cfg) {
  return op_entry([&] {
    std::string why;
    const moe_status st = validate(cfg, &why);
    if (st != MOE_OK) g_error = why;
    return st;
  });
}

moe_status moe_ortho_create(const moe_ortho_config* cfg, moe_ortho** out) {
  moe_ortho* h = nullptr;
  const moe_status st = op_entry([&] { return create(cfg, out, h); });
  if (h) {
    h->free_all();
    delete h;
  }
  return st;
}

moe_status moe_ortho_forward(moe_ortho* h, const void* g, int64_t ldg, int64_t step_g, int32_t n, void* out, int64_t ldo,
                             int64_t step_o, void* stream) {
  return op_entry([&] { return forward(h, g, ldg, step_g, n, out, ldo, step_o, stream); });
}

moe_status moe_ortho_device_status(moe_ortho* h, void* stream) {
  return op_entry([&] { return h ? h->read_status(stream) : MOE_ERR_INVALID_ARG; });
}

int64_t moe_ortho_device_bytes(const moe_ortho* h) { return h ? h->bytes : 0; }

int32_t moe_ortho_last_launch_count(const moe_ortho* h) { return h ? h->last_launches : 0; }

moe_status moe_ortho_destroy(moe_ortho* h) {
  if (!h) return MOE_OK;
  {
    DeviceScope dev(h->device);
    cudaDeviceSynchronize();
    h->free_all();
  }
  delete h;
  return MOE_OK;
}

const char* moe_ortho_last_error(const moe_ortho* h) { return h ? h->last_error.c_str() : g_error.c_str(); }

}  // extern "C"
