// Orthogonalised updates (moe_ortho_* in include/moe_layer.h): host side and C ABI.
#include "moe_ortho_plan.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "moe_op_host.h"

using namespace moe_op;

struct moe_ortho : OpHandle {
  moe_ortho_config cfg{};
  int m = 0;                        // the smaller side: A and B are [m, m]
  int64_t ld_x = 0, ld_a = 0;       // row strides of X and of A, B
  int q = 0;                        // scale of X: 2^q
  int workers[3] = {0, 0, 0};       // resident CTAs, and pairs of them, by the CTAs of a tile
  unsigned short *hi[2] = {nullptr, nullptr}, *a = nullptr, *b = nullptr;   // rows, as tensor copies read them
  unsigned short* lo = nullptr;     // X's second term in 32 x 32 pieces, as epilogues read it
  float *d = nullptr, *e = nullptr, *sums = nullptr;
  unsigned* done = nullptr;
  unsigned* arrived = nullptr;
  CUtensorMap tx[2], ta, tb;
  bool tall() const { return cfg.rows > cfg.cols; }
  int64_t step_x() const { return cfg.rows * ld_x; }
  int64_t step_a() const { return m * ld_a; }
  int64_t step_lo() const { return (cfg.rows + 31) / 32 * (ld_x / 32) * 1024; }
};

namespace {

thread_local std::string g_error;

constexpr int kMaxSide = 32768;
constexpr int kMaxSteps = 64;

// The largest |singular value| and |b l + c l^2| (l its square) that the steps can
// reach from singular values in [0, 1].  Each step maps [0, top] by p on a grid.  Rounding may
// leave a singular value above the largest that the definition has, by less than 2^-9 of
// it a step (hi, O and P by 2^-11 each), and where p repels from there the next steps take it away: with
// (2.5, -3.5, 2), p(1) = 1 and p'(1) = 2, a matrix of rank one went to infinity in 30 steps.
constexpr double kRounding = 1.0 / 512;
struct Reach {
  double x = 1.0, b = 0.0;
};
Reach reach(const moe_ortho_config& c) {
  Reach R;
  double top = 1.0 + kRounding;
  for (int i = 0; i < c.steps && top < 64.0; ++i) {
    double next = 0.0;
    for (int j = 0; j <= 2048; ++j) {
      const double s = top * j / 2048, l = s * s, b = c.b * l + c.c * l * l;
      next = std::max(next, std::fabs((c.a + b) * s));
      R.b = std::max(R.b, std::fabs(b));
    }
    R.x = std::max(R.x, next);
    top = next * (1.0 + kRounding);
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
  if (or_parts(c->rows, 128) * or_parts(c->cols, 128) * c->max_matrices > (1 << 24))
    return fail(MOE_ERR_UNSUPPORTED, "more than 2^24 tiles of 128 x 128 in all matrices");
  const Reach R = reach(*c);
  if (R.x > 4.0 || R.b > 64.0) return fail(MOE_ERR_UNSUPPORTED, "the coefficients let singular values of 1 and less grow above 4");
  return MOE_OK;
}

using Kernel = void (*)(const OrthoArgs);

Kernel kernel_of(int cg, bool tall) {
  if (tall) return cg == 2 ? k_ortho<2, true> : k_ortho<1, true>;
  return cg == 2 ? k_ortho<2, false> : k_ortho<1, false>;
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
  const int m = h->m;
  const double scale = std::ldexp(1.0, h->q);

  OrthoStart t{};
  t.g = g;
  t.dt = c.dtype;
  t.ldg = ldg;
  t.step_g = step_g;
  t.M = c.rows;
  t.N = c.cols;
  t.ctas = or_start_ctas(R, C, n, h->num_sms);
  t.part = h->sums;
  t.hi = h->hi[0];
  t.lo = h->lo;
  t.step_lo = h->step_lo();
  t.cols_lo = static_cast<int>(h->ld_x / 32);
  t.ld_x = h->ld_x;
  t.step_x = h->step_x();
  t.vec = reinterpret_cast<uintptr_t>(g) % 16 == 0 && (R == 1 || ldg * gb % 16 == 0) && step_g * gb % 16 == 0;
  t.s = scale;
  t.eps = c.eps;
  t.done = h->done;
  t.arrived = h->arrived;
  t.n_arrived = ortho_counters(h->num_sms);
  cudaError_t e = cudaSuccess;
  for (int z = 0; z < n && e == cudaSuccess; z += 65535) {   // (a grid's second dimension)
    const int nz = std::min(n - z, 65535);
    OrthoStart p = t;
    p.g = gp + z * step_g * gb;
    p.part += static_cast<int64_t>(z) * t.ctas * 3;
    p.hi += z * t.step_x;
    p.lo += z * t.step_lo;
    p.done += 3ll * z;
    const dim3 grid(static_cast<unsigned>(t.ctas), static_cast<unsigned>(nz));
    if (t.ctas > 1) {
      e = launch_chained(k_ortho_norm, grid, 256, 0, 1, s, p);
      ++h->last_launches;
    }
    if (e == cudaSuccess) e = launch_chained(k_ortho_start, grid, 256, 0, 1, s, p);
    ++h->last_launches;
  }

  const OrthoPlan P = ortho_plan(c.rows, c.cols, n, h->workers);
  OrthoArgs a{};
  for (int i = 0; i < 2; ++i) {
    a.tx[i] = h->tx[i];
    a.x[i] = h->hi[i];
  }
  a.ta = h->ta;
  a.tb = h->tb;
  a.a = h->a;
  a.b = h->b;
  a.ld_x = h->ld_x;
  a.ld_a = h->ld_a;
  a.step_x = h->step_x();
  a.step_a = h->step_a();
  a.out = static_cast<unsigned short*>(out);
  a.ld_out = ldo;
  a.step_out = step_o;
  a.vec_out = reinterpret_cast<uintptr_t>(out) % 32 == 0 && ldo % 16 == 0 && step_o % 16 == 0;
  const int busy = ortho_phases(P, c.rows, c.cols, n, h->workers, h->part, h->arrived, &a);
  a.steps = c.steps;
  a.stages = OR_MAX_STAGES;
  while (or_smem_bytes(a.stages) > OR_SMEM_MAX) --a.stages;
  a.lo = h->lo;
  a.step_lo = t.step_lo;
  a.cols_lo = t.cols_lo;
  a.d = h->d;
  a.e = h->e;
  a.step_diag = h->ld_a;
  a.ka = c.a;
  a.ka_lo = c.a / OR_LO;
  a.kb = c.b;
  a.kc = static_cast<float>(c.c / (scale * scale));
  a.inv_s = static_cast<float>(1.0 / scale);
  a.inv_s2 = static_cast<float>(1.0 / (scale * scale));
  a.done = h->done;
  a.status = h->status;
  if (e == cudaSuccess) {
    // all CTAs resident at once: they wait for one another
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(busy * P.cg));
    cfg.blockDim = dim3(OR_THREADS);
    cfg.dynamicSmemBytes = static_cast<size_t>(or_smem_bytes(a.stages));
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeCooperative;
    at[0].val.cooperative = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = static_cast<unsigned>(P.cg);
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = P.cg > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kernel_of(P.cg, h->tall()), a);
    ++h->last_launches;
  }
  if (e != cudaSuccess) {
    h->last_error = std::string("launch: ") + cudaGetErrorString(e);
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
  if (e == cudaSuccess) e = h->alloc(reinterpret_cast<void**>(&h->lo), n * h->step_lo() * 2);
  for (unsigned short** p : {&h->a, &h->b})
    if (e == cudaSuccess) e = h->alloc(reinterpret_cast<void**>(p), a);
  for (float** p : {&h->d, &h->e})
    if (e == cudaSuccess) e = h->alloc(reinterpret_cast<void**>(p), n * h->ld_a * 4);
  if (e == cudaSuccess) e = h->alloc(reinterpret_cast<void**>(&h->sums), static_cast<size_t>(or_norm_parts(c.rows, c.cols, c.max_matrices, sms)) * 3 * 4);
  if (e == cudaSuccess) e = h->alloc(reinterpret_cast<void**>(&h->done), n * 3 * 4);
  if (e == cudaSuccess) e = h->alloc(reinterpret_cast<void**>(&h->arrived), static_cast<size_t>(ortho_counters(sms)) * 4);
  for (int cg = 1; cg <= 2 && e == cudaSuccess; ++cg) {
    const Kernel k = kernel_of(cg, h->tall());
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(k), cudaFuncAttributeMaxDynamicSharedMemorySize, OR_SMEM_MAX);
    if (e != cudaSuccess) break;
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3(static_cast<unsigned>(sms / cg * cg));
    lc.blockDim = dim3(OR_THREADS);
    lc.dynamicSmemBytes = OR_SMEM_MAX;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(cg);
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    lc.attrs = at;
    lc.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&h->workers[cg], k, &lc);
    h->workers[cg] = std::min(h->workers[cg], sms / cg);
    if (e == cudaSuccess && h->workers[cg] < 1) e = cudaErrorInvalidConfiguration;
  }
  for (int i = 1; i <= std::min(c.max_matrices, sms) && e == cudaSuccess; ++i)   // (more matrices: no splits)
    h->part_bytes = std::max(h->part_bytes, ortho_plan(c.rows, c.cols, i, h->workers).part_bytes(i));
  if (e == cudaSuccess && h->part_bytes) e = h->alloc(reinterpret_cast<void**>(&h->part), h->part_bytes);
  auto rows_of = [&](CUtensorMap* map, const void* p, int64_t cols, int64_t rows, int64_t ld) {
    return encode_stack16(map, p, cols, rows, ld, c.max_matrices, rows * ld, 64);
  };
  if (e == cudaSuccess && !(rows_of(&h->tx[0], h->hi[0], c.cols, c.rows, h->ld_x) && rows_of(&h->tx[1], h->hi[1], c.cols, c.rows, h->ld_x) &&
                            rows_of(&h->ta, h->a, h->m, h->m, h->ld_a) && rows_of(&h->tb, h->b, h->m, h->m, h->ld_a)))
    e = cudaErrorInvalidValue;
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
