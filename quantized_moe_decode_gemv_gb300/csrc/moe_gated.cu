// Gated feed-forward block with 16-bit weights (moe_gated_* in
// include/moe_layer.h): the forward pass, the backward pass, the C ABI.
#include <cuda_runtime.h>

#include <algorithm>
#include <new>

#include "moe_op_host.h"
#include "moe_outer.cuh"
#include "moe_stream16.cuh"

using namespace moe_op;

struct moe_gated : OpHandle {
  moe_gated_config cfg{};
  unsigned short* dg = nullptr;   // training: [max_tokens, N] gradients of the pre-activations
  unsigned short* du = nullptr;
};

namespace {

thread_local std::string g_error;

// Gradients of the pre-activations, eight elements a thread:
//   SwiGLU  p = 1 / (1 + exp(-g)):  du = e g p,  dg = e u p (1 + g (1 - p))
//   ReLU2   du = 2 e max(u, 0)
// Bound by memory: it reads g and u in fp32 and e in 16 bits, and writes dg and
// du in 16 bits, the type of the tensor-core products they feed.  g and u come
// in fp32 because a 16-bit copy of them would add its own rounding to that of
// dg and du, and 40% to the gradients' error, for 4 bytes an element less.
// Measured on 4096 x 8192 (470 MB): 78 us as what it adds to a backward pass, 65
// with part of its inputs still in L2.
// (No __restrict__: it would let the compiler take the inputs for constant while
// the kernel runs and read them before the wait, where the kernel before this one
// may still write them.)
template <bool GATED>
__global__ void __launch_bounds__(256) k_gated_grad(const float* g, const float* u, const unsigned short* e, int64_t lde,
                                                    int e_vec, int T, int N, int dt, unsigned short* dg,
                                                    unsigned short* du) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int q = N / 8;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= static_cast<int64_t>(T) * q) return;
  const int64_t r = i / q;
  const int c = static_cast<int>(i - r * q) * 8;
  const int64_t o = r * N + c;
  float uv[8], gv[8], ev[8];
  *reinterpret_cast<float4*>(uv) = *reinterpret_cast<const float4*>(u + o);
  *reinterpret_cast<float4*>(uv + 4) = *reinterpret_cast<const float4*>(u + o + 4);
  if (GATED) {
    *reinterpret_cast<float4*>(gv) = *reinterpret_cast<const float4*>(g + o);
    *reinterpret_cast<float4*>(gv + 4) = *reinterpret_cast<const float4*>(g + o + 4);
  }
  const unsigned short* ep = e + r * lde + c;
  if (e_vec) {
    const uint4 v = *reinterpret_cast<const uint4*>(ep);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      ev[2 * j] = lo16(w[j], dt);
      ev[2 * j + 1] = hi16(w[j], dt);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) ev[j] = lo16(ep[j], dt);
  }
  uint32_t ow[4], gw[4];
  float a[8], b[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (GATED) {
      const float p = 1.0f / (1.0f + __expf(-gv[j]));
      a[j] = ev[j] * gv[j] * p;
      b[j] = ev[j] * uv[j] * p * (1.0f + gv[j] * (1.0f - p));
    } else {
      a[j] = uv[j] < 0.0f ? ev[j] * 0.0f : 2.0f * ev[j] * uv[j];
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    ow[j] = pack2(a[2 * j], a[2 * j + 1], dt);
    if (GATED) gw[j] = pack2(b[2 * j], b[2 * j + 1], dt);
  }
  *reinterpret_cast<uint4*>(du + o) = make_uint4(ow[0], ow[1], ow[2], ow[3]);
  if (GATED) *reinterpret_cast<uint4*>(dg + o) = make_uint4(gw[0], gw[1], gw[2], gw[3]);
}

moe_status validate(const moe_gated_config* c, std::string* why) {
  auto fail = [&](moe_status s, const char* msg) {
    *why = msg;
    return s;
  };
  if (!c) return fail(MOE_ERR_INVALID_ARG, "config is NULL");
  if (c->in_features < 1 || c->out_features < 1 || c->max_tokens < 1)
    return fail(MOE_ERR_INVALID_ARG, "in_features, out_features and max_tokens must be positive");
  if (c->act != MOE_ACT_SWIGLU && c->act != MOE_ACT_RELU2) return fail(MOE_ERR_INVALID_ARG, "unknown activation");
  if (c->act_dtype < 0 || c->act_dtype > 2) return fail(MOE_ERR_INVALID_ARG, "unknown dtype");
  if (c->in_features % 8 || c->out_features % 8)
    return fail(MOE_ERR_SHAPE, "in_features and out_features must be multiples of 8");
  if (c->act_dtype == MOE_DTYPE_FP32) return fail(MOE_ERR_UNSUPPORTED, "fp32 activations");
  if (c->in_features > 65536) return fail(MOE_ERR_UNSUPPORTED, "in_features above 65536");
  if (c->out_features > (1 << 24)) return fail(MOE_ERR_UNSUPPORTED, "out_features above 2^24");
  return MOE_OK;
}

using StreamKernel = void (*)(const Stream16Args);

template <bool FP16>
StreamKernel stream_kernel_t(bool gated, int nt) {
  if (gated) return nt == 1 ? k_stream16<FP16, true, 1> : k_stream16<FP16, true, 2>;
  return nt == 1 ? k_stream16<FP16, false, 1> : k_stream16<FP16, false, 2>;
}
StreamKernel stream_kernel(bool fp16, bool gated, int nt) {
  return fp16 ? stream_kernel_t<true>(gated, nt) : stream_kernel_t<false>(gated, nt);
}

using OuterKernel = void (*)(const OuterArgs);

template <bool FP16>
OuterKernel outer_kernel(int T) {
  const int ks = (T + 15) / 16;
  return ks == 1 ? k_outer<FP16, 1> : ks == 2 ? k_outer<FP16, 2> : k_outer<FP16, 3>;
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Bytes from the first to past the last element of T rows of `cols` 16-bit elements.
int64_t span(int64_t T, int64_t ld, int64_t cols) { return ((T - 1) * ld + cols) * 2; }
bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
  return x && y && x < y + nb && y < x + na;
}

}  // namespace

static moe_status validate_entry(const moe_gated_config* cfg) {
  std::string why;
  const moe_status st = validate(cfg, &why);
  if (st != MOE_OK) g_error = why;
  return st;
}

// (h: the handle while it is not the caller's, for the entry point to free when an exception ends this)
static moe_status create(const moe_gated_config* cfg, moe_gated** out, moe_gated*& h) {
  if (out) *out = nullptr;
  std::string why;
  moe_status st = validate(cfg, &why);
  if (st == MOE_OK && !out) {
    st = MOE_ERR_INVALID_ARG;
    why = "out must not be NULL";
  }
  int device = 0, sms = 0;
  if (st == MOE_OK) st = op_device(&device, &sms, &why);
  if (st == MOE_OK && !gemm16_setup(&why)) st = MOE_ERR_CUDA;
  if (st != MOE_OK) {
    g_error = why;
    return st;
  }
  h = new (std::nothrow) moe_gated();
  if (!h) {
    g_error = "host memory";
    return MOE_ERR_OOM;
  }
  h->device = device;
  h->num_sms = sms;
  h->cfg = *cfg;
  const moe_gated_config& c = h->cfg;
  const bool gated = c.act == MOE_ACT_SWIGLU;
  cudaError_t e = h->alloc(reinterpret_cast<void**>(&h->status), 64);
  if (e == cudaSuccess) e = cudaMemset(h->status, 0, 64);
  if (c.training || c.max_tokens > ST_MAX_T) {   // else every call streams and splits nothing
    h->part_bytes = gemm16_part_bytes(c.max_tokens, std::max<int64_t>(c.out_features * (gated ? 2ll : 1ll),
                                                                      c.training ? c.in_features : 0), sms);
    if (e == cudaSuccess) e = h->alloc(reinterpret_cast<void**>(&h->part), h->part_bytes);
  }
  const size_t grad = static_cast<size_t>(c.max_tokens) * c.out_features * 2;
  if (c.training && e == cudaSuccess) e = h->alloc(reinterpret_cast<void**>(&h->du), grad);
  if (c.training && gated && e == cudaSuccess) e = h->alloc(reinterpret_cast<void**>(&h->dg), grad);
  for (int nt = 1; nt <= 2 && e == cudaSuccess; ++nt)
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(stream_kernel(c.act_dtype == MOE_DTYPE_FP16, gated, nt)),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, S16_SMEM_MAX);
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

static moe_status forward(moe_gated* h, const void* x, int64_t ldx, int32_t T, const void* gate_w, const void* up_w,
                             void* out, int64_t ldo, float* save_gate, float* save_up, void* stream) {
  if (!h) return MOE_ERR_INVALID_ARG;
  const moe_gated_config& c = h->cfg;
  const bool gated = c.act == MOE_ACT_SWIGLU;
  const int K = c.in_features, N = c.out_features;
  auto fail = [&](moe_status st, const char* msg) {
    h->last_error = msg;
    return st;
  };
  if (T < 0 || T > c.max_tokens) return fail(MOE_ERR_INVALID_ARG, "T must be in 0..max_tokens");
  h->last_launches = 0;
  if (T == 0) return MOE_OK;
  if (!x || !out || !up_w || (gated && !gate_w)) return fail(MOE_ERR_INVALID_ARG, "x, out and the weights must not be NULL");
  if (!gated && (gate_w || save_gate)) return fail(MOE_ERR_SHAPE, "a squared-ReLU block takes no gate matrix");
  if (gated && (save_gate == nullptr) != (save_up == nullptr))
    return fail(MOE_ERR_INVALID_ARG, "save_gate and save_up come together");
  if (ldx < K || ldx % 8 || !aligned16(x))
    return fail(MOE_ERR_INVALID_ARG, "x needs 16-byte aligned rows: ldx >= in_features, a multiple of 8");
  if (!aligned16(gate_w) || !aligned16(up_w) || !aligned16(save_gate) || !aligned16(save_up))
    return fail(MOE_ERR_INVALID_ARG, "the weights and the saved buffers must be 16-byte aligned");
  if (ldo < N || reinterpret_cast<uintptr_t>(out) % 2) return fail(MOE_ERR_INVALID_ARG, "ldo must be at least out_features");
  const int64_t no = span(T, ldo, N), nw = static_cast<int64_t>(K) * N * 2;
  if (rows_overlap(x, ldx, K, out, ldo, N, T) || overlap(out, no, up_w, nw) || overlap(out, no, gate_w, nw))
    return fail(MOE_ERR_INVALID_ARG, "out overlaps an input");
  const int64_t nx = span(T, ldx, K), ns = 4ll * T * N;
  for (const float* p : {save_gate, save_up})
    if (overlap(p, ns, x, nx) || overlap(p, ns, out, no) || overlap(p, ns, up_w, nw) || overlap(p, ns, gate_w, nw))
      return fail(MOE_ERR_INVALID_ARG, "a saved buffer overlaps an input or out");
  if (overlap(save_gate, ns, save_up, ns)) return fail(MOE_ERR_INVALID_ARG, "the saved buffers overlap");
  DeviceScope dev(h->device);
  if (!dev.ok) return fail(MOE_ERR_DEVICE, "the handle's device cannot be made current");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  std::string why;
  cudaError_t e = cudaSuccess;
  if (T <= ST_MAX_T) {
    Stream16Args a{};
    a.w_gate = gate_w;
    a.w_up = up_w;
    a.x = x;
    a.ldx = ldx;
    a.out = out;
    a.ldo = ldo;
    a.save_gate = save_gate;
    a.save_up = save_up;
    a.K = K;
    a.N = N;
    a.T = T;
    a.chunks = (K + 63) / 64;
    a.act = c.act;
    const Stream16Plan P = s16_plan(gated, T, N, h->num_sms);
    a.depth = P.depth;
    e = launch_chained(stream_kernel(c.act_dtype == MOE_DTYPE_FP16, gated, T > 8 ? 2 : 1), P.grid, S16_THREADS,
                       static_cast<size_t>(P.smem), 1, s, a);
    ++h->last_launches;
  } else {
    GemmCall g;
    g.M = T;
    g.N = N;
    g.K[0] = K;
    g.dual = gated;
    g.a[0] = x;
    g.lda = ldx;
    g.b[0] = gated ? gate_w : up_w;
    g.b[1] = up_w;
    g.ldb = K;
    g.dt = c.act_dtype;
    g.act = c.act;
    g.out[0] = out;
    g.ldo = ldo;
    g.save_gate = save_gate;
    g.save_up = save_up;
    e = gemm16_launch(g, *h, s, &h->last_launches, &why);
  }
  if (e != cudaSuccess) {
    h->last_error = why.empty() ? std::string("launch: ") + cudaGetErrorString(e) : why;
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

static moe_status backward(moe_gated* h, const void* d_out, int64_t ldd, int32_t T, const void* x, int64_t ldx,
                              const void* gate_w, const void* up_w, const float* save_gate, const float* save_up,
                              void* d_x, int64_t lddx, void* d_gate_w, void* d_up_w, void* stream) {
  if (!h) return MOE_ERR_INVALID_ARG;
  const moe_gated_config& c = h->cfg;
  const bool gated = c.act == MOE_ACT_SWIGLU;
  const int K = c.in_features, N = c.out_features;
  auto fail = [&](moe_status st, const char* msg) {
    h->last_error = msg;
    return st;
  };
  if (!c.training) return fail(MOE_ERR_UNSUPPORTED, "the handle was created without training");
  if (T < 0 || T > c.max_tokens) return fail(MOE_ERR_INVALID_ARG, "T must be in 0..max_tokens");
  if (!gated && (gate_w || save_gate || d_gate_w)) return fail(MOE_ERR_SHAPE, "a squared-ReLU block takes no gate matrix");
  if (!aligned16(d_x) || !aligned16(d_gate_w) || !aligned16(d_up_w))
    return fail(MOE_ERR_INVALID_ARG, "the gradients must be 16-byte aligned");
  DeviceScope dev(h->device);
  if (!dev.ok) return fail(MOE_ERR_DEVICE, "the handle's device cannot be made current");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t nw = static_cast<int64_t>(K) * N * 2;
  h->last_launches = 0;
  std::string why;
  cudaError_t e = cudaSuccess;
  if (T == 0) {
    if (d_gate_w) e = cudaMemsetAsync(d_gate_w, 0, static_cast<size_t>(nw), s);
    if (d_up_w && e == cudaSuccess) e = cudaMemsetAsync(d_up_w, 0, static_cast<size_t>(nw), s);
  } else {
    if (!d_out || !x || !up_w || !save_up || (gated && (!gate_w || !save_gate)))
      return fail(MOE_ERR_INVALID_ARG, "d_out, x, the weights and the saved buffers must not be NULL");
    if (ldx < K || ldx % 8 || !aligned16(x))
      return fail(MOE_ERR_INVALID_ARG, "x needs 16-byte aligned rows: ldx >= in_features, a multiple of 8");
    if (ldd < N || reinterpret_cast<uintptr_t>(d_out) % 2)
      return fail(MOE_ERR_INVALID_ARG, "ldd must be at least out_features");
    if (d_x && lddx < K) return fail(MOE_ERR_INVALID_ARG, "lddx must be at least in_features");
    if (!aligned16(gate_w) || !aligned16(up_w) || !aligned16(save_gate) || !aligned16(save_up))
      return fail(MOE_ERR_INVALID_ARG, "the weights and the saved buffers must be 16-byte aligned");
    struct Range { const void* p; int64_t n; };
    const Range in[6] = {{d_out, span(T, ldd, N)},          {x, span(T, ldx, K)},
                         {gate_w, nw},                      {up_w, nw},
                         {save_gate, 4ll * T * N},          {save_up, 4ll * T * N}};
    const Range outs[3] = {{d_x, span(T, lddx, K)}, {d_gate_w, nw}, {d_up_w, nw}};
    for (int o = 0; o < 3; ++o) {
      for (const Range& r : in)
        if (overlap(outs[o].p, outs[o].n, r.p, r.n)) return fail(MOE_ERR_INVALID_ARG, "a gradient overlaps an input");
      for (int p = 0; p < o; ++p)
        if (overlap(outs[o].p, outs[o].n, outs[p].p, outs[p].n))
          return fail(MOE_ERR_INVALID_ARG, "two gradients overlap");
    }
    const int64_t n = static_cast<int64_t>(T) * (N / 8);
    const int e_vec = aligned16(d_out) && ldd % 8 == 0;
    const unsigned short* ep = static_cast<const unsigned short*>(d_out);
    if (d_x || d_gate_w || d_up_w) {
      e = launch_chained(gated ? k_gated_grad<true> : k_gated_grad<false>, (n + 255) / 256, 256, 0, 1, s, save_gate, save_up,
                         ep, ldd, e_vec, T, N, c.act_dtype, h->dg, h->du);
      ++h->last_launches;
    }
    if (d_x && e == cudaSuccess) {
      GemmCall g;
      g.M = T;
      g.N = K;
      g.parts = gated ? 2 : 1;
      g.K[0] = g.K[1] = N;
      g.b_mn = true;
      g.a[0] = gated ? h->dg : h->du;
      g.a[1] = h->du;
      g.lda = N;
      g.b[0] = gated ? gate_w : up_w;
      g.b[1] = up_w;
      g.ldb = K;
      g.dt = c.act_dtype;
      g.out[0] = d_x;
      g.ldo = lddx;
      e = gemm16_launch(g, *h, s, &h->last_launches, &why);
    }
    if ((d_gate_w || d_up_w) && e == cudaSuccess && T <= OUT_MAX_T) {
      OuterArgs a{};
      a.d[0] = d_gate_w ? h->dg : h->du;
      a.d[1] = h->du;
      a.out[0] = static_cast<unsigned short*>(d_gate_w ? d_gate_w : d_up_w);
      a.out[1] = static_cast<unsigned short*>(d_up_w);
      a.x = static_cast<const unsigned short*>(x);
      a.ldx = ldx;
      a.T = T;
      a.N = N;
      a.K = K;
      e = launch_chained(c.act_dtype == MOE_DTYPE_FP16 ? outer_kernel<true>(T) : outer_kernel<false>(T),
                         dim3(static_cast<unsigned>((N + OUT_ROWS - 1) / OUT_ROWS),
                              static_cast<unsigned>((K + OUT_COLS - 1) / OUT_COLS), d_gate_w && d_up_w ? 2u : 1u),
                         256, 0, 1, s, a);
      ++h->last_launches;
    } else if ((d_gate_w || d_up_w) && e == cudaSuccess) {
      GemmCall g;
      g.M = N;
      g.N = K;
      g.K[0] = T;
      g.a_mn = g.b_mn = true;
      g.batches = (d_gate_w && d_up_w) ? 2 : 1;
      g.a[0] = d_gate_w ? h->dg : h->du;
      g.a[1] = h->du;
      g.lda = N;
      g.b[0] = x;
      g.ldb = ldx;
      g.dt = c.act_dtype;
      g.out[0] = d_gate_w ? d_gate_w : d_up_w;
      g.out[1] = d_up_w;
      g.ldo = K;
      e = gemm16_launch(g, *h, s, &h->last_launches, &why);
    }
  }
  if (e != cudaSuccess) {
    h->last_error = why.empty() ? std::string("launch: ") + cudaGetErrorString(e) : why;
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

extern "C" {

moe_status moe_gated_validate(const moe_gated_config* cfg) {
  return op_entry([&] { return validate_entry(cfg); });
}

moe_status moe_gated_create(const moe_gated_config* cfg, moe_gated** out) {
  moe_gated* h = nullptr;
  const moe_status st = op_entry([&] { return create(cfg, out, h); });
  if (h) {
    h->free_all();
    delete h;
  }
  return st;
}

moe_status moe_gated_forward(moe_gated* h, const void* x, int64_t ldx, int32_t T, const void* gate_w, const void* up_w,
                             void* out, int64_t ldo, float* save_gate, float* save_up, void* stream) {
  return op_entry([&] { return forward(h, x, ldx, T, gate_w, up_w, out, ldo, save_gate, save_up, stream); });
}

moe_status moe_gated_backward(moe_gated* h, const void* d_out, int64_t ldd, int32_t T, const void* x, int64_t ldx,
                              const void* gate_w, const void* up_w, const float* save_gate, const float* save_up,
                              void* d_x, int64_t lddx, void* d_gate_w, void* d_up_w, void* stream) {
  return op_entry([&] { return backward(h, d_out, ldd, T, x, ldx, gate_w, up_w, save_gate, save_up, d_x, lddx, d_gate_w, d_up_w, stream); });
}

moe_status moe_gated_device_status(moe_gated* h, void* stream) {
  return op_entry([&] { return h ? h->read_status(stream) : MOE_ERR_INVALID_ARG; });
}

int64_t moe_gated_device_bytes(const moe_gated* h) { return h ? h->bytes : 0; }

int32_t moe_gated_last_launch_count(const moe_gated* h) { return h ? h->last_launches : 0; }

moe_status moe_gated_destroy(moe_gated* h) {
  if (!h) return MOE_OK;
  {
    DeviceScope dev(h->device);
    cudaDeviceSynchronize();
    h->free_all();
  }
  delete h;
  return MOE_OK;
}

const char* moe_gated_last_error(const moe_gated* h) { return h ? h->last_error.c_str() : g_error.c_str(); }

}  // extern "C"
