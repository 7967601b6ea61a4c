// Linear operators with 4-bit weights (moe_qlinear_* in include/moe_layer.h):
// create-time re-layout, the choice of kernel per call, the C ABI.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "moe_op_host.h"
#include "moe_qgemm.cuh"

using namespace moe_op;

namespace {

thread_local std::string g_error;

// ---------------------------------------------------------------------------
// create-time kernels
// ---------------------------------------------------------------------------

// E4M3 byte -> (exponent + 9) << 3 | mantissa of the normalised magnitude
// (0..17 exponents), 0xFF for NaN; *zero when the magnitude is zero.
__device__ uint32_t e4m3_fields(uint32_t byte, bool* zero) {
  const uint32_t e = (byte >> 3) & 15u, m = byte & 7u;
  *zero = (byte & 0x7Fu) == 0u;
  if ((byte & 0x7Fu) == 0x7Fu) return 0xFFu;
  if (e) return ((e + 2u) << 3) | m;           // 2^(e - 7): exponent + 9 = e + 2
  if (m >= 4u) return (2u << 3) | ((m - 4u) << 1);   // m / 8 * 2^-6, normalised
  if (m >= 2u) return (1u << 3) | ((m - 2u) << 2);
  return 0u;                                    // m = 1: 2^-9
}

// The scale byte a kernel reads (fp4_scale): NVFP4 keeps five exponent and
// three mantissa bits, offset so that the 16-bit float they make is the scale
// times 2^106 (bf16) or 2^7 (fp16); MXFP4 keeps the exponent relative to the
// row's largest e0, as the float 2^(byte - e0 + 126) (bf16) or 2^(byte - e0 +
// 15) (fp16).  A scale below the type's range (2^-252, or 2^-29 of the row's
// largest) counts as zero; the weights themselves, v times it, are whole down to
// 2^-132 (bf16) or 2^-24 (fp16) of the largest scale.
template <int FMT, bool FP16>
__device__ uint32_t scale_byte(uint32_t byte, int e0, bool* zero) {
  if (FMT == W_NVFP4) {
    const uint32_t f = e4m3_fields(byte, zero);
    return f == 0xFFu ? f : (FP16 ? f + (13u << 3) : f);
  }
  const int v = static_cast<int>(byte) - e0 + (FP16 ? 30 : 253);
  *zero = v < 1 || byte == 255u;
  return *zero ? 0u : static_cast<uint32_t>(v);
}

// Per-row factors of the fp4 formats that close a row's sum: the matrix scale
// over the powers of two in the decoded weights, the row's block exponent e0,
// NaN for a row with a NaN scale.  One warp a row.
template <int FMT, bool FP16>
__global__ void ql_rows(const uint8_t* s, const float* matrix_scale, int N, int nblk, int* e0, float* factor) {
  const int row = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32, lane = threadIdx.x & 31;
  if (row >= N) return;
  int top = 0, bad = 0;
  for (int i = lane; i < nblk; i += 32) {
    const int b = s[static_cast<int64_t>(row) * nblk + i];
    if (FMT == W_NVFP4) {
      bad |= (b & 0x7F) == 0x7F;
    } else {
      bad |= b == 255;
      top = max(top, b == 255 ? 0 : b);
    }
  }
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  bad = __any_sync(0xFFFFFFFFu, bad);
  if (lane) return;
  float f;
  if (FMT == W_NVFP4) {
    f = *matrix_scale * (FP16 ? 0x1p7f : 0x1p20f);   // decoded: v s 2^-7 (fp16), v s 2^-20 (bf16)
  } else {
    e0[row] = top;
    // decoded: v 2^(byte - e0) (bf16), v 2^(byte - e0 + 1) (fp16)
    f = ldexpf(1.0f, top - 127 - (FP16 ? 1 : 0));
  }
  factor[row] = bad ? __int_as_float(0x7FC00000) : f;
}

// Row-major codes [N, K/8] and scales -> the streaming order of k_stream:
//   codes  [N/16][chunks][matrices][32 lanes][4 words], rows and columns past
//          the matrix zero
//   scales affine G = 32   [N/16][chunks][matrices][2 groups][8][2] words
//          affine G >= 64  [N/16][groups][matrices][8][2] words (scale low, bias high)
//          nvfp4           [N/16][chunks][matrices][8][4 blocks][2] bytes
//          mxfp4           [N/16][chunks][matrices][8][2 blocks][2] bytes
//          (the pair: rows g and g + 8)
// Word j of lane (g, t) holds four columns of rows g and g + 8: from 16 t + 4 j on,
// or, of affine codes in groups of 32, from 32 (j / 2) + 8 t + 4 (j % 2) on.
// One thread per (tile, chunk, lane) of matrix `m`.
template <int FMT, bool FP16>
__global__ void ql_tile(const uint32_t* q, const void* s, const void* b, const int* e0, int N, int K, int G, int chunks,
                        int mats, int m, uint4* codes, void* scales) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int tiles = (N + 15) / 16;
  if (i >= static_cast<int64_t>(tiles) * chunks * 32) return;
  const int lane = static_cast<int>(i & 31), g = lane >> 2, t = lane & 3;
  const int64_t tcx = i >> 5;
  const int c = static_cast<int>(tcx % chunks);
  const int64_t tile = tcx / chunks;
  const int64_t tc = (tile * chunks + c) * mats + m;
  const int kb = K / G;
  uint32_t words[4];
  uint32_t sbytes[2] = {0u, 0u};   // fp4: the lane's 16 columns share a block
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int col = c * 64 + (FMT == W_AFFINE && G == 32 ? 32 * (j >> 1) + 8 * t + 4 * (j & 1) : 16 * t + 4 * j);
    uint32_t half[2];   // four codes of rows g and g + 8
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t row = tile * 16 + g + 8 * h;
      const bool in = row < N && col < K;
      half[h] = in ? (q[row * (K / 8) + col / 8] >> (4 * (col & 4))) & 0xFFFFu : 0u;
      if (FMT != W_AFFINE && in) {
        const uint32_t by = static_cast<const uint8_t*>(s)[row * kb + col / G];
        bool zero = false;
        sbytes[h] = scale_byte<FMT, FP16>(by, FMT == W_MXFP4 ? e0[row] : 0, &zero);
        if (zero) half[h] = 0u;                                       // a zero scale: zero codes
        if (FMT == W_NVFP4 && (by & 0x80u)) half[h] ^= 0x8888u;       // a negative scale: negated codes
      }
    }
    // A registers: (row g: k 0, 1), (row g + 8: k 0, 1), (row g: k 2, 3), (row g + 8: k 2, 3);
    // code i of the low half word and code i of the high one make register i
    uint32_t w = 0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint32_t src = half[r & 1] >> (8 * (r >> 1));
      const uint32_t c0 = src & 15u, c1 = (src >> 4) & 15u;
      if (FMT == W_AFFINE)
        w |= (c0 << (4 * r)) | (c1 << (16 + 4 * r));
      else
        w |= fp4_place(c0, r, FP16) | (fp4_place(c1, r, FP16) << 16);
    }
    words[j] = w;
  }
  codes[tc * 32 + lane] = make_uint4(words[0], words[1], words[2], words[3]);
  if (FMT == W_AFFINE) {
    if (t == 0 || (G == 32 && t == 1)) {
      // t selects the group of the chunk (G = 32), or the chunk's only one
      const int64_t grp = G == 32 ? static_cast<int64_t>(c) * 2 + t : static_cast<int64_t>(c) * 64 / G;
      const int64_t ng = (static_cast<int64_t>(chunks) * 64 + G - 1) / G;
      uint32_t v[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t row = tile * 16 + g + 8 * h;
        const bool in = row < N && grp < kb;
        const uint32_t sv = in ? static_cast<const unsigned short*>(s)[row * kb + grp] : 0u;
        const uint32_t bv = in ? static_cast<const unsigned short*>(b)[row * kb + grp] : 0u;
        v[h] = sv | (bv << 16);
      }
      const int64_t o = G == 32 ? tc * 16 + t * 8 + g : ((tile * ng + grp) * mats + m) * 8 + g;
      static_cast<uint2*>(scales)[o] = make_uint2(v[0], v[1]);
    }
  } else if (FMT == W_NVFP4 || t % 2 == 0) {
    const int64_t o = FMT == W_NVFP4 ? tc * 32 + lane : tc * 16 + g * 2 + t / 2;
    static_cast<unsigned short*>(scales)[o] = static_cast<unsigned short>(sbytes[0] | (sbytes[1] << 8));
  }
}

}  // namespace

struct moe_qlinear : OpHandle {
  moe_qlinear_config cfg{};
  int mats = 1, chunks = 0;
  uint4* codes = nullptr;
  void* scales = nullptr;
  float* factor[2] = {nullptr, nullptr};   // fp4 per-row factors: gate, up
  void* bias = nullptr;
};

namespace {

moe_status validate(const moe_qlinear_config* c, const moe_qlinear_weights* w, std::string* why) {
  auto fail = [&](moe_status s, const char* msg) {
    *why = msg;
    return s;
  };
  if (!c) return fail(MOE_ERR_INVALID_ARG, "config is NULL");
  if (c->in_features < 1 || c->out_features < 1 || c->max_tokens < 1)
    return fail(MOE_ERR_INVALID_ARG, "in_features, out_features and max_tokens must be positive");
  if (c->act != MOE_QLINEAR_SWIGLU && c->act != MOE_QLINEAR_RELU2 && c->act != MOE_QLINEAR_NONE)
    return fail(MOE_ERR_INVALID_ARG, "unknown act");
  if (c->act_dtype < 0 || c->act_dtype > 2 || c->scale_dtype < 0 || c->scale_dtype > 2)
    return fail(MOE_ERR_INVALID_ARG, "unknown dtype");
  const int f = c->weight_format, G = c->group_size;
  if (f != MOE_WFMT_AFFINE && f != MOE_WFMT_NVFP4 && f != MOE_WFMT_MXFP4)
    return fail(MOE_ERR_INVALID_ARG, "unknown weight_format");
  if (f == MOE_WFMT_NVFP4 ? G != 16 : f == MOE_WFMT_MXFP4 ? G != 32 : (G != 32 && G != 64 && G != 128))
    return fail(MOE_ERR_SHAPE, "group_size must be 32, 64 or 128 (NVFP4: 16, MXFP4: 32)");
  if (c->in_features % G) return fail(MOE_ERR_SHAPE, "in_features must be a multiple of group_size");
  if (c->act_dtype == MOE_DTYPE_FP32) return fail(MOE_ERR_UNSUPPORTED, "fp32 activations");
  if (c->scale_dtype == MOE_DTYPE_FP32 && f == MOE_WFMT_AFFINE) return fail(MOE_ERR_UNSUPPORTED, "fp32 scales");
  if (c->in_features > 65536) return fail(MOE_ERR_UNSUPPORTED, "in_features above 65536");
  if (c->out_features > (1 << 24)) return fail(MOE_ERR_UNSUPPORTED, "out_features above 2^24");
  if (c->has_bias && c->act != MOE_QLINEAR_NONE)
    return fail(MOE_ERR_UNSUPPORTED, "a bias is defined without an activation only");
  if (w) {
    const bool need_b = f != MOE_WFMT_MXFP4, gated = c->act == MOE_QLINEAR_SWIGLU;
    if (!w->q || !w->s || (need_b && !w->b)) return fail(MOE_ERR_INVALID_ARG, "weights missing");
    if (gated && (!w->gate_q || !w->gate_s || (need_b && !w->gate_b)))
      return fail(MOE_ERR_INVALID_ARG, "SwiGLU needs gate weights");
    if (!gated && (w->gate_q || w->gate_s || w->gate_b)) return fail(MOE_ERR_SHAPE, "gate weights without SwiGLU");
    if (c->has_bias && !w->bias) return fail(MOE_ERR_INVALID_ARG, "bias missing");
    if (!c->has_bias && w->bias) return fail(MOE_ERR_SHAPE, "a bias given with has_bias = 0");
  }
  return MOE_OK;
}

// ---- k_stream launches ----

using StreamKernel = void (*)(const StreamArgs);

template <int FMT, bool FP16, int GB>
StreamKernel stream_kernel_g(bool gated, int nt) {
  if (gated) return nt == 1 ? k_stream<FMT, FP16, true, 1, GB> : k_stream<FMT, FP16, true, 2, GB>;
  return nt == 1 ? k_stream<FMT, FP16, false, 1, GB> : k_stream<FMT, FP16, false, 2, GB>;
}
template <bool FP16>
StreamKernel stream_kernel_t(const moe_qlinear_config& c, int nt) {
  const bool gated = c.act == MOE_QLINEAR_SWIGLU;
  if (c.weight_format == MOE_WFMT_NVFP4) return stream_kernel_g<W_NVFP4, FP16, 4>(gated, nt);
  if (c.weight_format == MOE_WFMT_MXFP4) return stream_kernel_g<W_MXFP4, FP16, 4>(gated, nt);
  return c.group_size == 32 ? stream_kernel_g<W_AFFINE, FP16, 2>(gated, nt) : stream_kernel_g<W_AFFINE, FP16, 4>(gated, nt);
}
StreamKernel stream_kernel(const moe_qlinear_config& c, int nt) {
  return c.act_dtype == MOE_DTYPE_FP16 ? stream_kernel_t<true>(c, nt) : stream_kernel_t<false>(c, nt);
}

int stream_format(const moe_qlinear_config& c) {
  return c.weight_format == MOE_WFMT_NVFP4 ? W_NVFP4 : c.weight_format == MOE_WFMT_MXFP4 ? W_MXFP4 : W_AFFINE;
}

// k_stream's plan for T rows; false when the call goes to the tensor-core GEMM:
// more rows than it takes, or wider ones than fit beside its rings.
bool stream_plan(const moe_qlinear& h, int T, StreamPlan* P) {
  const moe_qlinear_config& c = h.cfg;
  return T <= ST_MAX_T && st_plan(stream_format(c), h.mats == 2, c.group_size == 32 ? 2 : 4, h.chunks, T, c.out_features,
                                  h.num_sms, P);
}

cudaError_t run_stream(moe_qlinear& h, const StreamPlan& P, const void* x, int64_t ldx, int T, void* out, int64_t ldo,
                       cudaStream_t s) {
  const moe_qlinear_config& c = h.cfg;
  StreamArgs a{};
  a.codes = h.codes;
  a.scales = h.scales;
  a.nscale_gate = h.factor[0];
  a.nscale = h.factor[1];
  a.bias = h.bias;
  a.x = x;
  a.ldx = ldx;
  a.out = out;
  a.ldo = ldo;
  a.K = c.in_features;
  a.N = c.out_features;
  a.T = T;
  a.chunks = h.chunks;
  a.group = c.group_size;
  a.act = c.act;
  a.sdt = c.scale_dtype;
  a.depth = P.depth;
  a.status = h.status;
  ++h.last_launches;
  return launch_chained(stream_kernel(c, T > 8 ? 2 : 1), P.grid, ST_THREADS, static_cast<size_t>(P.smem), 1, s, a);
}

// ---- k_qgemm launches ----

using QGemmKernel = void (*)(const QGemmArgs);

template <bool FP16, bool GATED>
QGemmKernel qgemm_kernel_t(const moe_qlinear_config& c) {
  if (c.weight_format == MOE_WFMT_NVFP4) return k_qgemm<W_NVFP4, FP16, GATED, 4>;
  if (c.weight_format == MOE_WFMT_MXFP4) return k_qgemm<W_MXFP4, FP16, GATED, 4>;
  return c.group_size == 32 ? k_qgemm<W_AFFINE, FP16, GATED, 2> : k_qgemm<W_AFFINE, FP16, GATED, 4>;
}
QGemmKernel qgemm_kernel(const moe_qlinear_config& c) {
  const bool gated = c.act == MOE_QLINEAR_SWIGLU;
  if (c.act_dtype == MOE_DTYPE_FP16) return gated ? qgemm_kernel_t<true, true>(c) : qgemm_kernel_t<true, false>(c);
  return gated ? qgemm_kernel_t<false, true>(c) : qgemm_kernel_t<false, false>(c);
}

QGemmPlan qgemm_plan(const moe_qlinear& h, int T) {
  const moe_qlinear_config& c = h.cfg;
  return qg_plan(stream_format(c), c.group_size == 32 ? 2 : 4, h.mats, h.chunks, T, c.out_features, h.num_sms, h.part_bytes);
}

cudaError_t run_qgemm(moe_qlinear& h, const void* x, int64_t ldx, int T, void* out, int64_t ldo, cudaStream_t s,
                      std::string* why) {
  const moe_qlinear_config& c = h.cfg;
  const QGemmPlan P = qgemm_plan(h, T);
  QGemmArgs a{};
  if (!encode_rows16(&a.tx, x, c.in_features, T, ldx, P.ntok)) {
    *why = "tensor map of x refused";
    return cudaErrorInvalidValue;
  }
  a.codes = h.codes;
  a.scales = h.scales;
  a.nscale_gate = h.factor[0];
  a.nscale = h.factor[1];
  a.bias = h.bias;
  a.out = out;
  a.ldo = ldo;
  a.out_vec = ldo % 4 == 0 && reinterpret_cast<uintptr_t>(out) % 8 == 0;
  a.part = h.part;
  a.ld_part = static_cast<int64_t>((c.out_features + 3) / 4 * 4) * h.mats;
  a.status = h.status;
  a.T = T;
  a.N = c.out_features;
  a.chunks = h.chunks;
  a.group = c.group_size;
  a.sdt = c.scale_dtype;
  a.act = c.act;
  a.ntok = P.ntok;
  a.ksplit = P.ksplit;
  a.slots = P.slots;
  a.depth = P.depth;
  const size_t smem = static_cast<size_t>(qg_smem_bytes(stream_format(c), c.group_size == 32 ? 2 : 4, h.mats, P.ntok,
                                                        P.slots, P.depth));
  cudaError_t e = launch_chained(qgemm_kernel(c), std::min(P.units, h.num_sms), QG_THREADS, smem, 1, s, a);
  ++h.last_launches;
  if (e == cudaSuccess && P.ksplit > 1) {
    JoinCall j;
    j.part = a.part;
    j.ld_part = a.ld_part;
    j.ksplit = a.ksplit;
    j.M = T;
    j.N = a.N;
    j.dual = h.mats == 2;
    j.dt = c.act_dtype;
    j.act = c.act;
    j.out = out;
    j.ldo = ldo;
    j.nscale_gate = a.nscale_gate;
    j.nscale = a.nscale;
    j.bias = a.bias;
    e = gemm16_join(j, s);
    ++h.last_launches;
  }
  return e;
}

// ---- create-time launches ----

template <int FMT, bool FP16>
cudaError_t relay(moe_qlinear& h, const moe_qlinear_weights& w, int* e0, cudaStream_t s) {
  const moe_qlinear_config& c = h.cfg;
  const int N = c.out_features, K = c.in_features, G = c.group_size;
  for (int m = 0; m < h.mats; ++m) {
    const bool gate = h.mats == 2 && m == 0;
    const uint32_t* q = gate ? w.gate_q : w.q;
    const void* sc = gate ? w.gate_s : w.s;
    const void* b = gate ? w.gate_b : w.b;
    if constexpr (FMT != W_AFFINE)
      ql_rows<FMT, FP16><<<(N + 7) / 8, 256, 0, s>>>(static_cast<const uint8_t*>(sc), static_cast<const float*>(b), N,
                                                     K / G, e0, h.factor[gate ? 0 : 1]);
    const int64_t n = static_cast<int64_t>((N + 15) / 16) * h.chunks * 32;
    ql_tile<FMT, FP16><<<static_cast<unsigned>((n + 255) / 256), 256, 0, s>>>(q, sc, b, e0, N, K, G, h.chunks, h.mats, m,
                                                                             h.codes, h.scales);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

#define QL_BY_FORMAT(h, fn, ...)                                                              \
  ((h).cfg.act_dtype == MOE_DTYPE_FP16                                                        \
       ? ((h).cfg.weight_format == MOE_WFMT_NVFP4   ? fn<W_NVFP4, true>(__VA_ARGS__)          \
          : (h).cfg.weight_format == MOE_WFMT_MXFP4 ? fn<W_MXFP4, true>(__VA_ARGS__)          \
                                                    : fn<W_AFFINE, true>(__VA_ARGS__))        \
       : ((h).cfg.weight_format == MOE_WFMT_NVFP4   ? fn<W_NVFP4, false>(__VA_ARGS__)         \
          : (h).cfg.weight_format == MOE_WFMT_MXFP4 ? fn<W_MXFP4, false>(__VA_ARGS__)         \
                                                    : fn<W_AFFINE, false>(__VA_ARGS__)))

}  // namespace

static moe_status validate_entry(const moe_qlinear_config* cfg, const moe_qlinear_weights* w) {
  std::string why;
  const moe_status st = validate(cfg, w, &why);
  if (st != MOE_OK) g_error = why;
  return st;
}

// (h: the handle while it is not the caller's, for the entry point to free when an exception ends this)
static moe_status create(const moe_qlinear_config* cfg, const moe_qlinear_weights* w, void* stream,
                              moe_qlinear** out, moe_qlinear*& h) {
  if (out) *out = nullptr;
  std::string why;
  moe_status st = validate(cfg, w, &why);
  if (st == MOE_OK && (!out || !w)) {
    st = MOE_ERR_INVALID_ARG;
    why = "out and weights must not be NULL";
  }
  int device = 0, sms = 0;
  if (st == MOE_OK) st = op_device(&device, &sms, &why);
  if (st != MOE_OK) {
    g_error = why;
    return st;
  }
  h = new (std::nothrow) moe_qlinear();
  if (!h) {
    g_error = "host memory";
    return MOE_ERR_OOM;
  }
  h->device = device;
  h->num_sms = sms;
  h->cfg = *cfg;
  const moe_qlinear_config& c = h->cfg;
  const bool fp4 = c.weight_format != MOE_WFMT_AFFINE;
  h->mats = c.act == MOE_QLINEAR_SWIGLU ? 2 : 1;
  h->chunks = (c.in_features + 63) / 64;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t tc = static_cast<size_t>((c.out_features + 15) / 16) * h->chunks * h->mats;   // 16 x 64 tiles
  const size_t chunk_scales = c.weight_format == MOE_WFMT_MXFP4 ? 32 : c.weight_format == MOE_WFMT_NVFP4 ? 64
                              : c.group_size == 32              ? 128
                                                                : 64;
  int* e0 = nullptr;
  cudaError_t e = h->alloc(reinterpret_cast<void**>(&h->codes), tc * 512);
  if (e == cudaSuccess) e = h->alloc(&h->scales, tc * chunk_scales);
  if (e == cudaSuccess) e = h->alloc(reinterpret_cast<void**>(&h->status), 64);
  if (e == cudaSuccess) e = cudaMemsetAsync(h->status, 0, 64, s);
  if (fp4 && e == cudaSuccess) e = h->alloc(reinterpret_cast<void**>(&e0), static_cast<size_t>(c.out_features) * 4);
  for (int m = 2 - h->mats; fp4 && m < 2 && e == cudaSuccess; ++m)
    e = h->alloc(reinterpret_cast<void**>(&h->factor[m]), static_cast<size_t>(c.out_features) * 4);
  if (c.has_bias && e == cudaSuccess) {
    e = h->alloc(&h->bias, static_cast<size_t>(c.out_features) * 2);
    if (e == cudaSuccess)
      e = cudaMemcpyAsync(h->bias, w->bias, static_cast<size_t>(c.out_features) * 2, cudaMemcpyDeviceToDevice, s);
  }
  StreamPlan plan;
  bool streamed = true;   // whether k_stream takes every call
  for (int t = 1; t <= c.max_tokens && streamed; ++t) streamed = stream_plan(*h, t, &plan);
  if (!streamed && e == cudaSuccess) {
    if (!encoder_found(&why)) {
      st = MOE_ERR_CUDA;
      e = cudaErrorUnknown;
    }
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(reinterpret_cast<const void*>(qgemm_kernel(c)),
                               cudaFuncAttributeMaxDynamicSharedMemorySize, QG_SMEM_MAX);
    h->part_bytes = qg_part_bytes(stream_format(c), c.group_size == 32 ? 2 : 4, h->mats, h->chunks, c.max_tokens,
                                  c.out_features, sms);
    if (e == cudaSuccess && h->part_bytes) e = h->alloc(reinterpret_cast<void**>(&h->part), h->part_bytes);
  }
  for (int nt = 1; nt <= 2 && e == cudaSuccess; ++nt)
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(stream_kernel(c, nt)),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, ST_SMEM_MAX);
  if (e == cudaSuccess) e = QL_BY_FORMAT(*h, relay, *h, *w, e0, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) {
    if (why.empty()) why = std::string("create: ") + cudaGetErrorString(e);
    cudaStreamSynchronize(s);
    h->free_all();
    delete h;
    h = nullptr;
    g_error = why;
    return st != MOE_OK ? st : e == cudaErrorMemoryAllocation ? MOE_ERR_OOM : MOE_ERR_CUDA;
  }
  *out = h;
  h = nullptr;
  return MOE_OK;
}

static moe_status forward(moe_qlinear* h, const void* x, int64_t ldx, int32_t T, void* out, int64_t ldo,
                               void* stream) {
  if (!h) return MOE_ERR_INVALID_ARG;
  const moe_qlinear_config& c = h->cfg;
  auto fail = [&](moe_status st, const char* msg) {
    h->last_error = msg;
    return st;
  };
  if (T < 0 || T > c.max_tokens) return fail(MOE_ERR_INVALID_ARG, "T must be in 0..max_tokens");
  if (T == 0) {
    h->last_launches = 0;
    return MOE_OK;
  }
  if (!x || !out) return fail(MOE_ERR_INVALID_ARG, "x and out must not be NULL");
  if (ldx < c.in_features || ldx % 8 || reinterpret_cast<uintptr_t>(x) % 16)
    return fail(MOE_ERR_INVALID_ARG, "x needs 16-byte aligned rows: ldx >= in_features, a multiple of 8");
  if (ldo < c.out_features || reinterpret_cast<uintptr_t>(out) % 2)
    return fail(MOE_ERR_INVALID_ARG, "ldo must be at least out_features");
  if (rows_overlap(x, ldx, c.in_features, out, ldo, c.out_features, T))
    return fail(MOE_ERR_INVALID_ARG, "x and out overlap");
  DeviceScope dev(h->device);
  if (!dev.ok) return fail(MOE_ERR_DEVICE, "the handle's device cannot be made current");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  h->last_launches = 0;
  std::string why;
  cudaError_t e;
  StreamPlan plan;
  if (stream_plan(*h, T, &plan)) {
    e = run_stream(*h, plan, x, ldx, T, out, ldo, s);
  } else {
    e = run_qgemm(*h, x, ldx, T, out, ldo, s, &why);
  }
  if (e != cudaSuccess) {
    h->last_error = why.empty() ? std::string("launch: ") + cudaGetErrorString(e) : why;
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

extern "C" {

moe_status moe_qlinear_validate(const moe_qlinear_config* cfg, const moe_qlinear_weights* w) {
  return op_entry([&] { return validate_entry(cfg, w); });
}

moe_status moe_qlinear_create(const moe_qlinear_config* cfg, const moe_qlinear_weights* w, void* stream,
                              moe_qlinear** out) {
  moe_qlinear* h = nullptr;
  const moe_status st = op_entry([&] { return create(cfg, w, stream, out, h); });
  if (h) {
    h->free_all();
    delete h;
  }
  return st;
}

moe_status moe_qlinear_forward(moe_qlinear* h, const void* x, int64_t ldx, int32_t T, void* out, int64_t ldo,
                               void* stream) {
  return op_entry([&] { return forward(h, x, ldx, T, out, ldo, stream); });
}

moe_status moe_qlinear_device_status(moe_qlinear* h, void* stream) {
  return op_entry([&] { return h ? h->read_status(stream) : MOE_ERR_INVALID_ARG; });
}

int64_t moe_qlinear_device_bytes(const moe_qlinear* h) { return h ? h->bytes : 0; }

int32_t moe_qlinear_last_launch_count(const moe_qlinear* h) { return h ? h->last_launches : 0; }

moe_status moe_qlinear_destroy(moe_qlinear* h) {
  if (!h) return MOE_OK;
  {
    DeviceScope dev(h->device);
    cudaDeviceSynchronize();
    h->free_all();
  }
  delete h;
  return MOE_OK;
}

const char* moe_qlinear_last_error(const moe_qlinear* h) { return h ? h->last_error.c_str() : g_error.c_str(); }

}  // extern "C"
