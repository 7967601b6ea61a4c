// Linear operators with 4-bit weights (moe_qlinear_* in include/moe_layer.h):
// create-time re-layout, the choice of kernel per call, the C ABI.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "moe_op_host.h"
#include "moe_stream.cuh"

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
// largest) counts as zero.
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

template <int FMT>
__device__ __forceinline__ int ql_column(int j, int t) {
  return FMT == W_AFFINE ? 32 * (j >> 1) + 8 * t + 4 * (j & 1) : 16 * t + 4 * j;
}

// Row-major codes [N, K/8] and scales -> the streaming order of k_stream:
//   codes  [N/16][chunks][matrices][32 lanes][4 words], rows and columns past
//          the matrix zero
//   scales affine G = 32   [N/16][chunks][matrices][2 groups][8][2] words
//          affine G >= 64  [N/16][groups][matrices][8][2] words (scale low, bias high)
//          nvfp4           [N/16][chunks][matrices][8][4 blocks][2] bytes
//          mxfp4           [N/16][chunks][matrices][8][2 blocks][2] bytes
//          (the pair: rows g and g + 8)
// Word j of lane (g, t) holds four columns of rows g and g + 8: from 32 (j / 2)
// + 8 t + 4 (j % 2) on in an affine chunk, from 16 t + 4 j on in an fp4 one.
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
    const int col = c * 64 + ql_column<FMT>(j, t);
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

// The re-laid weights as 16-bit rows [matrix][N][chunks * 64] for k_gemm16: the
// affine value rounded once to the type (a relative error of at most 2^-9 or
// 2^-12 beside the output's own rounding of that size), the fp4 value times its
// block scale exactly.  One thread per (tile, chunk, matrix, lane).
template <int FMT, bool FP16>
__global__ void __launch_bounds__(256) ql_expand(const uint4* codes, const void* scales, int N, int G, int chunks,
                                                 int mats, int sdt, unsigned short* out) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int tiles = (N + 15) / 16;
  // (the call before this one may still read `out`)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  if (i >= static_cast<int64_t>(tiles) * chunks * mats * 32) return;
  constexpr int DT = FP16 ? DT_FP16 : DT_BF16;
  const int lane = static_cast<int>(i & 31), g = lane >> 2, t = lane & 3;
  const int64_t tc = i >> 5;
  const int m = static_cast<int>(tc % mats);
  const int64_t tcx = tc / mats;
  const int c = static_cast<int>(tcx % chunks);
  const int64_t tile = tcx / chunks;
  const uint4 w = codes[i];
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
  const int64_t ld = static_cast<int64_t>(chunks) * 64;
  const int64_t r0 = tile * 16 + g;
  unsigned short* p0 = out + (static_cast<int64_t>(m) * N + r0) * ld + c * 64;
  unsigned short* p1 = p0 + 8 * ld;
#pragma unroll
  for (int jj = 0; jj < 2; ++jj) {
    // words 2 jj and 2 jj + 1: eight consecutive columns of two rows
    uint32_t a[2][4];
    if constexpr (FMT == W_AFFINE) {
      const int64_t grp = (static_cast<int64_t>(c) * 64 + jj * 32) / G;
      const int64_t ng = (static_cast<int64_t>(chunks) * 64 + G - 1) / G;
      const int64_t o = G == 32 ? tc * 16 + jj * 8 + g : ((tile * ng + grp) * mats + m) * 8 + g;
      const uint2 v = __ldg(static_cast<const uint2*>(scales) + o);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        affine_word<FP16>(ws[2 * jj + j], a[j]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t sv = (r & 1) ? v.y : v.x;
          const float s = lo16(sv, sdt), b = hi16(sv, sdt), off = affine_offset<FP16>();
          a[j][r] = pack2(fmaf(lo16(a[j][r], DT) - off, s, b), fmaf(hi16(a[j][r], DT) - off, s, b), DT);
        }
      }
    } else {
      const int64_t o = FMT == W_NVFP4 ? tc * 32 + lane : tc * 16 + g * 2 + (t >> 1);
      const uint32_t sb = __ldg(static_cast<const unsigned short*>(scales) + o);
      const uint32_t s0 = fp4_scale<FMT, FP16>(sb, 0), s1 = fp4_scale<FMT, FP16>(sb, 1);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        fp4_word<FP16>(ws[2 * jj + j], a[j]);
#pragma unroll
        for (int r = 0; r < 4; ++r) a[j][r] = mul2<FP16>(a[j][r], (r & 1) ? s1 : s0);
      }
    }
    const int col = ql_column<FMT>(2 * jj, t);
    if (r0 < N) *reinterpret_cast<uint4*>(p0 + col) = make_uint4(a[0][0], a[0][2], a[1][0], a[1][2]);
    if (r0 + 8 < N) *reinterpret_cast<uint4*>(p1 + col) = make_uint4(a[0][1], a[0][3], a[1][1], a[1][3]);
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
  unsigned short* wide = nullptr;          // 16-bit weights of one call that k_stream does not take
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

template <int FMT, bool FP16>
cudaError_t expand(moe_qlinear& h, cudaStream_t s) {
  const moe_qlinear_config& c = h.cfg;
  const int64_t n = static_cast<int64_t>((c.out_features + 15) / 16) * h.chunks * h.mats * 32;
  ++h.last_launches;
  return launch_chained(ql_expand<FMT, FP16>, (n + 255) / 256, 256, 0, 1, s, static_cast<const uint4*>(h.codes),
                        static_cast<const void*>(h.scales), c.out_features, c.group_size, h.chunks, h.mats,
                        c.scale_dtype, h.wide);
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

extern "C" {

moe_status moe_qlinear_validate(const moe_qlinear_config* cfg, const moe_qlinear_weights* w) {
  std::string why;
  const moe_status st = validate(cfg, w, &why);
  if (st != MOE_OK) g_error = why;
  return st;
}

moe_status moe_qlinear_create(const moe_qlinear_config* cfg, const moe_qlinear_weights* w, void* stream,
                              moe_qlinear** out) {
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
  moe_qlinear* h = new (std::nothrow) moe_qlinear();
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
  if (!stream_plan(*h, c.max_tokens, &plan) && e == cudaSuccess) {
    if (!gemm16_setup(&why)) {
      st = MOE_ERR_CUDA;
      e = cudaErrorUnknown;
    }
    if (e == cudaSuccess)
      e = h->alloc(reinterpret_cast<void**>(&h->wide), static_cast<size_t>(h->mats) * c.out_features * h->chunks * 128);
    h->part_bytes = gemm16_part_bytes(c.max_tokens, static_cast<int64_t>(h->mats) * c.out_features);
    if (e == cudaSuccess) e = h->alloc(reinterpret_cast<void**>(&h->part), h->part_bytes);
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
    g_error = why;
    return st != MOE_OK ? st : e == cudaErrorMemoryAllocation ? MOE_ERR_OOM : MOE_ERR_CUDA;
  }
  *out = h;
  return MOE_OK;
}

moe_status moe_qlinear_forward(moe_qlinear* h, const void* x, int64_t ldx, int32_t T, void* out, int64_t ldo,
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
    e = QL_BY_FORMAT(*h, expand, *h, s);
    if (e == cudaSuccess) {
      GemmCall g;
      const int64_t ld = static_cast<int64_t>(h->chunks) * 64;
      g.M = T;
      g.N = c.out_features;
      g.K[0] = c.in_features;
      g.dual = h->mats == 2;
      g.a[0] = x;
      g.lda = ldx;
      g.b[0] = h->wide;
      g.b[1] = h->wide + static_cast<int64_t>(c.out_features) * ld;
      g.ldb = ld;
      g.dt = c.act_dtype;
      g.act = c.act;
      g.out[0] = out;
      g.ldo = ldo;
      g.nscale_gate = h->factor[0];
      g.nscale = h->factor[1];
      g.bias = h->bias;
      e = gemm16_launch(g, *h, s, &h->last_launches, &why);
    }
  }
  if (e != cudaSuccess) {
    h->last_error = why.empty() ? std::string("launch: ") + cudaGetErrorString(e) : why;
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

moe_status moe_qlinear_device_status(moe_qlinear* h, void* stream) {
  return h ? h->read_status(stream) : MOE_ERR_INVALID_ARG;
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
