// Host side of k_gemm16: tensor maps, tile and K-split choice, launches; and
// what the operator handles share (moe_op_host.h).
#include "moe_gemm16.cuh"

#include <cudaTypedefs.h>   // PFN_cuTensorMapEncodeTiled

#include <algorithm>
#include <mutex>

#include "moe_op_host.h"

namespace moe_op {

cudaError_t OpHandle::alloc(void** p, size_t n) {
  *p = nullptr;
  if (host_alloc_fails()) return cudaErrorMemoryAllocation;
  const cudaError_t e = cudaMalloc(p, n + 256);
  if (e == cudaSuccess) {
    allocs.push_back(*p);
    bytes += static_cast<int64_t>(n);
    host_count_allocs(1);
  }
  return e;
}

void OpHandle::free_all() {
  for (void* p : allocs) {
    cudaFree(p);
    host_count_allocs(-1);
  }
  allocs.clear();
  bytes = 0;
}

moe_status OpHandle::read_status(void* stream) {
  DeviceScope dev(device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int v = 0;
  cudaError_t e = dev.ok ? cudaMemcpyAsync(&v, status, sizeof(v), cudaMemcpyDeviceToHost, s) : cudaErrorInvalidDevice;
  if (e == cudaSuccess) e = cudaMemsetAsync(status, 0, sizeof(v), s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) {
    last_error = std::string("status read: ") + cudaGetErrorString(e);
    return MOE_ERR_CUDA;
  }
  if (v & STATUS_INDEX) {
    last_error = "an index read from data was out of range";
    return MOE_ERR_INDEX;
  }
  return (v & STATUS_TIMEOUT) ? MOE_ERR_TIMEOUT : MOE_OK;
}

moe_status op_device(int* device, int* num_sms, std::string* why) {
  int dev = 0, major = 0, minor = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    *why = "no CUDA device";
    return MOE_ERR_DEVICE;
  }
  if (!(major == 10 && minor == 3)) {
    *why = "device " + std::to_string(dev) + " is not compute capability 10.3";
    return MOE_ERR_DEVICE;
  }
  *device = dev;
  *num_sms = n;
  return MOE_OK;
}

namespace {

using Encoder = PFN_cuTensorMapEncodeTiled_v12000;

Encoder encoder() {
  static std::once_flag once;
  static Encoder fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<Encoder>(p);
  });
  return fn;
}

using Kernel = void (*)(const GemmArgs);

Kernel kernel_of(int cg, bool a_mn, bool b_mn) {
  if (cg == 2) {
    if (a_mn) return k_gemm16<2, true, true>;
    return b_mn ? k_gemm16<2, false, true> : k_gemm16<2, false, false>;
  }
  if (a_mn) return k_gemm16<1, true, true>;
  return b_mn ? k_gemm16<1, false, true> : k_gemm16<1, false, false>;
}

constexpr int kMaxSplit = 16;

struct Choice {
  int cg, bn, ksplit, sub;
};

// Tile shape and K split: the least estimated time in SM clocks.  A launch takes
// its waves over the SMs times a tile's K blocks, each the longest of its MMAs
// (2 BN clocks for 128 rows), its bytes (48 a clock and SM; rows past M are not
// fetched) and the issuing warp's wait and commit (400 clocks a slot), then the last
// accumulators' way out.  A K split adds the partial sums' way through memory and
// a launch: on 333 x 4096 x 3712, two splits of 256-column tiles took 22.0 us where
// one pass of 128-column tiles takes 16.5; on 9 x 11008 x 2048, one pass took 33 us
// where four splits take 12.
Choice choose(const GemmCall& c, int sms, size_t part_bytes) {
  Choice best{1, 64, 1, 2};
  double best_t = 1e30;
  const int nkb = (c.K[0] + 63) / 64 + (c.parts > 1 ? (c.K[1] + 63) / 64 : 0);
  for (int cg = 1; cg <= 2; ++cg) {
    if (cg == 2 && c.M <= 128) continue;
    for (int bn = 64; bn <= 256; bn *= 2) {
      if (c.b_mn && bn / cg < 64) continue;   // MN-major B comes in 64-column blocks
      const int bn_out = c.dual ? bn / 2 : bn, sub = bn == 256 ? 1 : 2;
      const int64_t tiles = static_cast<int64_t>((c.M + cg * 128 - 1) / (cg * 128)) * ((c.N + bn_out - 1) / bn_out) *
                            c.batches;
      const int slots = sms / cg;
      const double bytes = std::min(128, c.M) * 128.0 + bn / cg * 128.0;
      const double kb = std::max({2.0 * bn, bytes / 48.0, 400.0 / sub});
      for (int ks = 1; ks <= kMaxSplit; ++ks) {
        const int64_t ldp = static_cast<int64_t>((c.N + 3) / 4 * 4) * (c.dual ? 2 : 1);
        const double part = static_cast<double>(ks) * c.batches * c.M * ldp * 4;
        if (ks > 1 && (tiles * ks > slots || nkb / ks < 4 || part > static_cast<double>(part_bytes))) break;
        const double waves = static_cast<double>((tiles * ks + slots - 1) / slots);
        const double t = waves * ((nkb + ks - 1) / ks) * kb + bn * 12.0 + (waves - 1) * 1500.0 +
                         (ks > 1 ? 7000.0 + part * 2 / (sms * 30.0) : 0.0);
        if (t < best_t) {
          best_t = t;
          best = Choice{cg, bn, ks, sub};
        }
      }
    }
  }
  return best;
}

}  // namespace

bool encode_rows16(CUtensorMap* m, const void* p, int64_t cols, int64_t rows, int64_t ld, int box_rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t unit[2] = {1, 1};
  return encoder()(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(p), dims, strides, box, unit,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_stack16(CUtensorMap* m, const void* p, int64_t cols, int64_t rows, int64_t ld, int n, int64_t step, int box_rows) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(n)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(step) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t unit[3] = {1, 1, 1};
  return encoder()(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(p), dims, strides, box, unit,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t gemm16_join(const JoinCall& c, cudaStream_t s) {
  GemmFinishArgs f{};
  f.part = c.part;
  f.ld_part = c.ld_part;
  f.ksplit = c.ksplit;
  f.batches = 1;
  f.M = c.M;
  f.N = c.N;
  f.dual = c.dual;
  f.act = c.act;
  f.dt = c.dt;
  f.out[0] = c.out;
  f.ldo = c.ldo;
  f.out_vec = c.ldo % 8 == 0 && reinterpret_cast<uintptr_t>(c.out) % 16 == 0;
  f.nscale_gate = c.nscale_gate;
  f.nscale = c.nscale;
  f.bias = c.bias;
  const int64_t n = static_cast<int64_t>(c.M) * ((c.N + 3) / 4);
  return launch_chained(k_gemm16_finish, (n + 127) / 128, 128, 0, 1, s, f);
}

size_t gemm16_part_bytes(int M, int64_t ld_part, int sms) {
  // K is split only while the splits of all tiles run at once (choose): a tile of at
  // most 128 rows by 256 fp32 columns an SM, 19.9 MB on 152 SMs
  return std::min<size_t>(static_cast<size_t>(sms) * 128 * 256 * 4,
                          static_cast<size_t>(kMaxSplit) * M * ((ld_part + 7) / 4 * 4) * 4);
}

bool encoder_found(std::string* why) {
  if (encoder()) return true;
  *why = "the driver has no tensor-map encoder";
  return false;
}

bool gemm16_setup(std::string* why) {
  if (!encoder_found(why)) return false;
  for (int cg = 1; cg <= 2; ++cg)
    for (int k = 0; k < 3; ++k) {
      const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel_of(cg, k == 2, k >= 1)),
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, GM_SMEM_MAX);
      if (e != cudaSuccess) {
        *why = std::string("kernel attributes: ") + cudaGetErrorString(e);
        return false;
      }
    }
  return true;
}

cudaError_t gemm16_launch(const GemmCall& c, OpHandle& h, cudaStream_t s, int* launches, std::string* why) {
  if (c.M < 1 || c.N < 1) return cudaSuccess;
  const Choice ch = choose(c, h.num_sms, h.part_bytes);
  GemmArgs a{};
  a.M = c.M;
  a.N = c.N;
  a.BN = ch.bn;
  a.dual = c.dual;
  a.batches = c.batches;
  a.parts = c.parts;
  a.kb[0] = (c.K[0] + 63) / 64;
  a.kb[1] = c.parts > 1 ? (c.K[1] + 63) / 64 : 0;
  a.ksplit = ch.ksplit;
  a.dt = c.dt;
  a.act = c.act;
  a.ldo = c.ldo;
  a.out_vec = c.ldo % 16 == 0 ? 2 : c.ldo % 8 == 0 ? 1 : 0;
  for (int i = 0; i < 2; ++i) {
    a.out[i] = c.out[i];
    const uintptr_t at = reinterpret_cast<uintptr_t>(c.out[i]);
    if (at % 16) a.out_vec = 0;
    else if (at % 32 && a.out_vec == 2) a.out_vec = 1;
  }
  a.save_gate = c.save_gate;
  a.save_up = c.save_up;
  a.status = h.status;
  a.part = h.part;
  a.ld_part = static_cast<int64_t>((c.N + 3) / 4 * 4) * (c.dual ? 2 : 1);

  const int na = std::max(c.parts, c.batches), nbm = (c.parts > 1 || c.dual) ? 2 : 1;
  bool ok = true;
  for (int i = 0; i < na && ok; ++i) {
    const int64_t K = c.K[c.parts > 1 ? i : 0];
    ok = c.a_mn ? encode_rows16(&a.ta[i], c.a[i], c.M, K, c.lda, 64) : encode_rows16(&a.ta[i], c.a[i], K, c.M, c.lda, 128);
  }
  for (int i = 0; i < nbm && ok; ++i) {
    const int64_t K = c.K[c.parts > 1 ? i : 0];
    const int box = c.dual ? ch.bn / 2 : ch.bn / ch.cg;
    ok = c.b_mn ? encode_rows16(&a.tb[i], c.b[i], c.N, K, c.ldb, 64) : encode_rows16(&a.tb[i], c.b[i], K, c.N, c.ldb, box);
  }
  if (!ok) {
    *why = "tensor map refused (operands need 16-byte aligned bases and row strides)";
    return cudaErrorInvalidValue;
  }
  a.sub = ch.sub;
  a.stages = GM_MAX_STAGES;
  while (gm_smem_bytes(ch.bn, ch.cg, a.stages, a.sub) > GM_SMEM_MAX) --a.stages;
  const int bn_out = c.dual ? ch.bn / 2 : ch.bn;
  const int64_t units = static_cast<int64_t>((c.M + ch.cg * 128 - 1) / (ch.cg * 128)) * ((c.N + bn_out - 1) / bn_out) *
                        c.batches * ch.ksplit;
  const int64_t workers = std::min<int64_t>(units, h.num_sms / ch.cg);

  cudaError_t e = launch_chained(kernel_of(ch.cg, c.a_mn, c.b_mn), workers * ch.cg, GM_THREADS,
                                 static_cast<size_t>(gm_smem_bytes(ch.bn, ch.cg, a.stages, a.sub)), ch.cg, s, a);
  ++*launches;
  if (e == cudaSuccess && ch.ksplit > 1) {
    GemmFinishArgs f{};
    f.part = a.part;
    f.ld_part = a.ld_part;
    f.ksplit = a.ksplit;
    f.batches = a.batches;
    f.M = a.M;
    f.N = a.N;
    f.dual = a.dual;
    f.act = a.act;
    f.dt = a.dt;
    f.out_vec = a.out_vec;
    f.out[0] = a.out[0];
    f.out[1] = a.out[1];
    f.ldo = a.ldo;
    f.save_gate = a.save_gate;
    f.save_up = a.save_up;
    const int64_t n = static_cast<int64_t>(a.batches) * a.M * ((a.N + 3) / 4);
    e = launch_chained(k_gemm16_finish, (n + 127) / 128, 128, 0, 1, s, f);
    ++*launches;
  }
  if (e != cudaSuccess) *why = std::string("launch: ") + cudaGetErrorString(e);
  return e;
}

}  // namespace moe_op
