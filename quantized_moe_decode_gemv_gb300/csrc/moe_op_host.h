// Host side shared by the operator handles (moe_qlinear.cu, moe_gated.cu):
// tracked allocations, the device a handle lives on, the GEMM launcher.
#pragma once

#include <cuda.h>   // CUtensorMap
#include <cuda_runtime.h>
#include <stdint.h>

#include <new>
#include <string>
#include <vector>

#include "moe_layer.h"

namespace moe_op {

// Allocation accounting shared with the layer handles (moe_layer.cu): whether
// the injected failure is due, and the live count of moe_debug_live_allocations.
bool host_alloc_fails();
void host_count_allocs(int delta);

// Makes `device` current for a scope.
struct DeviceScope {
  int prev = -1;
  bool ok = true;
  explicit DeviceScope(int device) {
    int cur = -1;
    if (cudaGetDevice(&cur) != cudaSuccess) {
      ok = false;
    } else if (cur != device) {
      prev = cur;
      ok = cudaSetDevice(device) == cudaSuccess;
    }
  }
  ~DeviceScope() {
    if (prev >= 0) cudaSetDevice(prev);
  }
  DeviceScope(const DeviceScope&) = delete;
  DeviceScope& operator=(const DeviceScope&) = delete;
};

// Runs the body of a C entry point: no C++ exception leaves it.
template <typename F>
moe_status op_entry(F&& body) noexcept {
  try {
    return body();
  } catch (const std::bad_alloc&) {
    return MOE_ERR_OOM;   // host memory
  } catch (...) {
    return MOE_ERR_CUDA;
  }
}

// What every operator handle has.
struct OpHandle {
  int device = -1;
  int num_sms = 0;
  std::vector<void*> allocs;
  int64_t bytes = 0;
  std::string last_error;
  int last_launches = 0;
  int* status = nullptr;      // device word: STATUS_* bits
  float* part = nullptr;      // partial sums of products whose K is split
  size_t part_bytes = 0;

  OpHandle() { allocs.reserve(16); }
  cudaError_t alloc(void** p, size_t n);
  void free_all();
  moe_status read_status(void* stream);
};

// The current device and its SM count, or MOE_ERR_DEVICE with the reason.
moe_status op_device(int* device, int* num_sms, std::string* why);

// Whether T rows of ca 16-bit elements lda apart at a meet T rows of cb elements
// ldb apart at b.  Column ranges of one buffer (equal row strides) may interleave.
inline bool rows_overlap(const void* a, int64_t lda, int64_t ca, const void* b, int64_t ldb, int64_t cb, int64_t T) {
  const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
  if (!x || !y || T < 1) return false;
  if (x >= y + ((T - 1) * ldb + cb) * 2 || y >= x + ((T - 1) * lda + ca) * 2) return false;
  if (lda != ldb || T == 1) return true;
  const int64_t row = lda * 2;
  const int64_t off = ((y - x) % row + row) % row;   // b's first column, seen from a's rows
  return off < ca * 2 || off + cb * 2 > row;
}

// A launch that may begin while the kernel before it in the stream ends
// (programmatic dependent launch).  Every kernel launched so waits for that
// kernel (griddepcontrol.wait) before it touches what others write or read.
template <typename... P, typename... A>
cudaError_t launch_chained(void (*k)(P...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t s, const A&... a) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k, a...);
}

template <typename... P, typename... A>
cudaError_t launch_chained(void (*k)(P...), int64_t grid, int threads, size_t smem, int cluster, cudaStream_t s, const A&... a) {
  return launch_chained(k, dim3(static_cast<unsigned>(grid)), threads, smem, cluster, s, a...);
}

struct GemmCall {
  int M = 0, N = 0;
  int parts = 1, batches = 1;
  int K[2] = {0, 0};          // extent of each K part
  bool dual = false, a_mn = false, b_mn = false;
  const void* a[2] = {nullptr, nullptr};
  int64_t lda = 0;            // elements between rows as they lie in memory
  const void* b[2] = {nullptr, nullptr};
  int64_t ldb = 0;
  int dt = 0, act = 2;
  void* out[2] = {nullptr, nullptr};
  int64_t ldo = 0;
  float *save_gate = nullptr, *save_up = nullptr;
};

// Partial sums of a split K ([ksplit][M][ld_part] fp32, SwiGLU: gate at 0, up at
// ld_part / 2) added in order, and the epilogue.
struct JoinCall {
  const float* part = nullptr;
  int64_t ld_part = 0;
  int ksplit = 1, M = 0, N = 0;
  bool dual = false;
  int dt = 0, act = 2;
  void* out = nullptr;
  int64_t ldo = 0;
  const float *nscale_gate = nullptr, *nscale = nullptr;
  const void* bias = nullptr;
};
cudaError_t gemm16_join(const JoinCall& c, cudaStream_t s);

// Tensor map of a 16-bit matrix of `rows` memory rows of `cols` elements, ld
// apart; boxes of 64 columns (128 bytes, swizzled) by box_rows rows.  Elements
// outside read as zero.  False when the driver refuses it.  Needs encoder_found().
bool encode_rows16(CUtensorMap* m, const void* p, int64_t cols, int64_t rows, int64_t ld, int box_rows);

// Whether the driver has a tensor-map encoder (looked up once); false with the reason.
bool encoder_found(std::string* why);

// Launches the product on `s` (asynchronous); counts its kernel launches.
cudaError_t gemm16_launch(const GemmCall& c, OpHandle& h, cudaStream_t s, int* launches, std::string* why);
// Once per create, with the handle's device current: kernel attributes, the
// tensor-map encoder; false with the reason.
bool gemm16_setup(std::string* why);
// Bytes of OpHandle::part for the K splits of gemm16_launch with at most M rows
// and ld_part partial columns.
size_t gemm16_part_bytes(int M, int64_t ld_part, int sms);

}  // namespace moe_op
