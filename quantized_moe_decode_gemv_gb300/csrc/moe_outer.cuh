// Weight gradients of few token rows (k_outer):  dW[n, k] = sum_t d[t, n] x[t, k]
// for t < T <= 48, both gradients of a gated block in one launch.
//
// Writing dW is all the time there is: with T = 9 the products are 18 flops for
// each 2 bytes written.  A GEMM tile spends longer filling its pipeline and
// handing its accumulators over than on its one or two K blocks (19 us for
// 2 x 5504 x 2048 at T = 9, 45 MB written); here a CTA stages 128 columns of d and
// 256 of x once, and each of its 8 warps keeps the x fragments of 32 columns in
// registers and walks the 128 rows with warp-level MMAs (m16n8k16, T as k), whose
// results go straight out.  The MMA's columns are dealt so that a lane's results
// of four MMAs are eight consecutive columns of a row: 16-byte stores, four lanes
// to 64 bytes.  d comes transposed through ldmatrix.  Measured as what the
// weights' gradients add to a backward pass that writes d_x, passes back to back in a
// graph, this kernel and the GEMM: 2 x 5504 x 2048 at 9, 32 and 48 rows 8.7, 14.0 and
// 19.7 us (5.2 TB/s at 9) against 18.7, 20.3 and 20.4; at 48 rows 2 x 8192 x 4096 44.7
// against 52.8 and 3712 x 4096 14.3 against 17.4.  From 49 rows on the GEMM.
#pragma once

#include "moe_stream.cuh"   // mma_16816

namespace moe_op {

constexpr int OUT_MAX_T = 48;
constexpr int OUT_ROWS = 128, OUT_COLS = 256;

struct OuterArgs {
  const unsigned short* d[2];   // [T, N], rows N apart
  unsigned short* out[2];       // [N, K]
  const unsigned short* x;      // [T, K], rows ldx apart
  int64_t ldx;
  int T, N, K;
};

// KS: 16-token steps
template <bool FP16, int KS>
__global__ void __launch_bounds__(256) k_outer(const OuterArgs A) {
  __shared__ __align__(16) unsigned short ds[KS * 16][OUT_ROWS + 8];
  __shared__ __align__(16) unsigned short xs[KS * 16][OUT_COLS + 8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * OUT_ROWS, k0 = blockIdx.y * OUT_COLS, z = blockIdx.z;   // (N has up to 2^17 row blocks)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const unsigned short* d = z ? A.d[1] : A.d[0];
  // absent tokens, rows past N and columns past K: zeros
  for (int i = tid; i < KS * 16 * (OUT_ROWS / 8); i += 256) {
    const int r = i / (OUT_ROWS / 8), c = i % (OUT_ROWS / 8) * 8;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (r < A.T && n0 + c < A.N) v = *reinterpret_cast<const uint4*>(d + static_cast<int64_t>(r) * A.N + n0 + c);
    *reinterpret_cast<uint4*>(&ds[r][c]) = v;
  }
  for (int i = tid; i < KS * 16 * (OUT_COLS / 8); i += 256) {
    const int r = i / (OUT_COLS / 8), c = i % (OUT_COLS / 8) * 8;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (r < A.T && k0 + c < A.K) v = *reinterpret_cast<const uint4*>(A.x + static_cast<int64_t>(r) * A.ldx + k0 + c);
    *reinterpret_cast<uint4*>(&xs[r][c]) = v;
  }
  __syncthreads();
  // B: column n of MMA j is column 8 (n / 2) + 2 j + n % 2 of the warp's 32
  uint32_t b[KS][4][2];
#pragma unroll
  for (int s = 0; s < KS; ++s)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = warp * 32 + 8 * (g >> 1) + 2 * j + (g & 1), r = s * 16 + 8 * h + 2 * t;
        b[s][j][h] = static_cast<uint32_t>(xs[r][c]) | (static_cast<uint32_t>(xs[r + 1][c]) << 16);
      }
  unsigned short* out = (z ? A.out[1] : A.out[0]);
  const int col = k0 + warp * 32 + 8 * t;
  // this lane's row of the four 8 x 8 matrices of an A fragment: tokens 0-7 and 8-15 by rows 0-7 and 8-15
  const uint32_t a_at = smem_u32(&ds[(lane & 7) + (lane >> 4) * 8][((lane >> 3) & 1) * 8]);
  for (int m = 0; m < OUT_ROWS / 16 && n0 + m * 16 < A.N; ++m) {
    float acc[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      uint32_t a0, a1, a2, a3;
      asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                   : "=r"(a0), "=r"(a1), "=r"(a2), "=r"(a3)
                   : "r"(a_at + (s * 16 * (OUT_ROWS + 8) + m * 16) * 2)
                   : "memory");
#pragma unroll
      for (int j = 0; j < 4; ++j) mma_16816(acc[j], a0, a1, a2, a3, b[s][j][0], b[s][j][1], FP16);
    }
    constexpr int DT = FP16 ? DT_FP16 : DT_BF16;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = n0 + m * 16 + g + 8 * h;
      if (row < A.N && col < A.K)
        *reinterpret_cast<uint4*>(out + static_cast<int64_t>(row) * A.K + col) =
            make_uint4(pack2(acc[0][2 * h], acc[0][2 * h + 1], DT), pack2(acc[1][2 * h], acc[1][2 * h + 1], DT),
                       pack2(acc[2][2 * h], acc[2][2 * h + 1], DT), pack2(acc[3][2 * h], acc[3][2 * h + 1], DT));
    }
  }
}

}  // namespace moe_op
