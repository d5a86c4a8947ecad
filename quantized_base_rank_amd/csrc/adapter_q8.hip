// Adapter gradient from an 8-bit checkpoint of the layer's input:
//   dA[j][g] = sum_m du[m][j] xs[m] sum_{k in g} xq[m][k]
// (groups g of one column, or of 32 for the pooled adapter).  [QLoRA "The
// QLoRA recipe: quantize, then adapt": gradients reach the adapter only;
// QA-LoRA abstract for the pooled adapter]
#include "device_common.hpp"
#include "kernels.hpp"

namespace qlin {

namespace {

// One thread per column and 16 adapter rows.
__global__ __launch_bounds__(64) void k_da_q8(DaQ8Args a) {
  const int64_t k = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
  const int j0 = static_cast<int>(blockIdx.y) * 16;
  float acc[16] = {};
  for (int64_t m = 0; m < a.M; ++m) {
    const float x = static_cast<float>(a.xq[m * a.K + k]) * a.xs[m];
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j0 + j < a.r) acc[j] += a.du[m * a.r + j0 + j] * x;
  }
  const int64_t G = a.K / a.pool;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    float t = acc[j];
    if (a.pool == 32) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) t += __shfl_xor(t, o, 64);
      if ((threadIdx.x & 31) != 0) continue;
    }
    if (j0 + j < a.r) a.dA[(j0 + j) * G + k / a.pool] = f32_to_bf16(t);
  }
}

}  // namespace

hipError_t launch_da_q8(const DaQ8Args& a, hipStream_t stream) {
  hipLaunchKernelGGL(k_da_q8, dim3(static_cast<uint32_t>(a.K / 64), static_cast<uint32_t>((a.r + 15) / 16)), dim3(64), 0,
                     stream, a);
  return hipGetLastError();
}

}  // namespace qlin
