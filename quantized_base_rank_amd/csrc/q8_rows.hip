// 8-bit rows: int8 codes and one fp32 scale per row of a bf16 or fp32 matrix.
// [QLoRA "Background: what is quantization?": absmax scaling, here with one
// row as the block]
//
//   a = max_k |x_k|,  scale = RN32(a / 127),  code_k = round_half_even(127 x_k / a)
//
// taken on the exact real values; a row holding NaN or an infinity gets scale
// NaN and codes 0.
#include "device_common.hpp"
#include "kernels.hpp"
#include "q8_common.hpp"

namespace qlin {

namespace {

// One workgroup per row, two passes over it (the second reads it from cache).
template <bool F32>
__global__ __launch_bounds__(256) void k_quant_q8(Q8RowsArgs a) {
  __shared__ float s_red[4];
  const int tid = threadIdx.x;
  for (int64_t m = blockIdx.x; m < a.rows; m += gridDim.x) {
    auto at = [&](int64_t k) {
      return F32 ? static_cast<const float*>(a.x)[m * a.d + k]
                 : bf16_to_f32(static_cast<const uint16_t*>(a.x)[m * a.d + k]);
    };
    float mx = 0.0f;
    for (int64_t k = tid; k < a.d; k += 256) mx = max_abs_nan(mx, at(k));
    mx = block_max_nan<4>(mx, s_red);
    const float scale = q8_scale(mx);
    for (int64_t k = tid; k < a.d; k += 256) {
      const int q = q8_code_exact(at(k), mx);
      a.codes[m * a.d + k] = static_cast<int8_t>(q);
      if (a.values != nullptr) a.values[m * a.d + k] = f32_to_bf16(static_cast<float>(q) * scale);
    }
    if (tid == 0) a.scale[m] = scale;
  }
}

__global__ __launch_bounds__(256) void k_dequant_q8(const int8_t* codes, const float* scale, int64_t rows,
                                                    int64_t d, uint16_t* out) {
  for (int64_t m = blockIdx.x; m < rows; m += gridDim.x)
    for (int64_t k = threadIdx.x; k < d; k += 256)
      out[m * d + k] = f32_to_bf16(static_cast<float>(codes[m * d + k]) * scale[m]);
}

uint32_t row_grid(int64_t rows) { return static_cast<uint32_t>(rows < (1 << 20) ? rows : (1 << 20)); }

}  // namespace

hipError_t launch_quant_q8(const Q8RowsArgs& a, bool f32, hipStream_t stream) {
  if (f32)
    hipLaunchKernelGGL(k_quant_q8<true>, dim3(row_grid(a.rows)), dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL(k_quant_q8<false>, dim3(row_grid(a.rows)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_dequant_q8(const int8_t* codes, const float* scale, int64_t rows, int64_t d, uint16_t* out,
                             hipStream_t stream) {
  hipLaunchKernelGGL(k_dequant_q8, dim3(row_grid(rows)), dim3(256), 0, stream, codes, scale, rows, d, out);
  return hipGetLastError();
}

}  // namespace qlin
