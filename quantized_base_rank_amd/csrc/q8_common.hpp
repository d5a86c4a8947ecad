// Device helpers of the 8-bit row format (int8 codes, one fp32 scale per row).
#pragma once

#include "device_common.hpp"

namespace qlin {

// Running maximum of |v| that keeps a NaN once it has met one (fmaxf drops
// it): the bits of |v| order like the values, with NaN above infinity.
__device__ __forceinline__ float max_abs_nan(float m, float v) {
  const uint32_t a = __float_as_uint(m), b = __float_as_uint(v) & 0x7FFFFFFFu;
  return __uint_as_float(a > b ? a : b);
}

// Largest of non-negative values (NaN on top) over a workgroup of WAVES
// waves; `s` holds WAVES floats and is free again when every thread returns.
template <int WAVES>
__device__ __forceinline__ float block_max_nan(float v, float* s) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = max_abs_nan(v, __shfl_xor(v, o, 64));
  if (WAVES == 1) return v;
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  v = s[0];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) v = max_abs_nan(v, s[w]);
  __syncthreads();
  return v;
}

// Sum over a workgroup in a fixed order (waves' trees, then waves in order).
template <int WAVES>
__device__ __forceinline__ float block_sum(float v, float* s) {
  v = warp_sum(v);
  if (WAVES == 1) return v;
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  v = s[0];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) v += s[w];
  __syncthreads();
  return v;
}

__device__ __forceinline__ bool finite_f32(float v) { return (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u; }

// Scale of a row whose largest magnitude is mx (NaN if mx is not finite).
__device__ __forceinline__ float q8_scale(float mx) {
  return finite_f32(mx) ? mx / 127.0f : __uint_as_float(0x7FC00000u);
}

// round_half_even(127 v / mx), exact: 127 v has at most 31 significant bits,
// exact in fp64, and a quotient that is not a tie lies at least
// 1 / (2 * 127 * 2^24) relative from one, far more than fp64's rounding.
__device__ __forceinline__ int q8_code_exact(float v, float mx) {
  if (!finite_f32(mx) || mx == 0.0f) return 0;
  return static_cast<int>(rint(127.0 * static_cast<double>(v) / static_cast<double>(mx)));
}

}  // namespace qlin
