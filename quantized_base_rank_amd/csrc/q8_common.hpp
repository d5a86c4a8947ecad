// Device helpers of the 8-bit row format (int8 codes, one fp32 scale per row).
#pragma once

#include "device_common.hpp"

#include <type_traits>

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

// ------------------------------------------------------ rows in registers
// A row of at least eight elements is spread over T threads in vectors of
// eight: thread t holds vectors t, t + T, ...  Rows of any width and
// alignment go through the same branch-free 16-byte accesses (this target
// allows them at any address): a vector that would pass the row's end is
// moved back onto its last eight elements, so some of its elements are held
// twice, with the same values; they are stored twice alike and left out of
// sums (Vec::dup).
typedef u32x4 u32x4u __attribute__((aligned(2)));
typedef u32x2 u32x2u __attribute__((aligned(1)));

struct Vec {
  int k;    // first element
  int dup;  // elements k .. k + dup - 1 belong to an earlier vector (8: a vector past the row)
  bool in;  // holds elements of its own
};
__device__ __forceinline__ Vec row_vec(int v, int d) {
  const int k = 8 * v < d - 8 ? 8 * v : d - 8;
  const int dup = 8 * v - k;
  return Vec{k, dup < 8 ? dup : 8, dup < 8};
}
__device__ __forceinline__ u32x4 load8(const uint16_t* p) { return *reinterpret_cast<const u32x4u*>(p); }
__device__ __forceinline__ void store8(uint16_t* p, u32x4 v) { *reinterpret_cast<u32x4u*>(p) = v; }
__device__ __forceinline__ void store_codes8(int8_t* p, u32x2 v) { *reinterpret_cast<u32x2u*>(p) = v; }
__device__ __forceinline__ float elem8(u32x4 v, int e) { return (e & 1) ? bf16_hi(v[e >> 1]) : bf16_lo(v[e >> 1]); }

// Adding 1.5 * 2^23 rounds a value of less than 2^22 to the nearest integer
// (ties to even) and leaves that integer, in two's complement, in the low
// bits: the low byte is the code.
__device__ __forceinline__ uint32_t round_bits(float p) { return __float_as_uint(p + 12582912.0f); }
// low bytes of four words, in order
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return perm(perm(d, c, 0x0C0C0400u), perm(b, a, 0x0C0C0400u), 0x05040100u);
}
__device__ __forceinline__ float code_of(uint32_t word, int e) {
  return static_cast<float>(static_cast<int8_t>(word >> (8 * e)));
}

// bf16(code * scale) of eight codes.
__device__ __forceinline__ u32x4 values8(u32x2 c, float scale) {
  u32x4 o;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    o[j] = pack_bf16x2(code_of(c[j >> 1], 2 * (j & 1)) * scale, code_of(c[j >> 1], 2 * (j & 1) + 1) * scale);
  return o;
}

// A row's factors: y * pre * inv = 127 y / mx.  Rows below 2^-100 are first
// scaled by 2^64 (exact), so that inv stays inside fp32's range; rows that
// are zero or not finite have inv = 0 (codes 0, once their elements are made
// finite by the caller).
struct RowScale {
  float scale, pre, inv;
};
__device__ __forceinline__ RowScale row_scale(float mx) {
  RowScale r;
  r.scale = q8_scale(mx);
  r.pre = mx < 0x1p-100f ? 0x1p64f : 1.0f;
  r.inv = finite_f32(mx) && mx > 0.0f ? 127.0f / (mx * r.pre) : 0.0f;
  return r;
}

// Sizes of a row kernel's instantiations: threads per row, vectors of eight a
// thread.  One wave per row up to 1024 columns (several rows share a workgroup
// and nothing needs a barrier), then two or three vectors a thread up to 512
// threads, and beyond 8192 columns as many vectors as 512 threads need.  (4096
// rows to 8 bits, 512 threads against 1024 with two or four vectors: 11008
// columns 27 and 32 us, 28672 64 and 76; the norm at 11008 77 and 101 us, at
// 16384 112 and 129.  5120 columns: 256 x 3 14.6 us, 512 x 2 15.9.)  The
// gradient holds three rows and its sums, so its widest rows end at half the
// width.  Rows below eight columns or past the widest take the kernels that
// walk a row element by element.
constexpr int kRowMin = 8, kRowMax = 32768, kGradRowMax = 16384;
template <bool GRAD, typename F>
hipError_t by_row_width(int64_t d, F f) {
  if (d <= 512) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
  if (d <= 1024) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
  if (d <= 2048) return f(std::integral_constant<int, 128>{}, std::integral_constant<int, 2>{});
  if (d <= 4096) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
  if (d <= 6144) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 3>{});
  constexpr std::integral_constant<int, 512> wide{};
  if (d <= 8192) return f(wide, std::integral_constant<int, 2>{});
  if (d <= 12288) return f(wide, std::integral_constant<int, 3>{});
  if constexpr (GRAD) {
    return f(wide, std::integral_constant<int, 4>{});
  } else {
    if (d <= 16384) return f(wide, std::integral_constant<int, 4>{});
    if (d <= 20480) return f(wide, std::integral_constant<int, 5>{});
    if (d <= 24576) return f(wide, std::integral_constant<int, 6>{});
    if (d <= 28672) return f(wide, std::integral_constant<int, 7>{});
    return f(wide, std::integral_constant<int, 8>{});
  }
}
// Rows that share a workgroup: only rows of one wave, which need no barrier.
constexpr int rows_per_group(int threads) { return threads == 64 ? 4 : 1; }
// This thread's row of the group, known to be the same for its whole wave.
template <int T>
__device__ __forceinline__ int row_of_group() {
  return rows_per_group(T) == 1 ? 0 : __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / T);
}
// Workgroups for `rows` rows, `per` of them each; a longer queue is walked.
inline uint32_t row_grid(int64_t rows, int per) {
  const int64_t n = (rows + per - 1) / per;
  return static_cast<uint32_t>(n < (1 << 20) ? n : (1 << 20));
}

}  // namespace qlin
