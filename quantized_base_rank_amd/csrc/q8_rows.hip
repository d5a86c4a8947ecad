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

// Largest of two packed pairs of 16-bit magnitudes.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t max2_u16(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

// bf16 rows, held in registers between the maximum and the codes: one read
// of x.  HBM-bound: 3 bytes per element (5 with the values).  4096 x 28672:
// 59 us, 6.0 TB/s (reading the rows twice took 247 us); 16 rows of 28672, one
// workgroup each: 5.0 us, the latency of load, maximum and store.
template <int T, int NV>
__global__ __launch_bounds__(T * rows_per_group(T)) void k_quant_q8(Q8RowsArgs a) {
  constexpr int kRows = rows_per_group(T);
  __shared__ float s_red[T / 64];
  const int t = threadIdx.x % T, d = static_cast<int>(a.d);
  for (int64_t m = static_cast<int64_t>(blockIdx.x) * kRows + row_of_group<T>(); m < a.rows;
       m += static_cast<int64_t>(gridDim.x) * kRows) {
    const uint16_t* x = static_cast<const uint16_t*>(a.x) + m * a.d;
    u32x4 v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = load8(x + row_vec(t + T * i, d).k);
    uint32_t mx2 = 0u;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) mx2 = max2_u16(mx2, v[i][j] & 0x7FFF7FFFu);
    // (the halves' larger one, as the bits of an fp32 magnitude)
    const uint32_t hi = mx2 & 0xFFFF0000u, lo = mx2 << 16;
    const float mx = block_max_nan<T / 64>(__uint_as_float(hi > lo ? hi : lo), s_red);
    const RowScale s = row_scale(mx);
    const bool bad = !finite_f32(mx);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Vec q = row_vec(t + T * i, d);
      if (!q.in) continue;
      const u32x2 c = bad ? u32x2{0u, 0u} : codes8(v[i], s);
      store_codes8(a.codes + m * a.d + q.k, c);
      if (a.values != nullptr) store8(a.values + m * a.d + q.k, values8(c, s.scale));
    }
    if (t == 0) a.scale[m] = s.scale;
  }
}

// fp32 rows, and bf16 rows too short or too wide for the kernel above: two
// passes, the codes by one fp64 division each (weights, laid out once: 8192 x
// 28672 fp32 581 us; 512 rows of 65536 in bf16 164 us).
template <bool F32>
__global__ __launch_bounds__(256) void k_quant_q8_two_pass(Q8RowsArgs a) {
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

// values = bf16(code * scale), eight elements a thread and step: HBM-bound, 3
// bytes per element.  4096 x 28672: 72 us, 4.9 TB/s.
__global__ __launch_bounds__(256) void k_dequant_q8(const int8_t* codes, const float* scale, int64_t rows,
                                                    int64_t d, uint16_t* out) {
  const int dd = static_cast<int>(d);
  for (int64_t m = blockIdx.x; m < rows; m += gridDim.x) {
    const float s = scale[m];
    if (dd < kRowMin) {
      if (static_cast<int>(threadIdx.x) < dd)
        out[m * d + threadIdx.x] = f32_to_bf16(static_cast<float>(codes[m * d + threadIdx.x]) * s);
      continue;
    }
    for (int v = threadIdx.x; 8 * v < dd; v += 256) {
      const Vec q = row_vec(v, dd);
      store8(out + m * d + q.k, values8(*reinterpret_cast<const u32x2u*>(codes + m * d + q.k), s));
    }
  }
}

}  // namespace

hipError_t launch_quant_q8(const Q8RowsArgs& a, bool f32, hipStream_t stream) {
  if (f32) {
    hipLaunchKernelGGL(k_quant_q8_two_pass<true>, dim3(row_grid(a.rows, 1)), dim3(256), 0, stream, a);
    return hipGetLastError();
  }
  if (a.d < kRowMin || a.d > kRowMax) {
    hipLaunchKernelGGL(k_quant_q8_two_pass<false>, dim3(row_grid(a.rows, 1)), dim3(256), 0, stream, a);
    return hipGetLastError();
  }
  return by_row_width<false>(a.d, [&](auto t, auto nv) {
    constexpr int T = decltype(t)::value, NV = decltype(nv)::value, R = rows_per_group(T);
    hipLaunchKernelGGL((k_quant_q8<T, NV>), dim3(row_grid(a.rows, R)), dim3(T * R), 0, stream, a);
    return hipGetLastError();
  });
}

hipError_t launch_dequant_q8(const int8_t* codes, const float* scale, int64_t rows, int64_t d, uint16_t* out,
                             hipStream_t stream) {
  hipLaunchKernelGGL(k_dequant_q8, dim3(row_grid(rows, 1)), dim3(256), 0, stream, codes, scale, rows, d, out);
  return hipGetLastError();
}

}  // namespace qlin
