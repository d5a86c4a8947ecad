// Product of 8-bit rows: y[m][n] = xs[m] ws[n] sum_k xq[m][k] wq[n][k], the
// sum taken by the 8-bit matrix instructions in int32 (exact for
// K <= 131056, where 128 * 128 * K < 2^31).
#include "device_common.hpp"
#include "kernels.hpp"
#include "q8_common.hpp"

namespace qlin {

namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));

// One wave per 32 x 32 tile, operands straight from memory: lane (l, h) of
// the 32x32x32 instruction holds 16 consecutive k, from 16 h, of row l.
__global__ __launch_bounds__(64) void k_w8a8(W8A8Args a) {
  const int lane = threadIdx.x, l = lane & 31, h = lane >> 5;
  const int64_t n_tiles = (a.N + 31) / 32;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) / n_tiles * 32, n0 = static_cast<int64_t>(blockIdx.x) % n_tiles * 32;
  const int64_t mr = m0 + l < a.M ? m0 + l : a.M - 1, nr = n0 + l < a.N ? n0 + l : a.N - 1;
  i32x16 acc{};
  for (int64_t k = 16 * h; k < (a.K + 31) / 32 * 32; k += 32) {
    i32x4 av{}, bv{};
    if (k < a.K) {
      av = *reinterpret_cast<const i32x4*>(a.xq + mr * a.K + k);
      bv = *reinterpret_cast<const i32x4*>(a.wq + nr * a.K + k);
    }
    acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(av, bv, acc, 0, 0, 0);
  }
  // lane (l, h) holds D[m = 8 i + 4 h + v][n = l] at acc[4 i + v]
  if (n0 + l >= a.N) return;
  const float ws = a.ws[n0 + l];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t m = m0 + 8 * (i >> 2) + 4 * h + (i & 3);
    if (m < a.M) a.y[m * a.N + n0 + l] = f32_to_bf16(static_cast<float>(acc[i]) * a.xs[m] * ws);
  }
}

}  // namespace

hipError_t launch_w8a8(const W8A8Args& a, hipStream_t stream) {
  const int64_t tiles = (a.M + 31) / 32 * ((a.N + 31) / 32);
  hipLaunchKernelGGL(k_w8a8, dim3(static_cast<uint32_t>(tiles)), dim3(64), 0, stream, a);
  return hipGetLastError();
}

}  // namespace qlin
