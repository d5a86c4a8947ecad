// Root-mean-square norm of a residual sum, given out as 8-bit rows, and its
// gradient.
//
//   h = x + res,  rstd = 1 / sqrt(mean h^2 + eps),  y = h rstd gamma,
//   (codes, scale) = 8-bit rows of y
//   xh = h rstd,  g = dy gamma,
//   dx = rstd (g - xh mean(g xh)) + dh,   dgamma = sum_m dy xh
#include "device_common.hpp"
#include "kernels.hpp"
#include "q8_common.hpp"

namespace qlin {

namespace {

__global__ __launch_bounds__(256) void k_rmsnorm_q8(RmsNormArgs a) {
  __shared__ float s_red[4];
  const int tid = threadIdx.x;
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const int64_t row = m * a.d;
    auto sum_at = [&](int64_t k) {
      const float x = bf16_to_f32(a.x[row + k]);
      return a.res != nullptr ? x + bf16_to_f32(a.res[row + k]) : x;
    };
    float ss = 0.0f, hm = 0.0f;
    for (int64_t k = tid; k < a.d; k += 256) {
      const float h = sum_at(k);
      ss += h * h;
      if (a.h != nullptr) a.h[row + k] = f32_to_bf16(h);
    }
    ss = block_sum<4>(ss, s_red);
    float rstd = 1.0f / sqrtf(ss / static_cast<float>(a.d) + a.eps);
    if (!finite_f32(ss) || !finite_f32(rstd)) rstd = __uint_as_float(0x7FC00000u);
    for (int64_t k = tid; k < a.d; k += 256) hm = max_abs_nan(hm, sum_at(k) * rstd * bf16_to_f32(a.gamma[k]));
    const float mx = block_max_nan<4>(hm, s_red);
    const float scale = q8_scale(mx);
    const bool zero = !finite_f32(mx) || mx == 0.0f;
    for (int64_t k = tid; k < a.d; k += 256) {
      const float y = sum_at(k) * rstd * bf16_to_f32(a.gamma[k]);
      const int q = zero ? 0 : static_cast<int>(rintf(127.0f * y / mx));
      a.codes[row + k] = static_cast<int8_t>(q);
      if (a.values != nullptr) a.values[row + k] = f32_to_bf16(static_cast<float>(q) * scale);
    }
    if (tid == 0) {
      a.scale[m] = scale;
      if (a.rstd != nullptr) a.rstd[m] = rstd;
    }
  }
}

__global__ __launch_bounds__(256) void k_rmsnorm_dx(RmsNormBwdArgs a) {
  __shared__ float s_red[4];
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const int64_t row = m * a.d;
    const float rstd = a.rstd[m];
    float c = 0.0f;
    for (int64_t k = threadIdx.x; k < a.d; k += 256)
      c += bf16_to_f32(a.dy[row + k]) * bf16_to_f32(a.gamma[k]) * (bf16_to_f32(a.h[row + k]) * rstd);
    c = block_sum<4>(c, s_red) / static_cast<float>(a.d);
    for (int64_t k = threadIdx.x; k < a.d; k += 256) {
      const float xh = bf16_to_f32(a.h[row + k]) * rstd;
      float v = rstd * (bf16_to_f32(a.dy[row + k]) * bf16_to_f32(a.gamma[k]) - xh * c);
      if (a.dh != nullptr) v += bf16_to_f32(a.dh[row + k]);
      a.dx[row + k] = f32_to_bf16(v);
    }
  }
}

constexpr int kDgShares = 64;

// Columns' sums over a share of the tokens, then the shares' sum in order.
__global__ __launch_bounds__(256) void k_rmsnorm_dgamma_part(RmsNormBwdArgs a) {
  const int64_t k = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (k >= a.d) return;
  const int64_t per = (a.M + kDgShares - 1) / kDgShares;
  const int64_t m1 = (blockIdx.y + 1) * per < a.M ? (blockIdx.y + 1) * per : a.M;
  float t = 0.0f;
  for (int64_t m = blockIdx.y * per; m < m1; ++m)
    t += bf16_to_f32(a.dy[m * a.d + k]) * (bf16_to_f32(a.h[m * a.d + k]) * a.rstd[m]);
  a.partial[blockIdx.y * a.d + k] = t;
}
__global__ __launch_bounds__(256) void k_rmsnorm_dgamma_sum(RmsNormBwdArgs a) {
  const int64_t k = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (k >= a.d) return;
  float t = 0.0f;
  for (int s = 0; s < kDgShares; ++s) t += a.partial[s * a.d + k];
  a.dgamma[k] = t;
}

uint32_t row_grid(int64_t rows) { return static_cast<uint32_t>(rows < (1 << 20) ? rows : (1 << 20)); }

}  // namespace

hipError_t launch_rmsnorm_q8(const RmsNormArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(k_rmsnorm_q8, dim3(row_grid(a.M)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

int64_t rmsnorm_bwd_partial_floats(int64_t, int64_t d) { return kDgShares * d; }

hipError_t launch_rmsnorm_bwd(const RmsNormBwdArgs& a, hipStream_t stream) {
  const uint32_t cols = static_cast<uint32_t>((a.d + 255) / 256);
  hipLaunchKernelGGL(k_rmsnorm_dx, dim3(row_grid(a.M)), dim3(256), 0, stream, a);
  hipLaunchKernelGGL(k_rmsnorm_dgamma_part, dim3(cols, kDgShares), dim3(256), 0, stream, a);
  hipLaunchKernelGGL(k_rmsnorm_dgamma_sum, dim3(cols), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace qlin
