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

// Reciprocal root of the mean square; NaN marks a non-finite row.
__device__ __forceinline__ float norm_rstd(float ss, const RmsNormArgs& a) {
  const float r = 1.0f / sqrtf(ss / static_cast<float>(a.d) + a.eps);
  return finite_f32(ss) && finite_f32(r) ? r : __uint_as_float(0x7FC00000u);
}

// The row's sum h = x + res stays in registers as fp32 (one rounding, of the
// sum), so x and the residual are read once: HBM-bound, 9 bytes per element
// with every output.  T threads hold a row, NV vectors of eight each.
template <int T, int NV, bool RES>
__global__ __launch_bounds__(T * rows_per_group(T)) void k_rmsnorm_q8(RmsNormArgs a) {
  constexpr int kRows = rows_per_group(T);
  __shared__ float s_red[T / 64];
  const int t = threadIdx.x % T, d = static_cast<int>(a.d);
  for (int64_t m = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / T; m < a.M;
       m += static_cast<int64_t>(gridDim.x) * kRows) {
    const int64_t row = m * a.d;
    u32x4 xv[NV], rv[NV], gv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int k = row_vec(t + T * i, d).k;
      xv[i] = load8(a.x + row + k);
      if (RES) rv[i] = load8(a.res + row + k);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) gv[i] = load8(a.gamma + row_vec(t + T * i, d).k);
    float y[NV][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Vec q = row_vec(t + T * i, d);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[i][e] = RES ? elem8(xv[i], e) + elem8(rv[i], e) : elem8(xv[i], e);
        const float own = e >= q.dup ? y[i][e] : 0.0f;
        ss = __builtin_fmaf(own, own, ss);
      }
      if (RES && q.in) {
        u32x4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = pack_bf16x2(y[i][2 * j], y[i][2 * j + 1]);
        store8(a.h + row + q.k, o);
      }
    }
    const float rstd = norm_rstd(block_sum<T / 64>(ss, s_red), a);
    float mx = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[i][e] = y[i][e] * rstd * elem8(gv[i], e);
        mx = max_abs_nan(mx, y[i][e]);
      }
    mx = block_max_nan<T / 64>(mx, s_red);
    const RowScale s = row_scale(mx);
    const bool bad = !finite_f32(mx);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Vec v = row_vec(t + T * i, d);
      if (!v.in) continue;
      uint32_t q[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = round_bits(y[i][e] * s.pre * s.inv);
      u32x2 c{low_bytes(q[0], q[1], q[2], q[3]), low_bytes(q[4], q[5], q[6], q[7])};
      if (bad) c = u32x2{0u, 0u};
      store_codes8(a.codes + row + v.k, c);
      if (a.values != nullptr) store8(a.values + row + v.k, values8(c, s.scale));
    }
    if (t == 0) {
      a.scale[m] = s.scale;
      if (a.rstd != nullptr) a.rstd[m] = rstd;
    }
  }
}

// Rows too short or too wide for the kernel above: the input is read three times.
__global__ __launch_bounds__(256) void k_rmsnorm_q8_wide(RmsNormArgs a) {
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
    const float rstd = norm_rstd(ss, a);
    for (int64_t k = tid; k < a.d; k += 256) hm = max_abs_nan(hm, sum_at(k) * rstd * bf16_to_f32(a.gamma[k]));
    const float mx = block_max_nan<4>(hm, s_red);
    const RowScale s = row_scale(mx);
    const bool bad = !finite_f32(mx);
    for (int64_t k = tid; k < a.d; k += 256) {
      const float y = sum_at(k) * rstd * bf16_to_f32(a.gamma[k]);
      const int q = bad ? 0 : static_cast<int8_t>(round_bits(y * s.pre * s.inv));
      a.codes[row + k] = static_cast<int8_t>(q);
      if (a.values != nullptr) a.values[row + k] = f32_to_bf16(static_cast<float>(q) * s.scale);
    }
    if (tid == 0) {
      a.scale[m] = s.scale;
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

}  // namespace

hipError_t launch_rmsnorm_q8(const RmsNormArgs& a, hipStream_t stream) {
  if (a.d < kRowMin || a.d > kRowMax) {
    hipLaunchKernelGGL(k_rmsnorm_q8_wide, dim3(row_grid(a.M, 1)), dim3(256), 0, stream, a);
    return hipGetLastError();
  }
  return by_row_width(a.d, [&](auto t, auto nv) {
    constexpr int T = decltype(t)::value, NV = decltype(nv)::value, R = rows_per_group(T);
    const dim3 grid(row_grid(a.M, R)), block(T * R);
    if (a.res != nullptr)
      hipLaunchKernelGGL((k_rmsnorm_q8<T, NV, true>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((k_rmsnorm_q8<T, NV, false>), grid, block, 0, stream, a);
    return hipGetLastError();
  });
}

int64_t rmsnorm_bwd_partial_floats(int64_t, int64_t d) { return kDgShares * d; }

hipError_t launch_rmsnorm_bwd(const RmsNormBwdArgs& a, hipStream_t stream) {
  const uint32_t cols = static_cast<uint32_t>((a.d + 255) / 256);
  hipLaunchKernelGGL(k_rmsnorm_dx, dim3(row_grid(a.M, 1)), dim3(256), 0, stream, a);
  hipLaunchKernelGGL(k_rmsnorm_dgamma_part, dim3(cols, kDgShares), dim3(256), 0, stream, a);
  hipLaunchKernelGGL(k_rmsnorm_dgamma_sum, dim3(cols), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace qlin
