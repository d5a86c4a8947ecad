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

// Reciprocal root of the mean square; NaN marks a non-finite row.  A mean
// below the normal numbers has lost its bits (that of 2^-70 keeps nine); from
// 2^-126 on the squares that underflow in the sum cost it 2^-24 at most.
__device__ __forceinline__ float norm_rstd(float ss, const RmsNormArgs& a) {
  const float mean = ss / static_cast<float>(a.d) + a.eps;
  return finite_f32(ss) && mean >= 0x1p-126f ? 1.0f / sqrtf(mean) : __uint_as_float(0x7FC00000u);
}

// The row's sum h = x + res stays in registers as fp32 (one rounding, of the
// sum), so x and the residual are read once: HBM-bound, 9 bytes per element
// with every output.  T threads hold a row, NV vectors of eight each.  4096 x
// 8192 with the residual and the values: 53 us, 5.7 TB/s (202 us with a row
// re-read for each of its three passes); one token of 4096: 3.1 us; 777 x
// 5003 (rows at any alignment) 8.0 us, one round of workgroups' latency; 4096
// x 16384 112 us, 5.4 TB/s.
template <int T, int NV, bool RES>
__global__ __launch_bounds__(T * rows_per_group(T)) void k_rmsnorm_q8(RmsNormArgs a) {
  constexpr int kRows = rows_per_group(T);
  __shared__ float s_red[T / 64];
  const int t = threadIdx.x % T, d = static_cast<int>(a.d);
  for (int64_t m = static_cast<int64_t>(blockIdx.x) * kRows + row_of_group<T>(); m < a.M;
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

// Rows too short or too wide for the kernel above: the input is read three
// times, element by element (512 rows of 65536 with every output 367 us).
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

// Gradient, one pass over h, dy (and dh): a workgroup walks a run of rows, one
// at a time, with the next row's loads in flight during this row's sum, and
// keeps its share of dgamma in registers (each thread's columns are the same
// in every row).  Shares of dgamma go to the workspace; k_rmsnorm_dgamma adds
// them in order.  HBM-bound: 8 bytes per element with dh.  4096 x 8192: 51 us,
// 5.2 TB/s, and 5 us for the 256 shares of dgamma (dx and dgamma in passes of
// their own took 147 us); 250 x 4096: 5.4 + 4.6 us.
template <int T, int NV, bool DH>
__global__ __launch_bounds__(T * rows_per_group(T)) void k_rmsnorm_bwd(RmsNormBwdArgs a) {
  constexpr int kRows = rows_per_group(T);
  __shared__ float s_red[2][T / 64];
  const int t = threadIdx.x % T, sub = row_of_group<T>(), d = static_cast<int>(a.d);
  const int64_t share = static_cast<int64_t>(blockIdx.x) * kRows + sub;
  const int64_t m0 = share * a.per, m1 = m0 + a.per < a.M ? m0 + a.per : a.M;
  u32x4 gv[NV];
  float dg[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    gv[i] = load8(a.gamma + row_vec(t + T * i, d).k);
#pragma unroll
    for (int e = 0; e < 8; ++e) dg[i][e] = 0.0f;
  }
  // (four vectors a thread leave no room for the next row)
  constexpr int kAhead = NV < 4 ? 1 : 0;
  u32x4 hv[1 + kAhead][NV], yv[1 + kAhead][NV], ev[1 + kAhead][NV];
  float rs[1 + kAhead];
  auto load = [&](int64_t m, int p) {
    const int64_t row = (m < m1 ? m : a.M - 1) * a.d;  // (past the run: any row, unused)
    rs[p] = a.rstd[m < m1 ? m : a.M - 1];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int k = row_vec(t + T * i, d).k;
      hv[p][i] = load8(a.h + row + k);
      yv[p][i] = load8(a.dy + row + k);
      if (DH) ev[p][i] = load8(a.dh + row + k);
    }
  };
  const float inv_d = 1.0f / static_cast<float>(a.d);
  if (kAhead != 0) load(m0, 0);
  for (int64_t mm = m0; mm < m1; mm += 1 + kAhead) {
#pragma unroll
    for (int p = 0; p < 1 + kAhead; ++p) {
      const int64_t m = mm + p;
      const int turn = static_cast<int>(m & 1);
      if (m >= m1) break;
      load(m + kAhead, kAhead != 0 ? 1 - p : 0);
      const float rstd = rs[p];
      float c = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int dup = row_vec(t + T * i, d).dup;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float xh = elem8(hv[p][i], e) * rstd, dy = elem8(yv[p][i], e);
          dg[i][e] = __builtin_fmaf(dy, xh, dg[i][e]);
          c = __builtin_fmaf(e >= dup ? dy * elem8(gv[i], e) : 0.0f, xh, c);
        }
        if (NV >= 4) __builtin_amdgcn_sched_barrier(0);  // one vector unpacked at a time
      }
      // (two buffers take turns, so one barrier a row)
      c = warp_sum(c);
      if (T > 64) {
        if ((t & 63) == 0) s_red[turn][t >> 6] = c;
        __syncthreads();
        c = s_red[turn][0];
#pragma unroll
        for (int w = 1; w < T / 64; ++w) c += s_red[turn][w];
      }
      c *= inv_d;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        // (unpacked again from here: held over the sum as fp32 the row would
        // take twice the registers, of which the wide rows have none left)
        __asm__ volatile("" : "+v"(hv[p][i]), "+v"(yv[p][i]), "+v"(gv[i]));
        const Vec q = row_vec(t + T * i, d);
        u32x4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float v[2];
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const int e = 2 * j + z;
            const float xh = elem8(hv[p][i], e) * rstd;
            v[z] = rstd * (elem8(yv[p][i], e) * elem8(gv[i], e) - xh * c);
            if (DH) v[z] += elem8(ev[p][i], e);
          }
          o[j] = pack_bf16x2(v[0], v[1]);
        }
        if (q.in) store8(a.dx + m * a.d + q.k, o);
        if (NV >= 4) __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  if (m0 >= a.M) return;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const Vec q = row_vec(t + T * i, d);
    if (!q.in) continue;
#pragma unroll
    for (int e = 0; e < 8; ++e) a.partial[share * a.d + q.k + e] = dg[i][e];
  }
}

// Rows too short or too wide for the kernel above: dx row by row, dgamma's
// shares column by column (512 rows of 65536: 184 and 41 us).
__global__ __launch_bounds__(256) void k_rmsnorm_dx_wide(RmsNormBwdArgs a) {
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
__global__ __launch_bounds__(256) void k_rmsnorm_dgamma_wide(RmsNormBwdArgs a) {
  const int64_t k = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (k >= a.d) return;
  const int64_t m0 = blockIdx.y * a.per, m1 = m0 + a.per < a.M ? m0 + a.per : a.M;
  float t = 0.0f;
  for (int64_t m = m0; m < m1; ++m)
    t += bf16_to_f32(a.dy[m * a.d + k]) * (bf16_to_f32(a.h[m * a.d + k]) * a.rstd[m]);
  a.partial[blockIdx.y * a.d + k] = t;
}

// dgamma: 64 columns a workgroup, sixteen waves each adding every sixteenth
// share, their sums added in wave order.
__global__ __launch_bounds__(1024) void k_rmsnorm_dgamma(RmsNormBwdArgs a, int shares) {
  __shared__ float s_t[16][64];
  const int c = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t k = static_cast<int64_t>(blockIdx.x) * 64 + c;
  float t = 0.0f;
  if (k < a.d) {
#pragma unroll 8
    for (int s = w; s < shares; s += 16) t += a.partial[s * a.d + k];
  }
  s_t[w][c] = t;
  __syncthreads();
  if (w != 0 || k >= a.d) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) t += s_t[i][c];
  a.dgamma[k] = t;
}

// Rows per share: 256 shares, 512 of rows up to 2048 columns (whose shares are
// one or two waves each), at least two rows each so that a short batch does
// not write more partial sums than it reads rows.  4096 x 1000: 21.9 us with
// 256, 16.4 with 512, 16.0 with 1024; x 2048: 23.2, 20.3, 21.2; x 4096: 28.9,
// 29.2, 34.0; x 8192: 54, 59, 65.
int64_t bwd_rows(int64_t M, int64_t d) {
  const int64_t shares = d <= 2048 ? 512 : 256, per = (M + shares - 1) / shares;
  return per < 2 ? 2 : per;
}
int64_t bwd_shares(int64_t M, int64_t d) { return (M + bwd_rows(M, d) - 1) / bwd_rows(M, d); }

}  // namespace

hipError_t launch_rmsnorm_q8(const RmsNormArgs& a, hipStream_t stream) {
  if (a.d < kRowMin || a.d > kRowMax) {
    hipLaunchKernelGGL(k_rmsnorm_q8_wide, dim3(row_grid(a.M, 1)), dim3(256), 0, stream, a);
    return hipGetLastError();
  }
  return by_row_width<false>(a.d, [&](auto t, auto nv) {
    constexpr int T = decltype(t)::value, NV = decltype(nv)::value, R = rows_per_group(T);
    const dim3 grid(row_grid(a.M, R)), block(T * R);
    if (a.res != nullptr)
      hipLaunchKernelGGL((k_rmsnorm_q8<T, NV, true>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((k_rmsnorm_q8<T, NV, false>), grid, block, 0, stream, a);
    return hipGetLastError();
  });
}

int64_t rmsnorm_bwd_partial_floats(int64_t M, int64_t d) { return bwd_shares(M, d) * d; }

hipError_t launch_rmsnorm_bwd(const RmsNormBwdArgs& args, hipStream_t stream) {
  RmsNormBwdArgs a = args;
  a.per = bwd_rows(a.M, a.d);
  const int64_t shares = bwd_shares(a.M, a.d);
  hipError_t e;
  if (a.d < kRowMin || a.d > kGradRowMax) {
    hipLaunchKernelGGL(k_rmsnorm_dx_wide, dim3(row_grid(a.M, 1)), dim3(256), 0, stream, a);
    hipLaunchKernelGGL(k_rmsnorm_dgamma_wide, dim3(static_cast<uint32_t>((a.d + 255) / 256), static_cast<uint32_t>(shares)),
                       dim3(256), 0, stream, a);
    e = hipGetLastError();
  } else {
    e = by_row_width<true>(a.d, [&](auto t, auto nv) {
      constexpr int T = decltype(t)::value, NV = decltype(nv)::value, R = rows_per_group(T);
      const dim3 grid(static_cast<uint32_t>((shares + R - 1) / R)), block(T * R);
      if (a.dh != nullptr)
        hipLaunchKernelGGL((k_rmsnorm_bwd<T, NV, true>), grid, block, 0, stream, a);
      else
        hipLaunchKernelGGL((k_rmsnorm_bwd<T, NV, false>), grid, block, 0, stream, a);
      return hipGetLastError();
    });
  }
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_rmsnorm_dgamma, dim3(static_cast<uint32_t>((a.d + 63) / 64)), dim3(1024), 0, stream, a,
                     static_cast<int>(shares));
  return hipGetLastError();
}

}  // namespace qlin
