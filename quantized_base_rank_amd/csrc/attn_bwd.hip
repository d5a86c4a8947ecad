// Gradient of causal attention (attn_fwd.hip), the scores formed again from
// q, k and the forward's lse:
//     p_ij = exp(c q_i . k_j - lse_i),      delta_i = do_i . o_i,
//     ds_ij = p_ij (do_i . v_j - delta_i),  dv_j = sum_i p_ij do_i,
//     dk_j = c sum_i ds_ij q_i,             dq_i = c sum_j ds_ij k_j.
// Three launches: delta (and lse in powers of two), rows of one key head one
// behind the other; dk and dv, a workgroup for 128 keys, which walks the query
// rows of all heads that share them; dq, a workgroup for 128 query rows, which
// walks the keys.  Scores are formed twice; in return no sum needs atomics, so
// the results are the same from run to run.
//
// Roundings: p and ds to bf16 as operands of the products that sum over
// queries and keys; all sums fp32.
#include "attn_common.hpp"
#include "kernels.hpp"
#include "q8_common.hpp"

namespace qlin {

namespace {

constexpr int kBK = 128;  // keys, or query rows, of a workgroup
constexpr int kBQ = 64;   // query rows, or keys, of a step

// Sixteen lanes take a row.
__global__ __launch_bounds__(256) void k_attn_delta(AttnBwdArgs a) {
  const int lane = threadIdx.x & 15;
  const int64_t rows = static_cast<int64_t>(a.T) * a.Hq;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4); i < rows;
       i += static_cast<int64_t>(gridDim.x) * 16) {
    float sum = 0.0f;
    if (8 * lane < a.D) {
      const u32x4 x = *reinterpret_cast<const u32x4*>(a.o + i * a.D + 8 * lane);
      const u32x4 y = *reinterpret_cast<const u32x4*>(a.dout + i * a.D + 8 * lane);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += elem8(x, e) * elem8(y, e);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 16);
    if (lane == 0) {
      const int t = static_cast<int>(i / a.Hq), hq = static_cast<int>(i % a.Hq);
      const int64_t at = (static_cast<int64_t>(hq / a.g) * a.T + t) * a.g + hq % a.g;
      a.lse2[at] = a.lse[i] * kLog2e;
      a.delta[at] = sum;
    }
  }
}

template <int DP>
__global__ __launch_bounds__(256, 1) void k_attn_dkdv(AttnBwdArgs a) {
  constexpr int NP = DP / 8, KS = DP / 16, DB = DP / 32;
  __shared__ __attribute__((aligned(16))) uint8_t sq[kBQ * DP * 2];
  __shared__ __attribute__((aligned(16))) uint8_t sdo[kBQ * DP * 2];
  __shared__ __attribute__((aligned(16))) float s_lse[kBQ], s_delta[kBQ];

  const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kvh = static_cast<int>(blockIdx.x) % a.Hkv, D = a.D, g = a.g;
  RowTile rt;  // rows are keys here
  if (!find_rows(a.cu, a.B, a.T, 1, kBK, static_cast<int>(blockIdx.x) / a.Hkv, &rt)) return;
  const int rows = rt.n * g;  // query rows of the sequence

  const int key = rt.row0 + wave * 32 + l32;
  const bool in = key < rt.n;
  u32x4 kf[KS], vf[KS];
  const int64_t krow = rt.s0 + (in ? key : rt.row0);
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    const int c = 16 * s + 8 * h;
    kf[s] = in && c < D ? *reinterpret_cast<const u32x4*>(a.k + krow * a.k_ld + kvh * D + c) : u32x4{0, 0, 0, 0};
    vf[s] = in && c < D ? *reinterpret_cast<const u32x4*>(a.v + krow * a.v_ld + kvh * D + c) : u32x4{0, 0, 0, 0};
  }
  f32x16 dk[DB], dv[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) dk[d] = dv[d] = f32x16{};

  const float* lse2 = a.lse2 + (static_cast<int64_t>(kvh) * a.T + rt.s0) * g;
  const float* delta = a.delta + (static_cast<int64_t>(kvh) * a.T + rt.s0) * g;
  for (int r0 = rt.row0 * g; r0 < rows; r0 += kBQ) {
    const int t0 = r0 / g, rem = r0 - t0 * g;
#pragma unroll
    for (int i = 0; i < kBQ * NP / 256; ++i) {
      const int idx = tid + 256 * i, r = idx / NP, c = idx % NP;
      u32x4 q = {0, 0, 0, 0}, y = {0, 0, 0, 0};
      if (r0 + r < rows && 8 * c < D) {
        const int dt = small_div(rem + r, a.g_inv), hq = kvh * g + rem + r - dt * g;
        const int64_t row = rt.s0 + t0 + dt;
        q = *reinterpret_cast<const u32x4*>(a.q + row * a.q_ld + hq * D + 8 * c);
        y = *reinterpret_cast<const u32x4*>(a.dout + (row * a.Hq + hq) * D + 8 * c);
      }
      *reinterpret_cast<u32x4*>(sq + piece_at<DP>(r, c)) = q;
      *reinterpret_cast<u32x4*>(sdo + piece_at<DP>(r, c)) = y;
    }
    if (tid < kBQ) {
      const bool ok = r0 + tid < rows;
      s_lse[tid] = ok ? lse2[r0 + tid] : 0.0f;
      s_delta[tid] = ok ? delta[r0 + tid] : 0.0f;
    }
    __syncthreads();
    // rows from key's own token on count: row (key g) is the first
    const int64_t from = static_cast<int64_t>(key) * g - r0;
#pragma unroll
    for (int qb = 0; qb < 2; ++qb) {
      f32x16 s = {}, dp = {};
#pragma unroll
      for (int t = 0; t < KS; ++t) {
        s = mfma32(*reinterpret_cast<const u32x4*>(sq + piece_at<DP>(qb * 32 + l32, 2 * t + h)), kf[t], s);
        dp = mfma32(*reinterpret_cast<const u32x4*>(sdo + piece_at<DP>(qb * 32 + l32, 2 * t + h)), vf[t], dp);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int r = qb * 32 + acc_row(i, h);
        const bool on = in && r >= from && r0 + r < rows;
        const float p = on ? __builtin_amdgcn_exp2f(s[i] * a.c2 - s_lse[r]) : 0.0f;
        s[i] = p;
        dp[i] = on ? p * (dp[i] - s_delta[r]) : 0.0f;
      }
#pragma unroll
      for (int kg = 0; kg < 2; ++kg) {
        const u32x4 p = pack_operand(s, kg), ds = pack_operand(dp, kg);
#pragma unroll
        for (int d = 0; d < DB; ++d) {
          dv[d] = mfma32(column_operand<DP>(sdo, qb * 32 + 16 * kg, 32 * d, lane), p, dv[d]);
          dk[d] = mfma32(column_operand<DP>(sq, qb * 32 + 16 * kg, 32 * d, lane), ds, dk[d]);
        }
      }
    }
    __syncthreads();
  }
  if (!in) return;
  uint16_t* const odk = a.dk + krow * a.dk_ld + kvh * D;
  uint16_t* const odv = a.dv + krow * a.dv_ld + kvh * D;
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int c = 32 * d + acc_row(i, h);
      if (c >= D) continue;
      *reinterpret_cast<u32x2*>(odv + c) = u32x2{pack_bf16x2(dv[d][i], dv[d][i + 1]), pack_bf16x2(dv[d][i + 2], dv[d][i + 3])};
      *reinterpret_cast<u32x2*>(odk + c) = u32x2{pack_bf16x2(dk[d][i] * a.scale, dk[d][i + 1] * a.scale),
                                                 pack_bf16x2(dk[d][i + 2] * a.scale, dk[d][i + 3] * a.scale)};
    }
}

template <int DP>
__global__ __launch_bounds__(256, 1) void k_attn_dq(AttnBwdArgs a) {
  constexpr int NP = DP / 8, KS = DP / 16, DB = DP / 32;
  __shared__ __attribute__((aligned(16))) uint8_t sk[kBQ * DP * 2];
  __shared__ __attribute__((aligned(16))) uint8_t sv[kBQ * DP * 2];

  const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kvh = static_cast<int>(blockIdx.x) % a.Hkv, D = a.D, g = a.g;
  const int tiles = static_cast<int>(gridDim.x) / a.Hkv;
  RowTile rt;
  if (!find_rows(a.cu, a.B, a.T, g, kBK, tiles - 1 - static_cast<int>(blockIdx.x) / a.Hkv, &rt)) return;

  const int tok0 = rt.row0 / g, rem0 = rt.row0 - tok0 * g;
  const int x = rem0 + wave * 32 + l32, dt = small_div(x, a.g_inv);
  const bool in = rt.row0 + wave * 32 + l32 < rt.rows;
  const int tok = in ? tok0 + dt : tok0, hq = kvh * g + (in ? x - dt * g : 0);
  const int seen = in ? tok + 1 : 0;
  const int last = (rt.rows - rt.row0 < kBK ? rt.rows : rt.row0 + kBK) - 1;
  const int end = last / g + 1;

  u32x4 qf[KS], yf[KS];
  const int64_t t_row = rt.s0 + tok, o_row = t_row * a.Hq + hq;
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    const int c = 16 * s + 8 * h;
    qf[s] = c < D ? *reinterpret_cast<const u32x4*>(a.q + t_row * a.q_ld + hq * D + c) : u32x4{0, 0, 0, 0};
    yf[s] = c < D ? *reinterpret_cast<const u32x4*>(a.dout + o_row * D + c) : u32x4{0, 0, 0, 0};
  }
  const int64_t at = (static_cast<int64_t>(kvh) * a.T + rt.s0 + tok) * g + (in ? x - dt * g : 0);
  const float lse2 = a.lse2[at], delta = a.delta[at];
  f32x16 dq[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) dq[d] = f32x16{};

  for (int j0 = 0; j0 < end; j0 += kBQ) {
#pragma unroll
    for (int i = 0; i < kBQ * NP / 256; ++i) {
      const int idx = tid + 256 * i, r = idx / NP, c = idx % NP;
      u32x4 k = {0, 0, 0, 0}, v = {0, 0, 0, 0};
      if (j0 + r < rt.n && 8 * c < D) {
        const int64_t row = rt.s0 + j0 + r;
        k = *reinterpret_cast<const u32x4*>(a.k + row * a.k_ld + kvh * D + 8 * c);
        v = *reinterpret_cast<const u32x4*>(a.v + row * a.v_ld + kvh * D + 8 * c);
      }
      *reinterpret_cast<u32x4*>(sk + piece_at<DP>(r, c)) = k;
      *reinterpret_cast<u32x4*>(sv + piece_at<DP>(r, c)) = v;
    }
    __syncthreads();
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      f32x16 s = {}, dp = {};
#pragma unroll
      for (int t = 0; t < KS; ++t) {
        s = mfma32(*reinterpret_cast<const u32x4*>(sk + piece_at<DP>(kb * 32 + l32, 2 * t + h)), qf[t], s);
        dp = mfma32(*reinterpret_cast<const u32x4*>(sv + piece_at<DP>(kb * 32 + l32, 2 * t + h)), yf[t], dp);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const bool on = j0 + kb * 32 + acc_row(i, h) < seen;
        const float p = __builtin_amdgcn_exp2f(s[i] * a.c2 - lse2);
        s[i] = on ? p * (dp[i] - delta) : 0.0f;
      }
#pragma unroll
      for (int kg = 0; kg < 2; ++kg) {
        const u32x4 ds = pack_operand(s, kg);
#pragma unroll
        for (int d = 0; d < DB; ++d) dq[d] = mfma32(column_operand<DP>(sk, kb * 32 + 16 * kg, 32 * d, lane), ds, dq[d]);
      }
    }
    __syncthreads();
  }
  if (!in) return;
  uint16_t* const out = a.dq + t_row * a.dq_ld + hq * D;
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int c = 32 * d + acc_row(i, h);
      if (c < D)
        *reinterpret_cast<u32x2*>(out + c) = u32x2{pack_bf16x2(dq[d][i] * a.scale, dq[d][i + 1] * a.scale),
                                                   pack_bf16x2(dq[d][i + 2] * a.scale, dq[d][i + 3] * a.scale)};
    }
}

template <int DP>
hipError_t launch_bwd(const AttnBwdArgs& a, hipStream_t stream) {
  const int64_t key_tiles = static_cast<int64_t>(a.T) / kBK + a.B, row_tiles = static_cast<int64_t>(a.T) * a.g / kBK + a.B;
  hipLaunchKernelGGL((k_attn_dkdv<DP>), dim3(static_cast<uint32_t>(key_tiles * a.Hkv)), dim3(256), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_attn_dq<DP>), dim3(static_cast<uint32_t>(row_tiles * a.Hkv)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_bwd(const AttnBwdArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(k_attn_delta, dim3(row_grid(static_cast<int64_t>(a.T) * a.Hq, 16)), dim3(256), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return a.D <= 64 ? launch_bwd<64>(a, stream) : launch_bwd<128>(a, stream);
}

}  // namespace qlin
