// Adapter gradient from an 8-bit checkpoint of the layer's input:
//   dA[j][g] = sum_m z[m][j] sum_{k in g} xq[m][k],   z[m][j] = du[m][j] xs[m]
// (groups g of one column, or of 32 for the pooled adapter).  [QLoRA "The
// QLoRA recipe: quantize, then adapt": gradients reach the adapter only;
// QA-LoRA abstract for the pooled adapter]
//
// A code is exact in bf16 (8 significant bits), so the product runs on the
// bf16 matrix cores with z as two planes, hi = bf16(z) and lo = bf16(z - hi),
// which keeps z to 2^-17 relative.  It is one pass over the codes, bound by
// HBM up to rank 64: per step of 16 tokens a wave loads 8 rows per lane half
// of 32 FW columns (FW bytes a lane: column FW l + t of lane l belongs to
// matrix tile t), pairs the bytes of neighbouring tokens into bf16 operands
// in registers, and multiplies them with z's planes, which a small kernel has
// laid out in operand order.  No LDS and no barrier in the loop: the waves of
// a workgroup walk different tokens with the loads of kRing - 1 steps in
// flight, and their sums meet in LDS at the end, in wave order; token shares
// publish fp32 partial sums and the last workgroup of a strip (atomic ticket)
// adds them in share order.
#include "device_common.hpp"
#include "kernels.hpp"

#include <type_traits>

namespace qlin {

namespace {

constexpr int kStep = 16;  // tokens per step

// z's planes in operand order: [step][32-row tile of j][plane][lane (l, h)][8],
// lane (l, h) holding tokens 8 h .. 8 h + 7 of the step for row j = 32 tile + l.
// Rows past r and tokens past M are zero.
__global__ __launch_bounds__(256) void k_z_planes(const float* __restrict__ du, const float* __restrict__ xs,
                                                  int64_t M, int r, int jt, u32x4* __restrict__ out) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;  // (step, tile, lane)
  const int64_t steps = (M + kStep - 1) / kStep;
  if (i >= steps * jt * 64) return;
  const int lane = static_cast<int>(i & 63);
  const int64_t st = i / 64 / jt;
  const int tile = static_cast<int>(i / 64 % jt);
  const int j = 32 * tile + (lane & 31);
  const int64_t m0 = st * kStep + 8 * (lane >> 5);
  float hi[8], lo[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float z = j < r && m0 + e < M ? du[(m0 + e) * r + j] * xs[m0 + e] : 0.0f;
    split_bf16(z, hi[e], lo[e]);
  }
  u32x4 ph, pl;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    ph[e] = pack_bf16x2(hi[2 * e], hi[2 * e + 1]);
    pl[e] = pack_bf16x2(lo[2 * e], lo[2 * e + 1]);
  }
  u32x4* const dst = out + (st * jt + tile) * 128 + lane;
  dst[0] = ph;
  dst[64] = pl;
}

// Byte t of two words as a packed pair of bf16 (exact: the fp32 image of a
// code has nothing below its upper half).
template <int T>
__device__ __forceinline__ uint32_t code_pair(uint32_t a, uint32_t b) {
  const float fa = static_cast<float>(static_cast<int8_t>(a >> (8 * T)));
  const float fb = static_cast<float>(static_cast<int8_t>(b >> (8 * T)));
  return perm(__float_as_uint(fb), __float_as_uint(fa), 0x07060302u);
}

template <int JT, int FW>
__global__ __launch_bounds__(256, 1) void k_da_q8(DaQ8Args a) {
  constexpr int kCols = 32 * FW, kRing = 4, kW = FW / 4;
  __shared__ __attribute__((aligned(16))) f32x4 s_acc[4][FW][4][64];
  __shared__ uint32_t s_ticket;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  const int S = a.splits;
  const int strip = static_cast<int>(blockIdx.x) / S, share = static_cast<int>(blockIdx.x) % S;
  const int64_t M = a.M, K = a.K, k0 = static_cast<int64_t>(strip) * kCols;
  const int64_t steps = (M + kStep - 1) / kStep, per = (steps + 4 * S - 1) / (4 * S);
  const int64_t b0 = (share * 4 + wave) * per;
  const int64_t st0 = b0 < steps ? b0 : steps, st1 = b0 + per < steps ? b0 + per : steps;

  // Rows past M lie outside a step's resource; columns past K hold the next
  // row's codes (or zeros), whose outputs are never stored.
  const uint32_t xo = static_cast<uint32_t>(8 * h * K + k0 + FW * l32);
  const uint32_t zo = static_cast<uint32_t>(lane * 16);
  typedef uint32_t words_t __attribute__((ext_vector_type(kW == 1 ? 2 : kW)));
  words_t xv[kRing][8];
  u32x4 zv[kRing][JT][2];
  auto load = [&](int64_t st, words_t (&x)[8], u32x4 (&z)[JT][2]) {
    const int64_t sc = st < st1 ? st : 0, left = M - sc * kStep;
    const rsrc_t xr = uniform_rsrc(a.xq + sc * kStep * K, st < st1 ? static_cast<uint32_t>((left < kStep ? left : kStep) * K) : 0u);
    const rsrc_t zr = uniform_rsrc(a.z + sc * JT * 128, st < st1 ? JT * 2048u : 0u);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (kW == 2)
        x[e] = __builtin_amdgcn_raw_buffer_load_b64(xr, xo, static_cast<int>(e * K), 0);
      else
        x[e][0] = __builtin_amdgcn_raw_buffer_load_b32(xr, xo, static_cast<int>(e * K), 0);
    }
#pragma unroll
    for (int j = 0; j < JT; ++j)
#pragma unroll
      for (int p = 0; p < 2; ++p) z[j][p] = __builtin_amdgcn_raw_buffer_load_b128(zr, zo, (j * 2 + p) * 1024, 0);
  };

  f32x16 acc[JT][FW];
#pragma unroll
  for (int j = 0; j < JT; ++j)
#pragma unroll
    for (int t = 0; t < FW; ++t) acc[j][t] = f32x16{};
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) load(st0 + i, xv[i], zv[i]);
  for (int64_t st = st0; st < st1; st += kRing) {
#pragma unroll
    for (int i = 0; i < kRing; ++i) {
      load(st + i + kRing - 1, xv[(i + kRing - 1) % kRing], zv[(i + kRing - 1) % kRing]);
      __builtin_amdgcn_sched_barrier(0);
      auto tile = [&](auto T) {
        constexpr int t = decltype(T)::value;
        u32x4 b;
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = code_pair<t & 3>(xv[i][2 * e][t >> 2], xv[i][2 * e + 1][t >> 2]);
#pragma unroll
        for (int j = 0; j < JT; ++j) {
          acc[j][t] = mfma32(zv[i][j][0], b, acc[j][t]);
          acc[j][t] = mfma32(zv[i][j][1], b, acc[j][t]);
        }
      };
      tile(std::integral_constant<int, 0>{});
      tile(std::integral_constant<int, 1>{});
      tile(std::integral_constant<int, 2>{});
      tile(std::integral_constant<int, 3>{});
      if constexpr (FW == 8) {
        tile(std::integral_constant<int, 4>{});
        tile(std::integral_constant<int, 5>{});
        tile(std::integral_constant<int, 6>{});
        tile(std::integral_constant<int, 7>{});
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // Lane (l, h) holds row j = 32 jt + 8 q + 4 h + v of column k0 + FW l + t at
  // acc[jt][t][4 q + v].  The waves' sums, added in wave order: wave w ends
  // with the rows of q = w.
  f32x4 o[JT][FW];
#pragma unroll
  for (int j = 0; j < JT; ++j) {
    __syncthreads();
#pragma unroll
    for (int t = 0; t < FW; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        s_acc[wave][t][q][lane] = f32x4{acc[j][t][4 * q], acc[j][t][4 * q + 1], acc[j][t][4 * q + 2], acc[j][t][4 * q + 3]};
    __syncthreads();
#pragma unroll
    for (int t = 0; t < FW; ++t) {
      o[j][t] = s_acc[0][t][wave][lane];
#pragma unroll
      for (int w = 1; w < 4; ++w) o[j][t] += s_acc[w][t][wave][lane];
    }
  }
  if (S > 1) {
    // partial layout [strip][share][wave][jt][t][lane] x 16 bytes
    constexpr uint32_t kShare = 4u * JT * FW * 1024u;
    const rsrc_t pr = make_rsrc(reinterpret_cast<const uint8_t*>(a.partial) + static_cast<int64_t>(strip) * S * kShare);
    auto off = [&](int sp, int j, int t) {
      return static_cast<uint32_t>(sp) * kShare + static_cast<uint32_t>(((wave * JT + j) * FW + t) * 1024 + lane * 16);
    };
#pragma unroll
    for (int j = 0; j < JT; ++j)
#pragma unroll
      for (int t = 0; t < FW; ++t) st_sys16(pr, off(share, j, t), o[j][t]);
    if (publish_and_ticket(a.counters + strip, &s_ticket) != static_cast<uint32_t>(S - 1)) return;
#pragma unroll
    for (int j = 0; j < JT; ++j)
#pragma unroll
      for (int t = 0; t < FW; ++t) o[j][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int sp = 0; sp < S; ++sp) {
      f32x4 v[JT][FW];
#pragma unroll
      for (int j = 0; j < JT; ++j)
#pragma unroll
        for (int t = 0; t < FW; ++t) v[j][t] = ld_sys16(pr, off(sp, j, t));
#pragma unroll
      for (int j = 0; j < JT; ++j)
#pragma unroll
        for (int t = 0; t < FW; ++t) o[j][t] += v[j][t];
    }
    if (tid == 0) a.counters[strip] = 0u;
  }
  const int64_t k = k0 + FW * l32, G = K / a.pool;
#pragma unroll
  for (int j = 0; j < JT; ++j)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int row = 32 * j + 8 * wave + 4 * h + v;
      if (a.pool == 1) {
        if (row >= a.r || k >= K) continue;
        uint32_t p[FW / 2];
#pragma unroll
        for (int t = 0; t < FW; t += 2) p[t / 2] = pack_bf16x2(o[j][t][v], o[j][t + 1][v]);
        uint16_t* const dst = a.dA + row * K + k;  // 2 FW-byte aligned: K % 64 == 0
        if constexpr (FW == 8) *reinterpret_cast<u32x4*>(dst) = u32x4{p[0], p[1], p[2], p[3]};
        else *reinterpret_cast<u32x2*>(dst) = u32x2{p[0], p[1]};
      } else {
        // a group of 32 columns is 32 / FW lanes
        float t = 0.0f;
#pragma unroll
        for (int c = 0; c < FW; ++c) t += o[j][c][v];
#pragma unroll
        for (int x = 1; x < 32 / FW; x <<= 1) t += __shfl_xor(t, x, 64);
        if (row < a.r && k < K && l32 % (32 / FW) == 0) a.dA[row * G + k / 32] = f32_to_bf16(t);
      }
    }
}

// Columns a lane holds: 8 up to rank 64, 4 above (256 accumulator registers).
int da_fw(int r) { return r <= 64 ? 8 : 4; }

}  // namespace

int da_q8_strips(int64_t K, int r) { return static_cast<int>((K + 32 * da_fw(r) - 1) / (32 * da_fw(r))); }
// Token shares: about one workgroup per compute unit, each wave at least two
// steps.
int da_q8_splits(int64_t M, int64_t K, int r) {
  const int64_t steps = (M + kStep - 1) / kStep;
  int64_t s = 256 / da_q8_strips(K, r);
  if (s > steps / 8) s = steps / 8;
  return static_cast<int>(s < 1 ? 1 : s);
}
int64_t da_q8_partial_floats(int64_t M, int64_t K, int r) {
  const int64_t s = da_q8_splits(M, K, r);
  return s > 1 ? s * da_q8_strips(K, r) * 4 * ((r + 31) / 32) * da_fw(r) * 256 : 0;
}
int64_t da_q8_z_bytes(int64_t M, int r) { return (M + kStep - 1) / kStep * ((r + 31) / 32) * 2048; }

hipError_t launch_da_q8(const DaQ8Args& a, hipStream_t stream) {
  const int jt = (a.r + 31) / 32;
  const int64_t n = (a.M + kStep - 1) / kStep * jt * 64;
  hipLaunchKernelGGL(k_z_planes, dim3(static_cast<uint32_t>((n + 255) / 256)), dim3(256), 0, stream, a.du, a.xs, a.M,
                     a.r, jt, const_cast<u32x4*>(a.z));
  const dim3 grid(static_cast<uint32_t>(da_q8_strips(a.K, a.r) * a.splits)), block(256);
  switch (jt) {
    case 1: hipLaunchKernelGGL((k_da_q8<1, 8>), grid, block, 0, stream, a); break;
    case 2: hipLaunchKernelGGL((k_da_q8<2, 8>), grid, block, 0, stream, a); break;
    case 3: hipLaunchKernelGGL((k_da_q8<3, 4>), grid, block, 0, stream, a); break;
    default: hipLaunchKernelGGL((k_da_q8<4, 4>), grid, block, 0, stream, a); break;
  }
  return hipGetLastError();
}

}  // namespace qlin
