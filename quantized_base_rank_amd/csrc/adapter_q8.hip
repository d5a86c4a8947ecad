// Adapter gradients as streaming products on the bf16 matrix cores, with no
// LDS and no barrier in their loops.  [QLoRA "The QLoRA recipe: quantize,
// then adapt": gradients reach the adapter only; QA-LoRA abstract for the
// pooled adapter]
//
//   du[m][j] = s sum_n dY[m][n] B[n][j]                          k_du_stream
//   dB[n][j] = s sum_m u[m][j] dY[m][n]                          k_tokens<bf16>
//   dA[j][g] = sum_m du[m][j] xs[m] sum_{k in g} xq[m][k]        k_tokens<8-bit>
// (groups g of one column, or of 32 for the pooled adapter).
//
// An operand of the matrix instruction holds eight consecutive reduction
// indices of one column per lane.  Where the reduction runs along a matrix's
// rows, a lane loads 16 or 8 bytes of each of eight rows (several columns) and
// pairs neighbouring rows' values in registers: column FW l + t of lane l
// belongs to matrix tile t, so neither operand is transposed through memory.
// The waves of a workgroup walk different parts of the reduction with a ring
// of loads in flight; their sums meet in LDS at the end, in wave order, and
// shares of the reduction publish fp32 partial sums that the last workgroup
// of a tile (atomic ticket) adds in share order.
#include "device_common.hpp"
#include "kernels.hpp"

#include <type_traits>

namespace qlin {

namespace {

// Adds the four waves' sums in wave order: wave w ends with part w of each of
// the G groups of lane values.  s_acc holds 4 * G * 4 * 64 f32x4.
template <int G>
__device__ __forceinline__ void join_waves(f32x4* s_acc, int wave, int lane, const f32x4 (&v)[G][4], f32x4 (&o)[G]) {
  __syncthreads();
#pragma unroll
  for (int t = 0; t < G; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) s_acc[((wave * G + t) * 4 + q) * 64 + lane] = v[t][q];
  __syncthreads();
#pragma unroll
  for (int t = 0; t < G; ++t) {
    o[t] = s_acc[(t * 4 + wave) * 64 + lane];
#pragma unroll
    for (int w = 1; w < 4; ++w) o[t] += s_acc[((w * G + t) * 4 + wave) * 64 + lane];
  }
}

// Publishes a workgroup's G lane values per wave as share `share` of `S`;
// true in the last workgroup of `tile`, whose o then holds the shares' sum.
template <int G>
__device__ __forceinline__ bool join_shares(float* partial, uint32_t* counters, int tile, int share, int S, int wave,
                                            int lane, f32x4 (&o)[G], uint32_t* s_ticket) {
  constexpr uint32_t kShare = 4u * G * 1024u;
  const rsrc_t pr = make_rsrc(reinterpret_cast<const uint8_t*>(partial) + static_cast<int64_t>(tile) * S * kShare);
  auto off = [&](int sp, int t) {
    return static_cast<uint32_t>(sp) * kShare + static_cast<uint32_t>((wave * G + t) * 1024 + lane * 16);
  };
#pragma unroll
  for (int t = 0; t < G; ++t) st_sys16(pr, off(share, t), o[t]);
  if (publish_and_ticket(counters + tile, s_ticket) != static_cast<uint32_t>(S - 1)) return false;
#pragma unroll
  for (int t = 0; t < G; ++t) o[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int sp = 0; sp < S; ++sp) {
    f32x4 v[G];
#pragma unroll
    for (int t = 0; t < G; ++t) v[t] = ld_sys16(pr, off(sp, t));
#pragma unroll
    for (int t = 0; t < G; ++t) o[t] += v[t];
  }
  if (threadIdx.x == 0) counters[tile] = 0u;
  return true;
}

// ------------------------------------------------------- sums over the tokens

constexpr int kStep = 16;  // tokens per step

// Byte t of two words as a packed pair of bf16 (exact: the fp32 image of a
// code has nothing below its upper half).
template <int T>
__device__ __forceinline__ uint32_t code_pair(uint32_t a, uint32_t b) {
  const float fa = static_cast<float>(static_cast<int8_t>(a >> (8 * T)));
  const float fb = static_cast<float>(static_cast<int8_t>(b >> (8 * T)));
  return perm(__float_as_uint(fb), __float_as_uint(fa), 0x07060302u);
}

// C = Z^T X over the tokens: Z fp32 [M][r] (times xs[m] for 8-bit rows) as two
// bf16 planes, hi = bf16(z) and lo = bf16(z - hi), which keep z to 2^-17
// relative; X the codes (exact in bf16) or bf16 rows.  One pass over X, whose
// strip of 32 FW columns a workgroup takes for a share of the tokens: FW
// columns a lane, JT 32-row tiles of Z's columns, 16 JT FW accumulators.
// HBM-bound up to rank 64 (4096 x 28672 codes: TIME).
template <bool Q8, int JT, int FW>
__global__ __launch_bounds__(256, 1) void k_tokens(TokensArgs a) {
  constexpr int kCols = 32 * FW, kRing = Q8 ? 4 : 3;
  constexpr int kBytes = Q8 ? FW : 2 * FW, kW = kBytes / 4;  // of a lane's piece of a row
  __shared__ __attribute__((aligned(16))) f32x4 s_acc[4 * FW * 4 * 64];
  __shared__ uint32_t s_ticket;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  const int S = a.splits, r = a.r;
  const int strip = static_cast<int>(blockIdx.x) / S, share = static_cast<int>(blockIdx.x) % S;
  const int64_t M = a.M, P = a.P, p0 = static_cast<int64_t>(strip) * kCols;
  const int64_t steps = (M + kStep - 1) / kStep, per = (steps + 4 * S - 1) / (4 * S);
  const int64_t b0 = (share * 4 + wave) * per;
  const int64_t st0 = b0 < steps ? b0 : steps, st1 = b0 + per < steps ? b0 + per : steps;

  // Rows past M lie outside a step's resources (zeros).  Columns past P hold
  // the next row's values (or zeros), and rows of Z past r the last one's:
  // their outputs are never stored.
  constexpr int kEl = Q8 ? 1 : 2;
  const uint32_t xo = static_cast<uint32_t>((8 * h * P + p0 + FW * l32) * kEl);
  uint32_t zo[JT];
#pragma unroll
  for (int j = 0; j < JT; ++j) zo[j] = static_cast<uint32_t>((8 * h * r + (32 * j + l32 < r ? 32 * j + l32 : r - 1)) * 4);
  typedef uint32_t words_t __attribute__((ext_vector_type(kW == 1 ? 2 : kW)));
  struct Step {
    words_t x[8];
    float z[JT][8];
    f32x4 s[2];
  };
  Step ring[kRing];
  auto load = [&](int64_t st, Step& v) {
    const bool in = st < st1;
    const int64_t m = (in ? st : 0) * kStep;
    const uint32_t rows = in ? static_cast<uint32_t>(M - m < kStep ? M - m : kStep) : 0u;
    const rsrc_t xr = uniform_rsrc(static_cast<const uint8_t*>(a.X) + m * P * kEl, rows * static_cast<uint32_t>(P * kEl));
    const rsrc_t zr = uniform_rsrc(a.Z + m * r, rows * static_cast<uint32_t>(r * 4));
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int so = static_cast<int>(e * P * kEl);
      if constexpr (kW == 4) v.x[e] = __builtin_amdgcn_raw_buffer_load_b128(xr, xo, so, 0);
      else if constexpr (kW == 2) v.x[e] = __builtin_amdgcn_raw_buffer_load_b64(xr, xo, so, 0);
      else v.x[e][0] = __builtin_amdgcn_raw_buffer_load_b32(xr, xo, so, 0);
    }
#pragma unroll
    for (int j = 0; j < JT; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v.z[j][e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(zr, zo[j], e * r * 4, 0));
    if constexpr (Q8) {
      const rsrc_t sr = uniform_rsrc(a.xs + m, rows * 4u);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        v.s[i] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(sr, static_cast<uint32_t>(32 * h + 16 * i), 0, 0));
    }
  };

  f32x16 acc[JT][FW];
#pragma unroll
  for (int j = 0; j < JT; ++j)
#pragma unroll
    for (int t = 0; t < FW; ++t) acc[j][t] = f32x16{};
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) load(st0 + i, ring[i]);
  for (int64_t st = st0; st < st1; st += kRing) {
#pragma unroll
    for (int i = 0; i < kRing; ++i) {
      load(st + i + kRing - 1, ring[(i + kRing - 1) % kRing]);
      __builtin_amdgcn_sched_barrier(0);
      const Step& v = ring[i];
      u32x4 zh[JT], zl[JT];
#pragma unroll
      for (int j = 0; j < JT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float z0 = v.z[j][2 * e], z1 = v.z[j][2 * e + 1];
          if constexpr (Q8) {
            z0 *= v.s[e >> 1][2 * (e & 1)];
            z1 *= v.s[e >> 1][2 * (e & 1) + 1];
          }
          zh[j][e] = pack_bf16x2(z0, z1);
          zl[j][e] = pack_bf16x2(z0 - bf16_lo(zh[j][e]), z1 - bf16_hi(zh[j][e]));
        }
      auto tile = [&](auto T) {
        constexpr int t = decltype(T)::value;
        u32x4 b;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (Q8) b[e] = code_pair<t & 3>(v.x[2 * e][t >> 2], v.x[2 * e + 1][t >> 2]);
          else b[e] = perm(v.x[2 * e + 1][t >> 1], v.x[2 * e][t >> 1], (t & 1) ? 0x07060302u : 0x05040100u);
        }
#pragma unroll
        for (int j = 0; j < JT; ++j) {
          acc[j][t] = mfma32(zh[j], b, acc[j][t]);
          acc[j][t] = mfma32(zl[j], b, acc[j][t]);
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

  // Lane (l, h) holds row j = 32 jt + 8 q + 4 h + v of column p0 + FW l + t at
  // acc[jt][t][4 q + v]; wave w ends with the rows of q = w.
  f32x4 o[JT * FW];
#pragma unroll
  for (int j = 0; j < JT; ++j) {
    f32x4 v[FW][4], part[FW];
#pragma unroll
    for (int t = 0; t < FW; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q) v[t][q] = f32x4{acc[j][t][4 * q], acc[j][t][4 * q + 1], acc[j][t][4 * q + 2], acc[j][t][4 * q + 3]};
    join_waves<FW>(s_acc, wave, lane, v, part);
#pragma unroll
    for (int t = 0; t < FW; ++t) o[j * FW + t] = part[t];
  }
  if (S > 1 && !join_shares<JT * FW>(a.partial, a.counters, strip, share, S, wave, lane, o, &s_ticket)) return;
  const int64_t p = p0 + FW * l32, G = P / a.pool;
#pragma unroll
  for (int j = 0; j < JT; ++j) {
    const int row0 = 32 * j + 8 * wave + 4 * h;
    if constexpr (!Q8) {
      // dB[n][j]: four consecutive j of each of the lane's columns
#pragma unroll
      for (int t = 0; t < FW; ++t) {
        if (p + t >= P) continue;
        const f32x4 c = o[j * FW + t];
        uint16_t* const dst = a.C + (p + t) * r + row0;
        if (row0 + 4 <= r) {
          typedef u32x2 u32x2h __attribute__((aligned(2)));
          *reinterpret_cast<u32x2h*>(dst) = u32x2{pack_bf16x2(a.alpha * c[0], a.alpha * c[1]), pack_bf16x2(a.alpha * c[2], a.alpha * c[3])};
        } else {
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (row0 + v < r) dst[v] = f32_to_bf16(a.alpha * c[v]);
        }
      }
    } else {
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int row = row0 + v;
        if (a.pool == 1) {
          if (row >= r || p >= P) continue;
          uint32_t w[FW / 2];
#pragma unroll
          for (int t = 0; t < FW; t += 2) w[t / 2] = pack_bf16x2(a.alpha * o[j * FW + t][v], a.alpha * o[j * FW + t + 1][v]);
          uint16_t* const dst = a.C + row * P + p;  // 2 FW-byte aligned: P % 64 == 0
          if constexpr (FW == 8) *reinterpret_cast<u32x4*>(dst) = u32x4{w[0], w[1], w[2], w[3]};
          else *reinterpret_cast<u32x2*>(dst) = u32x2{w[0], w[1]};
        } else {
          // a group of 32 columns is 32 / FW lanes
          float t = 0.0f;
#pragma unroll
          for (int c = 0; c < FW; ++c) t += o[j * FW + c][v];
#pragma unroll
          for (int x = 1; x < 32 / FW; x <<= 1) t += __shfl_xor(t, x, 64);
          if (row < r && p < P && l32 % (32 / FW) == 0) a.C[row * G + p / 32] = f32_to_bf16(a.alpha * t);
        }
      }
    }
  }
}

// Columns a lane holds: 8 up to rank 64, 4 above (256 accumulator registers).
int tokens_fw(int r) { return r <= 64 ? 8 : 4; }

// ------------------------------------------------- sums over the output features

// du = s dY B: a workgroup takes 64 tokens (four 16-row operands of the
// 16x16x32 instruction, lane (l, g): 8 consecutive n from 8 g of row l, so 64
// bytes of each row a load) and a share of the n; B's rows are paired in
// registers, lane l holding columns c0 .. c0 + FW - 1 with c0 = FW l, moved
// back inside the row where it would pass r (those columns are then formed
// twice, alike).
template <int FW>
__global__ __launch_bounds__(256, 1) void k_du_stream(DuArgs a) {
  constexpr int kRing = FW == 8 ? 3 : 4, kW = FW >= 2 ? FW / 2 : 1;
  __shared__ __attribute__((aligned(16))) f32x4 s_acc[4 * FW * 4 * 64];
  __shared__ uint32_t s_ticket;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int S = a.splits, r = a.r;
  const int tile = static_cast<int>(blockIdx.x) / S, share = static_cast<int>(blockIdx.x) % S;
  const int64_t M = a.M, N = a.N, m0 = static_cast<int64_t>(tile) * 64;
  const int slices = static_cast<int>((N + 31) / 32), per = (slices + 4 * S - 1) / (4 * S);
  const int b0 = (share * 4 + wave) * per;
  const int s0 = b0 < slices ? b0 : slices, s1 = b0 + per < slices ? b0 + per : slices;
  const int64_t rows = M - m0 < 64 ? M - m0 : 64;
  const rsrc_t yr = uniform_rsrc(a.dy + m0 * N, static_cast<uint32_t>(rows * N * 2));
  const int c0 = FW * l16 + FW <= r ? FW * l16 : r - FW;
  uint32_t yo[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) yo[t] = static_cast<uint32_t>(((16 * t + l16) * N + 8 * g) * 2);
  typedef uint32_t words_t __attribute__((ext_vector_type(kW == 1 ? 2 : kW)));
  struct Slice {
    u32x4 y[4];
    words_t b[8];
  };
  Slice ring[kRing];
  auto load = [&](int sl, Slice& v) {
    // Past the wave's share, and past N (a multiple of 16) in the last slice:
    // dY reads as zero, B as its last rows, which are cleared.
    const bool in = sl < s1;
    const int64_t n = static_cast<int64_t>(in ? sl : 0) * 32 + 8 * g;
    const bool ok = in && n < N;
    const int so = in ? sl * 64 : 0;
#pragma unroll
    for (int t = 0; t < 4; ++t) v.y[t] = __builtin_amdgcn_raw_buffer_load_b128(yr, ok ? yo[t] : 0x80000000u, so, 0);
    const uint16_t* const bp = a.B + (n < N ? n : 0) * r + c0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint16_t* const q = bp + e * r;
      if constexpr (FW == 1) {
        v.b[e][0] = *q;
      } else {
        typedef words_t words_u __attribute__((aligned(2)));
        typedef uint32_t word_u __attribute__((aligned(2)));
        if constexpr (kW == 1) v.b[e][0] = *reinterpret_cast<const word_u*>(q);
        else v.b[e] = *reinterpret_cast<const words_u*>(q);
      }
    }
  };
  f32x4 acc[FW][4];  // [column of the lane][16 tokens]
#pragma unroll
  for (int t = 0; t < FW; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[t][q] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) load(s0 + i, ring[i]);
  for (int sl = s0; sl < s1; sl += kRing) {
#pragma unroll
    for (int i = 0; i < kRing; ++i) {
      load(sl + i + kRing - 1, ring[(i + kRing - 1) % kRing]);
      __builtin_amdgcn_sched_barrier(0);
      const Slice& v = ring[i];
      const bool ok = sl + i < s1 && static_cast<int64_t>(sl + i) * 32 + 8 * g < N;
#pragma unroll
      for (int t = 0; t < FW; ++t) {
        u32x4 b;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t w = perm(v.b[2 * e + 1][t >> 1], v.b[2 * e][t >> 1], (t & 1) ? 0x07060302u : 0x05040100u);
          b[e] = ok ? w : 0u;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[t][q] = mfma16(v.y[q], b, acc[t][q]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // lane (l, g) holds token 16 q + 4 g + v of column c0 + t; wave w ends with q = w
  f32x4 o[FW];
  join_waves<FW>(s_acc, wave, lane, acc, o);
  if (S > 1 && !join_shares<FW>(a.partial, a.counters, tile, share, S, wave, lane, o, &s_ticket)) return;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int64_t m = m0 + 16 * wave + 4 * g + v;
    if (m >= M || FW * l16 >= r) continue;
#pragma unroll
    for (int t = 0; t < FW; ++t) a.du[m * r + c0 + t] = a.s * o[t][v];
  }
}

int du_fw(int r) { return r <= 16 ? 1 : r <= 32 ? 2 : r <= 64 ? 4 : 8; }

}  // namespace

int64_t tokens_strips(int64_t P, int r) { return (P + 32 * tokens_fw(r) - 1) / (32 * tokens_fw(r)); }
// Token shares: about one workgroup per compute unit, each wave at least two
// steps.
int tokens_splits(int64_t M, int64_t P, int r) {
  const int64_t steps = (M + kStep - 1) / kStep;
  int64_t s = 256 / tokens_strips(P, r);
  if (s > steps / 8) s = steps / 8;
  return static_cast<int>(s < 1 ? 1 : s);
}
int64_t tokens_partial_floats(int64_t M, int64_t P, int r) {
  const int64_t s = tokens_splits(M, P, r);
  return s > 1 ? s * tokens_strips(P, r) * 4 * ((r + 31) / 32) * tokens_fw(r) * 256 : 0;
}

hipError_t launch_tokens(const TokensArgs& a, bool q8, hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>(tokens_strips(a.P, a.r) * a.splits)), block(256);
  switch ((a.r + 31) / 32) {
    case 1:
      if (q8) hipLaunchKernelGGL((k_tokens<true, 1, 8>), grid, block, 0, stream, a);
      else hipLaunchKernelGGL((k_tokens<false, 1, 8>), grid, block, 0, stream, a);
      break;
    case 2:
      if (q8) hipLaunchKernelGGL((k_tokens<true, 2, 8>), grid, block, 0, stream, a);
      else hipLaunchKernelGGL((k_tokens<false, 2, 8>), grid, block, 0, stream, a);
      break;
    case 3:
      if (q8) hipLaunchKernelGGL((k_tokens<true, 3, 4>), grid, block, 0, stream, a);
      else hipLaunchKernelGGL((k_tokens<false, 3, 4>), grid, block, 0, stream, a);
      break;
    default:
      if (q8) hipLaunchKernelGGL((k_tokens<true, 4, 4>), grid, block, 0, stream, a);
      else hipLaunchKernelGGL((k_tokens<false, 4, 4>), grid, block, 0, stream, a);
      break;
  }
  return hipGetLastError();
}

int64_t du_tiles(int64_t M) { return (M + 63) / 64; }
int du_splits(int64_t M, int64_t N) {
  int64_t s = 256 / du_tiles(M);
  const int64_t slices = (N + 31) / 32;
  if (s > slices / 8) s = slices / 8;
  return static_cast<int>(s < 1 ? 1 : s);
}
int64_t du_partial_floats(int64_t M, int64_t N, int r) {
  const int64_t s = du_splits(M, N);
  return s > 1 ? s * du_tiles(M) * 4 * du_fw(r) * 256 : 0;
}

hipError_t launch_du_stream(const DuArgs& a, hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>(du_tiles(a.M) * a.splits)), block(256);
  switch (du_fw(a.r)) {
    case 1: hipLaunchKernelGGL(k_du_stream<1>, grid, block, 0, stream, a); break;
    case 2: hipLaunchKernelGGL(k_du_stream<2>, grid, block, 0, stream, a); break;
    case 4: hipLaunchKernelGGL(k_du_stream<4>, grid, block, 0, stream, a); break;
    default: hipLaunchKernelGGL(k_du_stream<8>, grid, block, 0, stream, a); break;
  }
  return hipGetLastError();
}

}  // namespace qlin
