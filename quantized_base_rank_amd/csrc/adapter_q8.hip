// Adapter gradients as streaming products on the bf16 matrix cores, with no
// LDS and no barrier in their loops.  [QLoRA "The QLoRA recipe: quantize,
// then adapt": gradients reach the adapter only; QA-LoRA abstract for the
// pooled adapter]
//
//   du[m][j] = s sum_n dY[m][n] B[n][j]                          k_du
//   dB[n][j] = s sum_m u[m][j] dY[m][n]                          k_tokens
//   dA[j][g] = sum_m du[m][j] xs[m] sum_{k in g} xq[m][k]        k_tokens
// (groups g of one column, or of 32 for the pooled adapter).  Two launches:
// k_du also lays the factors of the sums over tokens, u and du xs, out as
// operands; k_tokens forms dB and dA.
//
// An operand of the matrix instruction holds eight consecutive reduction
// indices of one column per lane.  Where the reduction runs along a matrix's
// rows, a lane loads a few columns of each of eight rows and pairs
// neighbouring rows' values in registers: column FW l + t of lane l belongs
// to matrix tile t, so no operand is transposed through memory.  The waves of
// a workgroup walk different parts of the reduction with a ring of loads in
// flight; their sums meet in LDS at the end, in wave order, and shares of the
// reduction publish fp32 partial sums that the last workgroup of a tile
// (atomic ticket) adds in share order.
#include "device_common.hpp"
#include "kernels.hpp"

#include <type_traits>

namespace qlin {

namespace {

// Adds W waves' lane values in wave order: of each of the G groups of four,
// wave w < 4 ends with part w.  s_acc holds W * G * 4 * 64 f32x4.
template <int W, int G>
__device__ __forceinline__ void join_waves(f32x4* s_acc, int wave, int lane, const f32x4 (&v)[G][4], f32x4 (&o)[G]) {
  __syncthreads();
#pragma unroll
  for (int t = 0; t < G; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) s_acc[((wave * G + t) * 4 + q) * 64 + lane] = v[t][q];
  __syncthreads();
  if (wave >= 4) return;
#pragma unroll
  for (int t = 0; t < G; ++t) {
    o[t] = s_acc[(t * 4 + wave) * 64 + lane];
#pragma unroll
    for (int w = 1; w < W; ++w) o[t] += s_acc[((w * G + t) * 4 + wave) * 64 + lane];
  }
}

// o = the S shares' published values, added in share order, several shares'
// loads in flight (one after the other they cost over a microsecond each).
template <int G, typename Off>
__device__ __forceinline__ void add_shares(rsrc_t pr, int S, Off off, f32x4 (&o)[G]) {
  constexpr int kBatch = G >= 8 ? 2 : 16 / G;
#pragma unroll
  for (int t = 0; t < G; ++t) o[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int sp0 = 0; sp0 < S; sp0 += kBatch) {
    f32x4 v[kBatch][G];
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
#pragma unroll
      for (int t = 0; t < G; ++t) v[b][t] = ld_sys16(pr, off(sp0 + b < S ? sp0 + b : S - 1, t));
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      if (sp0 + b < S)
#pragma unroll
        for (int t = 0; t < G; ++t) o[t] += v[b][t];
  }
}

// Publishes the G lane values of a workgroup's first four waves as share
// `share` of `S`; true in the last workgroup of `tile`, whose o then holds the
// shares' sum.
template <int G>
__device__ __forceinline__ bool join_shares(float* partial, uint32_t* counters, int tile, int share, int S, int wave,
                                            int lane, f32x4 (&o)[G], uint32_t* s_ticket) {
  constexpr uint32_t kShare = 4u * G * 1024u;
  const rsrc_t pr = make_rsrc(reinterpret_cast<const uint8_t*>(partial) + static_cast<int64_t>(tile) * S * kShare);
  auto off = [&](int sp, int t) {
    return static_cast<uint32_t>(sp) * kShare + static_cast<uint32_t>((wave * G + t) * 1024 + lane * 16);
  };
  if (wave < 4)
#pragma unroll
    for (int t = 0; t < G; ++t) st_sys16(pr, off(share, t), o[t]);
  if (publish_and_ticket(counters + tile, s_ticket) != static_cast<uint32_t>(S - 1)) return false;
  if (threadIdx.x == 0) counters[tile] = 0u;
  if (wave < 4) add_shares<G>(pr, S, off, o);
  return true;
}

// A factor Z [M][r] of the sums over tokens as two bf16 planes, hi = bf16(z)
// and lo = bf16(z - hi) (z to 2^-17 relative), in operand order:
// [step of 16 tokens][32-column tile][plane][lane (l, h)][8], lane (l, h)
// holding tokens 8 h .. 8 h + 7 of column 32 tile + l.
constexpr int kStep = 16;

__device__ __forceinline__ void store_planes(u32x4* out, int64_t step, int jt, int tile, int lane, const float (&z)[8]) {
  u32x4 hi, lo;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    hi[e] = pack_bf16x2(z[2 * e], z[2 * e + 1]);
    lo[e] = pack_bf16x2(z[2 * e] - bf16_lo(hi[e]), z[2 * e + 1] - bf16_hi(hi[e]));
  }
  u32x4* const dst = out + (step * jt + tile) * 128 + lane;
  dst[0] = hi;
  dst[64] = lo;
}

// ------------------------------------------------------- sums over the tokens

// Byte t of two words as a packed pair of bf16 (exact: the fp32 image of a
// code has nothing below its upper half).
template <int T>
__device__ __forceinline__ uint32_t code_pair(uint32_t a, uint32_t b) {
  const float fa = static_cast<float>(static_cast<int8_t>(a >> (8 * T)));
  const float fb = static_cast<float>(static_cast<int8_t>(b >> (8 * T)));
  return perm(__float_as_uint(fb), __float_as_uint(fa), 0x07060302u);
}

// C = alpha Z^T X over the tokens, Z as planes, X the codes (exact in bf16) or
// bf16 rows: one pass over X, of which a workgroup takes a strip of 128
// columns (four a lane) and a share of the tokens.  Waves: two per SIMD up to
// rank 64 (128 accumulators each), so that one pairs its operands while the
// other multiplies; one above.  dB and dA of 4096 tokens, 8192 x 28672, rank
// 64 (184 MB): 58 us, 3.2 TB/s; the codes alone 35 us.  No one resource is
// full there: matrix cores busy 26 % of the cycles, half of the wave cycles
// waiting to issue.  L2 serves 495 MB for the 184 MB of operands, since every
// strip reads all of Z's planes again (288 strips, 1 MB each).  Timing copies:
// 50 us without Z's traffic, 44 without X's, 42 without either's, 35 with half
// of the matrix instructions besides; two rounds of workgroups pay start and
// join, some 7 us each.  Slower: eight columns a lane and one wave per SIMD
// 62-65 us, z's planes formed here from fp32 78 us, other numbers of shares
// 62-74 us.
constexpr int kFW = 4, kStrip = 32 * kFW;
constexpr int tokens_waves(int jt) { return jt <= 2 ? 8 : 4; }

template <bool Q8, int JT>
__device__ __forceinline__ void tokens_block(const TokensArgs& a, int block, f32x4* s_acc, uint32_t* s_ticket) {
  constexpr int kWaves = tokens_waves(JT), kRing = 3;
  constexpr int kEl = Q8 ? 1 : 2, kW = kEl;  // words of a lane's piece of a row
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  const int S = a.splits, r = a.r;
  const int strip = block / S, share = block % S;
  const int64_t M = a.M, P = a.P, p0 = static_cast<int64_t>(strip) * kStrip;
  const int64_t steps = (M + kStep - 1) / kStep, per = (steps + kWaves * S - 1) / (kWaves * S);
  const int64_t b0 = (share * kWaves + wave) * per;
  const int64_t st0 = b0 < steps ? b0 : steps;
  // this wave's steps
  const int n = __builtin_amdgcn_readfirstlane(static_cast<int>(b0 + per < steps ? per : steps - st0));

  // Rows past M lie outside a step's resource (zeros, as Z's planes there),
  // and so does everything past the wave's steps.  Columns past P hold the
  // next row's values (or zeros), and columns of Z past r zeros: their
  // outputs are never stored.  The loads take the steps in order, so bases
  // and rows left are carried along in scalar registers.
  const uint32_t xo = static_cast<uint32_t>((8 * h * P + p0 + kFW * l32) * kEl);
  const uint32_t zo = static_cast<uint32_t>(lane * 16);
  const int row_bytes = static_cast<int>(P * kEl);
  typedef uint32_t words_t __attribute__((ext_vector_type(2)));
  words_t x[kRing][8];
  u32x4 z[kRing][JT][2];
  const uint8_t* x_base = static_cast<const uint8_t*>(a.X) + st0 * kStep * row_bytes;
  const u32x4* z_base = a.Z + st0 * JT * 128;
  int x_rows = __builtin_amdgcn_readfirstlane(
      static_cast<int>(M - st0 * kStep < static_cast<int64_t>(n) * kStep ? M - st0 * kStep : static_cast<int64_t>(n) * kStep));
  int z_steps = n;
  auto load_x = [&](words_t (&v)[8]) {
    const int rows = x_rows < 0 ? 0 : x_rows < kStep ? x_rows : kStep;
    const rsrc_t xr = uniform_rsrc(x_base, static_cast<uint32_t>(rows) * static_cast<uint32_t>(row_bytes));
    x_base += kStep * static_cast<int64_t>(row_bytes);
    x_rows -= kStep;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (kW == 2) v[e] = __builtin_amdgcn_raw_buffer_load_b64(xr, xo, e * row_bytes, 0);
      else v[e][0] = __builtin_amdgcn_raw_buffer_load_b32(xr, xo, e * row_bytes, 0);
    }
  };
  auto load_z = [&](u32x4 (&v)[JT][2]) {
    const rsrc_t zr = uniform_rsrc(z_base, z_steps > 0 ? JT * 2048u : 0u);
    z_base += JT * 128;
    --z_steps;
#pragma unroll
    for (int j = 0; j < JT; ++j)
#pragma unroll
      for (int p = 0; p < 2; ++p) v[j][p] = __builtin_amdgcn_raw_buffer_load_b128(zr, zo, (j * 2 + p) * 1024, 0);
  };

  f32x16 acc[JT][kFW];
#pragma unroll
  for (int j = 0; j < JT; ++j)
#pragma unroll
    for (int t = 0; t < kFW; ++t) acc[j][t] = f32x16{};
  // (issued in the loop's own order: at the loop's head the compiler waits for
  // what both ways in leave pending)
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) {
    load_z(z[i]);
    load_x(x[i]);
    __builtin_amdgcn_sched_barrier(0);
  }
  for (int st = 0; st < n; st += kRing) {
#pragma unroll
    for (int i = 0; i < kRing; ++i) {
      load_z(z[(i + kRing - 1) % kRing]);
      load_x(x[(i + kRing - 1) % kRing]);
      __builtin_amdgcn_sched_barrier(0);
      auto tile = [&](auto T) {
        constexpr int t = decltype(T)::value;
        u32x4 b;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (Q8) b[e] = code_pair<t>(x[i][2 * e][0], x[i][2 * e + 1][0]);
          else b[e] = perm(x[i][2 * e + 1][t >> 1], x[i][2 * e][t >> 1], (t & 1) ? 0x07060302u : 0x05040100u);
        }
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int j = 0; j < JT; ++j) acc[j][t] = mfma32(z[i][j][p], b, acc[j][t]);
      };
      // (a branch may skip arithmetic; one past the loads would make the
      // compiler copy or spill what it carries round the loop)
      if (i == 0 || st + i < n) {
        tile(std::integral_constant<int, 0>{});
        tile(std::integral_constant<int, 1>{});
        tile(std::integral_constant<int, 2>{});
        tile(std::integral_constant<int, 3>{});
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // Lane (l, h) holds row j = 32 jt + 8 q + 4 h + v of column p0 + 4 l + t at
  // acc[jt][t][4 q + v]; wave w < 4 ends with the rows of q = w.
  f32x4 o[JT * kFW];
#pragma unroll
  for (int j = 0; j < JT; ++j) {
    f32x4 v[kFW][4], part[kFW];
#pragma unroll
    for (int t = 0; t < kFW; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q) v[t][q] = f32x4{acc[j][t][4 * q], acc[j][t][4 * q + 1], acc[j][t][4 * q + 2], acc[j][t][4 * q + 3]};
    join_waves<kWaves, kFW>(s_acc, wave, lane, v, part);
#pragma unroll
    for (int t = 0; t < kFW; ++t) o[j * kFW + t] = part[t];
  }
  if (S > 1 && !join_shares<JT * kFW>(a.partial, a.counters, strip, share, S, wave, lane, o, s_ticket)) return;
  if (wave >= 4) return;
  const int64_t p = p0 + kFW * l32, G = P / a.pool;
#pragma unroll
  for (int j = 0; j < JT; ++j) {
    const int row0 = 32 * j + 8 * wave + 4 * h;
    if constexpr (!Q8) {
      // dB[n][j]: four consecutive j of each of the lane's columns
      if (p >= P) continue;  // (P is a multiple of 16: all four columns or none)
#pragma unroll
      for (int t = 0; t < kFW; ++t) {
        const f32x4 c = o[j * kFW + t];
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
        const f32x4 c{o[j * kFW][v], o[j * kFW + 1][v], o[j * kFW + 2][v], o[j * kFW + 3][v]};
        if (a.pool == 1) {
          if (row < r && p < P)
            *reinterpret_cast<u32x2*>(a.C + row * P + p) =
                u32x2{pack_bf16x2(a.alpha * c[0], a.alpha * c[1]), pack_bf16x2(a.alpha * c[2], a.alpha * c[3])};
        } else {
          // a group of 32 columns is eight lanes
          float t = ((c[0] + c[1]) + c[2]) + c[3];
#pragma unroll
          for (int k = 1; k < 8; k <<= 1) t += __shfl_xor(t, k, 64);
          if (row < r && p < P && (l32 & 7) == 0) a.C[row * G + p / 32] = f32_to_bf16(a.alpha * t);
        }
      }
    }
  }
}

// dA's blocks, the longer ones, then dB's.
template <int JT>
__global__ __launch_bounds__(64 * tokens_waves(JT), tokens_waves(JT) / 4) void k_tokens(TokensArgs b, TokensArgs a) {
  __shared__ __attribute__((aligned(16))) f32x4 s_acc[tokens_waves(JT) * kFW * 4 * 64];
  __shared__ uint32_t s_ticket;
  const int block = static_cast<int>(blockIdx.x);
  if (block < a.blocks)
    tokens_block<true, JT>(a, block, s_acc, &s_ticket);
  else
    tokens_block<false, JT>(b, block - a.blocks, s_acc, &s_ticket);
}

// ------------------------------------------------- sums over the output features

// du = s dY B: a workgroup of 4 waves takes 16 RT tokens (RT operands of the
// 16x16x32 instruction, lane (l, g): 8 consecutive n from 8 g of row l, so 64
// bytes of each row a load) and a share of the n; B's rows are paired in
// registers, lane l holding columns c0 .. c0 + FW - 1 with c0 = FW l, moved
// back inside the row where it would pass r (those columns are then formed
// twice, alike).  The first share of a tile also lays u's planes out, the last
// one to finish those of du xs.  Fewer tokens a workgroup read B more often,
// more of them need more shares, whose join (write-through stores, ticket,
// reload) is a chain of some 6 us: at 4096 x 8192, rank 64, RT = 1, 2, 4 on
// 256 workgroups take 34, 29 and 32 us, on 512 38, 33 and 37.
constexpr int kDuWaves = 4;

template <int FW, int RT>
__global__ __launch_bounds__(64 * kDuWaves, FW == 8 ? 1 : 2) void k_du(DuArgs a) {
  constexpr int kThreads = 64 * kDuWaves, kRing = FW == 8 ? 3 : 4, kW = FW >= 2 ? FW / 2 : 1, kTok = 16 * RT;
  constexpr int kItems = FW * RT, kMine = (kItems + kDuWaves - 1) / kDuWaves;
  __shared__ __attribute__((aligned(16))) f32x4 s_acc[kDuWaves * kItems * 64];
  float* const s_du = reinterpret_cast<float*>(s_acc);  // (once the waves' sums are joined)
  static_assert(kTok * (16 * FW + 16 + 1) <= kDuWaves * kItems * 256, "32 jt <= 16 FW + 16 columns");
  __shared__ uint32_t s_ticket;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int S = a.splits, r = a.r, jt = (r + 31) / 32;
  const int64_t M = a.M, N = a.N;
  const int tile = static_cast<int>(blockIdx.x) / S, share = static_cast<int>(blockIdx.x) % S;
  const int64_t m0 = static_cast<int64_t>(tile) * kTok;
  const int slices = static_cast<int>((N + 31) / 32), per = (slices + kDuWaves * S - 1) / (kDuWaves * S);
  const int b0 = (share * kDuWaves + wave) * per;
  const int s0 = b0 < slices ? b0 : slices, s1 = b0 + per < slices ? b0 + per : slices;
  const int64_t rows = M - m0 < kTok ? M - m0 : kTok;
  const rsrc_t yr = uniform_rsrc(a.dy + m0 * N, static_cast<uint32_t>(rows * N * 2));
  const int c0 = FW * l16 + FW <= r ? FW * l16 : r - FW;
  uint32_t yo[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) yo[t] = static_cast<uint32_t>(((16 * t + l16) * N + 8 * g) * 2);
  typedef uint32_t words_t __attribute__((ext_vector_type(kW == 1 ? 2 : kW)));
  struct Slice {
    u32x4 y[RT];
    words_t b[8];
  };
  Slice ring[kRing];
  auto load = [&](int sl, Slice& v) {
    // Past the wave's share, and past N (a multiple of 16) in the last slice:
    // dY reads as zero, B as its first rows, which are cleared.
    const bool in = sl < s1;
    const int64_t n = static_cast<int64_t>(in ? sl : 0) * 32 + 8 * g;
    const bool ok = in && n < N;
    const int so = in ? sl * 64 : 0;
#pragma unroll
    for (int t = 0; t < RT; ++t) v.y[t] = __builtin_amdgcn_raw_buffer_load_b128(yr, ok ? yo[t] : 0x80000000u, so, 0);
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
  f32x4 acc[FW][RT];  // [column of the lane][16 tokens]
#pragma unroll
  for (int t = 0; t < FW; ++t)
#pragma unroll
    for (int q = 0; q < RT; ++q) acc[t][q] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) load(s0 + i, ring[i]);
  if (share == 0)
    for (int i = tid; i < RT * jt * 64; i += kThreads) {
      const int ln = i & 63, tj = i / 64 % jt, st = i / 64 / jt;
      const int j = 32 * tj + (ln & 31);
      const int64_t m = m0 + 16 * st + 8 * (ln >> 5);
      if (m0 + 16 * st >= M) continue;
      float z[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = j < r && m + e < M ? a.u[(m + e) * r + j] : 0.0f;
      store_planes(a.u_planes, m0 / kStep + st, jt, tj, ln, z);
    }
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
        for (int q = 0; q < RT; ++q) acc[t][q] = mfma16(v.y[q], b, acc[t][q]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // Lane (l, g) holds token 16 q + 4 g + v of column c0 + t: item t RT + q.
  // The waves' sums, in wave order; wave w ends with items w, w + 4, ...
#pragma unroll
  for (int t = 0; t < FW; ++t)
#pragma unroll
    for (int q = 0; q < RT; ++q) s_acc[(wave * kItems + t * RT + q) * 64 + lane] = acc[t][q];
  __syncthreads();
  f32x4 o[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int item = wave + kDuWaves * i < kItems ? wave + kDuWaves * i : kItems - 1;
    o[i] = s_acc[item * 64 + lane];
#pragma unroll
    for (int w = 1; w < kDuWaves; ++w) o[i] += s_acc[(w * kItems + item) * 64 + lane];
  }
  if (S > 1) {
    constexpr uint32_t kShare = kDuWaves * kMine * 1024u;
    const rsrc_t pr = make_rsrc(reinterpret_cast<const uint8_t*>(a.partial) + static_cast<int64_t>(tile) * S * kShare);
    auto off = [&](int sp, int i) { return static_cast<uint32_t>(sp) * kShare + static_cast<uint32_t>((wave * kMine + i) * 1024 + lane * 16); };
#pragma unroll
    for (int i = 0; i < kMine; ++i) st_sys16(pr, off(share, i), o[i]);
    if (publish_and_ticket(a.counters + tile, &s_ticket) != static_cast<uint32_t>(S - 1)) return;
    if (tid == 0) a.counters[tile] = 0u;
    add_shares<kMine>(pr, S, off, o);
  }
  // the tile as fp32 rows of 32 jt + 1 words, columns past r and tokens past M zero
  const int stride = 32 * jt + 1;
  __syncthreads();
  for (int i = tid; i < kTok * stride; i += kThreads) s_du[i] = 0.0f;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int item = wave + kDuWaves * i;
    if (item >= kItems) continue;
    const int t = item / RT, q = item % RT;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int mr = 16 * q + 4 * g + v;
      const int64_t m = m0 + mr;
      if (m >= M || FW * l16 >= r) continue;
      const float du = a.s * o[i][v];
      a.du[m * r + c0 + t] = du;
      s_du[mr * stride + c0 + t] = du * a.xs[m];
    }
  }
  __syncthreads();
  for (int i = tid; i < RT * jt * 64; i += kThreads) {
    const int ln = i & 63, tj = i / 64 % jt, st = i / 64 / jt;
    if (m0 + 16 * st >= M) continue;
    float z[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = s_du[(16 * st + 8 * (ln >> 5) + e) * stride + 32 * tj + (ln & 31)];
    store_planes(a.du_planes, m0 / kStep + st, jt, tj, ln, z);
  }
}

int du_fw(int r) { return r <= 16 ? 1 : r <= 32 ? 2 : r <= 64 ? 4 : 8; }
int du_rt(int64_t M) { return M < 16384 ? 2 : 4; }

}  // namespace

int64_t tokens_strips(int64_t P) { return (P + kStrip - 1) / kStrip; }
// Token shares of dB and dA, whose blocks share one launch (dA's first, one
// workgroup a unit): those with the shortest estimated end.  The constants
// were fitted to every pair of shares at 31 sizes (150 .. 4096 tokens, 512 ..
// 28672 columns, ranks 16 .. 128; the picks were 0.8 % off the fastest on
// average, 6 % at worst): a block takes 6 us and 0.5 per 32 ranks, its waves'
// steps, and with shares 7 us and 1 for every batch of their loads.  (As many
// shares as fit a round each, which leaves partial rounds and long joins: 2048
// x 4096 x 11008 rank 64 41 us with du, now 30; 3279 x 704 x 4928 rank 97 65
// and 39; 4096 x 2048 x 2176 rank 64 48 and 31.)
TokensShares tokens_shares(int64_t M, int64_t N, int64_t K, int r) {
  static const int kShares[] = {1, 2, 3, 4, 6, 8, 12};
  static const double kA[4] = {0.5, 0.85, 0.75, 1.3}, kB[4] = {0.7, 0.7, 0.7, 1.1};  // us a step, by 32 ranks
  const int jt = (r + 31) / 32, waves = tokens_waves(jt), batch = jt == 1 ? 4 : 2;
  const int64_t steps = (M + kStep - 1) / kStep, strips_a = tokens_strips(K), strips_b = tokens_strips(N);
  auto block_us = [&](int s, double step) {
    const double t = 6.0 + 0.5 * jt + static_cast<double>((steps + waves * s - 1) / (waves * s)) * step;
    return s > 1 ? t + 7.0 + static_cast<double>((s + batch - 1) / batch) : t;
  };
  // the end of na blocks of ta and then nb of tb on 256 units
  auto end_us = [](int64_t na, double ta, int64_t nb, double tb) {
    const int64_t rounds = na / 256, more = na % 256;
    double late = static_cast<double>(rounds + (more != 0 ? 1 : 0)) * ta, early = static_cast<double>(rounds) * ta;
    double end = late;
    while (nb > 0) {
      double& t = more != 0 && late <= early ? late : early;
      nb -= &t == &late ? more : 256 - more;
      t += tb;
      if (t > end) end = t;
    }
    return end;
  };
  TokensShares best;
  double best_t = 0.0;
  for (int sa : kShares) {
    if (sa > 1 && (steps < sa * waves || strips_a * sa > 512)) break;
    const double ta = block_us(sa, kA[jt - 1]);
    for (int sb : kShares) {
      if (sb > 1 && (steps < sb * waves || strips_b * sb > 512)) break;
      const double t = end_us(strips_a * sa, ta, strips_b * sb, block_us(sb, kB[jt - 1]));
      if (best_t == 0.0 || t < best_t) {
        best_t = t;
        best.dA = sa;
        best.dB = sb;
      }
    }
  }
  return best;
}
int64_t tokens_partial_floats(int64_t P, int r, int shares) {
  return shares > 1 ? shares * tokens_strips(P) * 4 * ((r + 31) / 32) * kFW * 256 : 0;
}
int64_t plane_bytes(int64_t M, int r) { return (M + kStep - 1) / kStep * ((r + 31) / 32) * 2048; }

hipError_t launch_tokens(const TokensArgs& b, TokensArgs a, hipStream_t stream) {
  a.blocks = static_cast<int32_t>(tokens_strips(a.P) * a.splits);
  const uint32_t grid = static_cast<uint32_t>(a.blocks + tokens_strips(b.P) * b.splits);
  switch ((a.r + 31) / 32) {
    case 1: hipLaunchKernelGGL(k_tokens<1>, dim3(grid), dim3(64 * tokens_waves(1)), 0, stream, b, a); break;
    case 2: hipLaunchKernelGGL(k_tokens<2>, dim3(grid), dim3(64 * tokens_waves(2)), 0, stream, b, a); break;
    case 3: hipLaunchKernelGGL(k_tokens<3>, dim3(grid), dim3(64 * tokens_waves(3)), 0, stream, b, a); break;
    default: hipLaunchKernelGGL(k_tokens<4>, dim3(grid), dim3(64 * tokens_waves(4)), 0, stream, b, a); break;
  }
  return hipGetLastError();
}

int64_t du_tiles(int64_t M) { return (M + 16 * du_rt(M) - 1) / (16 * du_rt(M)); }
// Shares of the n: about one workgroup per compute unit, each wave at least 16
// slices (fewer would not pay for the join).
int du_splits(int64_t M, int64_t N) {
  int64_t s = 256 / du_tiles(M);
  const int64_t most = (N + 31) / 32 / (4 * kDuWaves);
  if (s > most) s = most;
  return static_cast<int>(s < 1 ? 1 : s);
}
int64_t du_partial_floats(int64_t M, int64_t N, int r) {
  const int64_t s = du_splits(M, N), items = du_fw(r) * du_rt(M);
  return s > 1 ? s * du_tiles(M) * kDuWaves * ((items + kDuWaves - 1) / kDuWaves) * 256 : 0;
}

namespace {
template <int RT>
hipError_t launch_du_rt(const DuArgs& a, hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>(du_tiles(a.M) * a.splits)), block(64 * kDuWaves);
  switch (du_fw(a.r)) {
    case 1: hipLaunchKernelGGL((k_du<1, RT>), grid, block, 0, stream, a); break;
    case 2: hipLaunchKernelGGL((k_du<2, RT>), grid, block, 0, stream, a); break;
    case 4: hipLaunchKernelGGL((k_du<4, RT>), grid, block, 0, stream, a); break;
    default: hipLaunchKernelGGL((k_du<8, RT>), grid, block, 0, stream, a); break;
  }
  return hipGetLastError();
}
}  // namespace

hipError_t launch_du(const DuArgs& a, hipStream_t stream) {
  return du_rt(a.M) == 2 ? launch_du_rt<2>(a, stream) : launch_du_rt<4>(a, stream);
}

}  // namespace qlin
