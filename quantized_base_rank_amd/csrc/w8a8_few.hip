// Product of 8-bit rows for few tokens (M <= 64): the weight codes stream from
// HBM straight into the operands of the 8-bit matrix instructions.
//   y[m][n] = xs[m] ws[n] sum_k xq[m][k] wq[n][k],  exact in int32
//
// A workgroup of 8 waves owns 16 RT channels and a share of K; its waves
// divide the share's 64-byte slices, each walking a contiguous run with the
// loads of the next kAhead slices in flight in a register ring.  Per slice a
// wave loads RT weight operands (lane (r, g): 16 bytes from 16 g of row r,
// so 64 bytes of each of 16 rows) and MT token operands, which come from the
// cache.  The waves' int32 sums meet in LDS (integer addition: any order
// gives the same sum); shares of K publish theirs and the last workgroup of a
// tile (atomic ticket) adds them.
#include "device_common.hpp"
#include "kernels.hpp"
#include "q8_common.hpp"

namespace qlin {

namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

constexpr int kFewWaves = 8;
constexpr int kSlice = 64;  // bytes of K per matrix instruction
constexpr int kAhead = 6;   // slices in flight per wave

template <int RT, int MT>
__global__ __launch_bounds__(64 * kFewWaves, 2) void k_w8a8_few(W8A8Args a) {
  constexpr int kRows = 16 * RT, kTok = 16 * MT;
  __shared__ int32_t s_sum[kTok][kRows + 4];
  __shared__ uint32_t s_ticket;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int S = a.splits;
  const int tile = static_cast<int>(blockIdx.x) / S, share = static_cast<int>(blockIdx.x) % S;
  const int64_t M = a.M, N = a.N, K = a.K, n0 = static_cast<int64_t>(tile) * kRows;
  const int slices = static_cast<int>((K + kSlice - 1) / kSlice);
  // the slices of this wave
  const int per = (slices + S * kFewWaves - 1) / (S * kFewWaves);
  const int b0 = (share * kFewWaves + wave) * per;
  const int s_begin = b0 < slices ? b0 : slices, s_end = b0 + per < slices ? b0 + per : slices;

  for (int i = tid; i < kTok * (kRows + 4); i += 64 * kFewWaves) (&s_sum[0][0])[i] = 0;

  // Rows past the matrix lie outside the resource (zeros).  A weight piece
  // past K holds the next row's codes, against a token piece that is zero.
  const int64_t rows = N - n0 < kRows ? N - n0 : kRows;
  const rsrc_t wr = uniform_rsrc(a.wq + n0 * K, static_cast<uint32_t>(rows * K));
  const rsrc_t xr = uniform_rsrc(a.xq, static_cast<uint32_t>(M * K));
  uint32_t wo[RT], xo[MT], xo_tail[MT];
#pragma unroll
  for (int t = 0; t < RT; ++t) wo[t] = static_cast<uint32_t>((16 * t + l16) * K + 16 * g);
  const bool past = (slices - 1) * kSlice + 16 * g >= K;
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int64_t m = 16 * t + l16 < M ? 16 * t + l16 : M - 1;
    xo[t] = static_cast<uint32_t>(m * K + 16 * g);
    xo_tail[t] = xo[t] | (past ? 0x80000000u : 0u);
  }

  i32x4 wv[kAhead][RT], xv[kAhead][MT], acc[RT][MT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[r][m] = i32x4{};
  auto load = [&](int sl, i32x4 (&w)[RT], i32x4 (&x)[MT]) {
    // (a slice past the run lies outside the resources)
    const int so = sl < s_end ? sl * kSlice : 0x7FFFFFFF;
    const bool last = sl == slices - 1;
#pragma unroll
    for (int t = 0; t < RT; ++t)
      w[t] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(wr, wo[t], so, 0));
#pragma unroll
    for (int t = 0; t < MT; ++t)
      x[t] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(xr, last ? xo_tail[t] : xo[t], so, 0));
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load(s_begin + i, wv[i], xv[i]);
  for (int sl = s_begin; sl < s_end; sl += kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m)
          acc[r][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[i][r], xv[i][m], acc[r][m], 0, 0, 0);
      load(sl + kAhead + i, wv[i], xv[i]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // lane (l16, g) holds channel 16 r + 4 g + v of token 16 m + l16
  __syncthreads();
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int v = 0; v < 4; ++v) atomicAdd(&s_sum[16 * m + l16][16 * r + 4 * g + v], acc[r][m][v]);
  __syncthreads();
  if (S > 1) {
    int32_t* const part = reinterpret_cast<int32_t*>(a.partial) + static_cast<int64_t>(tile) * S * kTok * kRows;
    for (int i = tid; i < kTok * kRows; i += 64 * kFewWaves)
      st_sys(reinterpret_cast<float*>(part + share * kTok * kRows + i), __int_as_float(s_sum[i / kRows][i % kRows]));
    if (publish_and_ticket(a.counters + tile, &s_ticket) != static_cast<uint32_t>(S - 1)) return;
    for (int i = tid; i < kTok * kRows; i += 64 * kFewWaves) {
      int32_t t = 0;
      for (int sp = 0; sp < S; ++sp) t += __float_as_int(ld_sys(reinterpret_cast<const float*>(part + sp * kTok * kRows + i)));
      s_sum[i / kRows][i % kRows] = t;
    }
    if (tid == 0) a.counters[tile] = 0u;
    __syncthreads();
  }
  for (int i = tid; i < kTok * kRows; i += 64 * kFewWaves) {
    const int m = i / kRows, c = i % kRows;
    if (m < M && n0 + c < N)
      a.y[m * N + n0 + c] = f32_to_bf16(static_cast<float>(s_sum[m][c]) * a.xs[m] * a.ws[n0 + c]);
  }
}

// 32 channels per workgroup where that leaves at least one per compute unit.
int few_rt(int64_t N) { return (N + 31) / 32 >= 256 ? 2 : 1; }
int few_mt(int64_t M) { return M <= 16 ? 1 : M <= 32 ? 2 : 4; }

}  // namespace

int w8a8_few_tiles(int64_t N) { return static_cast<int>((N + 16 * few_rt(N) - 1) / (16 * few_rt(N))); }
// Shares of K: about one workgroup per compute unit, each wave at least two
// slices.
int w8a8_few_splits(int64_t N, int64_t K) {
  const int64_t tiles = w8a8_few_tiles(N), slices = (K + kSlice - 1) / kSlice;
  int64_t s = 256 / tiles;
  if (s > slices / (2 * kFewWaves)) s = slices / (2 * kFewWaves);
  return static_cast<int>(s < 1 ? 1 : s);
}
int64_t w8a8_few_partial_words(int64_t M, int64_t N, int64_t K) {
  const int64_t s = w8a8_few_splits(N, K);
  return s > 1 ? s * w8a8_few_tiles(N) * 16 * few_rt(N) * 16 * few_mt(M) : 0;
}

hipError_t launch_w8a8_few(const W8A8Args& a, hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>(w8a8_few_tiles(a.N) * a.splits)), block(64 * kFewWaves);
  const int rt = few_rt(a.N), mt = few_mt(a.M);
  if (rt == 2 && mt == 1) hipLaunchKernelGGL((k_w8a8_few<2, 1>), grid, block, 0, stream, a);
  else if (rt == 2 && mt == 2) hipLaunchKernelGGL((k_w8a8_few<2, 2>), grid, block, 0, stream, a);
  else if (rt == 2) hipLaunchKernelGGL((k_w8a8_few<2, 4>), grid, block, 0, stream, a);
  else if (mt == 1) hipLaunchKernelGGL((k_w8a8_few<1, 1>), grid, block, 0, stream, a);
  else if (mt == 2) hipLaunchKernelGGL((k_w8a8_few<1, 2>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((k_w8a8_few<1, 4>), grid, block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace qlin
