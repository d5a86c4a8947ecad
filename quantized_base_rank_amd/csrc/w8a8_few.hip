// Product of 8-bit rows for few tokens (M <= 64): the weight codes stream from
// HBM straight into the operands of the 8-bit matrix instructions.
//   y[m][n] = xs[m] ws[n] sum_k xq[m][k] wq[n][k],  exact in int32
//
// A workgroup of 8 waves owns 16 RT channels and a share of K, walked in
// chunks of kChunk bytes.  The chunk of all token rows is copied to LDS (two
// buffers, direct-to-LDS loads one chunk ahead): read from cache by every
// wave, the token operands cost as many load instructions as the weights (16
// tokens by 8192 x 28672: 54 us, against 50 through LDS).  Each wave takes a
// contiguous eighth of the chunk for all rows, in 64-byte slices: a weight
// operand is 16 bytes from 16 g of row r for lane (r, g).  The weights of two
// slices are loaded together, two chunks ahead into a register ring, so that
// both halves of a 128-byte line are asked for one behind the other (slice by
// slice the line came from L2 twice: 52.6 against 49.0 us, 4.8 TB/s).  The
// waves' int32 sums meet in LDS (integer addition: any order gives the same
// sum); shares of K publish theirs and the last workgroup of a tile (atomic
// ticket) adds them.
#include "device_common.hpp"
#include "kernels.hpp"
#include "q8_common.hpp"

namespace qlin {

namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

constexpr int kFewWaves = 8;
constexpr int kSlice = 64;  // bytes of K per matrix instruction
typedef __attribute__((address_space(3))) void* lds_ptr_t;

// Bytes of K per chunk: 32 or 64 KB of LDS per buffer.
constexpr int few_chunk(int mt) { return mt <= 2 ? 2048 : 1024; }

template <int RT, int MT>
__global__ __launch_bounds__(64 * kFewWaves, 2) void k_w8a8_few(W8A8Args a) {
  constexpr int kRows = 16 * RT, kTok = 16 * MT, kChunk = few_chunk(MT);
  constexpr int kSl = kChunk / kSlice / kFewWaves;         // slices per wave and chunk
  static_assert(kSl % 2 == 0, "whole lines");
  constexpr int kDma = kTok * kChunk / 1024 / kFewWaves;   // token loads per wave and chunk
  // one array per buffer: a read of one is not held for loads into the other
  __shared__ __attribute__((aligned(16))) uint8_t s_x0[kTok * kChunk];
  __shared__ __attribute__((aligned(16))) uint8_t s_x1[kTok * kChunk];
  __shared__ int32_t s_sum[kTok][kRows + 4];
  __shared__ uint32_t s_ticket;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int S = a.splits;
  const int tile = static_cast<int>(blockIdx.x) / S, share = static_cast<int>(blockIdx.x) % S;
  const int64_t M = a.M, N = a.N, n0 = static_cast<int64_t>(tile) * kRows;
  const int K = static_cast<int>(a.K);
  const int chunks = (K + kChunk - 1) / kChunk, per = (chunks + S - 1) / S;
  const int c_begin = share * per < chunks ? share * per : chunks;
  const int c_end = c_begin + per < chunks ? c_begin + per : chunks;

  // Rows past the matrices lie outside the resources (zeros), and whole
  // slices past K too.  A weight piece past K holds the next row's codes,
  // against a token piece that is zero.
  const int64_t rows = N - n0 < kRows ? N - n0 : kRows;
  const rsrc_t wr = uniform_rsrc(a.wq + n0 * K, static_cast<uint32_t>(rows * K));
  const rsrc_t xr = uniform_rsrc(a.xq, static_cast<uint32_t>(M * K));
  uint32_t wo[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) wo[t] = static_cast<uint32_t>((16 * t + l16) * K + 16 * g + wave * kSl * kSlice);

  // Token rows of a chunk: [token][kChunk / 16 pieces], piece p at
  // p ^ (token % 16), so that 16 tokens' reads of one piece take 16 distinct
  // bank groups.  Load i of wave w fills 1 KB: part (8 i + w) % (kChunk / 1024)
  // of token (8 i + w) / (kChunk / 1024).
  auto load_tokens = [&](int c, uint8_t* buf) {
#pragma unroll
    for (int i = 0; i < kDma; ++i) {
      const int ii = i * kFewWaves + wave;
      const int tok = ii / (kChunk / 1024), part = ii % (kChunk / 1024);
      const int k = c * kChunk + part * 1024 + ((lane ^ (tok & 15)) << 4);
      const uint32_t vo = c < c_end && k < K ? static_cast<uint32_t>(tok * K + k) : 0x80000000u;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, (lds_ptr_t)(buf + ii * 1024), 16, vo, 0, 0, 0);
    }
  };
  i32x4 wv[2][kSl][RT], acc[RT][MT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[r][m] = i32x4{};
  // slices i and i + 1 (i even): the halves of a row's 128-byte lines one
  // behind the other
  auto load_weights = [&](int c, int i, i32x4 (&w0)[RT], i32x4 (&w1)[RT]) {
    const int k = c * kChunk + i * kSlice, kw = k + wave * kSl * kSlice;
    const int so0 = c < c_end && kw < K ? k : 0x7FFFFFFF, so1 = c < c_end && kw + kSlice < K ? k + kSlice : 0x7FFFFFFF;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      w0[t] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(wr, wo[t], so0, 0));
      w1[t] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(wr, wo[t], so1, 0));
    }
  };
  load_tokens(c_begin, s_x0);
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int i = 0; i < kSl; i += 2) load_weights(c_begin + c, i, wv[c][i], wv[c][i + 1]);
  for (int i = tid; i < kTok * (kRows + 4); i += 64 * kFewWaves) (&s_sum[0][0])[i] = 0;

  // Chunk c: its token rows and this wave's weights have landed once at most
  // the weights of chunk c + 1 are in flight; past the barrier the other
  // buffer is free for the token rows of chunk c + 1.
  for (int c0 = c_begin; c0 < c_end; c0 += 2) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int c = c0 + p;
      uint8_t* const cur = p == 0 ? s_x0 : s_x1;
      uint8_t* const nxt = p == 0 ? s_x1 : s_x0;
      static_assert(kSl * RT <= 16, "the waits below");
      if constexpr (kSl * RT == 2) __asm__ volatile("s_waitcnt vmcnt(2) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      else if constexpr (kSl * RT == 4) __asm__ volatile("s_waitcnt vmcnt(4) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      else if constexpr (kSl * RT == 8) __asm__ volatile("s_waitcnt vmcnt(8) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      else __asm__ volatile("s_waitcnt vmcnt(16) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      static_assert(kSl * RT == 2 || kSl * RT == 4 || kSl * RT == 8 || kSl * RT == 16, "a wait for each");
      load_tokens(c + 1, nxt);
#pragma unroll
      for (int i = 0; i < kSl; ++i) {
        i32x4 xv[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m)
          xv[m] = *reinterpret_cast<const i32x4*>(cur + (16 * m + l16) * kChunk +
                                                  ((((wave * kSl + i) * 4 + g) ^ l16) << 4));
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int m = 0; m < MT; ++m)
            acc[r][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[p][i][r], xv[m], acc[r][m], 0, 0, 0);
        if (i % 2 != 0) load_weights(c + 2, i - 1, wv[p][i - 1], wv[p][i]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  // (the loads issued past the share land before the workgroup ends)
  __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");

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

// Share of the compute units' time that `groups` workgroups fill, in whole
// rounds of one per unit.
double few_fill(int64_t groups) { return static_cast<double>(groups) / (256.0 * static_cast<double>((groups + 255) / 256)); }

// 16-row tiles per workgroup.  More rows use each token operand more often
// but leave fewer workgroups.  Four where K has four chunks for each of the
// shares that fill the card (16 tokens by 8192 x 28672: 49 us, against 53 and
// 57 with two and one), and for more than 32 tokens where four fill the rounds
// about as well as two do (64 by 14336 x 4096: 22 against 25; 22016 x 2048,
// 344 groups: 23 against 22); else two where those fill them about as well as
// one (16 by 7168 x 4096: 9.8 against 10.7; 64 by 7168 x 4096: 13.6 against
// 17.1; 11008 x 4096, 344 groups: 16 against 15).
int few_rt(int64_t M, int64_t N, int64_t K) {
  const int64_t t4 = (N + 63) / 64, t2 = (N + 31) / 32, t1 = (N + 15) / 16, shares = t4 < 256 ? 256 / t4 : 1;
  if (t4 >= 128 && K >= shares * 4 * 2048) return 4;
  if (M > 32 && t4 >= 128 && few_fill(t4) > few_fill(t2) - 0.1) return 4;
  return t2 >= 128 && few_fill(t2) > few_fill(t1) - 0.1 ? 2 : 1;
}
int few_mt(int64_t M) { return M <= 16 ? 1 : M <= 32 ? 2 : 4; }

}  // namespace

int64_t w8a8_few_tiles(int64_t M, int64_t N, int64_t K) {
  const int rows = 16 * few_rt(M, N, K);
  return (N + rows - 1) / rows;
}
// Shares of K: about one workgroup per compute unit, each a chunk or
// more.
int w8a8_few_splits(int64_t M, int64_t N, int64_t K) {
  const int64_t tiles = w8a8_few_tiles(M, N, K), chunks = (K + 2047) / 2048;
  int64_t s = 256 / tiles;
  if (s > chunks) s = chunks;
  return static_cast<int>(s < 1 ? 1 : s);
}
int64_t w8a8_few_partial_words(int64_t M, int64_t N, int64_t K) {
  const int64_t s = w8a8_few_splits(M, N, K);
  return s > 1 ? s * w8a8_few_tiles(M, N, K) * 16 * few_rt(M, N, K) * 16 * few_mt(M) : 0;
}

namespace {

template <int RT>
hipError_t launch_few_rt(const W8A8Args& a, hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>(w8a8_few_tiles(a.M, a.N, a.K) * a.splits)), block(64 * kFewWaves);
  switch (few_mt(a.M)) {
    case 1: hipLaunchKernelGGL((k_w8a8_few<RT, 1>), grid, block, 0, stream, a); break;
    case 2: hipLaunchKernelGGL((k_w8a8_few<RT, 2>), grid, block, 0, stream, a); break;
    default: hipLaunchKernelGGL((k_w8a8_few<RT, 4>), grid, block, 0, stream, a); break;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_w8a8_few(const W8A8Args& a, hipStream_t stream) {
  switch (few_rt(a.M, a.N, a.K)) {
    case 1: return launch_few_rt<1>(a, stream);
    case 2: return launch_few_rt<2>(a, stream);
    default: return launch_few_rt<4>(a, stream);
  }
}

}  // namespace qlin
