// Product of 8-bit rows: y[m][n] = xs[m] ws[n] sum_k xq[m][k] wq[n][k], the
// sum taken by the 8-bit matrix instructions in int32 (exact for
// K <= 131056, where 128 * 128 * K < 2^31).
//
// Tile: 256 channels x 64 J tokens (J = 1 .. 4) per workgroup of 4 waves (one
// per SIMD), each wave 128 x 32 J in 64 J accumulator registers, so that at
// J = 4 a K slice of 32 bytes costs 8 LDS reads of 16 bytes per lane for 16
// matrix instructions.  Both operands stream through a ring of four
// 64-byte-deep half-stages (32 KB each at J = 4) by direct-to-LDS loads, the
// last of which are issued three half-stages ahead.  One barrier per
// half-stage, in its middle: by then every wave holds the half-stage's last
// fragments in registers, so its slot is free for the loads of the half-stage
// four on, and the next one has landed (counted wait), so the fragments of
// its first slice load while this one's last matrix instructions run.
//
// At 4096 x 8192 x 28672: 806-822 us, 2.34-2.39 PFLOP/s, matrix cores busy
// 56 % of the cycles at 2.0 GHz.  Timing copies: without the loads 615 us
// (the clock falls to 1.77 GHz: power), with every load hitting L2 740-770 us
// at 1.62 GHz, with zeros as data 434 us at 2.4 GHz.  So what remains above
// the power limit is the L2 misses' share, under 10 %; a fifth slot of the
// ring (160 KB) gained nothing.
#include "device_common.hpp"
#include "kernels.hpp"
#include "q8_common.hpp"

namespace qlin {

namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr int kTN = 256;    // channels per tile
constexpr int kHalf = 64;   // bytes of K per half-stage
constexpr int kWBytes = kTN * kHalf;

// Waits until at most two half-stages of this wave's loads (4 + J each) are
// in flight and its LDS reads are done, then meets the other waves.  One asm
// block: a fence would wait for every direct-to-LDS load in flight.
template <int J>
__device__ __forceinline__ void half_barrier() {
  static_assert(J >= 1 && J <= 4, "one wait for each");
  if constexpr (J == 1) __asm__ volatile("s_waitcnt vmcnt(10) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  if constexpr (J == 2) __asm__ volatile("s_waitcnt vmcnt(12) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  if constexpr (J == 3) __asm__ volatile("s_waitcnt vmcnt(14) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  if constexpr (J == 4) __asm__ volatile("s_waitcnt vmcnt(16) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Fragments of one 32-byte slice of K: lane (l, h) holds bytes 16 h .. of row
// l of each of the wave's 32-row tiles.
template <int J>
struct Frags {
  i32x4 w[4], x[J];
};

template <int J>
__device__ __forceinline__ void read_frags(const uint8_t* slot, uint32_t woff, uint32_t xoff, Frags<J>& f) {
#pragma unroll
  for (int t = 0; t < 4; ++t) f.w[t] = *reinterpret_cast<const i32x4*>(slot + woff + t * 32 * kHalf);
#pragma unroll
  for (int t = 0; t < J; ++t) f.x[t] = *reinterpret_cast<const i32x4*>(slot + xoff + t * 32 * kHalf);
}

// Order of a slice's instructions: its 4 + J LDS reads two by two behind the
// first matrix instructions, then a global load every other one.
template <int J, int LOADS>
__device__ __forceinline__ void slice_order() {
#pragma unroll
  for (int i = 0; i < (4 + J) / 2; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
  }
  if constexpr (J % 2 == 1) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, J >= 3 ? 2 : 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
  }
  constexpr int kLeft = 4 * J - (4 + J) / 2 - LOADS * (J >= 3 ? 2 : 1);
  if constexpr (kLeft > 0) __builtin_amdgcn_sched_group_barrier(0x008, kLeft, 0);
}

template <int J>
__global__ __launch_bounds__(256, 1) void k_w8a8_gemm(W8A8Args a) {
  constexpr int kTM = 64 * J, kLoads = 4 + J, kSlot = kWBytes + kTM * kHalf;
  // one array per slot: a read of one is not held for loads into another
  __shared__ __attribute__((aligned(16))) uint8_t s0[kSlot];
  __shared__ __attribute__((aligned(16))) uint8_t s1[kSlot];
  __shared__ __attribute__((aligned(16))) uint8_t s2[kSlot];
  __shared__ __attribute__((aligned(16))) uint8_t s3[kSlot];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  const int wn = wave & 1, wm = wave >> 1;
  const int64_t M = a.M, N = a.N, K = a.K;
  const int tiles_m = static_cast<int>((M + kTM - 1) / kTM), tiles_n = static_cast<int>((N + kTN - 1) / kTN);
  const int S = a.splits;
  const int work = xcd_round_order(static_cast<int>(blockIdx.x), tiles_m * tiles_n * S);
  const int share = work % S, tile = work / S;
  int tm, tn;
  grouped_tile(tile, tiles_m, tiles_n, tm, tn);
  const int64_t m0 = static_cast<int64_t>(tm) * kTM, n0 = static_cast<int64_t>(tn) * kTN;
  const int all = static_cast<int>((K + kHalf - 1) / kHalf), per = (all + S - 1) / S;
  const int h_begin = share * per < all ? share * per : all, h_end = h_begin + per < all ? h_begin + per : all;

  // Loads: instruction i of wave w fills rows 16 (4 i + w) .. +15 of an
  // operand, four 16-byte pieces a row; piece c of row r sits at
  // c ^ ((r / 4) % 4), which puts one piece of 16 consecutive rows in 16
  // distinct bank groups.  Rows past the matrix lie outside the resource and
  // read as zero, pieces past K get an offset outside it, half-stages past
  // the share an empty resource.
  const int64_t xrows = M - m0 < kTM ? M - m0 : kTM, wrows = N - n0 < kTN ? N - n0 : kTN;
  const rsrc_t xr = uniform_rsrc(a.xq + m0 * K, static_cast<uint32_t>(xrows * K));
  const rsrc_t wr = uniform_rsrc(a.wq + n0 * K, static_cast<uint32_t>(wrows * K));
  const rsrc_t none = uniform_rsrc(a.xq, 0u);
  const int piece = (lane & 3) ^ ((lane >> 4) & 3);
  const uint32_t voff = static_cast<uint32_t>((wave * 16 + (lane >> 2)) * K + piece * 16);
  const int tail = static_cast<int>(K % kHalf);
  const uint32_t voff_tail = voff | ((tail != 0 && piece * 16 >= tail) ? 0x80000000u : 0u);
  const int wslot = wave * 1024;
  auto load = [&](int hs, uint8_t* slot, int i) {  // i < 4: channels, else tokens
    const rsrc_t r = hs < h_end ? (i < 4 ? wr : xr) : none;
    const uint32_t vo = hs == all - 1 ? voff_tail : voff;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)(slot + i * 4096 + wslot), 16, vo,
                                             static_cast<int>((i & 3) * 64 * K + hs * kHalf), 0, 0);
  };

  // fragment offsets of the half-stage's two slices
  const int sw = (l32 >> 2) & 3;
  const uint32_t wrow = static_cast<uint32_t>((wn * 128 + l32) * kHalf);
  const uint32_t xrow = static_cast<uint32_t>(kWBytes + (wm * 32 * J + l32) * kHalf);
  const uint32_t c0 = static_cast<uint32_t>((h ^ sw) << 4), c1 = c0 ^ 32u;

  i32x16 acc[4][J];  // [channels][tokens]
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < J; ++j) acc[i][j] = i32x16{};
  auto mfmas = [&](const Frags<J>& f) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.w[i], f.x[j], acc[i][j], 0, 0, 0);
  };

  // The loads of the half-stage four on go out in two parts: four after the
  // barrier that frees the slot, the rest in the first slice of the next
  // half-stage (an even stream: 2 % over all of them after the barrier).
  Frags<J> f0, f1;
#pragma unroll
  for (int st = 0; st < 4; ++st)
#pragma unroll
    for (int i = 0; i < (st == 3 ? 4 : kLoads); ++i)
      load(h_begin + st, st == 0 ? s0 : st == 1 ? s1 : st == 2 ? s2 : s3, i);
  if constexpr (J == 1) __asm__ volatile("s_waitcnt vmcnt(14)\n\ts_barrier" ::: "memory");
  if constexpr (J == 2) __asm__ volatile("s_waitcnt vmcnt(16)\n\ts_barrier" ::: "memory");
  if constexpr (J == 3) __asm__ volatile("s_waitcnt vmcnt(18)\n\ts_barrier" ::: "memory");
  if constexpr (J == 4) __asm__ volatile("s_waitcnt vmcnt(20)\n\ts_barrier" ::: "memory");
  read_frags<J>(s0, wrow + c0, xrow + c0, f0);

  // whole turns of the ring: half-stages past the share hold zeros
  for (int hs0 = h_begin; hs0 < h_end; hs0 += 4) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      uint8_t* const cur = p == 0 ? s0 : p == 1 ? s1 : p == 2 ? s2 : s3;
      uint8_t* const prv = p == 0 ? s3 : p == 1 ? s0 : p == 2 ? s1 : s2;
      const uint8_t* const nxt = p == 0 ? s1 : p == 1 ? s2 : p == 2 ? s3 : s0;
      read_frags<J>(cur, wrow + c1, xrow + c1, f1);
#pragma unroll
      for (int i = 4; i < kLoads; ++i) load(hs0 + p + 3, prv, i);
      mfmas(f0);
      slice_order<J, J>();
      half_barrier<J>();
#pragma unroll
      for (int i = 0; i < 4; ++i) load(hs0 + p + 4, cur, i);
      read_frags<J>(nxt, wrow + c0, xrow + c0, f0);
      mfmas(f1);
      slice_order<J, 4>();
    }
  }
  __asm__ volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");

  const int64_t mw = m0 + wm * 32 * J, nw = n0 + wn * 128;
  if (S > 1) {
    // Shares of K: int32 sums [share][tile][wave][i][q][j][lane] x 16 bytes,
    // joined by k_w8a8_join.  Waves whose rows or channels all lie past the
    // matrix leave theirs out.
    if (mw >= M || nw >= N) return;
    i32x4* const part = reinterpret_cast<i32x4*>(a.partial) +
                        ((static_cast<int64_t>(share) * tiles_m * tiles_n + tile) * 4 + wave) * (16 * J * 64) + lane;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int j = 0; j < J; ++j)
          part[((i * 4 + q) * J + j) * 64] =
              i32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    return;
  }

  // Output: lane (l, h) holds channel 32 i + 8 q + 4 h + v of token 32 j + l
  // at acc[i][j][4 q + v].  Each wave turns its tile round in its slot as
  // bf16 rows of tokens (16-byte pieces XOR-swizzled by token), then stores
  // whole row segments, at any alignment of the rows.
  uint8_t* const out = wave == 0 ? s0 : wave == 1 ? s1 : wave == 2 ? s2 : s3;
  float xs[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int64_t m = mw + 32 * j + l32;
    xs[j] = m < M ? a.xs[m] : 0.0f;
  }
  // (channels past N read as zero)
  const rsrc_t wsr = uniform_rsrc(a.ws + nw, static_cast<uint32_t>(nw < N ? (N - nw < 128 ? N - nw : 128) * 4 : 0));
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = 32 * i + 8 * q + 4 * h;
      const f32x4 ws = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(wsr, static_cast<uint32_t>(c * 4), 0, 0));
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int m = 32 * j + l32;
        float o[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) o[v] = static_cast<float>(acc[i][j][4 * q + v]) * xs[j] * ws[v];
        *reinterpret_cast<u32x2*>(out + m * 256 + (((c >> 3) ^ (m & 15)) << 4) + h * 8) =
            u32x2{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
      }
    }
  for (int it = 0; it < 8 * J; ++it) {
    const int m = 4 * it + (lane >> 4), pc = lane & 15;
    const u32x4 v = *reinterpret_cast<const u32x4*>(out + m * 256 + ((pc ^ (m & 15)) << 4));
    const int64_t n = nw + 8 * pc;
    if (mw + m >= M || n >= N) continue;
    uint16_t* const dst = a.y + (mw + m) * N + n;
    if (n + 8 <= N) {
      store8(dst, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (n + e < N) dst[e] = static_cast<uint16_t>(v[e >> 1] >> (16 * (e & 1)));
    }
  }
}

// The shares' sums (integers: exact), scaled and rounded: a thread takes four
// channels of one token, as the matrix instruction left them.
template <int J>
__global__ __launch_bounds__(256) void k_w8a8_join(W8A8Args a) {
  const int tiles_m = static_cast<int>((a.M + 64 * J - 1) / (64 * J)), tiles_n = static_cast<int>((a.N + kTN - 1) / kTN);
  const int64_t per = 4 * 16 * J * 64;  // 16-byte pieces of a tile
  const int64_t total = per * tiles_m * tiles_n;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int tile = static_cast<int>(at / per), in = static_cast<int>(at % per);
  const int lane = in & 63, j = in / 64 % J, q = in / (64 * J) & 3, i = in / (256 * J) & 3, wave = in / (1024 * J);
  int tm, tn;
  grouped_tile(tile, tiles_m, tiles_n, tm, tn);
  const int64_t m = static_cast<int64_t>(tm) * 64 * J + (wave >> 1) * 32 * J + 32 * j + (lane & 31);
  const int64_t n = static_cast<int64_t>(tn) * kTN + (wave & 1) * 128 + 32 * i + 8 * q + 4 * (lane >> 5);
  if (m >= a.M || n >= a.N) return;
  const i32x4* part = reinterpret_cast<const i32x4*>(a.partial) + at;
  i32x4 t = part[0];
#pragma unroll 4
  for (int sp = 1; sp < a.splits; ++sp) t += part[sp * total];
  const float xs = a.xs[m];
  uint16_t* const dst = a.y + m * a.N + n;
  if (n + 4 <= a.N) {
    float o[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) o[v] = static_cast<float>(t[v]) * xs * a.ws[n + v];
    typedef u32x2 u32x2h __attribute__((aligned(2)));
    *reinterpret_cast<u32x2h*>(dst) = u32x2{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
  } else {
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (n + v < a.N) dst[v] = f32_to_bf16(static_cast<float>(t[v]) * xs * a.ws[n + v]);
  }
}

}  // namespace

int64_t w8a8_gemm_tiles(int64_t M, int64_t N, int j) { return (M + 64 * j - 1) / (64 * j) * ((N + kTN - 1) / kTN); }

// Tile height and shares of K by estimated time, from what the kernel
// measured: a half-stage of a lone workgroup takes 0.53, 0.59, 0.63, 0.67 us
// (J = 1 .. 4: the ring's depth over the memory's latency), of a full card
// 0.85 (two workgroups a unit, J = 1 only), 0.62, 0.725, 0.917 us; the
// weights stream at 4.6 TB/s at best; joining shares costs a launch and 8
// bytes per output and share at 3.5 TB/s.  (128 x 8192 x 28672: J = 2 in 8
// shares 62 us, against 79 for J = 1 in 4 and 301 for J = 4 in one; 333 x
// 32003 x 4096: J = 3 57 us, against 60 for J = 4.)
W8A8Shape w8a8_gemm_shape(int64_t M, int64_t N, int64_t K) {
  static const double kLone[4] = {0.53, 0.59, 0.63, 0.67}, kFull[4] = {0.85, 0.62, 0.725, 0.917};
  static const int kShares[] = {1, 2, 3, 4, 6, 8, 12, 16};
  const int64_t halves = (K + kHalf - 1) / kHalf;
  const double stream = static_cast<double>(K) * static_cast<double>(M + N) / 4.6e6;
  W8A8Shape best;
  double best_t = 0.0;
  for (int j = 4; j >= 1; --j) {
    const int64_t tiles = w8a8_gemm_tiles(M, N, j), slots = j == 1 ? 512 : 256;
    for (int s : kShares) {
      if (s > 1 && (halves < 8 * s || tiles * s > slots)) continue;
      const double fill = tiles * s < slots ? static_cast<double>(tiles * s) / static_cast<double>(slots) : 1.0;
      const double half = kLone[j - 1] + (kFull[j - 1] - kLone[j - 1]) * fill;
      const double rounds = static_cast<double>((tiles * s + slots - 1) / slots);
      double t = rounds * static_cast<double>((halves + s - 1) / s + 6) * half;
      if (t < stream) t = stream;
      if (s > 1) t += 4.0 + 8.0 * static_cast<double>(M) * static_cast<double>(N) * s / 3.5e6;
      if (best_t == 0.0 || t < best_t) {
        best_t = t;
        best.j = j;
        best.splits = s;
      }
    }
  }
  return best;
}
int64_t w8a8_gemm_partial_words(int64_t M, int64_t N, W8A8Shape s) {
  return s.splits > 1 ? w8a8_gemm_tiles(M, N, s.j) * s.splits * 64 * s.j * kTN : 0;
}

namespace {

template <int J>
hipError_t launch_gemm_j(const W8A8Args& a, hipStream_t stream) {
  const int64_t tiles = w8a8_gemm_tiles(a.M, a.N, J);
  hipLaunchKernelGGL(k_w8a8_gemm<J>, dim3(static_cast<uint32_t>(tiles * a.splits)), dim3(256), 0, stream, a);
  if (a.splits > 1)  // 4096 J pieces a tile, 256 a workgroup
    hipLaunchKernelGGL(k_w8a8_join<J>, dim3(static_cast<uint32_t>(tiles * 16 * J)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_w8a8_gemm(const W8A8Args& a, int j, hipStream_t stream) {
  switch (j) {
    case 1: return launch_gemm_j<1>(a, stream);
    case 2: return launch_gemm_j<2>(a, stream);
    case 3: return launch_gemm_j<3>(a, stream);
    default: return launch_gemm_j<4>(a, stream);
  }
}

}  // namespace qlin
