// Product of 8-bit rows: y[m][n] = xs[m] ws[n] sum_k xq[m][k] wq[n][k], the
// sum taken by the 8-bit matrix instructions in int32 (exact for
// K <= 131056, where 128 * 128 * K < 2^31).
//
// Tile: 256 channels x 64 J tokens (J = 1 .. 4) per workgroup of 4 waves (one
// per SIMD), each wave 128 x 32 J in 64 J accumulator registers, so that at
// J = 4 a K slice of 32 bytes costs 8 LDS reads of 16 bytes per lane for 16
// matrix instructions.  Both operands stream through a ring of 64-byte-deep
// half-stages (32 KB each at J = 4, five of them) by direct-to-LDS loads.
// One barrier per half-stage, in its middle: by then every wave holds the
// half-stage's last fragments in registers, so its slot is free for loads,
// and the next one has landed (counted wait), so the fragments of its first
// slice load while this one's last matrix instructions run.
//
// A 128-byte line holds two half-stages of a row.  Asked for one at a time,
// half a microsecond apart, it came from L2 twice (the rows of a pair of
// half-stages are twice the L1); so the loads of a pair go out together, the
// two halves of a line one behind the other, in four equal parts over the
// pair's four slices.  At 4096 x 8192 x 28672 one half-stage at a time took
// 846 us, pairs 784 us with the loads in two bursts, 721 in three, 704 in
// four equal parts (2.73 PFLOP/s); 4096 x 4096 x 4096: 64 to 62 us, 333 x
// 32003 x 4096 (J = 3): 59.7 to 53.3 us.  A ring of whole 128-byte stages,
// two deep (all that fits), took 876 us: its loads are short of time.
//
// What bounds the largest: power.  The matrix cores are busy 80 % of the
// cycles, at 1.63 GHz.  (Timing copies of the kernel that asked for half
// lines: without the loads 615 us at 1.77 GHz, with zeros as data 434 us at
// 2.4 GHz.)
#include <type_traits>

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

// Waits until at most N of this wave's loads are in flight and its LDS reads
// are done, then meets the other waves.  One asm block: a fence would wait
// for every direct-to-LDS load in flight.
template <int N>
__device__ __forceinline__ void ring_barrier() {
  __asm__ volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
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
// first matrix instructions, then a global load after every one or two of
// the next.  Nothing moves from one slice into another.
template <int J, int LOADS>
__device__ __forceinline__ void slice_order() {
  constexpr int kRest = 4 * J - (4 + J) / 2, kEach = kRest >= 2 * LOADS ? 2 : 1;
#pragma unroll
  for (int i = 0; i < (4 + J) / 2; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
  }
  if constexpr (J % 2 == 1) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    if (kEach * i < kRest) __builtin_amdgcn_sched_group_barrier(0x008, kEach, 0);
    __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
  }
  if constexpr (kRest > kEach * LOADS) __builtin_amdgcn_sched_group_barrier(0x008, kRest - kEach * LOADS, 0);
  __builtin_amdgcn_sched_barrier(0);
}

// The ring holds R half-stages; the loads of a pair of them (e, e + 1: e
// even) go out in four equal parts, the first after the barrier of half-stage
// e + 1 - R, which frees the pair's second slot, the others in the next three
// slices.
template <int J>
struct Ring {
  static constexpr int kSlots = J == 1 ? 4 : J == 2 ? 6 : 5;                      // what the LDS holds (J = 1: two workgroups)
  static constexpr int kTurn = kSlots % 2 == 0 ? kSlots : 2 * kSlots;             // half-stages after which slot and parity repeat
  static constexpr int kPair = 2 * (4 + J);                                       // loads of a pair
  static constexpr int kA = (kPair + 3) / 4, kB = (kPair + 2) / 4, kC = (kPair + 1) / 4;
  // loads of pair e that have gone out before the first half-stage
  static constexpr int before(int e) {
    const int start = e + 1 - kSlots;
    return start < -2 ? kPair : start == -2 ? kA + kB + kC : start == -1 ? kA : 0;
  }
  static constexpr int kAhead = before(2) + before(4);                            // .. of those, the ones behind pair 0's
  // loads in flight behind pair e's at the barrier of half-stage e - 1
  static constexpr int kBehind = (kSlots - 4) / 2 * kPair + (kSlots % 2 != 0 ? kA + kB : 0);
};

template <int J>
__global__ __launch_bounds__(256, 1) void k_w8a8_gemm(W8A8Args a) {
  constexpr int kTM = 64 * J, R = Ring<J>::kSlots, kSlot = kWBytes + kTM * kHalf;
  // one array per slot (those that the ring does not have are never named, so
  // take no room): a read of one is not held for loads into another
  __shared__ __attribute__((aligned(16))) uint8_t s0[kSlot];
  __shared__ __attribute__((aligned(16))) uint8_t s1[kSlot];
  __shared__ __attribute__((aligned(16))) uint8_t s2[kSlot];
  __shared__ __attribute__((aligned(16))) uint8_t s3[kSlot];
  __shared__ __attribute__((aligned(16))) uint8_t s4[kSlot];
  __shared__ __attribute__((aligned(16))) uint8_t s5[kSlot];

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
  const int all = static_cast<int>((K + kHalf - 1) / kHalf), per = ((all + S - 1) / S + 1) & ~1;
  const int h_begin = share * per < all ? share * per : all, h_end = h_begin + per < all ? h_begin + per : all;

  // Loads: instruction i of wave w fills rows 16 (4 i + w) .. +15 of an
  // operand, four 16-byte pieces a row; piece c of row r sits at
  // c ^ ((r / 4) % 4), which puts one piece of 16 consecutive rows in 16
  // distinct bank groups.  Rows past the matrix lie outside the resource and
  // read as zero; pieces past K and half-stages past the share get an offset
  // outside it.
  const int64_t xrows = M - m0 < kTM ? M - m0 : kTM, wrows = N - n0 < kTN ? N - n0 : kTN;
  const rsrc_t xr = uniform_rsrc(a.xq + m0 * K, static_cast<uint32_t>(xrows * K));
  const rsrc_t wr = uniform_rsrc(a.wq + n0 * K, static_cast<uint32_t>(wrows * K));
  const int piece = (lane & 3) ^ ((lane >> 4) & 3);
  const uint32_t voff = static_cast<uint32_t>((wave * 16 + (lane >> 2)) * K + piece * 16);
  const int tail = static_cast<int>(K % kHalf);
  const uint32_t voff_tail = voff | ((tail != 0 && piece * 16 >= tail) ? 0x80000000u : 0u);
  const int wslot = wave * 1024;
  auto slot = [&](int s) {
    return s % R == 0 ? s0 : s % R == 1 ? s1 : s % R == 2 ? s2 : s % R == 3 ? s3 : s % R == 4 ? s4 : s5;
  };
  // load i of the pair of half-stages hs, hs + 1: both halves of a row
  // group's 128-byte lines one behind the other; row groups < 4 are channels
  auto load = [&](int hs, int s, int i) {
    const int half = i & 1, row = i >> 1;
    const uint32_t vo = hs + half >= h_end ? 0x80000000u : hs + half == all - 1 ? voff_tail : voff;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(row < 4 ? wr : xr, (lds_ptr_t)(slot(s + half) + row * 4096 + wslot), 16, vo,
                                             static_cast<int>((row & 3) * 64 * K + (hs + half) * kHalf), 0, 0);
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

  using G = Ring<J>;
  Frags<J> f0, f1;
#pragma unroll
  for (int e = 0; e < R; e += 2)
#pragma unroll
    for (int i = 0; i < G::before(e); ++i) load(h_begin + e, e, i);
  __asm__ volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(G::kAhead) : "memory");
  read_frags<J>(s0, wrow + c0, xrow + c0, f0);

  int hs0 = h_begin;
  auto turn = [&](auto last) __attribute__((always_inline)) {
#pragma unroll
    for (int p = 0; p < G::kTurn; ++p) {
      if (decltype(last)::value && p % 2 == 0 && hs0 + p >= h_end) return;
      const bool starts = ((p + R) & 1) != 0;  // this half-stage's barrier frees a pair of slots
      read_frags<J>(slot(p), wrow + c1, xrow + c1, f1);
      if (starts) {
#pragma unroll
        for (int i = G::kA + G::kB + G::kC; i < G::kPair; ++i) load(hs0 + p + R - 3, p + R - 3, i);
      } else {
#pragma unroll
        for (int i = G::kA; i < G::kA + G::kB; ++i) load(hs0 + p + R - 2, p + R - 2, i);
      }
      mfmas(f0);
      if (starts)
        slice_order<J, G::kPair - G::kA - G::kB - G::kC>();
      else
        slice_order<J, G::kB>();
      if (p % 2 != 0)
        ring_barrier<G::kBehind>();
      else
        ring_barrier<63>();  // the next half-stage has landed with this one
      read_frags<J>(slot(p + 1), wrow + c0, xrow + c0, f0);
      if (starts) {
#pragma unroll
        for (int i = 0; i < G::kA; ++i) load(hs0 + p + R - 1, p + R - 1, i);
      } else {
#pragma unroll
        for (int i = G::kA + G::kB; i < G::kA + G::kB + G::kC; ++i) load(hs0 + p + R - 2, p + R - 2, i);
      }
      mfmas(f1);
      if (starts)
        slice_order<J, G::kA>();
      else
        slice_order<J, G::kC>();
    }
  };
  // whole turns of the ring, then the pairs that are left (an exit inside the
  // loop would move the sums about in it)
  for (; hs0 + G::kTurn <= h_end; hs0 += G::kTurn) turn(std::false_type{});
  turn(std::true_type{});
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
// channels of one token, as the matrix instruction left them.  128 x 8192 in
// eight shares: 8.0 us, 36 MB (4.5 TB/s).
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

// Tile height and shares of K by estimated time.  The constants were fitted
// to every allowed shape at 59 sizes (65 .. 4096 tokens, 512 .. 32942
// channels, K 256 .. 28672): a half-stage of a lone workgroup takes 0.47,
// 0.44, 0.46, 0.89 us (J = 1 .. 4), of a full card 0.67 (two workgroups a
// unit, J = 1 only), 0.51, 0.63, 0.73 us, start and end of a tile as long as
// 5, 9, 7, 26 half-stages; joining shares costs a launch and 8 bytes per
// output and share at 4.4 TB/s.  The operands stream no faster than 4.9 TB/s
// on a full card, 1.2 TB/s and its share of the rest on part of one; of
// shapes that this floor makes equal, the one with less work of its own.
// (With one floor of 4.5 TB/s for all, ties to the tallest, 128 x 8192 x 28672
// took J = 3 in 6 shares, 74 us, for J = 2 in 8, 62; over 75 sizes, 65 .. 4096
// tokens, the picks were 3.7 % off the fastest, 28 % at worst, now 1.5 and 15.)
// 333 x 32003 x 4096: J = 3 53 us, J = 4 62, J = 2 73; 2772 x 32768 x 512: J =
// 3 92, J = 4 101; 4096 x 8192 x 28672: J = 4 704, J = 3 815, J = 2 869.
W8A8Shape w8a8_gemm_shape(int64_t M, int64_t N, int64_t K) {
  static const double kLone[4] = {0.47, 0.44, 0.46, 0.89}, kFull[4] = {0.67, 0.51, 0.63, 0.73};
  static const double kEnds[4] = {5, 9, 7, 26};
  static const int kShares[] = {1, 2, 3, 4, 6, 8, 12, 16};
  const int64_t halves = (K + kHalf - 1) / kHalf;
  const double operands = static_cast<double>(K) * static_cast<double>(M + N);  // bytes
  W8A8Shape best;
  double best_t = 0.0, best_own = 0.0;
  for (int j = 4; j >= 1; --j) {
    const int64_t tiles = w8a8_gemm_tiles(M, N, j), slots = j == 1 ? 512 : 256;
    for (int s : kShares) {
      if (s > 1 && (halves < 8 * s || tiles * s > slots)) continue;
      const double fill = tiles * s < slots ? static_cast<double>(tiles * s) / static_cast<double>(slots) : 1.0;
      const double half = kLone[j - 1] + (kFull[j - 1] - kLone[j - 1]) * fill;
      const double rounds = static_cast<double>((tiles * s + slots - 1) / slots);
      const double own = rounds * (static_cast<double>((halves + s - 1) / s) + kEnds[j - 1]) * half;
      const double stream = operands / (1.2e6 + 3.7e6 * fill);
      double t = own < stream ? stream : own;
      if (s > 1) t += 3.8 + 8.0 * static_cast<double>(M) * static_cast<double>(N) * s / 4.4e6;
      if (best_t == 0.0 || t < best_t || (t == best_t && own < best_own)) {
        best_t = t;
        best_own = own;
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
