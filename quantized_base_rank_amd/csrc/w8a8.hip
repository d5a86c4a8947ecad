// Product of 8-bit rows: y[m][n] = xs[m] ws[n] sum_k xq[m][k] wq[n][k], the
// sum taken by the 8-bit matrix instructions in int32 (exact for
// K <= 131056, where 128 * 128 * K < 2^31).
//
// Tile: 256 channels x 256 tokens per workgroup of 4 waves (one per SIMD),
// each wave 128 x 128 in 256 accumulator registers, so that a K slice of 32
// bytes costs 8 LDS reads of 16 bytes per lane for 16 matrix instructions.
// Both operands stream through a ring of four 64-byte-deep half-stages (32 KB
// each) by direct-to-LDS loads issued three half-stages ahead.  One barrier
// per half-stage, in its middle: by then every wave holds the half-stage's
// last fragments in registers, so its slot is free for the loads of the
// half-stage four on, and the next one has landed (counted wait), so the
// fragments of its first slice load while this one's last matrix
// instructions run.
#include "device_common.hpp"
#include "kernels.hpp"
#include "q8_common.hpp"

namespace qlin {

namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr int kWT = 256;              // tile: channels, and tokens
constexpr int kHalf = 64;             // bytes of K per half-stage
constexpr int kOpBytes = kWT * kHalf; // one operand of a half-stage: 16 KB
constexpr int kSlotBytes = 2 * kOpBytes;

// Waits until at most two half-stages (16 loads) of this wave's loads are in
// flight and its LDS reads are done, then meets the other waves.  One asm
// block: a fence would wait for every direct-to-LDS load in flight.
__device__ __forceinline__ void half_barrier() {
  __asm__ volatile("s_waitcnt vmcnt(16) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Fragments of one 32-byte slice of K: lane (l, h) holds bytes 16 h .. of row
// l of each of the wave's four 32-row tiles.
struct Frags {
  i32x4 w[4], x[4];
};

__device__ __forceinline__ void read_frags(const uint8_t* slot, uint32_t woff, uint32_t xoff, Frags& f) {
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    f.w[t] = *reinterpret_cast<const i32x4*>(slot + woff + t * 32 * kHalf);
    f.x[t] = *reinterpret_cast<const i32x4*>(slot + xoff + t * 32 * kHalf);
  }
}

__global__ __launch_bounds__(256, 1) void k_w8a8_gemm(W8A8Args a) {
  // one array per slot: a read of one is not held for loads into another
  __shared__ __attribute__((aligned(16))) uint8_t s0[kSlotBytes];
  __shared__ __attribute__((aligned(16))) uint8_t s1[kSlotBytes];
  __shared__ __attribute__((aligned(16))) uint8_t s2[kSlotBytes];
  __shared__ __attribute__((aligned(16))) uint8_t s3[kSlotBytes];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  const int wn = wave & 1, wm = wave >> 1;
  const int64_t M = a.M, N = a.N, K = a.K;
  const int tiles_m = static_cast<int>((M + kWT - 1) / kWT), tiles_n = static_cast<int>((N + kWT - 1) / kWT);
  int tm, tn;
  grouped_tile(xcd_round_order(static_cast<int>(blockIdx.x), tiles_m * tiles_n), tiles_m, tiles_n, tm, tn);
  const int64_t m0 = static_cast<int64_t>(tm) * kWT, n0 = static_cast<int64_t>(tn) * kWT;
  const int halves = static_cast<int>((K + kHalf - 1) / kHalf);

  // Loads: instruction i of wave w fills rows 16 (4 i + w) .. +15 of an
  // operand, four 16-byte pieces a row; piece c of row r sits at
  // c ^ ((r / 4) % 4), which puts one piece of 16 consecutive rows in 16
  // distinct bank groups.  Rows past the matrix lie outside the resource and
  // read as zero, pieces past K get an offset outside it, half-stages past
  // the end an empty resource.
  const int64_t xrows = M - m0 < kWT ? M - m0 : kWT, wrows = N - n0 < kWT ? N - n0 : kWT;
  const rsrc_t xr = uniform_rsrc(a.xq + m0 * K, static_cast<uint32_t>(xrows * K));
  const rsrc_t wr = uniform_rsrc(a.wq + n0 * K, static_cast<uint32_t>(wrows * K));
  const rsrc_t none = uniform_rsrc(a.xq, 0u);
  const int piece = (lane & 3) ^ ((lane >> 4) & 3);
  const uint32_t voff = static_cast<uint32_t>((wave * 16 + (lane >> 2)) * K + piece * 16);
  const int tail = static_cast<int>(K % kHalf);
  const uint32_t voff_tail = voff | ((tail != 0 && piece * 16 >= tail) ? 0x80000000u : 0u);
  const int wslot = wave * 1024;
  auto load = [&](int hs, uint8_t* slot, int i) {  // i < 4: channels, else tokens
    const rsrc_t r = hs < halves ? (i < 4 ? wr : xr) : none;
    const uint32_t vo = hs == halves - 1 ? voff_tail : voff;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)(slot + i * 4096 + wslot), 16, vo,
                                             static_cast<int>((i & 3) * 64 * K + hs * kHalf), 0, 0);
  };

  // fragment offsets of the half-stage's two slices
  const int sw = (l32 >> 2) & 3;
  const uint32_t wrow = static_cast<uint32_t>((wn * 128 + l32) * kHalf);
  const uint32_t xrow = static_cast<uint32_t>(kOpBytes + (wm * 128 + l32) * kHalf);
  const uint32_t c0 = static_cast<uint32_t>((h ^ sw) << 4), c1 = c0 ^ 32u;

  i32x16 acc[4][4];  // [channels][tokens]
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = i32x16{};
  auto mfmas = [&](const Frags& f) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.w[i], f.x[j], acc[i][j], 0, 0, 0);
  };

  Frags f0, f1;
#pragma unroll
  for (int st = 0; st < 4; ++st)
#pragma unroll
    for (int i = 0; i < 8; ++i) load(st, st == 0 ? s0 : st == 1 ? s1 : st == 2 ? s2 : s3, i);
  __asm__ volatile("s_waitcnt vmcnt(24)\n\ts_barrier" ::: "memory");
  read_frags(s0, wrow + c0, xrow + c0, f0);

  // whole turns of the ring: half-stages past the end hold zeros
  for (int hs0 = 0; hs0 < halves; hs0 += 4) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      uint8_t* const cur = p == 0 ? s0 : p == 1 ? s1 : p == 2 ? s2 : s3;
      const uint8_t* const nxt = p == 0 ? s1 : p == 1 ? s2 : p == 2 ? s3 : s0;
      read_frags(cur, wrow + c1, xrow + c1, f1);
      mfmas(f0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
      }
      half_barrier();
#pragma unroll
      for (int i = 0; i < 8; ++i) load(hs0 + p + 4, cur, i);
      read_frags(nxt, wrow + c0, xrow + c0, f0);
      mfmas(f1);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      }
    }
  }
  __asm__ volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");

  // Output: lane (l, h) holds channel 32 i + 8 q + 4 h + v of token 32 j + l
  // at acc[i][j][4 q + v].  Each wave turns its 128 x 128 tile round in its
  // slot as bf16 rows of tokens (16-byte pieces XOR-swizzled by token), then
  // stores whole row segments.
  uint8_t* const out = wave == 0 ? s0 : wave == 1 ? s1 : wave == 2 ? s2 : s3;
  const int64_t mw = m0 + wm * 128, nw = n0 + wn * 128;
  float xs[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
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
      for (int j = 0; j < 4; ++j) {
        const int m = 32 * j + l32;
        float o[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) o[v] = static_cast<float>(acc[i][j][4 * q + v]) * xs[j] * ws[v];
        *reinterpret_cast<u32x2*>(out + m * 256 + (((c >> 3) ^ (m & 15)) << 4) + h * 8) =
            u32x2{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
      }
    }
  for (int it = 0; it < 32; ++it) {
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

}  // namespace

int w8a8_gemm_tiles(int64_t M, int64_t N) {
  return static_cast<int>((M + kWT - 1) / kWT * ((N + kWT - 1) / kWT));
}

hipError_t launch_w8a8_gemm(const W8A8Args& a, hipStream_t stream) {
  hipLaunchKernelGGL(k_w8a8_gemm, dim3(static_cast<uint32_t>(w8a8_gemm_tiles(a.M, a.N))), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace qlin
