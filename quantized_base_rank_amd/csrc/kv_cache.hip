// A paged cache of keys and values in 8-bit rows: a row is one token's key (or
// value) of one head, D codes and an fp32 scale, held as codes [pages][heads]
// [page][D] and scales [pages][heads][page].  Rounding and non-finite rows are
// those of the 8-bit rows (q8_rows.hip).
//
// A wave takes sixteen rows of one token (its key heads, then its value heads),
// sixteen lanes a row of up to 128 elements, so the token's sequence, place and
// page are looked up once for all of them.  HBM-bound: 4 x 4096 tokens, 8 heads
// of 128, 102 MB: written in 24 us (4.2 TB/s, every store behind its row's
// largest element), read back in 18.6 (5.5 TB/s).  One token of each of 64
// sequences: 4.9 and 4.0 us, the chain of lookups.
#include "attn_common.hpp"
#include "kernels.hpp"
#include "q8_common.hpp"

namespace qlin {

namespace {

constexpr int kRows = 16;  // rows of a wave, four at a time

// Row of the cache's rows, before the head's is added, of packed token t: the
// sequence's new tokens are the last of its cached ones.
struct Place {
  bool known;  // t belongs to a sequence
  int page;    // -1: not there
  int row;     // in the page
};
__device__ __forceinline__ Place place_of(const KvBatchArgs& s, const KvCacheArgs& c, int t) {
  const int b = seq_of(s.cu, s.B, s.T, t);
  if (b < 0) return Place{false, -1, 0};
  const int s0 = uniform_start(s.cu, b, s.T), s1 = uniform_start(s.cu, b + 1, s.T);
  const int64_t j = static_cast<int64_t>(uniform_i32(s.lens, b)) - (s1 - s0) + (t - s0);
  if (j < 0 || j > 0x7FFFFFFF) return Place{true, -1, 0};
  const int at = static_cast<int>(j);
  return Place{true, uniform_page(s.table, s.table_len, c.pages, c.page_shift, b, at), at & ((1 << c.page_shift) - 1)};
}

// f(token, first row) for every sixteen rows; a longer queue is walked.
template <typename F>
__device__ __forceinline__ void each_part(int T, int H, F f) {
  const int parts = (2 * H + kRows - 1) / kRows;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int64_t n = static_cast<int64_t>(T) * parts;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 4 + wave; i < n; i += static_cast<int64_t>(gridDim.x) * 4) {
    const int64_t t = i / parts;
    f(static_cast<int>(t), static_cast<int>(i - t * parts) * kRows);
  }
}

__global__ __launch_bounds__(256) void k_kv_write(KvWriteArgs a) {
  const int lane = threadIdx.x & 15, sub = (threadIdx.x & 63) >> 4, H = a.c.H, D = a.c.D;
  const bool in = 8 * lane < D;
  each_part(a.s.T, H, [&](int t, int r0) {
    u32x4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + 4 * i + sub;
      const uint16_t* const src = r < H ? a.k + t * a.k_ld + r * D : a.v + t * a.v_ld + (r - H) * D;
      x[i] = in && r < 2 * H ? *reinterpret_cast<const u32x4*>(src + 8 * lane) : u32x4{0, 0, 0, 0};
    }
    const Place p = place_of(a.s, a.c, t);
    if (p.page < 0) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + 4 * i + sub, head = r < H ? r : r - H;
      float mx = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) mx = max_abs_nan(mx, elem8(x[i], e));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) mx = max_abs_nan(mx, __shfl_xor(mx, o, 16));
      if (r >= 2 * H) continue;
      const RowScale s = row_scale(mx);
      const int64_t row = ((static_cast<int64_t>(p.page) * H + head) << a.c.page_shift) + p.row;
      if (in)
        *reinterpret_cast<u32x2*>((r < H ? a.c.k : a.c.v) + row * D + 8 * lane) =
            finite_f32(mx) ? codes8(x[i], s) : u32x2{0u, 0u};
      if (lane == 0) (r < H ? a.c.ks : a.c.vs)[row] = s.scale;
    }
  });
}

__global__ __launch_bounds__(256) void k_kv_read(KvReadArgs a) {
  // (lanes past D stay: the whole wave looks the token up)
  const int lane = threadIdx.x & 15, sub = (threadIdx.x & 63) >> 4, H = a.c.H, D = a.c.D;
  const bool in = 8 * lane < D;
  each_part(a.s.T, H, [&](int t, int r0) {
    const Place p = place_of(a.s, a.c, t);
    if (!p.known) return;
    u32x2 c[4];
    float s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + 4 * i + sub, head = r < H ? r : r - H;
      const int64_t row = ((static_cast<int64_t>(p.page) * H + head) << a.c.page_shift) + p.row;
      const bool there = in && p.page >= 0 && r < 2 * H;
      c[i] = there ? *reinterpret_cast<const u32x2*>((r < H ? a.c.k : a.c.v) + row * D + 8 * lane) : u32x2{0u, 0u};
      s[i] = there ? (r < H ? a.c.ks : a.c.vs)[row] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + 4 * i + sub, head = r < H ? r : r - H;
      if (in && r < 2 * H)
        *reinterpret_cast<u32x4*>((r < H ? a.k : a.v) + (static_cast<int64_t>(t) * H + head) * D + 8 * lane) = values8(c[i], s[i]);
    }
  });
}

// Workgroups for T tokens, four waves each.
uint32_t kv_grid(int64_t T, int H) { return row_grid(T * ((2 * H + kRows - 1) / kRows), 4); }

}  // namespace

hipError_t launch_kv_write(const KvWriteArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(k_kv_write, dim3(kv_grid(a.s.T, a.c.H)), dim3(256), 0, stream, a);
  return hipGetLastError();
}
hipError_t launch_kv_read(const KvReadArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(k_kv_read, dim3(kv_grid(a.s.T, a.c.H)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace qlin
