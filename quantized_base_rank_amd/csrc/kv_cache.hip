// A paged cache of keys and values in 8-bit rows: a row is one token's key (or
// value) of one head, D codes and an fp32 scale, held as codes [pages][heads]
// [page][D] and scales [pages][heads][page].  Rounding and non-finite rows are
// those of the 8-bit rows (q8_rows.hip).
//
// Sixteen lanes take a row of up to 128 elements, eight each, so a wave's
// four rows are four heads of one token or of neighbouring tokens.  HBM-bound.
#include "attn_common.hpp"
#include "kernels.hpp"
#include "q8_common.hpp"

namespace qlin {

namespace {

// Place of packed token t: the sequence's new tokens are the last of its
// cached ones.  b = -1: a row behind the last sequence.
struct Place {
  int b, j;
};
__device__ __forceinline__ Place place_of(const KvBatchArgs& s, int t) {
  const int b = seq_of(s.cu, s.B, s.T, t);
  if (b < 0) return Place{-1, 0};
  const int s0 = seq_start(s.cu, b, s.T), s1 = seq_start(s.cu, b + 1, s.T);
  const int64_t j = static_cast<int64_t>(s.lens[b]) - (s1 - s0) + (t - s0);
  return Place{b, j < 0 || j > 0x7FFFFFFF ? -1 : static_cast<int>(j)};
}

__global__ __launch_bounds__(256) void k_kv_write(KvWriteArgs a) {
  const int lane = threadIdx.x & 15;
  const int64_t rows = static_cast<int64_t>(a.s.T) * a.c.H * 2;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4); i < rows;
       i += static_cast<int64_t>(gridDim.x) * 16) {
    const int64_t th = i >> 1;
    const int t = static_cast<int>(th / a.c.H), h = static_cast<int>(th % a.c.H);
    const bool is_v = (i & 1) != 0;
    const Place p = place_of(a.s, t);
    const int pg = p.b < 0 ? -1 : page_of(a.s.table, a.s.table_len, a.c.pages, a.c.page_shift, p.b, p.j);
    if (pg < 0) continue;  // (sixteen lanes alike)
    const uint16_t* x = (is_v ? a.v + t * a.v_ld : a.k + t * a.k_ld) + h * a.c.D;
    const bool in = 8 * lane < a.c.D;
    const u32x4 v = in ? *reinterpret_cast<const u32x4*>(x + 8 * lane) : u32x4{0, 0, 0, 0};
    float mx = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) mx = max_abs_nan(mx, elem8(v, e));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) mx = max_abs_nan(mx, __shfl_xor(mx, o, 16));
    const RowScale s = row_scale(mx);
    const int64_t row = ((static_cast<int64_t>(pg) * a.c.H + h) << a.c.page_shift) + (p.j & ((1 << a.c.page_shift) - 1));
    if (in)
      *reinterpret_cast<u32x2*>((is_v ? a.c.v : a.c.k) + row * a.c.D + 8 * lane) =
          finite_f32(mx) ? codes8(v, s) : u32x2{0u, 0u};
    if (lane == 0) (is_v ? a.c.vs : a.c.ks)[row] = s.scale;
  }
}

__global__ __launch_bounds__(256) void k_kv_read(KvReadArgs a) {
  const int lane = threadIdx.x & 15;
  const int64_t rows = static_cast<int64_t>(a.s.T) * a.c.H * 2;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4); i < rows;
       i += static_cast<int64_t>(gridDim.x) * 16) {
    const int64_t th = i >> 1;
    const int t = static_cast<int>(th / a.c.H), h = static_cast<int>(th % a.c.H);
    const bool is_v = (i & 1) != 0;
    const Place p = place_of(a.s, t);
    if (p.b < 0 || 8 * lane >= a.c.D) continue;
    const int pg = page_of(a.s.table, a.s.table_len, a.c.pages, a.c.page_shift, p.b, p.j);
    u32x4 out = {0, 0, 0, 0};
    if (pg >= 0) {
      const int64_t row = ((static_cast<int64_t>(pg) * a.c.H + h) << a.c.page_shift) + (p.j & ((1 << a.c.page_shift) - 1));
      out = values8(*reinterpret_cast<const u32x2*>((is_v ? a.c.v : a.c.k) + row * a.c.D + 8 * lane),
                    (is_v ? a.c.vs : a.c.ks)[row]);
    }
    *reinterpret_cast<u32x4*>((is_v ? a.v : a.k) + th * a.c.D + 8 * lane) = out;
  }
}

// Workgroups for the rows of T tokens, sixteen rows each.
uint32_t kv_grid(int64_t rows) { return row_grid(rows, 16); }

}  // namespace

hipError_t launch_kv_write(const KvWriteArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(k_kv_write, dim3(kv_grid(2LL * a.s.T * a.c.H)), dim3(256), 0, stream, a);
  return hipGetLastError();
}
hipError_t launch_kv_read(const KvReadArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(k_kv_read, dim3(kv_grid(2LL * a.s.T * a.c.H)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace qlin
