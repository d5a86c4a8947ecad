// Causal attention with grouped heads: o_i = sum_j p_ij v_j over the keys at
// or before token i's place, p the softmax of c q_i . k_j, in one pass over
// the keys with a running maximum and sum per query row.
//
// A workgroup takes 128 query rows (32 per wave) of one sequence and key head
// and walks the keys 64 at a time.  The products are formed transposed,
// S^T = K Q^T and O^T = V^T P^T: a lane then holds scores of one query row
// only, so maximum and sum need a single exchange between the wave's halves,
// and the scores in its registers are, rounded to bf16, the operand of the
// second product as they stand.
//
// Roundings: p (0 .. 1) to bf16 for the second product, relative 2^-9 at most
// and independent from key to key, while the sum of p takes the unrounded
// values; everything else is fp32.  Over the cache, keys and values enter as
// their integer codes (exact in bf16); a key's scale multiplies its score and
// a value's scale its p, both in fp32.
//
// What is masked does not count whatever it holds: scores behind the mask are
// replaced, not multiplied, and in steps that the mask cuts, values that are
// not finite are left out of the product (0 times them is not 0) and added to
// the rows that see them.
#include "attn_common.hpp"
#include "kernels.hpp"

namespace qlin {

namespace {

constexpr int kBM = 128;  // query rows of a workgroup
constexpr int kBN = 64;   // keys of a step

template <int DP, bool PAGED>
__global__ __launch_bounds__(256, 1) void k_attn(AttnArgs a) {
  constexpr int NP = DP / 8, KS = DP / 16, DB = DP / 32;
  __shared__ __attribute__((aligned(16))) uint8_t sk[kBN * DP * 2];
  __shared__ __attribute__((aligned(16))) uint8_t sv[kBN * DP * 2];
  __shared__ __attribute__((aligned(16))) float s_ks[kBN], s_vs[kBN];

  const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kvh = static_cast<int>(blockIdx.x) % a.Hkv;
  const int tiles = static_cast<int>(gridDim.x) / a.Hkv;
  RowTile rt;
  if (!find_rows(a.s.cu, a.s.B, a.s.T, a.g, kBM, tiles - 1 - static_cast<int>(blockIdx.x) / a.Hkv, &rt)) return;
  const int D = a.D, len = PAGED ? cached_len(a.s.lens, rt.b, a.max_len) : rt.n;
  const int first = len - rt.n;  // place of the first new token

  // this lane's query row
  const int tok0 = rt.row0 / a.g, rem0 = rt.row0 - tok0 * a.g;
  const int in_tile = wave * 32 + l32;
  const bool in = rt.row0 + in_tile < rt.rows;
  const int x = rem0 + in_tile, dt = small_div(x, a.g_inv);
  const int tok = in ? tok0 + dt : tok0, hq = kvh * a.g + (in ? x - dt * a.g : 0);
  const int seen = in ? first + tok + 1 : 0;  // keys before this place count
  const int last_in = (rt.rows - rt.row0 < kBM ? rt.rows - rt.row0 : kBM) - 1;
  const int end = first + (rt.row0 + last_in) / a.g + 1;  // keys of the tile's last row
  const int w_last = wave * 32 + 31 < last_in ? wave * 32 + 31 : last_in;
  const int w_end = wave * 32 > last_in ? 0 : first + tok0 + small_div(rem0 + w_last, a.g_inv) + 1;
  const int w_all = wave * 32 + 31 > last_in ? 0 : first + tok0 + small_div(rem0 + wave * 32, a.g_inv) + 1;

  u32x4 qf[KS];
  const uint16_t* q = a.q + static_cast<int64_t>(rt.s0 + tok) * a.q_ld + hq * D;
#pragma unroll
  for (int s = 0; s < KS; ++s)
    qf[s] = 16 * s + 8 * h < D ? *reinterpret_cast<const u32x4*>(q + 16 * s + 8 * h) : u32x4{0, 0, 0, 0};

  f32x16 o[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) o[d] = f32x16{};
  float m = kMinusInf, l = 0.0f;

  for (int j0 = 0; j0 < end; j0 += kBN) {
    uint32_t there = 0xF;  // blocks of 16 keys whose page is there
    if constexpr (PAGED) {
      int pg[4];
      there = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        pg[i] = j0 + 16 * i < len
                    ? page_of(a.s.table, a.s.table_len, a.c.pages, a.c.page_shift, rt.b, j0 + 16 * i) : -1;
        there |= pg[i] >= 0 ? 1u << i : 0u;
      }
#pragma unroll
      for (int i = 0; i < kBN * NP / 256; ++i) {
        const int idx = tid + 256 * i, r = idx / NP, c = idx % NP, blk = r >> 4;
        const int p = blk == 0 ? pg[0] : blk == 1 ? pg[1] : blk == 2 ? pg[2] : pg[3];
        u32x2 ck = {0, 0}, cv = {0, 0};
        if (p >= 0 && 8 * c < D) {
          const int64_t row = ((static_cast<int64_t>(p) * a.c.H + kvh) << a.c.page_shift) +
                              ((j0 + r) & ((1 << a.c.page_shift) - 1));
          ck = *reinterpret_cast<const u32x2*>(a.c.k + row * D + 8 * c);
          cv = *reinterpret_cast<const u32x2*>(a.c.v + row * D + 8 * c);
          if (c == 0) {
            s_ks[r] = a.c.ks[row] * a.c2;
            s_vs[r] = a.c.vs[row];
          }
        }
        const u32x2 k0 = codes_bf16(ck.x), k1 = codes_bf16(ck.y), v0 = codes_bf16(cv.x), v1 = codes_bf16(cv.y);
        *reinterpret_cast<u32x4*>(sk + piece_at<DP>(r, c)) = u32x4{k0.x, k0.y, k1.x, k1.y};
        *reinterpret_cast<u32x4*>(sv + piece_at<DP>(r, c)) = u32x4{v0.x, v0.y, v1.x, v1.y};
      }
    } else {
#pragma unroll
      for (int i = 0; i < kBN * NP / 256; ++i) {
        const int idx = tid + 256 * i, r = idx / NP, c = idx % NP;
        u32x4 k = {0, 0, 0, 0}, v = {0, 0, 0, 0};
        if (j0 + r < len && 8 * c < D) {
          const int64_t row = rt.s0 + j0 + r;
          k = *reinterpret_cast<const u32x4*>(a.k + row * a.k_ld + kvh * D + 8 * c);
          v = *reinterpret_cast<const u32x4*>(a.v + row * a.v_ld + kvh * D + 8 * c);
        }
        *reinterpret_cast<u32x4*>(sk + piece_at<DP>(r, c)) = k;
        *reinterpret_cast<u32x4*>(sv + piece_at<DP>(r, c)) = v;
      }
    }
    __syncthreads();
    if (j0 < w_end) {
      f32x16 s[2];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        s[kb] = f32x16{};
#pragma unroll
        for (int t = 0; t < KS; ++t)
          s[kb] = mfma32(*reinterpret_cast<const u32x4*>(sk + piece_at<DP>(kb * 32 + l32, 2 * t + h)), qf[t], s[kb]);
      }
      const bool masked = j0 + kBN > w_all || there != 0xF;
      float top = kMinusInf;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int r = kb * 32 + acc_row(i, h);
          float t = s[kb][i] * (PAGED ? s_ks[r] : a.c2);
          if (masked && (j0 + r >= seen || (PAGED && (there >> (2 * kb + (i >> 3)) & 1) == 0))) t = kMinusInf;
          s[kb][i] = t;
          top = fmaxf(top, t);
        }
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      const float m_new = fmaxf(m, top), shift = m_new == kMinusInf ? 0.0f : m_new;
      const float alpha = __builtin_amdgcn_exp2f(m - shift);
      m = m_new;
      float sum = 0.0f;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float p = __builtin_amdgcn_exp2f(s[kb][i] - shift);
          sum += p;
          if constexpr (PAGED) {
            const int r = kb * 32 + acc_row(i, h);
            s[kb][i] = masked && s[kb][i] == kMinusInf ? 0.0f : p * s_vs[r];
          } else {
            s[kb][i] = p;
          }
        }
      l = l * alpha + sum;
#pragma unroll
      for (int d = 0; d < DB; ++d) o[d] *= alpha;
      uint32_t odd = 0;  // non-finite values behind some row's mask
#pragma unroll
      for (int kg = 0; kg < 4; ++kg) {
        const u32x4 p = pack_operand(s[kg >> 1], kg & 1);
#pragma unroll
        for (int d = 0; d < DB; ++d) {
          u32x4 v = column_operand<DP>(sv, 16 * kg, 32 * d, lane);
          if (!PAGED && masked) odd |= clear_nonfinite(v);
          o[d] = mfma32(v, p, o[d]);
        }
      }
      if (!PAGED && masked && __ballot(odd != 0) != 0) {
        // they reach, as they are, the rows that see them
        for (int j = 0; j < kBN; ++j) {
          if (j0 + j >= seen) break;
#pragma unroll
          for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int c = 32 * d + acc_row(i, h);
              const float x = bf16_to_f32(*reinterpret_cast<const uint16_t*>(sv + piece_at<DP>(j, c >> 3) + (c & 7) * 2));
              if ((__float_as_uint(x) & 0x7F800000u) == 0x7F800000u) o[d][i] += x;
            }
        }
      }
    }
    __syncthreads();
  }

  l += __shfl_xor(l, 32, 64);
  if (!in) return;
  const int64_t row = static_cast<int64_t>(rt.s0 + tok) * a.Hq + hq;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // (no key: 0; NaN stays)
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int c = 32 * d + acc_row(i, h);
      if (c < D)
        *reinterpret_cast<u32x2*>(a.o + row * D + c) =
            u32x2{pack_bf16x2(o[d][i] * inv, o[d][i + 1] * inv), pack_bf16x2(o[d][i + 2] * inv, o[d][i + 3] * inv)};
    }
  if (a.lse != nullptr && h == 0) a.lse[row] = l == 0.0f ? kMinusInf : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

}  // namespace

hipError_t launch_attn(const AttnArgs& a, bool paged, hipStream_t stream) {
  const int64_t tiles = static_cast<int64_t>(a.s.T) * a.g / kBM + a.s.B;
  const dim3 grid(static_cast<uint32_t>(tiles * a.Hkv));
  if (a.D <= 64) {
    if (paged)
      hipLaunchKernelGGL((k_attn<64, true>), grid, dim3(256), 0, stream, a);
    else
      hipLaunchKernelGGL((k_attn<64, false>), grid, dim3(256), 0, stream, a);
  } else if (paged) {
    hipLaunchKernelGGL((k_attn<128, true>), grid, dim3(256), 0, stream, a);
  } else {
    hipLaunchKernelGGL((k_attn<128, false>), grid, dim3(256), 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace qlin
