// Causal attention with grouped heads: o_i = sum_j p_ij v_j over the keys at
// or before token i's place, p the softmax of c q_i . k_j, in one pass over
// the keys with a running maximum and sum per query row.
//
// A workgroup takes 32 W query rows (32 per wave) of one sequence and key head
// and walks the keys 64 at a time.  The products are formed transposed,
// S^T = K Q^T and O^T = V^T P^T: a lane then holds scores of one query row
// only, so maximum and sum need a single exchange between the wave's halves,
// and the scores in its registers are, rounded to bf16, the operand of the
// second product as they stand.
//
// Steps are shifted by one: S of step j + 1 and O of step j are formed
// together (32 matrix instructions at D = 128), then the softmax of step j + 1.
// Of eight waves, two on each SIMD, four run their matrix phase while the
// other four run their softmax, with a barrier between phases.  Keys and values
// stream through three buffers each.
//
// Roundings: p (0 .. 1) to bf16 for the second product, relative 2^-8 at most
// and independent from key to key, while the sum of p takes the unrounded
// values; everything else is fp32.  Over the cache, keys and values enter as
// their integer codes (exact in bf16); a key's scale multiplies its score and
// a value's scale its p, both in fp32.
//
// The maximum that p refers to is raised only once a score passes it by 2^8:
// p then stays below 2^8 (relative roundings do not change), and most steps
// leave O and the sum as they are.
//
// What is masked does not count whatever it holds: scores behind the mask are
// replaced, not multiplied, and in steps that the mask cuts, values that are
// not finite are set to zero for the product (0 times them is not 0) and added
// to the rows that see them.
#include "attn_common.hpp"
#include "kernels.hpp"

namespace qlin {

namespace {

constexpr int kBN = 64;          // keys of a step
constexpr float kRaise = 8.0f;   // log2 of what p may reach

// Waits until at most VM of this wave's loads and LG of its LDS accesses are
// on their way (-1: any number), then meets the other waves.
template <int VM, int LG>
__device__ __forceinline__ void barrier() {
  if constexpr (VM == 0 && LG == 0)
    __asm__ volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  else if constexpr (VM == 0)
    __asm__ volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
  else if constexpr (LG == 0)
    __asm__ volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  else
    __asm__ volatile("s_barrier" ::: "memory");
}

template <int DP, bool PAGED, int W>
__global__ __launch_bounds__(64 * W, W == 8 ? 2 : 1) void k_attn(AttnArgs a) {
  constexpr int NP = DP / 8, KS = DP / 16, DB = DP / 32;
  constexpr int kBM = 32 * W, kTile = kBN * DP * 2, kLoads = kTile / 1024 / W;
  static_assert(kLoads >= 1, "every wave loads a part of each tile");
  constexpr int kRowsPer = 64 / NP;  // rows of a load
  // three buffers of keys and of values (an array each: a read of one is not
  // held for loads into another), and the scales of cached ones
  __shared__ __attribute__((aligned(16))) uint8_t sk0[kTile];
  __shared__ __attribute__((aligned(16))) uint8_t sk1[kTile];
  __shared__ __attribute__((aligned(16))) uint8_t sk2[kTile];
  __shared__ __attribute__((aligned(16))) uint8_t sv0[kTile];
  __shared__ __attribute__((aligned(16))) uint8_t sv1[kTile];
  __shared__ __attribute__((aligned(16))) uint8_t sv2[kTile];
  __shared__ __attribute__((aligned(16))) float s_scale[PAGED ? 3 * 2 * kBN : 1];
  __shared__ int s_odd[3];  // 1 + the step whose values in this buffer were not finite
  if (threadIdx.x < 3) s_odd[threadIdx.x] = 0;
  auto sk = [&](int buf) { return buf % 3 == 0 ? sk0 : buf % 3 == 1 ? sk1 : sk2; };
  auto sv = [&](int buf) { return buf % 3 == 0 ? sv0 : buf % 3 == 1 ? sv1 : sv2; };

  const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // the last tiles, which see the most keys, first
  const int kvh = static_cast<int>(blockIdx.x) % a.Hkv;
  int rest = static_cast<int>(gridDim.x / a.Hkv) - 1 - static_cast<int>(blockIdx.x) / a.Hkv;
  const int share = PAGED ? rest % a.splits : 0;
  if constexpr (PAGED) rest /= a.splits;
  RowTile rt;
  if (!find_rows(a.s.cu, a.s.B, a.s.T, a.g, kBM, rest, &rt)) return;
  const int D = a.D, len = PAGED ? clamp_len(uniform_i32(a.s.lens, rt.b), a.max_len) : rt.n;
  const int first = len - rt.n;  // place of the first new token
  // this share's keys: places base .. base + per - 1 (steps count from base)
  const int base = PAGED ? share * a.per : 0, until = PAGED ? base + a.per : 0x7FFFFFFF;
  if (base > 0 && base >= len) return;  // (k_attn_join counts a sequence's shares alike)
  auto inside = [&](int v) { return v < until ? v : until; };

  // this lane's query row
  const int tok0 = rt.row0 / a.g, rem0 = rt.row0 - tok0 * a.g;
  const int in_tile = wave * 32 + l32;
  const bool in = rt.row0 + in_tile < rt.rows;
  const int x = rem0 + in_tile, dt = small_div(x, a.g_inv);
  const int tok = in ? tok0 + dt : tok0, hq = kvh * a.g + (in ? x - dt * a.g : 0);
  const int seen = in ? inside(first + tok + 1) : 0;  // keys before this place count
  const int last_in = (rt.rows - rt.row0 < kBM ? rt.rows - rt.row0 : kBM) - 1;
  const int end = inside(first + tok0 + small_div(rem0 + last_in, a.g_inv) + 1);  // keys of the tile's last row
  const int w_last = wave * 32 + 31 < last_in ? wave * 32 + 31 : last_in;
  // keys of the wave's last row, and keys that all its rows see
  const int w_end = wave * 32 > last_in ? 0 : inside(first + tok0 + small_div(rem0 + w_last, a.g_inv) + 1);
  const int w_all = wave * 32 + 31 > last_in ? 0 : inside(first + tok0 + small_div(rem0 + wave * 32, a.g_inv) + 1);
  const int steps = end > base ? (end - base + kBN - 1) / kBN : 0;

  u32x4 qf[KS];
  const uint16_t* q = a.q + static_cast<int64_t>(rt.s0 + tok) * a.q_ld + hq * D;
#pragma unroll
  for (int s = 0; s < KS; ++s)
    qf[s] = 16 * s + 8 * h < D ? *reinterpret_cast<const u32x4*>(q + 16 * s + 8 * h) : u32x4{0, 0, 0, 0};

  // ---- loads of packed keys and values, straight into LDS: load i of a wave
  // fills kRowsPer rows; rows past the sequence and elements past D lie outside
  // the resource and read as zero
  uint32_t vo_k[kLoads], vo_v[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = (wave * kLoads + i) * kRowsPer + lane / NP;
    const int c = (lane % NP) ^ piece_swizzle<DP>(r);
    const uint32_t out = 8 * c < D ? 0u : 0x80000000u;
    vo_k[i] = (static_cast<uint32_t>(r) * static_cast<uint32_t>(a.k_ld * 2) + c * 16) | out;
    vo_v[i] = (static_cast<uint32_t>(r) * static_cast<uint32_t>(a.v_ld * 2) + c * 16) | out;
  }
  auto load_packed = [&](int j, int buf, bool values) {
    const int64_t ld = values ? a.v_ld : a.k_ld;
    const int left = len - j * kBN;
    const uint32_t bytes = left > 0 ? static_cast<uint32_t>(((left < kBN ? left : kBN) - 1) * ld + D) * 2u : 0u;
    const uint16_t* const src = (values ? a.v : a.k) + (static_cast<int64_t>(rt.s0) + j * kBN) * ld + kvh * D;
    uint8_t* const dst = (values ? sv(buf) : sk(buf)) + wave * kLoads * 1024;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) load_to_lds(src, bytes, dst + i * 1024, values ? vo_v[i] : vo_k[i]);
  };
  // ---- keys and values from the cache: 16 codes a thread, held in registers
  // for a step, then written to LDS as bf16.  A wave's rows of a load lie in
  // one block of 16 keys, so in one page.
  constexpr int kChunks = DP / 16, kHold = (kBN * kChunks + 64 * W - 1) / (64 * W);
  const int row_t = tid / kChunks, chunk = tid % kChunks;
  const int page_mask = (1 << a.c.page_shift) - 1;
  const bool holds = (kBN * kChunks >= 64 * W || tid < kBN * kChunks) && 16 * chunk < D;
  uint32_t queue = 0xFFFF;  // blocks of 16 keys that are there, four bits a step
  // Lane i % 4: the page of block i % 4 of step j, -1 if it is not there.  (A
  // vector load: waits for scalar ones would wait for LDS too.)
  auto pages_of = [&](int j) {
    const int place = base + j * kBN + 16 * (lane & 3), at = place >> a.c.page_shift;
    if (place >= end || at >= a.s.table_len) return -1;
    const int p = a.s.table[static_cast<int64_t>(rt.b) * a.s.table_len + at];
    return p < a.c.pages ? p : -1;
  };
  auto blocks = [&](int p) { return static_cast<uint32_t>(__ballot(p >= 0)) & 0xFu; };
  u32x4 held_k[kHold], held_v[kHold];
  float held_ks[kHold], held_vs[kHold];
  auto fetch = [&](int j, int p, bool values) {
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      const int r = row_t + i * (64 * W / kChunks);
      const int pg = __builtin_amdgcn_readlane(p, __builtin_amdgcn_readfirstlane(r >> 4) & 3);
      (values ? held_v : held_k)[i] = u32x4{0, 0, 0, 0};
      if (pg >= 0 && holds) {
        const int64_t row = ((static_cast<int64_t>(pg) * a.c.H + kvh) << a.c.page_shift) + ((base + j * kBN + r) & page_mask);
        (values ? held_v : held_k)[i] = *reinterpret_cast<const u32x4*>((values ? a.c.v : a.c.k) + row * D + 16 * chunk);
        if (!values && chunk == 0) {
          held_ks[i] = a.c.ks[row];
          held_vs[i] = a.c.vs[row];
        }
      }
    }
  };
  auto put = [&](int buf, bool values) {
    uint8_t* const dst = values ? sv(buf) : sk(buf);
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      if (kBN * kChunks < 64 * W && tid >= kBN * kChunks) break;
      const int r = row_t + i * (64 * W / kChunks);
      const u32x4 c = (values ? held_v : held_k)[i];
      const u32x2 w0 = codes_bf16(c.x), w1 = codes_bf16(c.y), w2 = codes_bf16(c.z), w3 = codes_bf16(c.w);
      *reinterpret_cast<u32x4*>(dst + piece_at<DP>(r, 2 * chunk)) = u32x4{w0.x, w0.y, w1.x, w1.y};
      *reinterpret_cast<u32x4*>(dst + piece_at<DP>(r, 2 * chunk + 1)) = u32x4{w2.x, w2.y, w3.x, w3.y};
      if (!values && chunk == 0) {
        s_scale[buf % 3 * 2 * kBN + r] = held_ks[i];
        s_scale[buf % 3 * 2 * kBN + kBN + r] = held_vs[i];
      }
    }
  };

  // ---- fragments
  const uint32_t k_at = static_cast<uint32_t>(piece_at<DP>(l32, h));
  const int p16 = lane & 15, vr = 4 * h + (p16 >> 2), vc = 16 * ((lane >> 4) & 1) + 4 * (p16 & 3);
  const uint32_t v_at = static_cast<uint32_t>(piece_at<DP>(vr, vc >> 3) + (vc & 7) * 2);

  f32x16 o[DB], s[2];
  u32x4 pf[4];
#pragma unroll
  for (int d = 0; d < DB; ++d) o[d] = f32x16{};
  float m = kMinusInf, l = 0.0f;

  auto key = [&](int buf, int kb, int t) {
    return *reinterpret_cast<const u32x4*>(sk(buf) + (k_at ^ (t << 5)) + kb * 32 * DP * 2);
  };
  auto value = [&](int buf, int kg, int d) {
    const uint8_t* const at = sv(buf) + (v_at ^ (d << 6)) + kg * 16 * DP * 2;
    const uint8_t* const at8 = sv(buf) + (v_at ^ (d << 6) ^ (DP == 128 ? 16 : 0)) + (kg * 16 + 8) * DP * 2;
    const u32x2 lo = ds_read_tr16(at), hi = ds_read_tr16(at8);
    return u32x4{lo.x, lo.y, hi.x, hi.y};
  };
  auto scores = [&](int buf) __attribute__((always_inline)) {
    s[0] = s[1] = f32x16{};
#pragma unroll
    for (int t = 0; t < KS; ++t)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) s[kb] = mfma32(key(buf, kb, t), qf[t], s[kb]);
  };
  auto values = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int kg = 0; kg < 4; ++kg)
#pragma unroll
      for (int d = 0; d < DB; ++d) o[d] = mfma32(value(buf, kg, d), pf[kg], o[d]);
  };
  // Values of step j that are not finite, where the mask cuts the step: set to
  // zero in LDS, by each wave in the part that it loaded, and noted ..
  auto clear_values = [&](int j, int buf) __attribute__((always_inline)) {
    uint32_t odd = 0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      u32x4* const at = reinterpret_cast<u32x4*>(sv(buf) + (wave * kLoads + i) * 1024 + lane * 16);
      u32x4 v = *at;
      const uint32_t bad = clear_nonfinite(v);
      if (bad != 0) *at = v;
      odd |= bad;
    }
    if (odd != 0) s_odd[buf % 3] = j + 1;
  };
  // .. and, as they are, added to the rows that see them
  auto add_nonfinite = [&](int j, int buf) {
    if (PAGED || s_odd[buf % 3] != j + 1) return;
    const int j0 = base + j * kBN;
    for (int jj = 0; jj < kBN && j0 + jj < seen; ++jj) {
      const uint16_t* const v = a.v + static_cast<int64_t>(rt.s0 + j0 + jj) * a.v_ld + kvh * D;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int c = 32 * d + acc_row(i, h);
          const float y = c < D ? bf16_to_f32(v[c]) : 0.0f;
          if ((__float_as_uint(y) & 0x7F800000u) == 0x7F800000u) o[d][i] += y;
        }
    }
  };
  auto softmax = [&](int j, int buf, uint32_t there) __attribute__((always_inline)) {
    const int j0 = base + j * kBN;
    const bool masked = j0 + kBN > w_all || there != 0xFu;
    const float* const sks = s_scale + (PAGED ? buf % 3 * 2 * kBN : 0);
    if constexpr (PAGED) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const f32x4 ks = *reinterpret_cast<const f32x4*>(sks + kb * 32 + acc_row(i, h));
#pragma unroll
          for (int e = 0; e < 4; ++e) s[kb][i + e] *= ks[e];
        }
    }
    if (masked) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int r = kb * 32 + acc_row(i, h);
          if (j0 + r >= seen || (PAGED && (there >> (2 * kb + (i >> 3)) & 1) == 0)) s[kb][i] = kMinusInf;
        }
    }
    float top = fmaxf(s[0][0], s[1][0]);
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(fmaxf(top, s[0][i]), s[1][i]);
    top = max_halves(top) * a.c2;
    if (__ballot(top > m + kRaise) != 0) {
      const float m_new = top > m + kRaise ? top : m;
      const float alpha = m_new == kMinusInf ? 1.0f : __builtin_amdgcn_exp2f(m - m_new);
      m = m_new;
      l *= alpha;
#pragma unroll
      for (int d = 0; d < DB; ++d) o[d] *= alpha;
    }
    const float shift = m == kMinusInf ? 0.0f : m;
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        f32x4 vs;
        if constexpr (PAGED) vs = *reinterpret_cast<const f32x4*>(sks + kBN + kb * 32 + acc_row(i, h));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float t = s[kb][i + e];
          const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(t, a.c2, -shift));
          sum[e & 1] += p;
          // (a masked value's scale may be anything)
          s[kb][i + e] = !PAGED ? p : masked && t == kMinusInf ? 0.0f : p * vs[e];
        }
      }
    }
    l += sum[0] + sum[1];
#pragma unroll
    for (int kg = 0; kg < 4; ++kg) pf[kg] = pack_operand(s[kg >> 1], kg & 1);
  };

  const bool second = W == 8 && wave >= 4;
  int page_k = -1, page_v = -1;  // pages of steps j + 4 and j + 3
  if (steps > 0) {
    if constexpr (PAGED) {
      const int q0 = pages_of(0), q1 = pages_of(1), q2 = pages_of(2), q3 = pages_of(3);
      fetch(0, q0, false);
      fetch(0, q0, true);
      put(0, false);
      put(0, true);
      fetch(1, q1, false);
      fetch(1, q1, true);
      put(1, false);
      put(1, true);
      fetch(2, q2, false);
      put(2, false);
      fetch(3, q3, false);
      fetch(2, q2, true);
      queue = blocks(q0) | blocks(q1) << 4 | blocks(q2) << 8 | blocks(q3) << 12;
      page_v = q3;
      page_k = pages_of(4);
      barrier<-1, 0>();
    } else {
      load_packed(0, 0, false);
      load_packed(0, 0, true);
      load_packed(1, 1, false);
      load_packed(1, 1, true);
      load_packed(2, 2, false);
      barrier<0, 0>();
    }
    // steps of which every row of the tile sees all keys, in whole turns of the
    // buffers, and with the next step to come
    const int sees_all = inside(first + tok0 + 1) - base;
    const int whole = sees_all >= 2 * kBN ? (sees_all / kBN - 1) / 3 * 3 : 0;
    if (!PAGED && whole == 0) {
      clear_values(0, 0);
      barrier<-1, 0>();
    }
    if (base < w_end) {
      scores(0);
      softmax(0, 0, queue & 0xFu);
    }
    if (second) barrier<-1, -1>();
    // the end of step j's matrix phase, and the softmax phase
    auto rest = [&](int j, int buf, bool cut) __attribute__((always_inline)) {
      if constexpr (W == 8) __builtin_amdgcn_s_setprio(0);
      __builtin_amdgcn_sched_barrier(0);
      if (!PAGED && cut) {
        __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
        clear_values(j + 1, buf + 1);
        barrier<-1, 0>();
      } else {
        barrier<PAGED ? -1 : 0, -1>();
      }
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (PAGED) {
        put(buf, false);
        put(buf + 2, true);
        queue = queue >> 4 | blocks(page_k) << 12;
        fetch(j + 4, page_k, false);
        fetch(j + 3, page_v, true);
        page_v = page_k;
        page_k = pages_of(j + 5);
      } else {
        load_packed(j + 3, buf, false);
        load_packed(j + 2, buf + 2, true);
      }
      if (base + (j + 1) * kBN < w_end) softmax(j + 1, buf + 1, queue & 0xFu);
      __builtin_amdgcn_sched_barrier(0);
      barrier<-1, PAGED ? 0 : -1>();
      __builtin_amdgcn_sched_barrier(0);
    };
    auto whole_step = [&](int j, int buf, bool last) __attribute__((always_inline)) {
      if constexpr (W == 8) __builtin_amdgcn_s_setprio(1);
      if (w_end > base) {
        scores(buf + 1);
        values(buf);
        // reads some instructions ahead of their use
        __builtin_amdgcn_sched_group_barrier(0x100, 6, 0);
#pragma unroll
        for (int i = 0; i < 2 * KS - 6; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
#pragma unroll
        for (int i = 0; i < 6; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        }
#pragma unroll
        for (int i = 0; i < 4 * DB; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        }
      }
      rest(j, buf, last);
    };
    auto cut_step = [&](int j, int buf) __attribute__((always_inline)) {
      if constexpr (W == 8) __builtin_amdgcn_s_setprio(1);
      if (base + (j + 1) * kBN < w_end) scores(buf + 1);
      if (base + j * kBN < w_end) {
        values(buf);
        add_nonfinite(j, buf);
      }
      rest(j, buf, true);
    };
    int j = 0;
    for (; j < whole; j += 3) {
      whole_step(j, 0, false);
      whole_step(j + 1, 1, false);
      whole_step(j + 2, 2, j + 3 == whole);
    }
    for (; j < steps; j += 3) {  // (steps past the last compute nothing)
      cut_step(j, 0);
      cut_step(j + 1, 1);
      cut_step(j + 2, 2);
    }
    if (!second && W == 8) barrier<-1, -1>();
    // (loads on their way into LDS end before the workgroup does)
    __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }
  l += swap_halves(l);
  if (!in) return;
  const int64_t row = static_cast<int64_t>(rt.s0 + tok) * a.Hq + hq;
  if (PAGED && a.splits > 1) {
    const int64_t part = static_cast<int64_t>(share) * a.s.T * a.Hq + row;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int c = 32 * d + acc_row(i, h);
        if (c < D) *reinterpret_cast<f32x4*>(a.part + part * D + c) = f32x4{o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]};
      }
    if (h == 0) *reinterpret_cast<f32x2*>(a.ml + 2 * part) = f32x2{m, l};
    return;
  }
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

template <int DP, bool PAGED, int W>
hipError_t launch(const AttnArgs& a, hipStream_t stream) {
  const int64_t tiles = static_cast<int64_t>(a.s.T) * a.g / (32 * W) + a.s.B;
  hipLaunchKernelGGL((k_attn<DP, PAGED, W>), dim3(static_cast<uint32_t>(tiles * (PAGED ? a.splits : 1) * a.Hkv)), dim3(64 * W), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn(const AttnArgs& a, bool paged, hipStream_t stream) {
  if (a.D <= 64) return paged ? launch<64, true, 8>(a, stream) : launch<64, false, 8>(a, stream);
  return paged ? launch<128, true, 8>(a, stream) : launch<128, false, 8>(a, stream);
}

}  // namespace qlin
