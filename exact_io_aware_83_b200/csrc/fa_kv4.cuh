// fa_kv4.cuh - a key/value cache held in 4 bits: writing new tokens into it, reading them
// back, and attention of a few new query rows over it, on sm_100a.
//
// Format (per batch entry and K/V head, one row per token; d channels in d / 32 groups):
//   codes  : d / 2 bytes, 32-bit words of 8 channels, the first channel in the lowest four
//            bits.  V's words follow the channels; K's word of channels 32 i + 8 c .. + 7
//            lies at place c * (d / 32) + i, so that the four lanes that share a key in the
//            score product each read one contiguous piece holding a word of every group.
//   params : two fp16 numbers per group, a step s and a minimum m.  V: (s, m) of group 0,
//            (s, m) of group 1, ...;  K: s of every group, then m of every group.
// A channel stands for m + n s, n its code.  For the 32 values x of a group (clamped to
// +-57344, so that m + 15 s stays inside fp16):
//   m = the largest fp16 number <= min x,   s = the smallest one with m + 15 s >= max x,
//   n = the number of k in 0..14 with x >= m + (k + 1/2) s   (0 where s = 0).
// So n is the nearest code, the upper one at a tie, and the stored bits depend on no rounding:
// every comparison is made exactly in fp32, in one of two forms.
//   x >= fl(m + h s), h = k + 1/2 or 15, where |m| >= 2^-8 s or m = 0: s has 11 significant
//     bits and s >= 2^-12 |m| (bf16 values that are not all equal span at least 2^-8 of their
//     largest magnitude), so the sum fits into 24 bits.
//   fl(x - h s) >= m, where 0 < |m| < 2^-8 s: a difference that is near m is a multiple of
//     2^-9 of s's unit and below s, hence exact; one that is not near m rounds to the same
//     side of it.
// A group that holds a NaN or an infinity gets m = NaN and reads back as NaN.
#pragma once

#include <cuda_fp16.h>

#include "fa_common.cuh"

namespace fa {

constexpr int kKV4Group = 32;           // channels per (s, m)
constexpr float kKV4Clamp = 57344.f;    // 1.75 * 2^15
constexpr int kKV4CapMultiple = 64;     // tokens of a cache: a multiple of this

struct KV4Params {
  uint8_t *kc, *vc;       // [B, Hkv, cap, d / 2]
  __half *kp, *vp;        // [B, Hkv, cap, 2 d / 32]
  __nv_bfloat16 *k, *v;   // [B, Hkv, n, d]: read by the write kernel, written by the read kernel
  const int *start;       // [B] first position of each batch entry (nullptr: 0)
  const int *counts;      // [B] tokens of each batch entry (nullptr: n), write only
  int B, Hkv, n, cap;
};

// One lane's eight bf16 values as fp32.
__device__ __forceinline__ void unpack_bf16x8(const uint4 &w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

// Position of token i of batch entry b, or -1 when it is not to be touched; positions
// outside the cache are reported.
__device__ __forceinline__ int kv4_position(const KV4Params &p, int b, int i) {
  if (p.counts && i >= p.counts[b]) return -1;
  const long long pos = static_cast<long long>(p.start ? p.start[b] : 0) + i;
  if (pos < 0 || pos >= p.cap) {
    report_bad_seqlens();
    return -1;
  }
  return static_cast<int>(pos);
}

// Which of the two exact forms of a comparison with m + h s holds (see the format).
__device__ __forceinline__ bool kv4_small_min(float m, float s) {
  return m != 0.f && fabsf(m) < s * 0.00390625f;
}

// Quantises the 32 values held by four lanes (8 each, lane c = lane % 4) and returns this
// lane's word of codes, and s, m.
__device__ __forceinline__ uint32_t kv4_quantise(float (&x)[8], __half &s_out, __half &m_out) {
  float lo = x[0], hi = x[0], bad = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
    bad = fmaf(x[i], 0.f, bad);  // NaN as soon as a value is not finite
  }
#pragma unroll
  for (int o = 1; o < 4; o *= 2) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    bad += __shfl_xor_sync(0xffffffffu, bad, o);
  }
  if (bad != 0.f) {  // NaN
    s_out = __ushort_as_half(0);
    m_out = __ushort_as_half(0x7FFF);
    return 0u;
  }
  lo = fminf(fmaxf(lo, -kKV4Clamp), kKV4Clamp);
  hi = fminf(fmaxf(hi, -kKV4Clamp), kKV4Clamp);
  const __half mh = __float2half_rd(lo);
  const float m = __half2float(mh);
  // The smallest fp16 s with m + 15 s >= hi: rounded up from the approximate quotient, which
  // is at most one step off either way.
  const unsigned short sb = __half_as_ushort(__float2half_ru((hi - m) * (1.f / 15.f)));
  auto reaches = [&](unsigned short bits) {
    const float t = __half2float(__ushort_as_half(bits));
    return kv4_small_min(m, t) ? fmaf(-15.f, t, hi) <= m : fmaf(15.f, t, m) >= hi;
  };
  const unsigned short sb1 = (sb > 0 && reaches(sb - 1)) ? sb - 1 : (reaches(sb) ? sb : sb + 1);
  const __half sh = __ushort_as_half(sb1);
  const float s = __half2float(sh);
  s_out = sh;
  m_out = mh;
  if (s == 0.f) return 0u;
  // t = (x - m) / s + 1/2 - 2^-8 in fp32 lies below the true quotient + 1/2 and above it
  // - 2^-7 (|m| / s <= 2^12, so rounding moves it by less than 2^-10), so its floor is n or
  // n - 1; one exact comparison with the border above it decides.
  const float inv = 1.f / s, c = fmaf(-m, inv, 0.5f - 0.00390625f);
  const float mh2 = fmaf(0.5f, s, m);  // border above code 0
  uint32_t word = 0;
  const bool small = kv4_small_min(m, s);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = fminf(fmaxf(x[i], -kKV4Clamp), kKV4Clamp);
    const float n0 = floorf(fmaf(v, inv, c));
    const bool above = small ? fmaf(-(n0 + 0.5f), s, v) >= m : v >= fmaf(n0, s, mh2);
    const float n1 = above ? n0 + 1.f : n0;
    word |= static_cast<uint32_t>(static_cast<int>(n1)) << (4 * i);
  }
  return word;
}

// Writes new tokens: four lanes per (token, group), 8 channels a lane, K then V.  Bound:
// HBM, 2 d bytes read and 5 d / 8 written per token for each of K and V.
template <int D>
__global__ void __launch_bounds__(256) fa_kv4_write_kernel(const KV4Params p) {
  constexpr int G = D / kKV4Group, T = D / 8;  // threads per token
  const long long rows = static_cast<long long>(p.B) * p.Hkv * p.n;
  const long long gid = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  long long row = gid / T;
  const int t = static_cast<int>(gid % T);  // word of the row: channels 8 t .. 8 t + 7
  const bool is_v = row >= rows;
  if (is_v) row -= rows;
  const bool live = row < rows;  // whole groups of T >= 8 threads
  int pos = -1;
  long long bh = 0;
  if (live) {
    bh = row / p.n;
    pos = kv4_position(p, static_cast<int>(bh / p.Hkv), static_cast<int>(row % p.n));
  }
  uint4 raw = make_uint4(0, 0, 0, 0);
  if (pos >= 0) raw = *reinterpret_cast<const uint4 *>((is_v ? p.v : p.k) + row * D + t * 8);
  float x[8];
  unpack_bf16x8(raw, x);
  __half s, m;
  const uint32_t word = kv4_quantise(x, s, m);
  if (pos < 0) return;
  const int gamma = t / 4, c = t % 4;
  const long long crow = bh * p.cap + pos;
  const int place = is_v ? t : c * G + gamma;
  reinterpret_cast<uint32_t *>((is_v ? p.vc : p.kc) + crow * (D / 2))[place] = word;
  if (c == 0) {
    __half *par = (is_v ? p.vp : p.kp) + crow * (2 * G);
    par[is_v ? 2 * gamma : gamma] = s;
    par[is_v ? 2 * gamma + 1 : G + gamma] = m;
  }
}

// Reads n tokens back as bf16: value = bf16(m + n s), the sum exact in fp32.
template <int D>
__global__ void __launch_bounds__(256) fa_kv4_read_kernel(const KV4Params p) {
  constexpr int G = D / kKV4Group, T = D / 8;
  const long long rows = static_cast<long long>(p.B) * p.Hkv * p.n;
  const long long gid = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  long long row = gid / T;
  const int t = static_cast<int>(gid % T);
  const bool is_v = row >= rows;
  if (is_v) row -= rows;
  if (row >= rows) return;
  const long long bh = row / p.n;
  const int pos = kv4_position(p, static_cast<int>(bh / p.Hkv), static_cast<int>(row % p.n));
  if (pos < 0) return;
  const int gamma = t / 4, c = t % 4;
  const long long crow = bh * p.cap + pos;
  const int place = is_v ? t : c * G + gamma;
  const uint32_t word = reinterpret_cast<const uint32_t *>((is_v ? p.vc : p.kc) + crow * (D / 2))[place];
  const __half *par = (is_v ? p.vp : p.kp) + crow * (2 * G);
  const float s = __half2float(par[is_v ? 2 * gamma : gamma]);
  const float m = __half2float(par[is_v ? 2 * gamma + 1 : G + gamma]);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = fmaf(static_cast<float>((word >> (8 * i)) & 15u), s, m);
    const float b = fmaf(static_cast<float>((word >> (8 * i + 4)) & 15u), s, m);
    w[i] = pack_bf16x2(a, b);
  }
  *reinterpret_cast<uint4 *>((is_v ? p.v : p.k) + row * D + t * 8) = make_uint4(w[0], w[1], w[2], w[3]);
}

// ============================================================================ attention
//
// fa_decode_kv4: for batch b, query head h and new row t < Nq, over the keys j < len
// (causal: j <= len - Nq + t),
//   x_j = scale q . k_j,  y_j = cap tanh(x_j / cap) (or x_j),  s_j = y_j - slope_h |len - Nq + t - j|,
//   O = sum_j softmax_j(s) v_j,  LSE = ln sum_j exp(s_j).
// The R = (Hq / Hkv) Nq rows that share a K/V head are processed together, 8 NT at a time.
//
//  * q . k_j = sum_i (s_ji sum_{c in group i} q_c n_jc + m_ji sum_{c in group i} q_c): the
//    codes go into the matrix product as whole numbers, exactly, and s, m are applied to the
//    fp32 sums.  q is scaled by a power of two per row and converted to fp16 (8 significant
//    bits of 11: exact but for entries below 2^-21 of the row's largest).
//  * v_jc = m + n s in fp16 (one rounding, 2^-11 relative), p_j in fp16 (p_j <= 2^8).
//  * The matrix products are warp-level m16n8k16: S^T = K Q^T with 16 keys as rows, O^T = V^T
//    P^T with 16 channels as rows.  The codes are unpacked from registers straight into the
//    operand layout (two lanes of work per instruction), which no shared-memory operand could
//    take without writing the widened values out and reading them back: 4 bytes a value
//    through shared memory against half a byte from HBM.
//  * Bound: HBM, 5 d / 4 bytes per key (K and V with their params).
struct KV4DecodeParams {
  const __nv_bfloat16 *q;  // [B, Hq, Nq, D]
  const uint8_t *kc, *vc;
  const __half *kp, *vp;
  const int *lens;         // [B] (nullptr: all `cap`), clamped to [0, cap]
  const float *slopes;     // [Hq] or nullptr
  __nv_bfloat16 *o;        // splits == 1
  float *lse;
  float *o_part;           // [splits, B * Hq * Nq, D] fp32 (splits > 1)
  float *lse_part;
  int B, Hkv, Nq, R, cap;
  int splits, chunk;       // split s covers keys [s * chunk, (s + 1) * chunk)
  int causal;
  float scale, sl2;        // scale, scale * log2(e)
  float softcap;           // 0: none
};

constexpr int kKV4Warps = 8;
constexpr int kKV4Keys = 32;  // keys per warp and iteration

// The score in log2 units from x = scale q . k: capped, y = cap tanh(x / cap) log2(e).
// tanh(u) = sign(u) (1 - w) / (1 + w), w = exp(-2 |u|): no cancellation that matters, the
// absolute error stays below 2^-22 for every u.
__device__ __forceinline__ float softcap_log2(float x, float inv_cap2, float cap_log2) {
  // inv_cap2 = 2 log2(e) / cap
  const float w = ex2_approx(-fabsf(x) * inv_cap2);
  return copysignf(cap_log2 * __fdividef(1.f - w, 1.f + w), x);
}

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t h2_u32(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 u32_h2(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }

// The codes at bits 4 i .. 4 i + 3 of both halves of w, i = 0 (LOW) or 1, as fp16 whole
// numbers: or-ed into the mantissa of 1024 (i = 0) or of 64 (i = 1, unit 2^-4), which is
// then subtracted (exactly).
template <int I>
__device__ __forceinline__ __half2 codes_h2(uint32_t w) {
  constexpr uint32_t mask = I ? 0x00F000F0u : 0x000F000Fu;
  constexpr uint32_t magic = I ? 0x54005400u : 0x64006400u;
  return __hsub2(u32_h2((w & mask) | magic), u32_h2(magic));
}

template <int D>
struct KV4Layout {
  static constexpr int G = D / 32;    // groups
  static constexpr int KW = G;        // K words per lane and key
  static constexpr int VW = D / 64;   // V words per lane and key
  static constexpr int MT = VW * 4;   // 16-channel tiles of O^T
};

// Key of row r of a 16-key step: the rows 2c, 2c+1, 2c+8, 2c+9 of lane group c of the second
// product are the keys c, c+4, c+8, c+12, so that its four loads cover consecutive tokens.
__device__ __forceinline__ int kv4_key_of_row(int r) { return ((r & 7) >> 1) + 4 * (r & 1) + (r & 8); }

template <int D, int NT>
__global__ void __launch_bounds__(kKV4Warps * 32) fa_decode_kv4_kernel(const KV4DecodeParams p) {
  using L = KV4Layout<D>;
  constexpr int G = L::G, KW = L::KW, VW = L::VW, MT = L::MT;
  constexpr int ROWS = 8 * NT;
  __shared__ float sm_o[kKV4Warps][ROWS][D / 8];  // combined in 8 passes over the channels
  __shared__ float sm_m[kKV4Warps][ROWS], sm_l[kKV4Warps][ROWS];

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, c = lane % 4;
  const int split = blockIdx.x, bh = blockIdx.y, r0 = blockIdx.z * ROWS;
  const int b = bh / p.Hkv, kvh = bh % p.Hkv;
  const int grp = p.R / p.Nq;  // query heads per K/V head
  int len = p.lens ? p.lens[b] : p.cap;
  len = len < 0 ? 0 : (len > p.cap ? p.cap : len);
  const int k_begin = split * p.chunk;
  const int k_end = min(k_begin + p.chunk, len);
  const long long rows_total = static_cast<long long>(p.B) * p.Hkv * p.R;
  const long long row0 = static_cast<long long>(bh) * p.R + r0;
  const int pos0 = len - p.Nq;

  // ---- Q fragments: row g of each 8-row tile, this lane's 8 channels of every group, scaled
  uint32_t qf[NT][G][4];         // [2 t + e]: channels (2t + e, 2t + e + 4) of the word
  float fac[NT][2];              // rows 2c, 2c+1: scale (or scale log2 e without a cap) / row scaling
  float qsum[NT][G][2];          // rows 2c, 2c+1: sum of the scaled q over each group
  float slope2[NT][2];
  int rpos[NT][2];               // position of the row
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = nt * 8 + g;
    const bool rv = r0 + r < p.R;
    float x[G][8];
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < G; ++i) {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (rv) w = *reinterpret_cast<const uint4 *>(p.q + (row0 + r) * D + 32 * i + 8 * c);
      unpack_bf16x8(w, x[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[i][e]));
    }
#pragma unroll
    for (int o = 1; o < 4; o *= 2) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    // largest magnitude into [128, 256)
    const int ex = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -100);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + 7 - ex) << 23);
    const float down = __uint_as_float(static_cast<uint32_t>(127 - 7 + ex) << 23);
#pragma unroll
    for (int i = 0; i < G; ++i) {
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[i][e] *= up;
        s += x[i][e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) qf[nt][i][e] = pack_f16x2(x[i][e], x[i][e + 4]);
#pragma unroll
      for (int o = 1; o < 4; o *= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
      qsum[nt][i][0] = __shfl_sync(0xffffffffu, s, 8 * c);
      qsum[nt][i][1] = __shfl_sync(0xffffffffu, s, 8 * c + 4);
    }
    const float f = (p.softcap > 0.f ? p.scale : p.sl2) * down;
    fac[nt][0] = __shfl_sync(0xffffffffu, f, 8 * c);
    fac[nt][1] = __shfl_sync(0xffffffffu, f, 8 * c + 4);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rr = r0 + nt * 8 + 2 * c + e;
      const int h = kvh * grp + min(rr / p.Nq, grp - 1);
      slope2[nt][e] = p.slopes ? p.slopes[h] * 1.4426950408889634f : 0.f;
      rpos[nt][e] = pos0 + rr % p.Nq;
    }
  }
  const float inv_cap2 = p.softcap > 0.f ? 2.f * 1.4426950408889634f / p.softcap : 0.f;
  const float cap_log2 = p.softcap * 1.4426950408889634f;

  float acc[MT][NT][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][nt][e] = 0.f;
  float m_run[NT][2], l_run[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m_run[nt][0] = m_run[nt][1] = -INFINITY;
    l_run[nt][0] = l_run[nt][1] = 0.f;
  }

  const long long crow0 = static_cast<long long>(bh) * p.cap;
  const int ka = kv4_key_of_row(g);  // key of row g; row g + 8 is ka + 8
  const int vgroup = (g * VW) / 4;   // group of this lane's V channels

  for (int kb = k_begin + warp * kKV4Keys; kb < k_end; kb += kKV4Warps * kKV4Keys) {
    float y[2][NT][4];  // [step][tile][key A: rows 2c, 2c+1; key B: rows 2c, 2c+1]
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      const int key0 = kb + 16 * st;
      const long long krow = crow0 + key0 + ka;
      uint32_t w[2][KW];
      __half sc[2][G], mn[2][G];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t *src = reinterpret_cast<const uint32_t *>(p.kc + (krow + 8 * e) * (D / 2)) + c * KW;
        if constexpr (KW == 2) {
          *reinterpret_cast<uint2 *>(w[e]) = *reinterpret_cast<const uint2 *>(src);
        } else {
#pragma unroll
          for (int i = 0; i < KW; i += 4) *reinterpret_cast<uint4 *>(w[e] + i) = *reinterpret_cast<const uint4 *>(src + i);
        }
        const __half *par = p.kp + (krow + 8 * e) * (2 * G);
#pragma unroll
        for (int i = 0; i < G; ++i) {
          sc[e][i] = par[i];
          mn[e][i] = par[G + i];
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[st][nt][e] = 0.f;
#pragma unroll
      for (int i = 0; i < G; ++i) {
        float part[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) part[nt][e] = 0.f;
        uint32_t a[2][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          a[e][0] = h2_u32(codes_h2<0>(w[e][i]));
          a[e][1] = h2_u32(codes_h2<1>(w[e][i]));
          a[e][2] = h2_u32(codes_h2<0>(w[e][i] >> 8));
          a[e][3] = h2_u32(codes_h2<1>(w[e][i] >> 8));
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16_16816(part[nt], a[0][0], a[1][0], a[0][1], a[1][1], qf[nt][i][0], qf[nt][i][1]);
          mma_f16_16816(part[nt], a[0][2], a[1][2], a[0][3], a[1][3], qf[nt][i][2], qf[nt][i][3]);
        }
        const float sA = __half2float(sc[0][i]), sB = __half2float(sc[1][i]);
        const float mA = __half2float(mn[0][i]), mB = __half2float(mn[1][i]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          y[st][nt][0] = fmaf(sA, part[nt][0], fmaf(mA, qsum[nt][i][0], y[st][nt][0]));
          y[st][nt][1] = fmaf(sA, part[nt][1], fmaf(mA, qsum[nt][i][1], y[st][nt][1]));
          y[st][nt][2] = fmaf(sB, part[nt][2], fmaf(mB, qsum[nt][i][0], y[st][nt][2]));
          y[st][nt][3] = fmaf(sB, part[nt][3], fmaf(mB, qsum[nt][i][1], y[st][nt][3]));
        }
      }
      // ---- cap, bias, mask: the scores in log2 units
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = key0 + ka + 8 * (e / 2);
          float v = y[st][nt][e] * fac[nt][e & 1];
          if (p.softcap > 0.f) v = softcap_log2(v, inv_cap2, cap_log2);
          if (p.slopes) v = fmaf(-slope2[nt][e & 1], fabsf(static_cast<float>(rpos[nt][e & 1] - key)), v);
          if (key >= k_end || (p.causal && key > rpos[nt][e & 1])) v = -INFINITY;
          y[st][nt][e] = v;
        }
    }
    // ---- running maximum: moved (for the whole warp) only when a row's rises by more than 2^8
    bool up = false;
    float mx[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[nt][e] = fmaxf(fmaxf(y[0][nt][e], y[0][nt][e + 2]), fmaxf(y[1][nt][e], y[1][nt][e + 2]));
        up |= mx[nt][e] > m_run[nt][e] + 8.f;
      }
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float alpha[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = mx[nt][e];
#pragma unroll
          for (int o = 4; o < 32; o *= 2) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
          const float mn = fmaxf(m_run[nt][e], v);
          alpha[e] = mn == m_run[nt][e] ? 1.f : ex2_approx(m_run[nt][e] - mn);  // 0 at the first keys
          m_run[nt][e] = mn;
          l_run[nt][e] *= alpha[e];
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][nt][e] *= alpha[e & 1];
      }
    }
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      uint32_t pb[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float pr[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float mu = m_run[nt][e & 1] == -INFINITY ? 0.f : m_run[nt][e & 1];
          pr[e] = ex2_approx(y[st][nt][e] - mu);
          l_run[nt][e & 1] += pr[e];
        }
        pb[nt][0] = movmatrix_trans(pack_f16x2(pr[0], pr[1]));
        pb[nt][1] = movmatrix_trans(pack_f16x2(pr[2], pr[3]));
      }
      const int key0 = kb + 16 * st;
      uint32_t wv[4][VW], sm[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = key0 + c + 4 * e;
        const uint32_t *src = reinterpret_cast<const uint32_t *>(p.vc + (crow0 + key) * (D / 2)) + g * VW;
        if constexpr (VW == 1) wv[e][0] = *src;
        else if constexpr (VW == 2) *reinterpret_cast<uint2 *>(wv[e]) = *reinterpret_cast<const uint2 *>(src);
        else *reinterpret_cast<uint4 *>(wv[e]) = *reinterpret_cast<const uint4 *>(src);
        sm[e] = reinterpret_cast<const uint32_t *>(p.vp + (crow0 + key) * (2 * G))[vgroup];
        if (key >= k_end) sm[e] = 0u;  // rows behind the last key hold anything; 0 * NaN would spread
      }
      __half2 sp[2], mp[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sp[e] = u32_h2(__byte_perm(sm[2 * e], sm[2 * e + 1], 0x5410));
        mp[e] = u32_h2(__byte_perm(sm[2 * e], sm[2 * e + 1], 0x7632));
      }
#pragma unroll
      for (int w = 0; w < VW; ++w)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t x[2];  // key pairs; the four codes of two bytes in each half
#pragma unroll
          for (int e = 0; e < 2; ++e) x[e] = __byte_perm(wv[2 * e][w], wv[2 * e + 1][w], half ? 0x7632 : 0x5410);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const uint32_t x0 = t ? x[0] >> 8 : x[0], x1 = t ? x[1] >> 8 : x[1];
            const uint32_t a0 = h2_u32(__hfma2(codes_h2<0>(x0), sp[0], mp[0]));
            const uint32_t a1 = h2_u32(__hfma2(codes_h2<1>(x0), sp[0], mp[0]));
            const uint32_t a2 = h2_u32(__hfma2(codes_h2<0>(x1), sp[1], mp[1]));
            const uint32_t a3 = h2_u32(__hfma2(codes_h2<1>(x1), sp[1], mp[1]));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16_16816(acc[w * 4 + half * 2 + t][nt], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
          }
        }
    }
  }

  // ---- combine the warps: m, l of every row, then O an eighth of the channels at a time
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int o = 4; o < 32; o *= 2) l_run[nt][e] += __shfl_xor_sync(0xffffffffu, l_run[nt][e], o);
      if (g == 0) {
        sm_m[warp][nt * 8 + 2 * c + e] = m_run[nt][e];
        sm_l[warp][nt * 8 + 2 * c + e] = l_run[nt][e];
      }
    }
  // Accumulator tile w * 4 + q of lane (g, c): channels 8 (g VW + w) + 2 q (+ 1), rows 2c, 2c+1.
#pragma unroll 1
  for (int pass = 0; pass < 8; ++pass) {
    __syncthreads();
    if (g == pass) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) sm_o[warp][nt * 8 + 2 * c + (e & 1)][2 * i + e / 2] = acc[i][nt][e];
    }
    __syncthreads();
    for (int idx = threadIdx.x; idx < ROWS * (D / 8); idx += blockDim.x) {
      const int r = idx / (D / 8), ch = idx % (D / 8);
      if (r0 + r >= p.R) continue;
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kKV4Warps; ++w) m = fmaxf(m, sm_m[w][r]);
      const float mu = m == -INFINITY ? 0.f : m;
      float l = 0.f, o = 0.f;
#pragma unroll
      for (int w = 0; w < kKV4Warps; ++w) {
        const float f = ex2_approx(sm_m[w][r] - mu);
        l = fmaf(f, sm_l[w][r], l);
        o = fmaf(f, sm_o[w][r][ch], o);
      }
      o = l == 0.f ? 0.f : o / l;  // a row without keys: 0; NaN stays NaN
      const float lse = l == 0.f ? -INFINITY : (mu + log2f(l)) * kLn2;
      const long long row = row0 + r;
      if (p.splits == 1) {
        p.o[row * D + pass * (D / 8) + ch] = __float2bfloat16_rn(o);
        if (pass == 0 && ch == 0) p.lse[row] = lse;
      } else {
        const long long prow = static_cast<long long>(split) * rows_total + row;
        p.o_part[prow * D + pass * (D / 8) + ch] = o;
        if (pass == 0 && ch == 0) p.lse_part[prow] = lse;
      }
    }
  }
}

}  // namespace fa
