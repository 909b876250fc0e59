// fa_score.cuh - scores that are changed before the softmax: capped by a tanh, lowered with
// the distance between query and key, or hidden outside a key range of the query's own.
//
// For query i and key j of head h, with x = scale q_i . k_j:
//   y = cap tanh(x / cap)   (cap = 0: y = x),      s_ij = y - slope_h |i - j|,
// and key j is visible to query i iff lo_i <= j < hi_i (and j <= i when causal).  Documents
// packed into one row, visible prefixes, padding and their combinations are such ranges.
// The kernels work in units of log2: s_ij log2(e).
//
// The gradient: with t = tanh(x / cap), d s_ij / d x = 1 - t^2; the bias is a constant.
//
// tanh.  MUFU.TANH is off by 2^-11 of its value: at cap = 50 a score of 20 would be off by
// 0.01 and its probability by 1%.  Instead, chosen per warp and block by the largest
// |u| = |x| / cap in it (the coefficients are this library's own minimax fits):
//  * t = u P(u^2), P of degree 3 up to |u| = 0.5 (relative error 5.4e-7) or of degree 5 up to 1
//    (5.9e-7).  In blocks without hidden keys and without a bias, scale, cap and log2(e) are
//    folded into the coefficients and the softmax's offset into the last product, so that a
//    capped pair of scores costs five or seven packed operations where a plain one costs one;
//  * beyond: t = sign(u) (1 - w) / (1 + w), w = 2^(-2 log2(e) |u|): two MUFU operations.
//    1 - t^2 is then 4 w / (1 + w)^2, which keeps its relative accuracy where t is near 1
//    (1 - t t would be all rounding there).  Near u = 0 the difference 1 - w cancels: t is off by
//    up to 2^-22 and the score by cap 2^-22, however small it is - 1.5e-5 at a cap of 64, less than
//    the products' own fp32 error, but 0.2 at 1e6.  So beyond a cap of 64 (kCapNear) each u up to
//    0.5 takes the polynomial of degree 3 instead: a relative error of 2^-20 or less for every u.
//    Up to 64 that is left out, by variants of the kernels that choose between the forms: taken
//    always it costs 7-13% of the saturated forward (cap 1, B = 2, Hq = 32, Hkv = 8, N = 4096,
//    d = 128: 655 against 740 us), and as a branch in one kernel 7%.  (One rational function for
//    every u, with one MUFU operation, measured 720.)
#pragma once

#include "fa_common.cuh"

namespace fa {

struct ScoreCfg {
  float cap_in;         // scale / cap (0: no cap)
  float cap_log2;       // cap * log2(e)
  // |q . k| up to which the folded polynomials of degree 3 and 5 hold (negative: not used, products
  // of 0 included), and their coefficients: score in log2 units = r (k[0] + k[1] r^2 + k[2] r^4 +
  // ...), r = q . k
  float raw3, raw5;
  float k3[4], k5[6];
  const float *slopes;  // [Hq] or nullptr
  const int2 *range;    // [B, N] (lo, hi) or nullptr
  int causal;
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTanhPolyMax = 1.f, kTanhPoly3Max = 0.5f;
constexpr float kCapNear = 64.f;
__host__ __device__ constexpr float tanh_coef(int i) {
  return i == 0 ? 0.9999994136f : i == 1 ? -0.3332904238f : i == 2 ? 0.1328143387f : i == 3 ? -0.05160567377f : i == 4 ? 0.01674311481f : -0.003067060224f;
}
__host__ __device__ constexpr float tanh3_coef(int i) {
  return i == 0 ? 0.9999994557708327f : i == 1 ? -0.33326317935183836f : i == 2 ? 0.13190296595162188f : -0.044402225913669886f;
}

template <int D>
struct Degree {
  static constexpr int value = D;
};
template <bool B>
struct Flag {
  static constexpr bool value = B;
};

// tanh of a pair, |u| <= kTanhPolyMax.
__device__ __forceinline__ uint64_t f2_tanh_poly(uint64_t u) {
  const uint64_t z = f2_mul(u, u);
  uint64_t q = f2_pack(tanh_coef(5), tanh_coef(5));
#pragma unroll
  for (int i = 4; i >= 0; --i) q = f2_fma(q, z, f2_pack(tanh_coef(i), tanh_coef(i)));
  return f2_mul(q, u);
}

// tanh of any u, and 1 - tanh^2.  FAR: accurate near u = 0 too, relative to tanh.
template <bool FAR>
__device__ __forceinline__ float tanh_any(float u, float &grad) {
  const float w = ex2_approx(fabsf(u) * (-2.f * kLog2e));
  const float r = __fdividef(1.f, 1.f + w);
  grad = 4.f * w * r * r;
  const float t = copysignf((1.f - w) * r, u);
  if constexpr (!FAR) return t;
  const float z = u * u;
  const float p = fmaf(fmaf(fmaf(tanh3_coef(3), z, tanh3_coef(2)), z, tanh3_coef(1)), z, tanh3_coef(0)) * u;
  return fabsf(u) <= kTanhPoly3Max ? p : t;
}

// P(r^2) of the folded polynomial of degree DEG for a pair of raw products r.
template <int DEG>
__device__ __forceinline__ uint64_t f2_cap_poly(uint64_t r, const ScoreCfg &c) {
  const uint64_t z = f2_mul(r, r);
  auto k = [&](int i) {
    const float v = DEG == 3 ? c.k3[i & 3] : c.k5[i];
    return f2_pack(v, v);
  };
  uint64_t q = k(DEG);
#pragma unroll
  for (int i = DEG - 1; i >= 0; --i) q = f2_fma(q, z, k(i));
  return q;
}
// The same for one product, operation by operation (so that the result has the same bits).
__device__ __forceinline__ float cap_poly(int deg, float r, const ScoreCfg &c) {
  const float z = r * r;
  if (deg == 3) return fmaf(fmaf(fmaf(c.k3[3], z, c.k3[2]), z, c.k3[1]), z, c.k3[0]);
  float q = c.k5[5];
#pragma unroll
  for (int i = 4; i >= 0; --i) q = fmaf(q, z, c.k5[i]);
  return q;
}
// The folded polynomial that holds for every product of the warp, |r| <= amax: 3, 5 or 0 (none).
__device__ __forceinline__ int cap_degree(float amax, const ScoreCfg &c) {
  if (__all_sync(0xffffffffu, amax <= c.raw3)) return 3;
  return __all_sync(0xffffffffu, amax <= c.raw5) ? 5 : 0;
}

// The visible keys of query row i (hi <= lo: none).
__device__ __forceinline__ void row_range(const ScoreCfg &c, int b, int i, int N, int &lo, int &hi) {
  lo = 0;
  hi = N;
  if (i >= N) {
    hi = 0;
    return;
  }
  if (c.range) {
    const int2 r = c.range[static_cast<size_t>(b) * N + i];
    lo = min(max(r.x, 0), N);  // both into 0 .. N: users of lo and hi subtract key positions
    hi = min(max(r.y, 0), N);
  }
  if (c.causal) hi = min(hi, i + 1);
}

// Smallest of N raw scores.
template <int N>
__device__ __forceinline__ float row_min(const uint32_t (&s)[N]) {
  float m0 = INFINITY, m1 = INFINITY;
#pragma unroll
  for (int c = 0; c < N; c += 4) {
    m0 = fmin3(m0, __uint_as_float(s[c + 0]), __uint_as_float(s[c + 1]));
    m1 = fmin3(m1, __uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]));
  }
  return fminf(m0, m1);
}

// P = 2^(score - m) of N raw products by the folded polynomial, packed to bf16 pairs and
// stored to TMEM at tP, and their fp32 sum (the capped counterpart of exp_block).
template <int N, int DEG>
__device__ __forceinline__ float exp_block_capped(const uint32_t (&s)[N], const ScoreCfg &cfg, float m, uint32_t tP) {
  const uint64_t negm2 = f2_pack(-m, -m);
  uint64_t l0 = 0, l1 = 0;  // packed (0.f, 0.f)
#pragma unroll
  for (int h = 0; h < N / 64; ++h) {
    uint32_t pk[32];
#pragma unroll
    for (int q = 0; q < 32; ++q) {
      const int pp = h * 32 + q;
      const uint64_t r = f2_pack(__uint_as_float(s[2 * pp]), __uint_as_float(s[2 * pp + 1]));
      float x0, x1;
      f2_unpack(f2_fma(r, f2_cap_poly<DEG>(r, cfg), negm2), x0, x1);
      const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
      pk[q] = pack_bf16x2(p0, p1);
      if (pp & 1)
        l1 = f2_add(l1, f2_pack(p0, p1));
      else
        l0 = f2_add(l0, f2_pack(p0, p1));
    }
    tmem_st_x32(tP + h * 32, pk);
  }
  float a, b;
  f2_unpack(f2_add(l0, l1), a, b);
  return a + b;
}

// Largest |s| of N raw scores.
template <int N>
__device__ __forceinline__ float row_absmax(const uint32_t (&s)[N]) {
  float m0 = 0.f, m1 = 0.f;
#pragma unroll
  for (int c = 0; c < N; c += 4) {
    m0 = fmax3(m0, fabsf(__uint_as_float(s[c + 0])), fabsf(__uint_as_float(s[c + 1])));
    m1 = fmax3(m1, fabsf(__uint_as_float(s[c + 2])), fabsf(__uint_as_float(s[c + 3])));
  }
  return fmaxf(m0, m1);
}

// Turns the raw products s[c] = q . k of one fixed index (row or key) `at` with N consecutive
// others `first` + c into scores in log2 units, in place.  `side`: -1 when every other index
// is <= at, +1 when every one is >= at, 0 otherwise (the same for the whole warp).  With GRAD
// and a cap, grad[c] = 1 - tanh^2.  FAR: the cap may lie beyond kCapNear.  POLY = false leaves the
// polynomial for all of them out.
template <int N, bool GRAD, bool FAR, bool POLY = true>
__device__ __forceinline__ void score_log2(uint32_t (&s)[N], float (&grad)[GRAD ? N : 1], const ScoreCfg &cfg,
                                           float sl2, float slope2, int at, int first, int side) {
  if (cfg.cap_in > 0.f) {
    bool poly = false;
    if constexpr (POLY) poly = __all_sync(0xffffffffu, row_absmax<N>(s) * cfg.cap_in <= kTanhPolyMax);
    if (poly) {
      const uint64_t in2 = f2_pack(cfg.cap_in, cfg.cap_in), out2 = f2_pack(cfg.cap_log2, cfg.cap_log2);
#pragma unroll
      for (int c = 0; c < N; c += 2) {
        const uint64_t u = f2_mul(f2_pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), in2);
        const uint64_t t = f2_tanh_poly(u);
        float a, b;
        f2_unpack(f2_mul(t, out2), a, b);
        s[c] = __float_as_uint(a);
        s[c + 1] = __float_as_uint(b);
        if constexpr (GRAD)
          f2_unpack(f2_fma(f2_mul(t, f2_pack(-1.f, -1.f)), t, f2_pack(1.f, 1.f)), grad[c], grad[c + 1]);
      }
    } else {
#pragma unroll
      for (int c = 0; c < N; ++c) {
        float slope;
        s[c] = __float_as_uint(cfg.cap_log2 * tanh_any<FAR>(__uint_as_float(s[c]) * cfg.cap_in, slope));
        if constexpr (GRAD) grad[c] = slope;
      }
    }
  } else if (!cfg.slopes || side == 0) {
    const uint64_t k2 = f2_pack(sl2, sl2);
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      float a, b;
      f2_unpack(f2_mul(f2_pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), k2), a, b);
      s[c] = __float_as_uint(a);
      s[c + 1] = __float_as_uint(b);
    }
  }
  if (cfg.slopes) {
    if (side != 0) {
      // -slope |at - (first + c)| = g c + g (first - at), g = slope below `at`, -slope above: four
      // running sums with step 8 g, added in the product with the scale where no cap came first
      const float g = side < 0 ? slope2 : -slope2;
      const float base = g * static_cast<float>(first - at);
      const uint64_t k2 = cfg.cap_in > 0.f ? f2_pack(1.f, 1.f) : f2_pack(sl2, sl2), step = f2_pack(8.f * g, 8.f * g);
      uint64_t bias[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        bias[k] = f2_pack(fmaf(static_cast<float>(2 * k), g, base), fmaf(static_cast<float>(2 * k + 1), g, base));
#pragma unroll
      for (int c = 0; c < N; c += 2) {
        uint64_t &bk = bias[(c / 2) & 3];
        float a, b;
        f2_unpack(f2_fma(f2_pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), k2, bk), a, b);
        bk = f2_add(bk, step);
        s[c] = __float_as_uint(a);
        s[c + 1] = __float_as_uint(b);
      }
    } else {
      const float d0 = static_cast<float>(first - at);
#pragma unroll
      for (int c = 0; c < N; ++c)
        s[c] = __float_as_uint(fmaf(-slope2, fabsf(d0 + static_cast<float>(c)), __uint_as_float(s[c])));
    }
  }
}

// P = 2^(score - lse) of N raw products of one fixed index with N others whose LSE (log2 units)
// is lse4, as in the backward: calls out(c, p, g) for each four of them, g = P (1 - tanh^2).
template <int N, bool FAR, typename Out>
__device__ __forceinline__ void score_probs(uint32_t (&s)[N], const float4 *lse4, const ScoreCfg &cfg, float sl2,
                                            float slope2, int at, int first, int side, Out out) {
  if (cfg.cap_in <= 0.f && !cfg.slopes) {
#pragma unroll
    for (int c = 0; c < N; c += 4) {
      const float4 l = lse4[c / 4];
      float p[4];
      p[0] = ex2_approx(fmaf(__uint_as_float(s[c + 0]), sl2, -l.x));
      p[1] = ex2_approx(fmaf(__uint_as_float(s[c + 1]), sl2, -l.y));
      p[2] = ex2_approx(fmaf(__uint_as_float(s[c + 2]), sl2, -l.z));
      p[3] = ex2_approx(fmaf(__uint_as_float(s[c + 3]), sl2, -l.w));
      out(c, p, p);
    }
    return;
  }
  if (cfg.cap_in <= 0.f) {  // a bias alone
    const uint64_t k2 = f2_pack(sl2, sl2);
    if (side != 0) {  // see score_log2
      const float g = side < 0 ? slope2 : -slope2;
      const float base = g * static_cast<float>(first - at);
      const uint64_t step = f2_pack(8.f * g, 8.f * g);
      uint64_t bias[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        bias[k] = f2_pack(fmaf(static_cast<float>(2 * k), g, base), fmaf(static_cast<float>(2 * k + 1), g, base));
#pragma unroll
      for (int c = 0; c < N; c += 4) {
        const float4 l = lse4[c / 4];
        float p[4];
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          uint64_t &bk = bias[((c + k) / 2) & 3];
          const uint64_t r = f2_pack(__uint_as_float(s[c + k]), __uint_as_float(s[c + k + 1]));
          float x0, x1;
          f2_unpack(f2_add(f2_fma(r, k2, bk), k ? f2_pack(-l.z, -l.w) : f2_pack(-l.x, -l.y)), x0, x1);
          bk = f2_add(bk, step);
          p[k] = ex2_approx(x0);
          p[k + 1] = ex2_approx(x1);
        }
        out(c, p, p);
      }
    } else {
      const float d0 = static_cast<float>(first - at);
#pragma unroll
      for (int c = 0; c < N; c += 4) {
        const float4 l = lse4[c / 4];
        const float ll[4] = {l.x, l.y, l.z, l.w};
        float p[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          p[k] = ex2_approx(fmaf(-slope2, fabsf(d0 + static_cast<float>(c + k)), fmaf(__uint_as_float(s[c + k]), sl2, -ll[k])));
        out(c, p, p);
      }
    }
    return;
  }
  const int deg = cfg.slopes ? 0 : cap_degree(row_absmax<N>(s), cfg);
  const float inv = __fdividef(1.f, cfg.cap_log2);
  auto folded = [&](auto d) {
    constexpr int DEG = decltype(d)::value;
    const uint64_t inv2 = f2_pack(inv, inv), one = f2_pack(1.f, 1.f), neg = f2_pack(-inv, -inv);
#pragma unroll
    for (int c = 0; c < N; c += 4) {
      const float4 l = lse4[c / 4];
      float p[4], g[4];
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        const uint64_t r = f2_pack(__uint_as_float(s[c + k]), __uint_as_float(s[c + k + 1]));
        const uint64_t y = f2_mul(r, f2_cap_poly<DEG>(r, cfg));
        float x0, x1, g0, g1;
        f2_unpack(f2_add(y, k ? f2_pack(-l.z, -l.w) : f2_pack(-l.x, -l.y)), x0, x1);
        f2_unpack(f2_fma(f2_mul(y, inv2), f2_mul(y, neg), one), g0, g1);  // 1 - t^2
        p[k] = ex2_approx(x0);
        p[k + 1] = ex2_approx(x1);
        g[k] = p[k] * g0;
        g[k + 1] = p[k + 1] * g1;
      }
      out(c, p, g);
    }
  };
  if (deg == 3) {
    folded(Degree<3>{});
  } else if (deg == 5) {
    folded(Degree<5>{});
  } else {
    // Sixteen at a time: the scores, their derivatives and both results of more would not fit a
    // thread's registers.
#pragma unroll
    for (int h = 0; h < N / 16; ++h) {
      uint32_t (&s16)[16] = *reinterpret_cast<uint32_t(*)[16]>(&s[16 * h]);
      float grad[16];
      score_log2<16, true, FAR>(s16, grad, cfg, sl2, slope2, at, first + 16 * h, side);
#pragma unroll
      for (int c = 0; c < 16; c += 4) {
        const float4 l = lse4[4 * h + c / 4];
        const float ll[4] = {l.x, l.y, l.z, l.w};
        float p[4], g[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          p[k] = ex2_approx(__uint_as_float(s16[c + k]) - ll[k]);
          g[k] = p[k] * grad[c + k];
        }
        out(16 * h + c, p, g);
      }
    }
  }
}

// Smallest lo and largest hi over the rows of a 128-row query block that see a key
// ((INT_MAX, 0) when none does), by one warp: the backward's key blocks pick their query blocks
// by it.
__device__ __forceinline__ int2 score_block_span(const ScoreCfg &cfg, int b, int qb, int N, int lane) {
  int lo = INT_MAX, hi = 0;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    int l, h;
    row_range(cfg, b, qb * 128 + r * 32 + lane, N, l, h);
    if (h > l) {
      lo = min(lo, l);
      hi = max(hi, h);
    }
  }
  return make_int2(__reduce_min_sync(0xffffffffu, lo), __reduce_max_sync(0xffffffffu, hi));
}

}  // namespace fa
