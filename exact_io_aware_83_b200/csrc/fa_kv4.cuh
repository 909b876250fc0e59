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
#include "fa_decode_line.cuh"

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

// Eight bf16 values as fp32.
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

__device__ __forceinline__ __nv_bfloat162 u32_bf2(uint32_t u) { return *reinterpret_cast<__nv_bfloat162 *>(&u); }

// Quantises a group of 32 bf16 values (16 words): four words of codes, and s, m.
__device__ __forceinline__ void kv4_quantise(const uint32_t (&x)[16], uint32_t (&codes)[4], __half &s_out,
                                             __half &m_out) {
  __nv_bfloat162 l2 = u32_bf2(x[0]), h2 = l2;
#pragma unroll
  for (int i = 1; i < 16; ++i) {
    l2 = __hmin2_nan(l2, u32_bf2(x[i]));
    h2 = __hmax2_nan(h2, u32_bf2(x[i]));
  }
  float lo = __bfloat162float(__hmin_nan(l2.x, l2.y)), hi = __bfloat162float(__hmax_nan(h2.x, h2.y));
#pragma unroll
  for (int i = 0; i < 4; ++i) codes[i] = 0u;
  s_out = __ushort_as_half(0);
  m_out = __ushort_as_half(0x7FFF);
  if (!(fabsf(lo) < INFINITY) || !(fabsf(hi) < INFINITY)) return;  // a NaN or an infinity
  const bool clamp = lo < -kKV4Clamp || hi > kKV4Clamp;
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
  s_out = __ushort_as_half(sb1);
  m_out = mh;
  const float s = __half2float(s_out);
  if (s == 0.f) return;
  // t = (x - m) / s + 1/2 - 2^-8 in fp32 lies below the true quotient + 1/2 and above it
  // - 2^-7 (|m| / s <= 2^12, so rounding moves it by less than 2^-10), so its floor is n or
  // n - 1; one exact comparison with the border above it decides.  The floor: adding 2^23,
  // rounded down, leaves it in the low bits.
  const float inv = __fdividef(1.f, s), c = fmaf(-m, inv, 0.5f - 0.00390625f);
  const float mh2 = fmaf(0.5f, s, m);  // border above code 0
  const bool small = kv4_small_min(m, s);
  auto code = [&](float v, bool small_, bool clamp_) -> uint32_t {
    if (clamp_) v = fminf(fmaxf(v, -kKV4Clamp), kKV4Clamp);
    const float f = __fadd_rd(fmaf(v, inv, c), 8388608.f);
    const float n0 = f - 8388608.f;
    const bool above = small_ ? fmaf(-(n0 + 0.5f), s, v) >= m : v >= fmaf(n0, s, mh2);
    return (__float_as_uint(f) & 15u) + (above ? 1u : 0u);
  };
  if (small || clamp) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      codes[i / 4] |= (code(__uint_as_float(x[i] << 16), small, clamp) |
                       (code(__uint_as_float(x[i] & 0xFFFF0000u), small, clamp) << 4)) << (8 * (i % 4));
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      codes[i / 4] |= (code(__uint_as_float(x[i] << 16), false, false) |
                       (code(__uint_as_float(x[i] & 0xFFFF0000u), false, false) << 4)) << (8 * (i % 4));
  }
}

// Writes new tokens: a thread per (token, group), K's threads before V's.  Bound: HBM, 2 d
// bytes read and 5 d / 8 written per token for each of K and V; a group per thread
// spreads the search for s and m over 32 values and needs no exchange between lanes.
template <int D>
__global__ void __launch_bounds__(256) fa_kv4_write_kernel(const KV4Params p) {
  constexpr int G = D / kKV4Group;
  const unsigned rows = static_cast<unsigned>(p.B) * p.Hkv * p.n;  // below 2^31
  const unsigned long long gid = static_cast<unsigned long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  unsigned row = static_cast<unsigned>(gid / G);
  const int gamma = static_cast<int>(gid % G);
  const bool is_v = row >= rows;
  if (is_v) row -= rows;
  if (row >= rows) return;
  const unsigned bh = row / static_cast<unsigned>(p.n);
  const int pos = kv4_position(p, static_cast<int>(bh / static_cast<unsigned>(p.Hkv)),
                               static_cast<int>(row - bh * static_cast<unsigned>(p.n)));
  if (pos < 0) return;
  uint32_t x[16];
  const uint4 *src = reinterpret_cast<const uint4 *>((is_v ? p.v : p.k) + static_cast<size_t>(row) * D) + gamma * 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4 *>(x + 4 * i) = __ldcs(src + i);
  uint32_t codes[4];
  __half s, m;
  kv4_quantise(x, codes, s, m);
  const size_t crow = static_cast<size_t>(bh) * p.cap + pos;
  if (is_v) {
    *reinterpret_cast<uint4 *>(p.vc + crow * (D / 2) + gamma * 16) = make_uint4(codes[0], codes[1], codes[2], codes[3]);
    reinterpret_cast<__half2 *>(p.vp + crow * (2 * G))[gamma] = __halves2half2(s, m);
  } else {
    uint32_t *dst = reinterpret_cast<uint32_t *>(p.kc + crow * (D / 2));
#pragma unroll
    for (int c = 0; c < 4; ++c) dst[c * G + gamma] = codes[c];
    p.kp[crow * (2 * G) + gamma] = s;
    p.kp[crow * (2 * G) + G + gamma] = m;
  }
}

// Reads n tokens back as bf16: value = bf16(m + n s), the sum rounded once in fp32.  A thread
// takes the same word of 8 channels of four tokens (blockDim / words apart), all their loads
// before the first use.
constexpr int kKV4ReadTokens = 4;

template <int D>
__global__ void __launch_bounds__(256) fa_kv4_read_kernel(const KV4Params p) {
  constexpr int G = D / kKV4Group, T = D / 8, U = kKV4ReadTokens, P = 256 / T;
  const unsigned rows = static_cast<unsigned>(p.B) * p.Hkv * p.n;
  const int t = static_cast<int>(threadIdx.x % T), gamma = t / 4, c = t % 4;
  const bool is_v = blockIdx.y != 0;
  const uint8_t *codes = is_v ? p.vc : p.kc;
  const __half *params = is_v ? p.vp : p.kp;
  uint32_t word[U];
  float s[U], m[U];
  unsigned row[U];
  bool live[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    row[u] = (blockIdx.x * U + u) * P + threadIdx.x / T;
    live[u] = row[u] < rows;
    if (!live[u]) continue;
    const unsigned bh = row[u] / static_cast<unsigned>(p.n);
    const int pos = kv4_position(p, static_cast<int>(bh / static_cast<unsigned>(p.Hkv)),
                                 static_cast<int>(row[u] - bh * static_cast<unsigned>(p.n)));
    live[u] = pos >= 0;
    if (!live[u]) continue;
    const size_t crow = static_cast<size_t>(bh) * p.cap + pos;
    word[u] = reinterpret_cast<const uint32_t *>(codes + crow * (D / 2))[is_v ? t : c * G + gamma];
    const __half *par = params + crow * (2 * G);
    if (is_v) {
      const float2 sm = __half22float2(reinterpret_cast<const __half2 *>(par)[gamma]);
      s[u] = sm.x;
      m[u] = sm.y;
    } else {
      s[u] = __half2float(par[gamma]);
      m[u] = __half2float(par[G + gamma]);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (!live[u]) continue;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = fmaf(static_cast<float>((word[u] >> (8 * i)) & 15u), s[u], m[u]);
      const float b = fmaf(static_cast<float>((word[u] >> (8 * i + 4)) & 15u), s[u], m[u]);
      w[i] = pack_bf16x2(a, b);
    }
    __stcs(reinterpret_cast<uint4 *>((is_v ? p.v : p.k) + static_cast<size_t>(row[u]) * D + t * 8),
           make_uint4(w[0], w[1], w[2], w[3]));
  }
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
//    codes go into the matrix product as whole numbers, exactly, and s is applied to the fp32
//    sums.  q is scaled by a power of two per row and converted to fp16 (8 significant bits of
//    11: exact but for entries below 2^-20 of the row's largest).  The second part is a product
//    over the groups, the sums of q split in two fp16 numbers.  (e4m3 products, whose operand
//    bytes the codes already are, measured slower: sm_100 runs the warp-level form as fp16.)
//  * v_jc = m + n s in fp16 (one rounding, 2^-11 relative), p_j in fp16 (p_j <= 2^8).
//  * The matrix products are warp-level m16n8k16: S^T = K Q^T with 16 keys as rows, O^T = V^T
//    P^T with 16 channels as rows.  The codes are unpacked from registers straight into the
//    operand layout (two lanes of work per instruction), which no shared-memory operand could
//    take without writing the widened values out and reading them back: 4 bytes a value
//    through shared memory against half a byte from HBM.
//  * Bound: HBM, 5 d / 4 bytes per key (K and V with their params).
//  * Work: blocks of 256 keys in equal pieces (fa_decode_line.cuh).  More rows than 8 NT are
//    segments of their own, far apart on the line, and read the cache again: B = 4, Hkv = 8, 64k
//    tokens, d = 128, 16, 32 and 128 rows per K/V head 121, 227 and 869 us, against 161, 169 and
//    650 of the bf16 decode.
//  * Blocks stream through a ring of shared-memory stages, across segments, four bulk copies
//    each (the rows of one head are contiguous); every warp takes 32 keys of a block, and the
//    warps take turns at refilling the stage that all have left.
struct KV4DecodeParams : LineParams {
  const uint8_t *kc, *vc;
  const __half *kp, *vp;
};

constexpr int kKV4Warps = 8;
constexpr int kKV4Keys = 32;                        // keys per warp and step
constexpr int kKV4Block = kKV4Warps * kKV4Keys;     // keys per block

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with C = 0 (the sums of one group, or over the groups of 8 or 16).
__device__ __forceinline__ void mma_f16_16816_z(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t h2_u32(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 u32_h2(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }

// The codes at bits 4 i .. 4 i + 3 of both halves of w, i = 0 (LOW) or 1, as fp16 whole
// numbers: or-ed into the mantissa of 1024 (i = 0) or of 64 (i = 1, unit 2^-4), which is
// then subtracted (exactly).
// (Kim et al., "Who Says Elephants Can't Run", 2022, widen whole-number weights this way.)
// The two magic numbers live in registers (a three-input logic operation takes one immediate,
// and the compiler would otherwise spend two of them).
template <int I>
__device__ __forceinline__ uint32_t codes_biased(uint32_t w, uint32_t magic) {
  constexpr uint32_t mask = I ? 0x00F000F0u : 0x000F000Fu;
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "n"(mask), "r"(magic));  // (w & mask) | magic
  return r;
}
template <int I>
__device__ __forceinline__ __half2 codes_h2(uint32_t w, uint32_t magic) {
  return __hsub2(u32_h2(codes_biased<I>(w, magic)), u32_h2(I ? 0x54005400u : 0x64006400u));
}

template <int D, int NT>
struct KV4Layout {
  static constexpr int G = D / 32;    // groups
  static constexpr int KW = G;        // K words per lane and key
  static constexpr int VW = D / 64;   // V words per lane and key
  static constexpr int MT = VW * 4;   // 16-channel tiles of O^T
  static constexpr int ROWS = 8 * NT;
  static constexpr int kCtas = NT == 1 && D <= 128 ? 2 : 1;  // CTAs per SM
  // One stage of the ring: codes and params of a block.
  static constexpr int kOffKC = 0;
  static constexpr int kOffVC = kOffKC + kKV4Block * D / 2;
  static constexpr int kOffKP = kOffVC + kKV4Block * D / 2;
  static constexpr int kOffVP = kOffKP + kKV4Block * 4 * G;
  static constexpr int kStageBytes = kOffVP + kKV4Block * 4 * G;
  static constexpr int kPartBytes = kKV4Warps / 2 * ROWS * D * 4;  // O of half the warps, where a segment ends
  static constexpr int kFixed = kPartBytes + 2 * kKV4Warps * ROWS * 4 + 2 * 8 * 8 + 64 + 128;
  static constexpr int kFit = ((kCtas == 2 ? 232448 / 2 - 1024 : 232448) - kFixed) / kStageBytes;
  static constexpr int kStages = kFit > 4 ? 4 : kFit;
  static constexpr int kOffPart = kStages * kStageBytes;
  static constexpr int kOffM = kOffPart + kPartBytes;      // [warp][row] m, then l
  static constexpr int kOffBar = kOffM + 2 * kKV4Warps * ROWS * 4;  // full[8], empty[8]
  static constexpr int kOffMisc = kOffBar + 2 * 8 * 8;
  static constexpr int kSmemBytes = kOffMisc + 64 + 128;   // + slack for 128-byte alignment
  static_assert(kStages >= 2 && kStages <= 8, "ring");
};

// Key of row r of a 16-key step: the rows 2c, 2c+1, 2c+8, 2c+9 of lane group c of the second
// product are the keys c, c+4, c+8, c+12, so that its four loads touch consecutive tokens
// and no two lanes of a load the same bank.
__device__ __forceinline__ int kv4_key_of_row(int r) { return ((r & 7) >> 1) + 4 * (r & 1) + (r & 8); }

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

template <int D, int NT, bool CHANGED>  // CHANGED: capped scores or a distance bias
__global__ void __launch_bounds__(kKV4Warps * 32, KV4Layout<D, NT>::kCtas)
    fa_decode_kv4_kernel(const KV4DecodeParams p) {
  using L = KV4Layout<D, NT>;
  constexpr int G = L::G, KW = L::KW, VW = L::VW, MT = L::MT, S = L::kStages, ROWS = L::ROWS;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 127u) & ~127u;
  uint8_t *smem = smem_raw + (base - smem_u32(smem_raw));
  float *sm_o = reinterpret_cast<float *>(smem + L::kOffPart);
  float *sm_m = reinterpret_cast<float *>(smem + L::kOffM);
  // [0] abort flag, [1] blocks whose copies have been started, [2] blocks of the piece, [6..11]
  // the block that is loaded next
  int *misc = reinterpret_cast<int *>(smem + L::kOffMisc);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, c = lane % 4;
  const uint32_t full = base + L::kOffBar, empty = full + 64;
  volatile int *abort_flag = misc;

  // ---- this piece of the line: blocks [x0, x1), and the segment that x0 lies in
  if (threadIdx.x < S) {
    mbar_init(full + 8 * threadIdx.x, 1);
    mbar_init(empty + 8 * threadIdx.x, kKV4Warps);
    fence_mbar_init();
  }
  if (warp == 0) {
    const LinePiece at = line_piece<kKV4Block>(p, blockIdx.x, lane);
    if (lane == 0) {
      misc[0] = misc[1] = 0;
      misc[2] = at.blocks;
      *reinterpret_cast<LineCursor<kKV4Block> *>(misc + 6) = line_cursor<kKV4Block>(p, at);
    }
  }
  __syncthreads();
  launch_dependents();        // the joining kernel
  const int total = misc[2];  // blocks of the piece
  int todo = total, taken = 0;
  LineCursor<kKV4Block> cur = *reinterpret_cast<LineCursor<kKV4Block> *>(misc + 6);  // what is computed next
  __syncthreads();            // the cursor moves on with the first copies
  bool ok = true;

  // Starts the copies of the piece's next block (one thread; the cursor passes from one issuer
  // to the next through the barriers of the stage).
  auto issue = [&]() {
    LineCursor<kKV4Block> *ahead = reinterpret_cast<LineCursor<kKV4Block> *>(misc + 6);
    LineCursor<kKV4Block> a = *ahead;
    const int st = misc[1] % S;
    const uint32_t dst = base + st * L::kStageBytes, bar = full + 8 * st;
    const int kb = a.blk * kKV4Block;
    const int n = min(kKV4Block, (a.len - kb + kKV4Keys - 1) / kKV4Keys * kKV4Keys);  // within cap, a multiple of 64
    if (n > 0) {
      const long long row = static_cast<long long>(a.b * p.Hkv + a.kvh) * p.cap + kb;
      mbar_arrive_expect_tx(bar, static_cast<uint32_t>(n) * (D + 8 * G));
      bulk_load(dst + L::kOffKC, p.kc + row * (D / 2), n * (D / 2), bar);
      bulk_load(dst + L::kOffVC, p.vc + row * (D / 2), n * (D / 2), bar);
      bulk_load(dst + L::kOffKP, p.kp + row * (2 * G), n * (4 * G), bar);
      bulk_load(dst + L::kOffVP, p.vp + row * (2 * G), n * (4 * G), bar);
    } else {
      mbar_arrive(bar);  // a segment without keys
    }
    a.next(p);
    *ahead = a;
    ++misc[1];
  };
  if (threadIdx.x == 0)
    for (int i = 0; i < min(S, total); ++i) issue();

  uint32_t magic0, magic1;  // 1024 and 64, twice
  asm volatile("mov.b32 %0, 0x64006400;" : "=r"(magic0));
  asm volatile("mov.b32 %0, 0x54005400;" : "=r"(magic1));
  const int grp = p.R / p.Nq;  // query heads per K/V head
  const float inv_cap = p.softcap > 0.f ? 1.f / p.softcap : 0.f;
  const float cap_log2 = p.softcap * kLog2e;
  const int ka = kv4_key_of_row(g);  // key of row g; row g + 8 is ka + 8
  const int vgroup = (g * VW) / 4;   // group of this lane's V channels

  while (todo > 0) {
    // ---- one segment, or the part of it that lies in this piece
    const int blk0 = cur.blk, count = min(cur.nblk - blk0, todo), len = cur.len;
    const bool began_before = blk0 > 0, ends_after = blk0 + count < cur.nblk;
    const int kvh = cur.kvh, r0 = cur.rt * ROWS;
    const long long row0 = static_cast<long long>(cur.b * p.Hkv + kvh) * p.R + r0;
    const int pos0 = len - p.Nq;

    // Q fragments: row g of each 8-row tile, this lane's 8 channels of every group, scaled
    uint32_t qf[NT][G][4];         // [e]: channels (e, e + 4) of the word
    uint32_t qs[NT][G == 8 ? 4 : 2];  // B operand of the product over the groups
    float raw[NT][2], fac[NT][2];  // rows 2c, 2c+1: from the products to scores, and from those to log2
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
      // largest magnitude into [8, 16): 64 times the sum of 16 of them stays inside fp16
      const int ex = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -100);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + 3 - ex) << 23);
      const float down = __uint_as_float(static_cast<uint32_t>(127 - 3 + ex) << 23);
      float qsum[G], qodd[G];  // sums of the scaled q over each group, and -64 times those of pairs 1 and 3
#pragma unroll
      for (int i = 0; i < G; ++i) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] *= up;
        float odd = (x[i][1] + x[i][3]) + (x[i][5] + x[i][7]);
        s = odd + ((x[i][0] + x[i][2]) + (x[i][4] + x[i][6]));
#pragma unroll
        for (int e = 0; e < 4; ++e) qf[nt][i][e] = pack_f16x2(x[i][e], x[i][e + 4]);
#pragma unroll
        for (int o = 1; o < 4; o *= 2) {
          s += __shfl_xor_sync(0xffffffffu, s, o);
          odd += __shfl_xor_sync(0xffffffffu, odd, o);
        }
        qsum[i] = s;
        qodd[i] = -64.f * odd;
      }
      // Row k of the operand that meets the groups' m: the sum of group k, its fp16 rounding
      // first, then what is left (8 groups: in the second half of 16 rows; fewer: in rows
      // G .. 2 G - 1 of 8).  The rows that meet s hold the other sums the same way.
      {
        constexpr int H = G == 8 ? 4 : G / 2;  // lanes that hold a pair of groups each
        float a = 0.f, bq = 0.f, ao = 0.f, bo = 0.f;
#pragma unroll
        for (int i = 0; i < G; i += 2)
          if (c % H == i / 2) {
            a = qsum[i];
            bq = qsum[i + 1];
            ao = qodd[i];
            bo = qodd[i + 1];
          }
        auto split = [&](float u, float v, uint32_t &hi, uint32_t &lo) {
          hi = pack_f16x2(u, v);
          lo = pack_f16x2(u - __low2float(u32_h2(hi)), v - __high2float(u32_h2(hi)));
        };
        uint32_t hi, lo, hi_o, lo_o;
        split(a, bq, hi, lo);
        split(ao, bo, hi_o, lo_o);
        if constexpr (G == 8) {
          qs[nt][0] = hi;
          qs[nt][1] = lo;
          qs[nt][2] = hi_o;
          qs[nt][3] = lo_o;
        } else {
          qs[nt][0] = c < H ? hi : (c < 2 * H ? lo : 0u);
          qs[nt][1] = c < H ? hi_o : (c < 2 * H ? lo_o : 0u);
        }
      }
      // (never 0: hidden scores are -inf and stay so)
      const float f = fmaxf((p.softcap > 0.f ? p.scale : p.sl2) * down, 1e-37f);
      raw[nt][0] = __shfl_sync(0xffffffffu, f, 8 * c);
      raw[nt][1] = __shfl_sync(0xffffffffu, f, 8 * c + 4);
      fac[nt][0] = CHANGED ? 1.f : raw[nt][0];
      fac[nt][1] = CHANGED ? 1.f : raw[nt][1];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rr = r0 + nt * 8 + 2 * c + e;
        const int h = kvh * grp + min(rr / p.Nq, grp - 1);
        slope2[nt][e] = p.slopes ? p.slopes[h] * kLog2e : 0.f;
        rpos[nt][e] = pos0 + rr % p.Nq;
      }
    }

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

    int kb = blk0 * kKV4Block + warp * kKV4Keys;
#pragma unroll 1
    for (int i = 0; i < count; ++i, ++taken, kb += kKV4Block) {
      // The stage that the block before this one was in is refilled, by one warp in turn.
      if (taken > 0 && taken + S - 1 < total && warp == taken % kKV4Warps && lane == 0 &&
          wait_bounded(empty + 8 * ((taken - 1) % S), ((taken - 1) / S) & 1, abort_flag, wait_site(5, 8 + (taken - 1) % S, taken)))
        issue();
      __syncwarp();
      const int st_ = taken % S;
      if (ok) ok = warp_wait_bounded(full + 8 * st_, (taken / S) & 1, abort_flag, wait_site(5, st_, taken));
      if (ok && kb < len) {  // !ok: the flag is up, nothing of this call is valid any more
      const uint8_t *stage = smem + st_ * L::kStageBytes + warp * (kKV4Keys * D / 2);
      const uint8_t *stage_par = smem + st_ * L::kStageBytes + L::kOffKP + warp * (kKV4Keys * 4 * G);
      float y[2][NT][4];  // [step][tile][key A: rows 2c, 2c+1; key B: rows 2c, 2c+1]
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        uint32_t w[2][KW], sc[2][G / 2], mn[2], sn[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int key = 16 * st + ka + 8 * e;
          const uint32_t *src = reinterpret_cast<const uint32_t *>(stage + L::kOffKC + key * (D / 2)) + c * KW;
          const uint32_t *ps = reinterpret_cast<const uint32_t *>(stage_par + key * (4 * G));
          if constexpr (KW == 2) {
            *reinterpret_cast<uint2 *>(w[e]) = *reinterpret_cast<const uint2 *>(src);
            sc[e][0] = ps[0];
          } else {
#pragma unroll
            for (int i = 0; i < KW; i += 4) *reinterpret_cast<uint4 *>(w[e] + i) = *reinterpret_cast<const uint4 *>(src + i);
            if constexpr (KW == 4) *reinterpret_cast<uint2 *>(sc[e]) = *reinterpret_cast<const uint2 *>(ps);
            else *reinterpret_cast<uint4 *>(sc[e]) = *reinterpret_cast<const uint4 *>(ps);
          }
          mn[e] = ps[G / 2 + (G == 8 ? c : c % (G / 2))];
          sn[e] = ps[G == 8 ? c : c % (G / 2)];
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if constexpr (G == 8) {
            mma_f16_16816_z(y[st][nt], mn[0], mn[1], mn[0], mn[1], qs[nt][0], qs[nt][1]);
            mma_f16_16816(y[st][nt], sn[0], sn[1], sn[0], sn[1], qs[nt][2], qs[nt][3]);
          } else {
            mma_f16_16816_z(y[st][nt], mn[0], mn[1], sn[0], sn[1], qs[nt][0], qs[nt][1]);
          }
        }
#pragma unroll
        for (int i = 0; i < G; ++i) {
          uint32_t a[2][4];  // pairs 1 and 3 stay 64 too large; the product over the groups takes that off
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            a[e][0] = h2_u32(codes_h2<0>(w[e][i], magic0));
            a[e][1] = codes_biased<1>(w[e][i], magic1);
            a[e][2] = h2_u32(codes_h2<0>(w[e][i] >> 8, magic0));
            a[e][3] = codes_biased<1>(w[e][i] >> 8, magic1);
          }
          auto pick = [](uint32_t u, int hi) { return hi ? __high2float(u32_h2(u)) : __low2float(u32_h2(u)); };
          const float sA = pick(sc[0][i / 2], i & 1), sB = pick(sc[1][i / 2], i & 1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float part[4];
            mma_f16_16816_z(part, a[0][0], a[1][0], a[0][1], a[1][1], qf[nt][i][0], qf[nt][i][1]);
            mma_f16_16816(part, a[0][2], a[1][2], a[0][3], a[1][3], qf[nt][i][2], qf[nt][i][3]);
            y[st][nt][0] = fmaf(sA, part[0], y[st][nt][0]);
            y[st][nt][1] = fmaf(sA, part[1], y[st][nt][1]);
            y[st][nt][2] = fmaf(sB, part[2], y[st][nt][2]);
            y[st][nt][3] = fmaf(sB, part[3], y[st][nt][3]);
          }
        }
      }
      // ---- cap and bias: the scores in log2 units (without them the factor goes into the exponent)
      if constexpr (CHANGED) {
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) y[st][nt][e] *= raw[nt][e & 1];
        auto cap_all = [&](auto far) {
#pragma unroll
          for (int st = 0; st < 2; ++st)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                y[st][nt][e] = softcap_log2<decltype(far)::value>(y[st][nt][e], inv_cap, cap_log2);
        };
        if (p.softcap > kCapNear) cap_all(Flag<true>{});
        else if (p.softcap > 0.f) cap_all(Flag<false>{});
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float v = y[st][nt][e];
              const int key = kb + 16 * st + ka + 8 * (e / 2);
              y[st][nt][e] = fmaf(-slope2[nt][e & 1], fabsf(static_cast<float>(rpos[nt][e & 1] - key)), v);
            }
      }
      if (kb + kKV4Keys > (p.causal ? min(len, pos0 + 1) : len)) {  // some key is hidden from some row
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = kb + 16 * st + ka + 8 * (e / 2);
              if (key >= len || (p.causal && key > rpos[nt][e & 1])) y[st][nt][e] = -INFINITY;
            }
      }
      // ---- running maximum: moved (for the whole warp) only when a row's rises by more than 2^8
      bool up = false;
      float mx[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[nt][e] = fmaxf(fmaxf(y[0][nt][e], y[0][nt][e + 2]), fmaxf(y[1][nt][e], y[1][nt][e + 2])) * fac[nt][e];
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
      float mu[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) mu[nt][e] = m_run[nt][e] == -INFINITY ? 0.f : m_run[nt][e];
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float pr[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            pr[e] = ex2_approx(fmaf(y[st][nt][e], fac[nt][e & 1], -mu[nt][e & 1]));
            l_run[nt][e & 1] += pr[e];
          }
          pb[nt][0] = movmatrix_trans(pack_f16x2(pr[0], pr[1]));
          pb[nt][1] = movmatrix_trans(pack_f16x2(pr[2], pr[3]));
        }
        uint32_t wv[4][VW], sm[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = 16 * st + c + 4 * e;
          const uint32_t *src = reinterpret_cast<const uint32_t *>(stage + L::kOffVC + key * (D / 2)) + g * VW;
          if constexpr (VW == 1) wv[e][0] = *src;
          else if constexpr (VW == 2) *reinterpret_cast<uint2 *>(wv[e]) = *reinterpret_cast<const uint2 *>(src);
          else *reinterpret_cast<uint4 *>(wv[e]) = *reinterpret_cast<const uint4 *>(src);
          sm[e] = reinterpret_cast<const uint32_t *>(stage_par + (L::kOffVP - L::kOffKP) + key * (4 * G))[vgroup];
        }
        if (kb + kKV4Keys > len) {
          // rows behind the last key hold anything; 0 * NaN would spread
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (kb + 16 * st + c + 4 * e >= len) sm[e] = 0u;
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
              const uint32_t a0 = h2_u32(__hfma2(codes_h2<0>(x0, magic0), sp[0], mp[0]));
              const uint32_t a1 = h2_u32(__hfma2(codes_h2<1>(x0, magic1), sp[0], mp[0]));
              const uint32_t a2 = h2_u32(__hfma2(codes_h2<0>(x1, magic0), sp[1], mp[1]));
              const uint32_t a3 = h2_u32(__hfma2(codes_h2<1>(x1, magic1), sp[1], mp[1]));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16_16816(acc[w * 4 + half * 2 + t][nt], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
            }
          }
      }
      }
      __syncwarp();  // every lane has read the stage
      if (lane == 0) mbar_arrive(empty + 8 * st_);
    }

    // Accumulator tile w * 4 + q of lane (g, c): channels 8 (g VW + w) + 2 q (+ 1), rows 2c, 2c+1.
    line_join<D, NT, kKV4Warps>(p, sm_o, sm_m, m_run, l_run, r0, row0, began_before, ends_after, abort_flag,
                                [&](float *row, float f, int nt, int e, bool add) {
                                  float4 *dst = reinterpret_cast<float4 *>(row + 8 * g * VW);
#pragma unroll
                                  for (int i = 0; i < MT; i += 2) {
                                    float4 v = add ? dst[i / 2] : make_float4(0.f, 0.f, 0.f, 0.f);
                                    v.x = fmaf(f, acc[i][nt][e], v.x);
                                    v.y = fmaf(f, acc[i][nt][e + 2], v.y);
                                    v.z = fmaf(f, acc[i + 1][nt][e], v.z);
                                    v.w = fmaf(f, acc[i + 1][nt][e + 2], v.w);
                                    dst[i / 2] = v;
                                  }
                                });
    todo -= count;
    cur.blk = cur.nblk - 1;  // to the next segment
    cur.next(p);
  }
  // No copy may still be landing in shared memory when the CTA exits.
  if (*abort_flag != 0 && threadIdx.x == 0)
    for (int i = max(0, misc[1] - S); i < misc[1]; ++i) wait_drain(full + 8 * (i % S), (i / S) & 1, 100000000ull);
}

}  // namespace fa
