// fa_api_score.cu - host side of the entry points for changed scores (fa_fwd_score,
// fa_bwd_score, fa_decode_score) and for the 4-bit cache (fa_kv4_write, fa_kv4_read,
// fa_decode_kv4): argument checks, TMA tensor maps, launches.  Declared, with their
// contracts, in include/fa.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <mutex>

#include "fa.h"
#include "fa_common.cuh"
#include "fa_fwd.cuh"
#include "fa_fwd_d256.cuh"
#include "fa_bwd.cuh"
#include "fa_bwd_plan.cuh"
#include "fa_bwd_q128.cuh"
#include "fa_decode.cuh"
#include "fa_decode_score.cuh"
#include "fa_kv4.cuh"
#include "fa_host.h"

namespace {

using namespace fa_host;

struct ScoreState {
  std::once_flag once;
  bool ok = false;
  std::atomic<bool> ready{false};  // ok, for readers outside of call_once
};
ScoreState g_score_dev[kMaxDevices];

// One-time kernel attribute setup on the current device.
bool score_ready() {
  int dev = 0;
  if (!device_ready() || !cuda_ok(cudaGetDevice(&dev), "cudaGetDevice") || dev < 0 || dev >= kMaxDevices) return false;
  ScoreState &st = g_score_dev[dev];
  std::call_once(st.once, [&] {
    bool ok = true;
    ok = ok && set_smem(fa::fa_bwd_q128_kernel<fa::kAttnFull, true>, fa::Q128Layout::kSmemBytes);
    ok = ok && set_smem(fa::fa_bwd_q128_kernel<fa::kAttnCausal, true>, fa::Q128Layout::kSmemBytes);
    ok = ok && set_smem(fa::fa_fwd_kernel<64, fa::kAttnScore>, fa::FwdLayout<64>::kSmemBytesScore);
    ok = ok && set_smem(fa::fa_fwd_kernel<64, fa::kAttnScoreFar>, fa::FwdLayout<64>::kSmemBytesScore);
    ok = ok && set_smem(fa::fa_fwd_kernel<128, fa::kAttnScore>, fa::FwdLayout<128>::kSmemBytesScore);
    ok = ok && set_smem(fa::fa_fwd_kernel<128, fa::kAttnScoreFar>, fa::FwdLayout<128>::kSmemBytesScore);
    ok = ok && regs_at_least(fa::fa_fwd_kernel<64, fa::kAttnScore>, fa::kFwdRegsLaunch);
    ok = ok && regs_at_least(fa::fa_fwd_kernel<64, fa::kAttnScoreFar>, fa::kFwdRegsLaunch);
    ok = ok && regs_at_least(fa::fa_fwd_kernel<128, fa::kAttnScore>, fa::kFwdRegsLaunch);
    ok = ok && regs_at_least(fa::fa_fwd_kernel<128, fa::kAttnScoreFar>, fa::kFwdRegsLaunch);
    ok = ok && set_smem(fa::fa_fwd_d256_kernel<fa::kAttnScore>, fa::FwdD256Layout::kSmemBytesScore);
    ok = ok && set_smem(fa::fa_fwd_d256_kernel<fa::kAttnScoreFar>, fa::FwdD256Layout::kSmemBytesScore);
    ok = ok && set_smem(fa::fa_bwd_main_kernel<64, 64, 64, fa::kAttnScore>, fa::BwdLayout<64, 64, 64>::kSmemBytesScore);
    ok = ok && set_smem(fa::fa_bwd_main_kernel<64, 64, 64, fa::kAttnScoreFar>, fa::BwdLayout<64, 64, 64>::kSmemBytesScore);
    ok = ok && set_smem(fa::fa_bwd_main_kernel<64, 64, 64, fa::kAttnScoreParts>, fa::BwdLayout<64, 64, 64>::kSmemBytesScore);
    ok = ok && set_smem(fa::fa_bwd_main_kernel<64, 64, 64, fa::kAttnScorePartsFar>, fa::BwdLayout<64, 64, 64>::kSmemBytesScore);
    ok = ok && set_smem(fa::fa_bwd_main_kernel<128, 128, 64, fa::kAttnScore>, fa::BwdLayout<128, 128, 64>::kSmemBytesScore);
    ok = ok && set_smem(fa::fa_bwd_main_kernel<128, 128, 64, fa::kAttnScoreFar>, fa::BwdLayout<128, 128, 64>::kSmemBytesScore);
    ok = ok && set_smem(fa::fa_bwd_main_kernel<128, 128, 64, fa::kAttnScoreParts>, fa::BwdLayout<128, 128, 64>::kSmemBytesScore);
    ok = ok && set_smem(fa::fa_bwd_main_kernel<128, 128, 64, fa::kAttnScorePartsFar>, fa::BwdLayout<128, 128, 64>::kSmemBytesScore);
    ok = ok && set_smem(fa::fa_bwd_main_kernel<256, 128, 64, fa::kAttnScore>, fa::BwdLayout<256, 128, 64>::kSmemBytesScore);
    ok = ok && set_smem(fa::fa_bwd_main_kernel<256, 128, 64, fa::kAttnScoreFar>, fa::BwdLayout<256, 128, 64>::kSmemBytesScore);
    ok = ok && set_smem(fa::fa_bwd_main_kernel<256, 128, 64, fa::kAttnScoreParts>, fa::BwdLayout<256, 128, 64>::kSmemBytesScore);
    ok = ok && set_smem(fa::fa_bwd_main_kernel<256, 128, 64, fa::kAttnScorePartsFar>, fa::BwdLayout<256, 128, 64>::kSmemBytesScore);
    ok = ok && set_smem(fa::fa_decode_kernel<64, 32, true>, fa::DecodeLayout<64, 32>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_kernel<64, 32, true, true>, fa::DecodeLayout<64, 32>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_kernel<64, 64, true>, fa::DecodeLayout<64, 64>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_kernel<64, 64, true, true>, fa::DecodeLayout<64, 64>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_kernel<64, 128, true>, fa::DecodeLayout<64, 128>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_kernel<64, 128, true, true>, fa::DecodeLayout<64, 128>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_kernel<128, 32, true>, fa::DecodeLayout<128, 32>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_kernel<128, 32, true, true>, fa::DecodeLayout<128, 32>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_kernel<128, 64, true>, fa::DecodeLayout<128, 64>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_kernel<128, 64, true, true>, fa::DecodeLayout<128, 64>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_kernel<128, 128, true>, fa::DecodeLayout<128, 128>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_kernel<128, 128, true, true>, fa::DecodeLayout<128, 128>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_kernel<256, 16, true>, fa::DecodeLayout<256, 16>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_kernel<256, 16, true, true>, fa::DecodeLayout<256, 16>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_kernel<256, 32, true>, fa::DecodeLayout<256, 32>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_kernel<256, 32, true, true>, fa::DecodeLayout<256, 32>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_kernel<256, 64, true>, fa::DecodeLayout<256, 64>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_kernel<256, 64, true, true>, fa::DecodeLayout<256, 64>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_kv4_kernel<64, 1, false>, fa::KV4Layout<64, 1>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_kv4_kernel<64, 1, true>, fa::KV4Layout<64, 1>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_kv4_kernel<64, 2, false>, fa::KV4Layout<64, 2>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_kv4_kernel<64, 2, true>, fa::KV4Layout<64, 2>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_kv4_kernel<128, 1, false>, fa::KV4Layout<128, 1>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_kv4_kernel<128, 1, true>, fa::KV4Layout<128, 1>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_kv4_kernel<128, 2, false>, fa::KV4Layout<128, 2>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_kv4_kernel<128, 2, true>, fa::KV4Layout<128, 2>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_kv4_kernel<256, 1, false>, fa::KV4Layout<256, 1>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_kv4_kernel<256, 1, true>, fa::KV4Layout<256, 1>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_score_kernel<64, 1>, fa::DecScoreLayout<64, 1>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_score_kernel<64, 2>, fa::DecScoreLayout<64, 2>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_score_kernel<128, 1>, fa::DecScoreLayout<128, 1>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_score_kernel<128, 2>, fa::DecScoreLayout<128, 2>::kSmemBytes);
    ok = ok && set_smem(fa::fa_decode_score_kernel<256, 1>, fa::DecScoreLayout<256, 1>::kSmemBytes);
    st.ok = ok;
    st.ready.store(ok);
  });
  return st.ok;
}

// The two arguments that change the scores: a cap (0: none) and a slope per query head
// (nullptr: none).
int check_score_args(float softcap, const float *slopes) {
  if (!(softcap >= 0.f) || !std::isfinite(softcap)) return FA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(slopes) & 3u) return FA_ERR_ALIGN;
  return FA_OK;
}

// Caps outside 2^-100 .. 2^100 count as the nearer end, so that 1 / cap, cap log2(e) and their
// products stay finite: below, the scores are equal to fp32 either way; above, a cap changes no
// score under 2^88 by more than its rounding.
float usable_cap(float softcap) {
  return softcap > 0.f ? std::fmin(std::fmax(softcap, 0x1p-100f), 0x1p100f) : softcap;
}

fa::ScoreCfg make_score(float softcap, const float *slopes, const int *key_range, int causal, float scale) {
  fa::ScoreCfg c{};
  softcap = usable_cap(softcap);
  c.raw3 = c.raw5 = -1.f;
  if (softcap > 0.f) {
    const double u = static_cast<double>(scale) / softcap, a = softcap * 1.4426950408889634;
    c.cap_in = static_cast<float>(std::fmin(u, FLT_MAX));
    c.cap_log2 = static_cast<float>(a);
    // tanh(u) / u as a polynomial of u^2: minimax fits on |u| <= 0.5 (degree 3, relative error
    // 5.4e-7) and |u| <= 1 (degree 5, 5.9e-7), with a and the powers of scale / cap folded in;
    // used where every coefficient is a normal fp32 number.
    constexpr double t3[4] = {0.9999994557708327, -0.33326317935183836, 0.13190296595162188, -0.044402225913669886};
    constexpr double t5[6] = {0.9999994135990478, -0.3332904237749518, 0.13281433872551196, -0.05160567377480486, 0.016743114805512608, -0.003067060223737072};
    auto fold = [&](const double *t, int deg, float *k) {
      double f = a * u;
      for (int i = 0; i <= deg; ++i, f *= u * u) {
        const double x = t[i] * f;
        if (!(std::fabs(x) > 0x1p-120 && std::fabs(x) < 0x1p120)) return false;
        k[i] = static_cast<float>(x);
      }
      return true;
    };
    if (fold(t3, 3, c.k3)) c.raw3 = static_cast<float>(0.5 / u);
    if (fold(t5, 5, c.k5)) c.raw5 = static_cast<float>(1.0 / u);
  }
  c.slopes = slopes;
  c.range = reinterpret_cast<const int2 *>(key_range);
  c.causal = causal;
  return c;
}

// Changed scores: the backward keeps one bit per 128-row query block in shared memory.
int check_score_bwd(int N, int d) {
  const long long words = ((N + 127) / 128 + 31) / 32;
  const int cap = d == 64 ? fa::BwdLayout<64, 64, 64>::kScoreBitmapBytes
                  : d == 128 ? fa::BwdLayout<128, 128, 64>::kScoreBitmapBytes
                             : fa::BwdLayout<256, 128, 64>::kScoreBitmapBytes;
  return words * 4 > cap ? FA_ERR_UNSUPPORTED : FA_OK;
}

// ---- forward

// A cap beyond which a score needs the other form of the tanh (fa_score.cuh).
bool far_cap(const fa::ScoreCfg &c) { return c.cap_log2 > fa::kCapNear * fa::kLog2e; }

template <int D, int MODE>
void launch_fwd_mode(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const CUtensorMap &to,
                     const fa::FwdParams &p, unsigned units, cudaStream_t s) {
  if constexpr (D == 256)
    fa::fa_fwd_d256_kernel<MODE><<<units, fa::kFwdD256Threads, fa::FwdD256Layout::kSmemBytesScore, s>>>(tq, tk, tv, to, p);
  else
    fa::fa_fwd_kernel<D, MODE><<<units, fa::kFwdThreads, fa::FwdLayout<D>::kSmemBytesScore, s>>>(tq, tk, tv, to, p);
}

template <int D>
void launch_fwd_score(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const CUtensorMap &to,
                      const fa::FwdParams &p, unsigned units, cudaStream_t s) {
  if (far_cap(p.score)) launch_fwd_mode<D, fa::kAttnScoreFar>(tq, tk, tv, to, p, units, s);
  else launch_fwd_mode<D, fa::kAttnScore>(tq, tk, tv, to, p, units, s);
}

// ---- backward

struct BwdScoreArgs {
  const void *q, *k, *v, *o;
  const float *lse;
  const void *dout;
  void *dq, *dk, *dv, *workspace;
  int B, Hq, Hkv, N, right;
  float scale;
  fa::ScoreCfg score;
  cudaStream_t s;
};

template <int D, int DH, int BQ>
int launch_bwd_score(const BwdScoreArgs &a) {
  using L = fa::BwdLayout<D, DH, BQ>;
  const auto enc = encode_fn();
  const long long rows = static_cast<long long>(a.B) * a.Hq * a.N;
  float *delta = static_cast<float *>(a.workspace);
  float *dqacc = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + fa::pad256(static_cast<size_t>(rows) * 4));
  const long long hq = static_cast<long long>(a.B) * a.Hq, hkv = static_cast<long long>(a.B) * a.Hkv;

  fa::BwdParams p{};
  p.lse = a.lse;
  p.delta = delta;
  p.B = a.B;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.N = a.N;
  p.nkb = (a.N + 127) / 128;
  p.left = -1;
  p.right = a.right;
  p.scale = a.scale;
  p.sl2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
  p.score = a.score;
  // Behind the dQ accumulator: the spans of the query blocks, then the plan.
  char *behind = static_cast<char *>(a.workspace) + fa::bwd_workspace_bytes(a.B, a.Hq, a.N, D);
  int2 *blocks = reinterpret_cast<int2 *>(behind);
  const int max_parts = fa::plan_max_parts(a.B, a.Hkv, a.N, D);
  const fa::PlanLayout plan = fa::plan_layout(a.B, a.Hkv, a.N, D, max_parts);
  behind += fa::pad256(static_cast<size_t>(a.B) * p.nkb * 8);
  int *parts = reinterpret_cast<int *>(behind + plan.parts);
  const auto *ob = static_cast<const __nv_bfloat16 *>(a.o), *dob = static_cast<const __nv_bfloat16 *>(a.dout);
  if (max_parts > 0 || a.score.range) {
    int4 *items = reinterpret_cast<int4 *>(behind + plan.items);
    const fa::PlanParams pp{a.score, a.B, a.N, p.nkb, a.Hq / a.Hkv, 128 / BQ, (a.N - (p.nkb - 1) * 128 + BQ - 1) / BQ,
                            a.Hkv * (D / DH), max_parts, D == 256 ? 6 : 12, blocks, parts, items};
    const unsigned ctas = static_cast<unsigned>(fa::front_blocks(max_parts > 0, a.B, p.nkb) +
                                                (rows + fa::kPlanThreads / 32 - 1) / (fa::kPlanThreads / 32));
    if (max_parts > 0) {
      fa::fa_bwd_front_kernel<D, true><<<ctas, fa::kPlanThreads, 0, a.s>>>(pp, ob, dob, delta, dqacc, rows);
      p.items = items;
      p.parts = reinterpret_cast<float *>(behind + plan.sums);
    } else {
      fa::fa_bwd_front_kernel<D, false><<<ctas, fa::kPlanThreads, 0, a.s>>>(pp, ob, dob, delta, dqacc, rows);
    }
  } else {
    fa::fa_bwd_pre_kernel<D><<<static_cast<unsigned>((rows + 7) / 8), 256, 0, a.s>>>(ob, dob, delta, dqacc, rows);
  }
  if (a.score.range) p.blocks = blocks;
  const fa::BwdOrder order = bwd_order(a.B, a.Hkv, a.N, a.score.range ? a.N : -1, a.right);
  const int tiers = order.tiers < 1 ? 1 : order.tiers, heads = a.B * a.Hkv;
  p.tsz = (p.nkb + tiers - 1) / tiers;
  p.tail = order.tail < 0 ? 0 : (order.tail < heads ? order.tail : heads - 1);

  // With slopes, no key ranges and no plan, d = 128 runs with 128-query steps from N = 4096 on, as plain
  // scores do: causal B = 2, Hq = 32, Hkv = 8, N = 4096 915 us against 978 with slopes, 1359
  // against 1454 with both.  A cap alone fits the 64-query steps better as long as most scores
  // stay in its shorter polynomials (1089 against 1055 us at cap 50 and standard normal q and k;
  // 1152 against 1177 at cap 5).  A cap beyond kCapNear takes those too.
  const bool far = far_cap(a.score);
  const bool wide = a.score.slopes && !far && !a.score.range && max_parts == 0 && D == 128 && a.N >= fa::kQ128MinN;
  bool launched = true;
  const int tslot = timer_start(1, a.s);
  if (wide) {
    const auto e = reinterpret_cast<fa::EncodeTiledFnBwd>(enc);
    launched = a.right == 0 ? fa::bwd_launch_q128<fa::kAttnCausal, true>(e, a.q, a.k, a.v, a.dout, a.dk, a.dv, dqacc, a.B,
                                                                       a.Hq, a.Hkv, a.N, p, a.s)
                            : fa::bwd_launch_q128<fa::kAttnFull, true>(e, a.q, a.k, a.v, a.dout, a.dk, a.dv, dqacc, a.B,
                                                                     a.Hq, a.Hkv, a.N, p, a.s);
  } else {
    const auto e = reinterpret_cast<fa::EncodeTiledFnBwd>(enc);
    CUtensorMap tq, tk, tv, tdo, tdk, tdv, tdq;
    launched = fa::bwd_map(e, &tq, a.q, false, D, a.N, hq, 64, BQ) && fa::bwd_map(e, &tdo, a.dout, false, D, a.N, hq, 64, BQ) &&
               fa::bwd_map(e, &tk, a.k, false, D, a.N, hkv, 64, 128) && fa::bwd_map(e, &tv, a.v, false, D, a.N, hkv, 64, 128) &&
               fa::bwd_map(e, &tdk, a.dk, false, D, a.N, hkv, 64, 128) && fa::bwd_map(e, &tdv, a.dv, false, D, a.N, hkv, 64, 128) &&
               fa::bwd_map(e, &tdq, dqacc, true, D, a.N, hq, L::kDQCols, BQ);
    const unsigned grid = static_cast<unsigned>(a.B) * a.Hkv * p.nkb * (D / DH) * (max_parts > 0 ? max_parts : 1);
    if (launched && max_parts > 0 && far)
      fa::bwd_launch_main<D, DH, BQ, fa::kAttnScorePartsFar>(tq, tk, tv, tdo, tdk, tdv, tdq, p, grid, a.s);
    else if (launched && max_parts > 0)
      fa::bwd_launch_main<D, DH, BQ, fa::kAttnScoreParts>(tq, tk, tv, tdo, tdk, tdv, tdq, p, grid, a.s);
    else if (launched && far)
      fa::bwd_launch_main<D, DH, BQ, fa::kAttnScoreFar>(tq, tk, tv, tdo, tdk, tdv, tdq, p, grid, a.s);
    else if (launched)
      fa::bwd_launch_main<D, DH, BQ, fa::kAttnScore>(tq, tk, tv, tdo, tdk, tdv, tdq, p, grid, a.s);
  }
  timer_stop(1, tslot, a.s);
  if (!launched) return FA_ERR_CUDA;
  const long long n8 = rows * D / 8;
  if (max_parts > 0) {
    const long long ctas = (n8 + 255) / 256 + hkv * p.nkb * (D / 8);
    fa::fa_bwd_join_kernel<D><<<static_cast<unsigned>(ctas), 256, 0, a.s>>>(
        dqacc, static_cast<__nv_bfloat16 *>(a.dq), reinterpret_cast<const float4 *>(p.parts), parts,
        static_cast<__nv_bfloat16 *>(a.dk), static_cast<__nv_bfloat16 *>(a.dv), a.scale, static_cast<int>(hkv), a.Hkv, a.N,
        p.nkb, n8);
    return cuda_ok(cudaGetLastError(), "fa_bwd_score launch") ? FA_OK : FA_ERR_CUDA;
  }
  fa::fa_bwd_post_kernel<<<static_cast<unsigned>((n8 + 255) / 256), 256, 0, a.s>>>(
      dqacc, static_cast<__nv_bfloat16 *>(a.dq), wide ? a.scale / fa::kGradUp : a.scale, n8);
  return cuda_ok(cudaGetLastError(), "fa_bwd_score launch") ? FA_OK : FA_ERR_CUDA;
}

// ---- decode with more rows per K/V head than the pieces take

template <int D, int RP>
void launch_decode(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const fa::DecodeParams &p,
                   unsigned grid, cudaStream_t s) {
  constexpr int smem = fa::DecodeLayout<D, RP>::kSmemBytes;
  if (far_cap(p.score)) fa::fa_decode_kernel<D, RP, true, true><<<grid, fa::kDecodeThreads, smem, s>>>(tq, tk, tv, p);
  else fa::fa_decode_kernel<D, RP, true><<<grid, fa::kDecodeThreads, smem, s>>>(tq, tk, tv, p);
}

template <int D>
void launch_decode_d(int RP, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                     const fa::DecodeParams &p, unsigned grid, cudaStream_t s) {
  if constexpr (D == 256) {
    if (RP == 16) launch_decode<D, 16>(tq, tk, tv, p, grid, s);
  }
  if (RP == 32) launch_decode<D, 32>(tq, tk, tv, p, grid, s);
  else if (RP == 64) launch_decode<D, 64>(tq, tk, tv, p, grid, s);
  else if constexpr (D != 256) {
    if (RP == 128) launch_decode<D, 128>(tq, tk, tv, p, grid, s);
  }
}

// fa_decode's tcgen05 kernel with changed scores.
int run_decode(const void *q, const void *k, const void *v, void *o, float *lse, const int *seqlens_k,
               void *workspace, size_t workspace_bytes, int B, int Hq, int Hkv, int Nq, int Nk, int d,
               int causal, int num_splits, float scale, void *stream, const fa::ScoreCfg &score) {
  if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
  if (num_splits < 1 || num_splits > kMaxDecodeSplits) return FA_ERR_INVALID_ARG;
  int rc = check_decode_sizes(B, Hq, Hkv, Nq, Nk, d, scale);
  if (rc != FA_OK) return rc;
  if (static_cast<long long>(B) * Hkv * num_splits >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  const size_t need = decode_workspace(B, Hq, Nq, d, num_splits);
  if (need > 0 && (!workspace || workspace_bytes < need)) return FA_ERR_WORKSPACE;
  const void *ptrs[] = {q, k, v, o, lse};
  for (const void *ptr : ptrs)
    if (!aligned16(ptr)) return FA_ERR_ALIGN;
  if ((need > 0 && !aligned16(workspace)) || (reinterpret_cast<uintptr_t>(seqlens_k) & 3u)) return FA_ERR_ALIGN;
  if (!score_ready()) return FA_ERR_CUDA;

  const int g = Hq / Hkv, R = g * Nq, RP = decode_rows_padded(R);
  CUtensorMap tq, tk, tv;
  // Q viewed as [B * Hkv][R][d]: the rows of the query heads that share a K/V head.
  if (!make_map_bf16(&tq, q, d, R, static_cast<long long>(B) * Hkv, RP) ||
      !make_map_bf16(&tk, k, d, Nk, static_cast<long long>(B) * Hkv, 128) ||
      !make_map_bf16(&tv, v, d, Nk, static_cast<long long>(B) * Hkv, 128)) {
    if (debug_enabled()) std::fprintf(stderr, "[fa] cuTensorMapEncodeTiled failed (fa_decode)\n");
    return FA_ERR_CUDA;
  }
  const size_t rows = static_cast<size_t>(B) * Hq * Nq;
  fa::DecodeParams p;
  p.lens = seqlens_k;
  p.o = static_cast<__nv_bfloat16 *>(o);
  p.lse = lse;
  p.o_part = num_splits > 1 ? static_cast<float *>(workspace) : nullptr;
  p.lse_part = num_splits > 1
                   ? reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                               fa::pad256(static_cast<size_t>(num_splits) * rows * d * 4))
                   : nullptr;
  p.B = B;
  p.Hkv = Hkv;
  p.Nq = Nq;
  p.Nk = Nk;
  p.R = R;
  p.splits = num_splits;
  const int per = (Nk + num_splits - 1) / num_splits;
  p.chunk = (per + 127) / 128 * 128;
  p.causal = causal;
  p.sl2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.score = score;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(B) * Hkv * num_splits;
  const int tslot = timer_start(2, s);
  if (d == 64) launch_decode_d<64>(RP, tq, tk, tv, p, grid, s);
  else if (d == 128) launch_decode_d<128>(RP, tq, tk, tv, p, grid, s);
  else launch_decode_d<256>(RP, tq, tk, tv, p, grid, s);
  timer_stop(2, tslot, s);
  if (num_splits > 1) launch_merge(p.o_part, p.lse_part, o, lse, num_splits, static_cast<long long>(rows), d, s);
  return cuda_ok(cudaGetLastError(), "fa_decode launch") ? FA_OK : FA_ERR_CUDA;
}

// ---- the 4-bit cache

int check_kv4_sizes(int B, int Hkv, int cap, int d) {
  if (B < 1 || Hkv < 1 || cap < 1) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128 && d != 256) return FA_ERR_UNSUPPORTED;
  if (cap % fa::kKV4CapMultiple != 0 || cap > (1 << 30) || static_cast<long long>(B) * Hkv * cap >= (1ll << 31))
    return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

int check_kv4_decode(int B, int Hq, int Hkv, int Nq, int cap, int d, float scale) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Nq < 1) return FA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  int rc = check_kv4_sizes(B, Hkv, cap, d);
  if (rc != FA_OK) return rc;
  if (Hq % Hkv != 0) return FA_ERR_GQA;
  if (static_cast<long long>(Hq / Hkv) * Nq > 128 || static_cast<long long>(B) * Hq * Nq >= (1ll << 31))
    return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// 8-row tiles of query rows that one CTA takes together.
int line_row_tiles(int R, int d) { return R > 8 && d != 256 ? 2 : 1; }

// Writes (store) or reads n tokens of the cache.
int run_kv4_copy(bool store, fa::KV4Params &p, int d, cudaStream_t s) {
  const long long rows = static_cast<long long>(p.B) * p.Hkv * p.n;  // below 2^31
  if (store) {  // a thread per token and group of 32 channels, of K and of V
    const unsigned gr = static_cast<unsigned>((2 * rows * (d / fa::kKV4Group) + 255) / 256);
    if (d == 64) fa::fa_kv4_write_kernel<64><<<gr, 256, 0, s>>>(p);
    else if (d == 128) fa::fa_kv4_write_kernel<128><<<gr, 256, 0, s>>>(p);
    else fa::fa_kv4_write_kernel<256><<<gr, 256, 0, s>>>(p);
  } else {  // a thread per word of 8 channels of four tokens; K and V in y
    const int per = 256 / (d / 8) * fa::kKV4ReadTokens;
    const dim3 gr(static_cast<unsigned>((rows + per - 1) / per), 2);
    if (d == 64) fa::fa_kv4_read_kernel<64><<<gr, 256, 0, s>>>(p);
    else if (d == 128) fa::fa_kv4_read_kernel<128><<<gr, 256, 0, s>>>(p);
    else fa::fa_kv4_read_kernel<256><<<gr, 256, 0, s>>>(p);
  }
  return cuda_ok(cudaGetLastError(), store ? "fa_kv4_write launch" : "fa_kv4_read launch") ? FA_OK : FA_ERR_CUDA;
}

// Scratch for the partial results of `pieces` pieces (fa_decode_line.cuh).
size_t line_workspace(int R, int d, int pieces) {
  return pieces > 1 ? fa::pad256(static_cast<size_t>(pieces) * 2 * 8 * line_row_tiles(R, d) * (d + 2) * 4) : 0;
}

// One piece per CTA that fits on the current device at once, but no more than there are blocks.
int line_pieces(int B, int Hkv, int R, int cap, int d, int block, int ctas_per_sm) {
  int sms = 148, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) {
    (void)cudaGetLastError();
    sms = 148;
  }
  const int rows = 8 * line_row_tiles(R, d);
  const long long slots = static_cast<long long>(sms) * ctas_per_sm;
  const long long blocks = static_cast<long long>(B) * Hkv * ((R + rows - 1) / rows) * ((cap + block - 1) / block);
  const long long s = blocks < slots ? blocks : slots;
  return static_cast<int>(s < kMaxDecodeSplits ? s : kMaxDecodeSplits);
}

// The joining kernel, launched while the pieces are computed (it waits for them itself).
template <int D, int KB>
bool launch_line_merge_d(const fa::LineParams &p, int tile_rows, cudaStream_t s) {
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.B) * p.Hkv * p.R);  // rows, below 2^31
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cuda_ok(cudaLaunchKernelEx(&cfg, fa::fa_line_merge_kernel<D, KB>, p, tile_rows), "fa_line_merge launch");
}

template <int KB64, int KB128, int KB256>
bool launch_line_merge(const fa::LineParams &p, int d, cudaStream_t s) {
  const int tile_rows = 8 * line_row_tiles(p.R, d);
  if (d == 64) return launch_line_merge_d<64, KB64>(p, tile_rows, s);
  if (d == 128) return launch_line_merge_d<128, KB128>(p, tile_rows, s);
  return launch_line_merge_d<256, KB256>(p, tile_rows, s);
}

// What a line of blocks needs besides the cache: sizes, lengths, scores, results.
void fill_line(fa::LineParams &p, const void *q, void *o, float *lse, const int *lens, const float *slopes,
               void *workspace, int B, int Hq, int Hkv, int Nq, int cap, int d, int causal, int pieces, float softcap,
               float scale) {
  p.q = static_cast<const __nv_bfloat16 *>(q);
  p.lens = lens;
  p.slopes = slopes;
  p.o = static_cast<__nv_bfloat16 *>(o);
  p.lse = lse;
  p.part = static_cast<float *>(workspace);
  p.B = B;
  p.Hkv = Hkv;
  p.Nq = Nq;
  p.R = Hq / Hkv * Nq;
  p.cap = cap;
  const int tile_rows = 8 * line_row_tiles(p.R, d);
  p.row_tiles = (p.R + tile_rows - 1) / tile_rows;
  p.pieces = pieces;
  p.causal = causal;
  p.scale = scale;
  p.sl2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.softcap = usable_cap(softcap);
}

// Decode with changed scores: rows per K/V head up to which the pieces of fa_decode_score.cuh
// serve it.  Beyond, a second tile of rows would read the cache again, and the tcgen05 kernel,
// which takes up to 128 rows at once, is used with its fixed key ranges.
bool score_in_pieces(int R, int d) { return R <= (d == 256 ? 8 : 16); }
constexpr int score_block(int d) { return d == 256 ? fa::DecScoreLayout<256, 1>::kBlock : fa::DecScoreLayout<128, 1>::kBlock; }

template <int D, int NT>
void launch_score_d(const CUtensorMap &tk, const CUtensorMap &tv, const fa::LineParams &p, cudaStream_t s) {
  using L = fa::DecScoreLayout<D, NT>;
  static_assert(L::kBlock == score_block(D), "block");
  fa::fa_decode_score_kernel<D, NT><<<static_cast<unsigned>(p.pieces), L::W * 32, L::kSmemBytes, s>>>(tk, tv, p);
}

template <int D, int NT>
void launch_kv4(const fa::KV4DecodeParams &p, cudaStream_t s) {
  constexpr int smem = fa::KV4Layout<D, NT>::kSmemBytes;
  const unsigned grid = static_cast<unsigned>(p.pieces);
  if (p.softcap > 0.f || p.slopes)
    fa::fa_decode_kv4_kernel<D, NT, true><<<grid, fa::kKV4Warps * 32, smem, s>>>(p);
  else
    fa::fa_decode_kv4_kernel<D, NT, false><<<grid, fa::kKV4Warps * 32, smem, s>>>(p);
}

}  // namespace

namespace fa_host {
int take_score_status() {
  int status = 0, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices || !g_score_dev[dev].ready.load()) return FA_OK;  // no kernel of this unit has run
  if (cudaMemcpyFromSymbol(&status, fa::g_fa_status, sizeof(int)) != cudaSuccess) return FA_ERR_CUDA;
  if (status != FA_OK) {
    const int zero = 0;
    const unsigned long long zero64 = 0;
    if (cudaMemcpyToSymbol(fa::g_fa_status, &zero, sizeof(int)) != cudaSuccess ||
        cudaMemcpyToSymbol(fa::g_fa_status_site, &zero64, sizeof(zero64)) != cudaSuccess)
      return FA_ERR_CUDA;
  }
  return status;
}
}  // namespace fa_host

extern "C" {

int fa_fwd_score(const void *q, const void *k, const void *v, void *o, float *lse, const float *alibi_slopes,
                 const int *key_range, int B, int Hq, int Hkv, int N, int d, int causal, float softcap, float scale,
                 void *stream) {
  if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
  int rc = check_sizes(B, Hq, Hkv, N, d, scale);
  if (rc == FA_OK) rc = check_score_args(softcap, alibi_slopes);
  if (rc != FA_OK) return rc;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse) ||
      (reinterpret_cast<uintptr_t>(key_range) & 7u))
    return FA_ERR_ALIGN;
  if (!score_ready()) return FA_ERR_CUDA;
  const int kv_rows = d == 256 ? 64 : 128;
  CUtensorMap tq, tk, tv, to;
  if (!make_map_bf16(&tq, q, d, N, static_cast<long long>(B) * Hq, 128) ||
      !make_map_bf16(&tk, k, d, N, static_cast<long long>(B) * Hkv, kv_rows) ||
      !make_map_bf16(&tv, v, d, N, static_cast<long long>(B) * Hkv, kv_rows) ||
      !make_map_bf16(&to, o, d, N, static_cast<long long>(B) * Hq, 128))
    return FA_ERR_CUDA;
  fa::FwdParams p{};
  p.lse = lse;
  p.o = static_cast<__nv_bfloat16 *>(o);
  p.cu_q = p.cu_k = nullptr;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.N = N;
  p.total_q = p.total_k = 0;
  p.nqb = (N + 127) / 128;
  p.left = p.right = -1;
  p.sl2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.score = make_score(softcap, alibi_slopes, key_range, causal, scale);
  // Blocks go level by level (the key ranges, not the position, decide what is heavy).
  const int g = Hq / Hkv;
  p.tail = 0;
  p.tsz = 1;
  p.drop = fa::DropCfg{};
  p.bmask = nullptr;
  p.pair_heads = d != 256 && g % 2 == 0 ? 1 : 0;
  const unsigned units = d == 256 ? static_cast<unsigned>(B) * Hq * p.nqb
                                  : p.pair_heads ? static_cast<unsigned>(B) * (Hq / 2) * p.nqb
                                                 : static_cast<unsigned>(B) * Hq * ((p.nqb + 1) / 2);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int tslot = timer_start(0, s);
  if (d == 64) launch_fwd_score<64>(tq, tk, tv, to, p, units, s);
  else if (d == 128) launch_fwd_score<128>(tq, tk, tv, to, p, units, s);
  else launch_fwd_score<256>(tq, tk, tv, to, p, units, s);
  const bool launched = cuda_ok(cudaGetLastError(), "fa_fwd_score launch");
  timer_stop(0, tslot, s);
  return launched ? FA_OK : FA_ERR_CUDA;
}

size_t fa_bwd_score_workspace_bytes(int B, int Hq, int Hkv, int N, int d) {
  if (check_sizes(B, Hq, Hkv, N, d, 1.0f) != FA_OK) return 0;
  return fa::bwd_workspace_bytes(B, Hq, N, d) + fa::pad256(static_cast<size_t>(B) * ((N + 127) / 128) * 8) +
         fa::pad256(fa::plan_layout(B, Hkv, N, d, fa::plan_max_parts(B, Hkv, N, d)).total);
}

int fa_bwd_score(const void *q, const void *k, const void *v, const void *o, const float *lse, const void *dout,
                 void *dq, void *dk, void *dv, void *workspace, size_t workspace_bytes, const float *alibi_slopes,
                 const int *key_range, int B, int Hq, int Hkv, int N, int d, int causal, float softcap, float scale,
                 void *stream) {
  if (!q || !k || !v || !o || !lse || !dout || !dq || !dk || !dv) return FA_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
  int rc = check_sizes(B, Hq, Hkv, N, d, scale);
  if (rc == FA_OK) rc = check_score_args(softcap, alibi_slopes);
  if (rc == FA_OK) rc = check_score_bwd(N, d);
  if (rc != FA_OK) return rc;
  if (!workspace || workspace_bytes < fa_bwd_score_workspace_bytes(B, Hq, Hkv, N, d)) return FA_ERR_WORKSPACE;
  const void *ptrs[] = {q, k, v, o, lse, dout, dq, dk, dv, workspace};
  for (const void *ptr : ptrs)
    if (!aligned16(ptr)) return FA_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(key_range) & 7u) return FA_ERR_ALIGN;
  if (!score_ready()) return FA_ERR_CUDA;
  const BwdScoreArgs a{q, k, v, o, lse, dout, dq, dk, dv, workspace, B, Hq, Hkv, N, causal ? 0 : -1, scale,
                       make_score(softcap, alibi_slopes, key_range, causal, scale), static_cast<cudaStream_t>(stream)};
  if (d == 64) return launch_bwd_score<64, 64, 64>(a);
  if (d == 128) return launch_bwd_score<128, 128, 64>(a);
  return launch_bwd_score<256, 128, 64>(a);
}

int fa_decode_score_num_splits(int B, int Hq, int Hkv, int Nq, int Nk, int d) {
  if (check_decode_sizes(B, Hq, Hkv, Nq, Nk, d, 1.0f) != FA_OK) return 0;
  const int R = Hq / Hkv * Nq;
  if (!score_in_pieces(R, d)) return fa_decode_num_splits(B, Hq, Hkv, Nq, Nk, d);
  return line_pieces(B, Hkv, R, Nk, d, score_block(d), 1);
}

size_t fa_decode_score_workspace_bytes(int B, int Hq, int Hkv, int Nq, int Nk, int d, int num_splits) {
  if (check_decode_sizes(B, Hq, Hkv, Nq, Nk, d, 1.0f) != FA_OK) return 0;
  if (num_splits < 1 || num_splits > kMaxDecodeSplits) return 0;
  const int R = Hq / Hkv * Nq;
  return score_in_pieces(R, d) ? line_workspace(R, d, num_splits) : decode_workspace(B, Hq, Nq, d, num_splits);
}

int fa_decode_score(const void *q, const void *k, const void *v, void *o, float *lse, const int *seqlens_k,
                    const float *alibi_slopes, void *workspace, size_t workspace_bytes, int B, int Hq, int Hkv,
                    int Nq, int Nk, int d, int causal, int num_splits, float softcap, float scale, void *stream) {
  if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
  if (num_splits < 1 || num_splits > kMaxDecodeSplits) return FA_ERR_INVALID_ARG;
  int rc = check_decode_sizes(B, Hq, Hkv, Nq, Nk, d, scale);
  if (rc == FA_OK) rc = check_score_args(softcap, alibi_slopes);
  if (rc != FA_OK) return rc;
  const int R = Hq / Hkv * Nq;
  if (!score_in_pieces(R, d)) {
    const fa::ScoreCfg score = make_score(softcap, alibi_slopes, nullptr, causal, scale);
    return run_decode(q, k, v, o, lse, seqlens_k, workspace, workspace_bytes, B, Hq, Hkv, Nq, Nk, d, causal, num_splits,
                      scale, stream, score);
  }
  const size_t need = line_workspace(R, d, num_splits);
  if (need > 0 && (!workspace || workspace_bytes < need)) return FA_ERR_WORKSPACE;
  const void *ptrs[] = {q, k, v, o, lse};
  for (const void *ptr : ptrs)
    if (!aligned16(ptr)) return FA_ERR_ALIGN;
  if ((need > 0 && !aligned16(workspace)) || (reinterpret_cast<uintptr_t>(seqlens_k) & 3u)) return FA_ERR_ALIGN;
  if (!score_ready()) return FA_ERR_CUDA;
  CUtensorMap tk, tv;
  if (!make_map_bf16(&tk, k, d, Nk, static_cast<long long>(B) * Hkv, score_block(d)) ||
      !make_map_bf16(&tv, v, d, Nk, static_cast<long long>(B) * Hkv, score_block(d))) {
    if (debug_enabled()) std::fprintf(stderr, "[fa] cuTensorMapEncodeTiled failed (fa_decode_score)\n");
    return FA_ERR_CUDA;
  }
  fa::LineParams p{};
  fill_line(p, q, o, lse, seqlens_k, alibi_slopes, workspace, B, Hq, Hkv, Nq, Nk, d, causal, num_splits, softcap, scale);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool two = line_row_tiles(R, d) == 2;
  const int tslot = timer_start(2, s);
  if (d == 64) two ? launch_score_d<64, 2>(tk, tv, p, s) : launch_score_d<64, 1>(tk, tv, p, s);
  else if (d == 128) two ? launch_score_d<128, 2>(tk, tv, p, s) : launch_score_d<128, 1>(tk, tv, p, s);
  else launch_score_d<256, 1>(tk, tv, p, s);
  timer_stop(2, tslot, s);
  bool joined = true;
  if (num_splits > 1 && Nk > score_block(d))  // segments of one block are never shared
    joined = launch_line_merge<score_block(64), score_block(128), score_block(256)>(p, d, s);
  return cuda_ok(cudaGetLastError(), "fa_decode_score launch") && joined ? FA_OK : FA_ERR_CUDA;
}

int fa_kv4_write(const void *k, const void *v, void *k_codes, void *k_params, void *v_codes, void *v_params,
                 const int *start, const int *counts, int B, int Hkv, int n, int cap, int d, void *stream) {
  if (!k || !v || !k_codes || !k_params || !v_codes || !v_params || n < 0) return FA_ERR_INVALID_ARG;
  int rc = check_kv4_sizes(B, Hkv, cap, d);
  if (rc != FA_OK) return rc;
  if (n > cap) return FA_ERR_UNSUPPORTED;
  const void *ptrs[] = {k, v, k_codes, k_params, v_codes, v_params};
  for (const void *ptr : ptrs)
    if (!aligned16(ptr)) return FA_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(start) & 3u) || (reinterpret_cast<uintptr_t>(counts) & 3u)) return FA_ERR_ALIGN;
  if (!score_ready()) return FA_ERR_CUDA;
  if (n == 0) return FA_OK;
  fa::KV4Params p{};
  p.kc = static_cast<uint8_t *>(k_codes);
  p.vc = static_cast<uint8_t *>(v_codes);
  p.kp = static_cast<__half *>(k_params);
  p.vp = static_cast<__half *>(v_params);
  p.k = static_cast<__nv_bfloat16 *>(const_cast<void *>(k));
  p.v = static_cast<__nv_bfloat16 *>(const_cast<void *>(v));
  p.start = start;
  p.counts = counts;
  p.B = B;
  p.Hkv = Hkv;
  p.n = n;
  p.cap = cap;
  return run_kv4_copy(true, p, d, static_cast<cudaStream_t>(stream));
}

int fa_kv4_read(const void *k_codes, const void *k_params, const void *v_codes, const void *v_params, void *k,
                void *v, const int *start, int B, int Hkv, int n, int cap, int d, void *stream) {
  if (!k || !v || !k_codes || !k_params || !v_codes || !v_params || n < 0) return FA_ERR_INVALID_ARG;
  int rc = check_kv4_sizes(B, Hkv, cap, d);
  if (rc != FA_OK) return rc;
  if (n > cap) return FA_ERR_UNSUPPORTED;
  const void *ptrs[] = {k, v, k_codes, k_params, v_codes, v_params};
  for (const void *ptr : ptrs)
    if (!aligned16(ptr)) return FA_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(start) & 3u) return FA_ERR_ALIGN;
  if (!score_ready()) return FA_ERR_CUDA;
  if (n == 0) return FA_OK;
  fa::KV4Params p{};
  p.kc = static_cast<uint8_t *>(const_cast<void *>(k_codes));
  p.vc = static_cast<uint8_t *>(const_cast<void *>(v_codes));
  p.kp = static_cast<__half *>(const_cast<void *>(k_params));
  p.vp = static_cast<__half *>(const_cast<void *>(v_params));
  p.k = static_cast<__nv_bfloat16 *>(k);
  p.v = static_cast<__nv_bfloat16 *>(v);
  p.start = start;
  p.B = B;
  p.Hkv = Hkv;
  p.n = n;
  p.cap = cap;
  return run_kv4_copy(false, p, d, static_cast<cudaStream_t>(stream));
}

int fa_decode_kv4_num_splits(int B, int Hq, int Hkv, int Nq, int cap, int d) {
  if (check_kv4_decode(B, Hq, Hkv, Nq, cap, d, 1.0f) != FA_OK) return 0;
  const int R = Hq / Hkv * Nq;
  // two CTAs an SM up to 8 rows and d = 128
  return line_pieces(B, Hkv, R, cap, d, fa::kKV4Block, line_row_tiles(R, d) == 1 && d <= 128 ? 2 : 1);
}

size_t fa_decode_kv4_workspace_bytes(int B, int Hq, int Hkv, int Nq, int cap, int d, int num_splits) {
  if (check_kv4_decode(B, Hq, Hkv, Nq, cap, d, 1.0f) != FA_OK) return 0;
  if (num_splits < 1 || num_splits > kMaxDecodeSplits) return 0;
  return line_workspace(Hq / Hkv * Nq, d, num_splits);
}

int fa_decode_kv4(const void *q, const void *k_codes, const void *k_params, const void *v_codes, const void *v_params,
                  void *o, float *lse, const int *seqlens_k, const float *alibi_slopes, void *workspace,
                  size_t workspace_bytes, int B, int Hq, int Hkv, int Nq, int cap, int d, int causal, int num_splits,
                  float softcap, float scale, void *stream) {
  if (!q || !k_codes || !k_params || !v_codes || !v_params || !o || !lse) return FA_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
  if (num_splits < 1 || num_splits > kMaxDecodeSplits) return FA_ERR_INVALID_ARG;
  int rc = check_kv4_decode(B, Hq, Hkv, Nq, cap, d, scale);
  if (rc == FA_OK) rc = check_score_args(softcap, alibi_slopes);
  if (rc != FA_OK) return rc;
  const size_t need = line_workspace(Hq / Hkv * Nq, d, num_splits);
  if (need > 0 && (!workspace || workspace_bytes < need)) return FA_ERR_WORKSPACE;
  const void *ptrs[] = {q, k_codes, k_params, v_codes, v_params, o, lse};
  for (const void *ptr : ptrs)
    if (!aligned16(ptr)) return FA_ERR_ALIGN;
  if ((need > 0 && !aligned16(workspace)) || (reinterpret_cast<uintptr_t>(seqlens_k) & 3u)) return FA_ERR_ALIGN;
  if (!score_ready()) return FA_ERR_CUDA;

  fa::KV4DecodeParams p{};
  fill_line(p, q, o, lse, seqlens_k, alibi_slopes, workspace, B, Hq, Hkv, Nq, cap, d, causal, num_splits, softcap, scale);
  p.kc = static_cast<const uint8_t *>(k_codes);
  p.vc = static_cast<const uint8_t *>(v_codes);
  p.kp = static_cast<const __half *>(k_params);
  p.vp = static_cast<const __half *>(v_params);
  const bool two = line_row_tiles(p.R, d) == 2;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int tslot = timer_start(2, s);
  if (d == 64) two ? launch_kv4<64, 2>(p, s) : launch_kv4<64, 1>(p, s);
  else if (d == 128) two ? launch_kv4<128, 2>(p, s) : launch_kv4<128, 1>(p, s);
  else launch_kv4<256, 1>(p, s);
  timer_stop(2, tslot, s);
  bool joined = true;
  if (num_splits > 1 && cap > fa::kKV4Block)  // segments of one block are never shared
    joined = launch_line_merge<fa::kKV4Block, fa::kKV4Block, fa::kKV4Block>(p, d, s);
  return cuda_ok(cudaGetLastError(), "fa_decode_kv4 launch") && joined ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
