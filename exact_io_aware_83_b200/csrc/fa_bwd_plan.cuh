// fa_bwd_plan.cuh - parts of key blocks, for a backward with changed scores that has fewer units
// (b, K/V head, key block, d half) than the GPU has SMs.
//
// A key block's CTA walks every (query head of the group, query block) that sees the block, one
// step after the other.  With few key blocks most SMs stay idle, and the few steps that key
// ranges or a causal mask leave are spread unevenly.  So a plan is made on the device, from the
// spans of the query blocks:
//   T_e    steps of key block e = (batch entry, 128 keys), the same for every K/V head;
//   cut    each key block into ceil(T_e / c) parts of (nearly) equal numbers of steps, for one
//          length c = ceil(max T / s), s = 1 .. max_parts, the same for all; every part is a CTA
//          of its own, and its dK and dV go to fp32 buffers that fa_bwd_join_kernel adds up
//          in the order of the parts (a key block in one part is written as bf16 at once);
//   choose the s whose estimated time is smallest: a part costs its steps and part_steps more
//          (K, V, the pipeline's start, the epilogue, the sums), the parts share the SMs evenly,
//          and the last one runs on for half a part; or the longest part alone when all fit at once;
//   order  the parts by length, longest first.
// Calls in a graph, us, without and with it: B = 2, Hq = 6, Hkv = 2, N = 1000, d = 64, prefixes
// and slopes 94 and 32; B = 1, Hq = 8, Hkv = 1, N = 4096, d = 128, causal, cap 50, 991 and 160;
// B = 1, H = 4, N = 4096, d = 128, prefixes and slopes, 135 and 99.  With more units it is left
// out: cutting cost more than it levelled (B = 2, H = 4, N = 4096, d = 128, documents of 400
// rows: 70 us whole, 91 in halves), and the order alone gave up the locality of a head's key
// blocks (B = 4, Hq = 32, Hkv = 8, N = 4096, documents of 500 rows: 697 us in unit_order's order,
// 781 longest first).
#pragma once

#include "fa_bwd.cuh"

namespace fa {

constexpr int kPlanMaxParts = 8;
constexpr int kPlanSMs = 148;
constexpr int kPlanThreads = 1024;

// Parts a key block may have (enough CTAs for four rounds on all SMs), or 0: no plan.
inline int plan_max_parts(int B, int Hkv, int N, int d) {
  const long long units = static_cast<long long>(B) * Hkv * ((N + 127) / 128) * (d == 256 ? 2 : 1);
  if (units >= kPlanSMs) return 0;
  const int s = static_cast<int>(4 * kPlanSMs / units);
  return s > kPlanMaxParts ? kPlanMaxParts : s;
}

struct PlanLayout {  // byte offsets behind the spans of the query blocks
  size_t parts, items, sums, total;
};

inline PlanLayout plan_layout(int B, int Hkv, int N, int d, int max_parts) {
  const size_t entries = max_parts > 0 ? static_cast<size_t>(B) * ((N + 127) / 128) : 0;
  PlanLayout l;
  l.parts = 0;
  l.items = pad256(entries * 4);
  l.sums = l.items + pad256(entries * 16 * max_parts);
  l.total = l.sums + entries * 128 * max_parts * Hkv * d * 8;
  return l;
}

// Blocks of fa_bwd_front_kernel that come before those of the rows.
__host__ __device__ inline int front_blocks(bool plan, int B, int nkb) {
  return plan ? 1 : static_cast<int>((static_cast<long long>(B) * nkb + kPlanThreads / 32 - 1) / (kPlanThreads / 32));
}

struct PlanParams {
  ScoreCfg cfg;
  int B, N, nkb, g;     // g: query heads per K/V head
  int nsub, nsub_last;  // steps per 128-row query block and in the last one
  int heads;            // CTAs per part: K/V heads, times the halves of d = 256
  int max_parts, part_steps;
  int2 *blocks;
  int *parts;
  int4 *items;
};

// The plan, by one CTA; B nkb < kPlanSMs.  Writes the spans of the query blocks, the parts of each
// key block and max_parts B nkb items, those behind the last part with no parts.
__device__ __forceinline__ void bwd_plan(const PlanParams &p) {
  const ScoreCfg &cfg = p.cfg;
  const int B = p.B, N = p.N, nkb = p.nkb, g = p.g, nsub = p.nsub, nsub_last = p.nsub_last, heads = p.heads;
  const int max_parts = p.max_parts, part_steps = p.part_steps;
  int2 *blocks = p.blocks;
  int *parts = p.parts;
  int4 *items = p.items;
  __shared__ int2 span[kPlanSMs];
  __shared__ int steps[kPlanSMs];
  __shared__ float cost[kPlanMaxParts];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = kPlanThreads / 32;
  const int entries = B * nkb;
  for (int e = warp; e < entries; e += warps) {
    const int b = e / nkb, qb = e - b * nkb;
    const int2 r = score_block_span(cfg, b, qb, N, lane);
    if (lane == 0) blocks[e] = span[e] = r;
  }
  __syncthreads();
  for (int e = warp; e < entries; e += warps) {
    const int b = e / nkb, kb = e - b * nkb;
    int n = 0;
    for (int qb = lane; qb < nkb; qb += 32) {
      const int2 r = span[b * nkb + qb];
      if ((!cfg.causal || qb >= kb) && r.x < kb * 128 + 128 && r.y > kb * 128) n += qb == nkb - 1 ? nsub_last : nsub;
    }
    n = __reduce_add_sync(0xffffffffu, n) * g;
    if (lane == 0) steps[e] = n;
  }
  __syncthreads();
  int most = 1;
  for (int e = lane; e < entries; e += 32) most = max(most, steps[e]);
  most = __reduce_max_sync(0xffffffffu, most);
  if (warp < max_parts) {
    const int c = (most + warp) / (warp + 1);
    int n = 0, total = 0;
    for (int e = lane; e < entries; e += 32) {
      n += max(1, (steps[e] + c - 1) / c);
      total += steps[e];
    }
    n = __reduce_add_sync(0xffffffffu, n) * heads;
    total = __reduce_add_sync(0xffffffffu, total);
    if (lane == 0)
      cost[warp] = n <= kPlanSMs ? static_cast<float>(c + part_steps)
                                 : (static_cast<float>(total) * heads + static_cast<float>(part_steps) * n) / kPlanSMs + 0.5f * c;
  }
  __syncthreads();
  int s = 0;
  for (int i = 1; i < max_parts; ++i)
    if (cost[i] < cost[s]) s = i;
  const int c = (most + s) / (s + 1);
  for (int e = warp; e < entries; e += warps) {
    const int n = max(1, (steps[e] + c - 1) / c), len = steps[e] / n, b = e / nkb;
    int at = 0, all = 0;  // parts before this block's, and all of them
    for (int f = lane; f < entries; f += 32) {
      const int m = max(1, (steps[f] + c - 1) / c), other = steps[f] / m;
      all += m;
      at += other > len || (other == len && f < e) ? m : 0;
    }
    at = __reduce_add_sync(0xffffffffu, at);
    all = __reduce_add_sync(0xffffffffu, all);
    if (lane < n) items[at + lane] = make_int4(e - b * nkb, b, lane, n);
    if (lane == 0) parts[e] = n;
    if (e == 0)
      for (int i = all + lane; i < entries * max_parts; i += 32) items[i] = make_int4(0, 0, 0, 0);
  }
}

// The first kernel of a backward with a plan or with key ranges.  The first blocks make the plan
// (one block) or, without one, find the spans of the query blocks (a warp each); the others do
// what fa_bwd_pre_kernel does (Delta_i = <dO_i, O_i>, a zeroed dQ accumulator), a warp per row.
// (One after the other, plan and rows took 4 and 8 us and a launch more.)
template <int D, bool PLAN>
static __global__ void __launch_bounds__(kPlanThreads, 2)
    fa_bwd_front_kernel(const PlanParams plan, const __nv_bfloat16 *__restrict__ o, const __nv_bfloat16 *__restrict__ dout,
                       float *__restrict__ delta, float *__restrict__ dqacc, long long rows) {
  constexpr int kWarps = kPlanThreads / 32;
  const int lane = threadIdx.x % 32, front = front_blocks(PLAN, plan.B, plan.nkb);
  const long long row = static_cast<long long>(static_cast<int>(blockIdx.x) - front) * kWarps + threadIdx.x / 32;
  if (row < 0) {
    if constexpr (PLAN) {
      bwd_plan(plan);
    } else {
      const int e = static_cast<int>(blockIdx.x) * kWarps + static_cast<int>(threadIdx.x / 32), b = e / plan.nkb;
      if (b < plan.B) {
        const int2 r = score_block_span(plan.cfg, b, e - b * plan.nkb, plan.N, lane);
        if (lane == 0) plan.blocks[e] = r;
      }
    }
    return;
  }
  constexpr int kPairs = D / 64;  // bf16 pairs per lane
  if (row >= rows) return;
  const __nv_bfloat162 *orow = reinterpret_cast<const __nv_bfloat162 *>(o + row * D) + lane * kPairs;
  const __nv_bfloat162 *drow = reinterpret_cast<const __nv_bfloat162 *>(dout + row * D) + lane * kPairs;
  float acc = 0.f;
#pragma unroll
  for (int e = 0; e < kPairs; ++e) {
    const float2 a = __bfloat1622float2(orow[e]), c = __bfloat1622float2(drow[e]);
    acc += a.x * c.x + a.y * c.y;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
  if (lane == 0) delta[row] = acc;
#pragma unroll
  for (int c = lane * 4; c < D; c += 128) *reinterpret_cast<float4 *>(dqacc + row * D + c) = make_float4(0.f, 0.f, 0.f, 0.f);
}

// dQ = bf16(scale dQacc), and dV = bf16(sum of the parts), dK = bf16(scale sum of the parts) for
// key blocks in several parts.  Eight columns a thread; in the sums, a warp takes 8 rows and 4
// times 8 columns, so that it reads whole 128 bytes and writes whole 64.
template <int D>
static __global__ void __launch_bounds__(256)
    fa_bwd_join_kernel(const float *__restrict__ dqacc, __nv_bfloat16 *__restrict__ dq, const float4 *__restrict__ sums,
                       const int *__restrict__ parts, __nv_bfloat16 *__restrict__ dk, __nv_bfloat16 *__restrict__ dv,
                       float scale, int BH, int Hkv, int N, int nkb, long long n8) {
  const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  auto store = [](__nv_bfloat16 *dst, const float4 &a, const float4 &c, float mul) {
    *reinterpret_cast<uint4 *>(dst) = make_uint4(pack_bf16x2(a.x * mul, a.y * mul), pack_bf16x2(a.z * mul, a.w * mul),
                                                 pack_bf16x2(c.x * mul, c.y * mul), pack_bf16x2(c.z * mul, c.w * mul));
  };
  const long long front = (n8 + 255) / 256;
  if (blockIdx.x < front) {
    if (i < n8)
      store(dq + 8 * i, reinterpret_cast<const float4 *>(dqacc)[2 * i], reinterpret_cast<const float4 *>(dqacc)[2 * i + 1],
            scale);
    return;
  }
  // A key block's dV, then its dK: 128 rows of D / 8 threads each.
  constexpr int kTile = 128 * (D / 8), kWide = D / 32;
  const long long j = i - front * 256, tile = j / kTile;  // (head * nkb + kb) * 2 + (0: dV, 1: dK)
  const long long unit = tile / 2, head = unit / nkb;
  if (head >= BH) return;
  const int kb = static_cast<int>(unit - head * nkb), is_dk = static_cast<int>(tile & 1);
  const int n = parts[(head / Hkv) * nkb + kb];
  if (n < 2) return;
  const int w = static_cast<int>(j % kTile) / 32, lane = threadIdx.x % 32;
  const int row = (w / kWide) * 8 + lane % 8, col8 = (w % kWide) * 4 + lane / 8;
  if (kb * 128 + row >= N) return;
  const size_t per_part = static_cast<size_t>(BH) * nkb * 2 * (D / 4) * 128;
  const float4 *src = sums + (static_cast<size_t>(tile) * (D / 4) + 2 * col8) * 128 + row;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f), c = a;
  for (int s = 0; s < n; ++s, src += per_part) {
    const float4 x = src[0], y = src[128];
    a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
    c.x += y.x, c.y += y.y, c.z += y.z, c.w += y.w;
  }
  store((is_dk ? dk : dv) + (static_cast<size_t>(head) * N + kb * 128 + row) * D + 8 * col8, a, c, is_dk ? scale : 1.f);
}

}  // namespace fa
