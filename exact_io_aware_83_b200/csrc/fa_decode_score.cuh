// fa_decode_score.cuh - decode with changed scores over a bf16 cache, for up to 16 query rows
// per K/V head, on sm_100a.
//
// For batch b, query head h and new row t < Nq, over the keys j < len (causal: j <= len - Nq + t),
//   x_j = scale q . k_j,  y_j = cap tanh(x_j / cap) (or x_j),  s_j = y_j - slope_h |len - Nq + t - j|,
//   O = sum_j softmax_j(s) v_j,  LSE = ln sum_j exp(s_j).
//
//  * Work in equal pieces of the line of key blocks (fa_decode_line.cuh): the cache's bytes are
//    the bound (4 d per key), and fixed ranges of the longest entry leave SMs idle when the
//    lengths differ (64k cache, four entries of 16k-64k: 238 us with 4 ranges each).
//  * K and V blocks arrive by TMA, 128-byte swizzled, in a ring of stages; a warp takes 16 keys
//    of a block.  The products are warp-level m16n8k16: S^T = K Q^T with the keys as rows,
//    its operand read as 16 bytes per key (the channels of an instruction are those of four
//    such pieces, Q permuted alike), and O^T = V^T P^T with V transposed by ldmatrix.  With at
//    most 16 query rows the tensor core idles either way; the warps stay independent until a
//    segment ends, which tcgen05 and its shared accumulator would not allow.
//  * P is the sum of two bf16 numbers, so that O carries the rounding of its result alone.
//  * Rows of V behind the last key are cleared in registers: a cache may hold anything there.
#pragma once

#include "fa_decode_line.cuh"

namespace fa {

template <int D, int NT>
struct DecScoreLayout {
  static constexpr int W = D == 256 ? 4 : 8;   // warps
  static constexpr int kKeys = 16;             // keys per warp and step
  static constexpr int kBlock = W * kKeys;     // keys per block
  static constexpr int kChunk = kBlock * 128;  // [block x 64] bf16 box
  static constexpr int kTile = D / 64 * kChunk;
  static constexpr int kStageBytes = 2 * kTile;
  static constexpr int ROWS = 8 * NT;
  static constexpr int kPartBytes = W / 2 * ROWS * D * 4;
  static constexpr int kFixed = kPartBytes + 2 * W * ROWS * 4 + 2 * 8 * 8 + 64 + 1024;
  static constexpr int kFit = (232448 - kFixed) / kStageBytes;
  static constexpr int kStages = kFit > 6 ? 6 : kFit;
  static constexpr int kOffPart = kStages * kStageBytes;
  static constexpr int kOffM = kOffPart + kPartBytes;
  static constexpr int kOffBar = kOffM + 2 * W * ROWS * 4;  // full[8], empty[8]
  static constexpr int kOffMisc = kOffBar + 2 * 8 * 8;
  static constexpr int kSmemBytes = kOffMisc + 64 + 1024;   // + slack for 1024-byte alignment
  static_assert(kStages >= 2, "ring");
};

__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

template <int D, int NT>
__global__ void __launch_bounds__(DecScoreLayout<D, NT>::W * 32, 1)
    fa_decode_score_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                           const LineParams p) {
  using L = DecScoreLayout<D, NT>;
  constexpr int G = D / 32, MT = D / 16, S = L::kStages, ROWS = L::ROWS, W = L::W, KB = L::kBlock;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
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

  if (threadIdx.x < S) {
    mbar_init(full + 8 * threadIdx.x, 1);
    mbar_init(empty + 8 * threadIdx.x, W);
    fence_mbar_init();
  }
  if (warp == 0) {
    const LinePiece at = line_piece<KB>(p, blockIdx.x, lane);
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      misc[0] = misc[1] = 0;
      misc[2] = at.blocks;
      *reinterpret_cast<LineCursor<KB> *>(misc + 6) = line_cursor<KB>(p, at);
    }
  }
  __syncthreads();
  launch_dependents();        // the joining kernel
  const int total = misc[2];  // blocks of the piece
  int todo = total, taken = 0;
  LineCursor<KB> cur = *reinterpret_cast<LineCursor<KB> *>(misc + 6);  // what is computed next
  __syncthreads();            // the cursor moves on with the first copies
  bool ok = true;

  // Starts the copies of the piece's next block (one thread; the cursor passes from one issuer
  // to the next through the barriers of the stage).  Rows past the cache arrive as zeros.
  auto issue = [&]() {
    LineCursor<KB> *ahead = reinterpret_cast<LineCursor<KB> *>(misc + 6);
    LineCursor<KB> a = *ahead;
    const int st = misc[1] % S;
    const uint32_t dst = base + st * L::kStageBytes, bar = full + 8 * st;
    if (a.len > 0) {
      mbar_arrive_expect_tx(bar, L::kStageBytes);
#pragma unroll
      for (int ch = 0; ch < D / 64; ++ch) {
        tma_load_3d(dst + ch * L::kChunk, &tm_k, bar, ch * 64, a.blk * KB, a.b * p.Hkv + a.kvh);
        tma_load_3d(dst + L::kTile + ch * L::kChunk, &tm_v, bar, ch * 64, a.blk * KB, a.b * p.Hkv + a.kvh);
      }
    } else {
      mbar_arrive(bar);  // a segment without keys
    }
    a.next(p);
    *ahead = a;
    ++misc[1];
  };
  if (threadIdx.x == 0)
    for (int i = 0; i < min(S, total); ++i) issue();

  const int grp = p.R / p.Nq;  // query heads per K/V head
  const float inv_cap = p.softcap > 0.f ? 1.f / p.softcap : 0.f;
  const float cap_log2 = p.softcap * kLog2e;
  const float raw = p.softcap > 0.f ? p.scale : p.sl2;
  // This lane's piece of K: 16 bytes of key g (and g + 8), and its row of V for ldmatrix.
  const uint32_t krow = static_cast<uint32_t>(warp * 16 + g) * 128;
  const int vkey = warp * 16 + (lane / 16) * 8 + lane % 8;
  const uint32_t vrow = static_cast<uint32_t>(vkey) * 128;

  while (todo > 0) {
    // ---- one segment, or the part of it that lies in this piece
    const int blk0 = cur.blk, count = min(cur.nblk - blk0, todo), len = cur.len;
    const bool began_before = blk0 > 0, ends_after = blk0 + count < cur.nblk;
    const int kvh = cur.kvh, r0 = cur.rt * ROWS;
    const long long row0 = static_cast<long long>(cur.b * p.Hkv + kvh) * p.R + r0;
    const int pos0 = len - p.Nq;

    uint32_t qf[NT][G][4];  // row g of each 8-row tile: channels 32 i + 8 c .. + 7, in pairs
    float slope2[NT][2];    // rows 2c, 2c+1
    int rpos[NT][2];        // position of the row
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = nt * 8 + g;
#pragma unroll
      for (int i = 0; i < G; ++i) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (r0 + r < p.R) w = *reinterpret_cast<const uint4 *>(p.q + (row0 + r) * D + 32 * i + 8 * c);
        *reinterpret_cast<uint4 *>(qf[nt][i]) = w;
      }
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

    int kb = blk0 * KB + warp * 16;
#pragma unroll 1
    for (int i = 0; i < count; ++i, ++taken, kb += KB) {
      // The stage that the block before this one was in is refilled, by one warp in turn.
      if (taken > 0 && taken + S - 1 < total && warp == taken % W && lane == 0 &&
          wait_bounded(empty + 8 * ((taken - 1) % S), ((taken - 1) / S) & 1, abort_flag, wait_site(6, 8 + (taken - 1) % S, taken)))
        issue();
      __syncwarp();
      const int st = taken % S;
      if (ok) ok = warp_wait_bounded(full + 8 * st, (taken / S) & 1, abort_flag, wait_site(6, st, taken));
      if (ok && kb < len) {  // !ok: the flag is up, nothing of this call is valid any more
        const uint32_t sk = base + st * L::kStageBytes, sv = sk + L::kTile;
        float y[NT][4];  // key g: rows 2c, 2c+1; key g + 8: rows 2c, 2c+1
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) y[nt][e] = 0.f;
#pragma unroll
        for (int u = 0; u < G; ++u) {
          const uint32_t at = sk + (u / 2) * L::kChunk + krow + (((4 * (u & 1) + c) ^ g) << 4);
          uint32_t a[4], b[4];
          ld_shared_v4(at, a[0], a[1], a[2], a[3]);
          ld_shared_v4(at + 8 * 128, b[0], b[1], b[2], b[3]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_bf16_16816(y[nt], a[0], b[0], a[1], b[1], qf[nt][u][0], qf[nt][u][1]);
            mma_bf16_16816(y[nt], a[2], b[2], a[3], b[3], qf[nt][u][2], qf[nt][u][3]);
          }
        }
        // ---- cap, bias, mask: the scores in log2 units
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = kb + g + 8 * (e / 2);
            float v = y[nt][e] * raw;
            if (p.softcap > 0.f) v = softcap_log2<true>(v, inv_cap, cap_log2);
            v = fmaf(-slope2[nt][e & 1], fabsf(static_cast<float>(rpos[nt][e & 1] - key)), v);
            y[nt][e] = (key >= len || (p.causal && key > rpos[nt][e & 1])) ? -INFINITY : v;
          }
        // ---- running maximum: moved (for the whole warp) only when a row's rises by more than 2^8
        bool up = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) up |= fmaxf(y[nt][e], y[nt][e + 2]) > m_run[nt][e] + 8.f;
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float alpha[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float v = fmaxf(y[nt][e], y[nt][e + 2]);
#pragma unroll
              for (int o = 4; o < 32; o *= 2) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
              const float mn = fmaxf(m_run[nt][e], v);
              alpha[e] = mn == m_run[nt][e] ? 1.f : ex2_approx(m_run[nt][e] - mn);  // 0 at the first keys
              m_run[nt][e] = mn;
              l_run[nt][e] *= alpha[e];
            }
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[t][nt][e] *= alpha[e & 1];
          }
        }
        uint32_t ph[NT][2], pl[NT][2];  // P^T operand: its bf16 rounding and what is left
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float pr[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            pr[e] = ex2_approx(y[nt][e] - (m_run[nt][e & 1] == -INFINITY ? 0.f : m_run[nt][e & 1]));
            l_run[nt][e & 1] += pr[e];
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t hi = pack_bf16x2(pr[2 * k], pr[2 * k + 1]);
            const uint32_t lo = pack_bf16x2(pr[2 * k] - __uint_as_float(hi << 16),
                                            pr[2 * k + 1] - __uint_as_float(hi & 0xFFFF0000u));
            ph[nt][k] = movmatrix_trans(hi);
            pl[nt][k] = movmatrix_trans(lo);
          }
        }
        const bool tail = kb + 16 > len;
        // keys 2c, 2c+1 (and + 8) of this lane's V operand that count
        const uint32_t keep0 = (kb + 2 * c < len ? 0xFFFFu : 0u) | (kb + 2 * c + 1 < len ? 0xFFFF0000u : 0u);
        const uint32_t keep1 = (kb + 2 * c + 8 < len ? 0xFFFFu : 0u) | (kb + 2 * c + 9 < len ? 0xFFFF0000u : 0u);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const int unit = 2 * t + ((lane / 8) & 1);
          uint32_t v[4];
          ldmatrix_x4_trans(sv + (t / 4) * L::kChunk + vrow + (((unit & 7) ^ (vkey & 7)) << 4), v);
          if (tail) {
            v[0] &= keep0;
            v[1] &= keep0;
            v[2] &= keep1;
            v[3] &= keep1;
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_bf16_16816(acc[t][nt], v[0], v[1], v[2], v[3], ph[nt][0], ph[nt][1]);
            mma_bf16_16816(acc[t][nt], v[0], v[1], v[2], v[3], pl[nt][0], pl[nt][1]);
          }
        }
      }
      __syncwarp();  // every lane has read the stage
      if (lane == 0) mbar_arrive(empty + 8 * st);
    }

    // Accumulator tile t of lane (g, c): channels 16 t + g (+ 8), rows 2c, 2c+1.
    line_join<D, NT, W>(p, sm_o, sm_m, m_run, l_run, r0, row0, began_before, ends_after, abort_flag,
                        [&](float *row, float f, int nt, int e, bool add) {
#pragma unroll
                          for (int t = 0; t < MT; ++t) {
                            row[16 * t + g] = fmaf(f, acc[t][nt][e], add ? row[16 * t + g] : 0.f);
                            row[16 * t + 8 + g] = fmaf(f, acc[t][nt][e + 2], add ? row[16 * t + 8 + g] : 0.f);
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
