// fa_decode_line.cuh - how decode's work is cut into equal pieces, and how the parts are joined.
//
// A segment is a (batch entry, K/V head, tile of query rows).  Its valid keys are cut into
// blocks of KB keys, the blocks of all segments are laid end to end (batch entry by batch
// entry, head by head), and this line is cut into `pieces` equal ranges, one CTA each, so that
// lengths that differ leave no SM idle.  The lengths are in device memory, so every CTA finds
// its range itself.  A segment inside one piece is written by its CTA; one that several pieces
// share leaves a partial result (O, m, l) per piece in the workspace, and fa_line_merge_kernel
// joins them.
#pragma once

#include "fa_fwd.cuh"
#include "fa_score.cuh"

namespace fa {

struct LineParams {
  const __nv_bfloat16 *q;  // [B, Hq, Nq, D]
  const int *lens;         // [B] (nullptr: all `cap`), clamped to [0, cap]
  const float *slopes;     // [Hq] or nullptr
  __nv_bfloat16 *o;
  float *lse;
  float *part;             // [pieces][2][rows of a tile][D + 2] fp32 (O, then m and l)
  int B, Hkv, Nq, R, cap;  // R = (Hq / Hkv) Nq rows share a K/V head; cap: rows of the cache
  int row_tiles, pieces;
  int causal;
  float scale, sl2;        // scale, scale * log2(e)
  float softcap;           // 0: none
};

__device__ __forceinline__ int line_len(const LineParams &p, int b) {
  const int len = p.lens ? p.lens[b] : p.cap;
  return len < 0 ? 0 : (len > p.cap ? p.cap : len);
}
// Blocks of a segment: one at least, so that a segment without keys is written too.
template <int KB>
__device__ __forceinline__ int line_blocks(int len) {
  return len > 0 ? (len + KB - 1) / KB : 1;
}

// Sum over the batch entries before `upto` of their blocks, times segments per entry (whole warp).
template <int KB>
__device__ __forceinline__ long long line_blocks_before(const LineParams &p, int upto, int lane) {
  long long n = 0;
  for (int b = lane; b < upto; b += 32) n += line_blocks<KB>(line_len(p, b));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n * (static_cast<long long>(p.Hkv) * p.row_tiles);
}

// First block of piece i of P over T blocks, and the piece that holds block x.  P <= T: with
// fewer blocks than pieces the last CTAs have no work, so that no piece is empty.
__device__ __forceinline__ int line_pieces_used(const LineParams &p, long long T) {
  return T < p.pieces ? static_cast<int>(T) : p.pieces;
}
__device__ __forceinline__ long long line_div(long long a, long long b) {  // a, b >= 0; most fit 32 bits
  return ((a | b) >> 32) == 0 ? static_cast<long long>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}
__device__ __forceinline__ long long line_piece_begin(long long T, int P, int i) { return line_div(T * i, P); }
__device__ __forceinline__ int line_piece_of(long long T, int P, long long x) {
  return static_cast<int>(line_div((x + 1) * P - 1, T));
}

// The kernel that follows in the stream may be launched (and wait) from here on; and: wait until
// the kernel before this one has completed and its writes are visible.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The piece that CTA i works on: its number of blocks, and where the first one lies.
struct LinePiece {
  int blocks, b, seg, blk;  // seg: kvh * row_tiles + row tile
};

// (whole warp)
template <int KB>
__device__ __forceinline__ LinePiece line_piece(const LineParams &p, int i, int lane) {
  const long long per = static_cast<long long>(p.Hkv) * p.row_tiles;
  const long long T = p.lens ? line_blocks_before<KB>(p, p.B, lane) : p.B * per * line_blocks<KB>(p.cap);
  const int P = line_pieces_used(p, T);
  if (i >= P) return LinePiece{0, 0, 0, 0};
  const long long x0 = line_piece_begin(T, P, i), x1 = line_piece_begin(T, P, i + 1);
  // the batch entry that holds block x0: 32 entries at a time
  long long before = 0;
  int b = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const long long n = b0 + lane < p.B ? line_blocks<KB>(line_len(p, b0 + lane)) * per : 0;
    long long sum = n;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const long long t = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += t;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, before + sum > x0 && n > 0);
    if (hit) {
      const int l = __ffs(hit) - 1;
      b = b0 + l;
      before += __shfl_sync(0xffffffffu, sum - n, l);
      break;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  const int nblk = line_blocks<KB>(line_len(p, b));
  const long long in = x0 - before;
  const int seg = static_cast<int>(line_div(in, nblk));
  return LinePiece{static_cast<int>(x1 - x0), b, seg, static_cast<int>(in - static_cast<long long>(seg) * nblk)};
}

// A block of the line: its segment and its place in it.
template <int KB>
struct LineCursor {
  int b, kvh, rt, blk, nblk, len;  // rt: row tile
  __device__ __forceinline__ void enter(const LineParams &p, int b_) {
    b = b_;
    len = line_len(p, b);
    nblk = line_blocks<KB>(len);
  }
  __device__ __forceinline__ void next(const LineParams &p) {
    if (++blk < nblk) return;
    blk = 0;
    if (++rt < p.row_tiles) return;
    rt = 0;
    if (++kvh < p.Hkv) return;
    kvh = 0;
    if (b + 1 < p.B) enter(p, b + 1);
  }
};

template <int KB>
__device__ __forceinline__ LineCursor<KB> line_cursor(const LineParams &p, const LinePiece &at) {
  LineCursor<KB> c;
  c.enter(p, at.b);
  c.kvh = at.seg / p.row_tiles;
  c.rt = at.seg % p.row_tiles;
  c.blk = at.blk;
  return c;
}

// The score in log2 units from x = scale q . k: capped, y = cap tanh(x / cap) log2(e).  FAR: the
// cap may lie beyond kCapNear.
template <bool FAR>
__device__ __forceinline__ float softcap_log2(float x, float inv_cap, float cap_log2) {
  float grad;
  return cap_log2 * tanh_any<FAR>(x * inv_cap, grad);
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}

// Where a segment, or the part of it that lies in this piece, ends: joins the CTA's W warps
// (those without keys have m = -inf, l = 0, O = 0) and writes the result or the partial one.
// Lane (g, c) of a warp holds m and (its share of) l of rows 8 nt + 2 c + e.  `put` brings the
// warp's O of row 8 nt + 2 c + e, times f, to a row of D fp32 in shared memory, adding to what
// is there or not: the second half of the warps hands its O, brought to the common maximum,
// to the first half, which adds its own; then every thread sums W / 2 of them.
// sm_o: [W / 2][8 NT][D], sm_m: m of [W][8 NT], then l.
template <int D, int NT, int W, typename Put>
__device__ __forceinline__ void line_join(const LineParams &p, float *sm_o, float *sm_m, const float (&m_run)[NT][2],
                                          float (&l_run)[NT][2], int r0, long long row0, bool began_before,
                                          bool ends_after, volatile int *abort_flag, Put put) {
  constexpr int ROWS = 8 * NT;
  float *sm_l = sm_m + W * ROWS;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, c = lane % 4;
  __syncthreads();  // sm_* of the previous segment have been read
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int o = 4; o < 32; o *= 2) l_run[nt][e] += __shfl_xor_sync(0xffffffffu, l_run[nt][e], o);
      if (g == 0) {
        sm_m[warp * ROWS + nt * 8 + 2 * c + e] = m_run[nt][e];
        sm_l[warp * ROWS + nt * 8 + 2 * c + e] = l_run[nt][e];
      }
    }
  __syncthreads();
  float scale_w[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < W; ++w) m = fmaxf(m, sm_m[w * ROWS + nt * 8 + 2 * c + e]);
      scale_w[nt][e] = ex2_approx(m_run[nt][e] - (m == -INFINITY ? 0.f : m));
    }
#pragma unroll
  for (int turn = 0; turn < 2; ++turn) {
    if (warp / (W / 2) == 1 - turn) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = nt * 8 + 2 * c + e;
          if (r0 + r >= p.R) continue;
          put(sm_o + ((warp % (W / 2)) * ROWS + r) * D, scale_w[nt][e], nt, e, turn == 1);
        }
    }
    __syncthreads();
  }
  if (*abort_flag == 0) {
    const bool direct = !began_before && !ends_after;
    float *part = p.part + (static_cast<long long>(blockIdx.x) * 2 + (began_before ? 0 : 1)) * (ROWS * (D + 2));
    for (int idx = threadIdx.x; idx < ROWS * (D / 2); idx += blockDim.x) {
      const int r = idx / (D / 2), ch = 2 * (idx % (D / 2));
      if (r0 + r >= p.R) break;
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < W; ++w) m = fmaxf(m, sm_m[w * ROWS + r]);
      const float mu = m == -INFINITY ? 0.f : m;
      float l = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) l = fmaf(ex2_approx(sm_m[w * ROWS + r] - mu), sm_l[w * ROWS + r], l);
#pragma unroll
      for (int w = 0; w < W / 2; ++w) {
        const float2 o = *reinterpret_cast<const float2 *>(sm_o + (w * ROWS + r) * D + ch);
        o0 += o.x;
        o1 += o.y;
      }
      if (direct) {
        const float inv = l == 0.f ? 0.f : 1.f / l;  // a row without keys: 0; NaN stays NaN
        *reinterpret_cast<uint32_t *>(p.o + (row0 + r) * D + ch) = pack_bf16x2(o0 * inv, o1 * inv);
        if (ch == 0) p.lse[row0 + r] = l == 0.f ? -INFINITY : (mu + log2f(l)) * kLn2;
      } else {
        float *dst = part + r * (D + 2);
        *reinterpret_cast<float2 *>(dst + ch) = make_float2(o0, o1);
        if (ch == 0) {
          dst[D] = m;
          dst[D + 1] = l;
        }
      }
    }
  }
}

// Joins the partial results of the segments that several pieces share, one CTA of four warps
// per row: with the pieces' m_i (log2 units), l_i and unnormalised O_i,
//   m = max m_i,  l = sum 2^(m_i - m) l_i,  O = sum 2^(m_i - m) O_i / l,  LSE = (m + log2 l) ln 2.
// Launched while the pieces are still being computed: it finds its pieces first, then waits.
// (One warp per row, one piece after the other, took 11-15 us for 16 pieces a row.)
template <int D, int KB>
__global__ void __launch_bounds__(128) fa_line_merge_kernel(const LineParams p, int tile_rows) {
  constexpr int kPer = D / 32;
  __shared__ float sm_acc[4][D], sm_l[4];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const long long row = blockIdx.x;
  const int bh = static_cast<int>(blockIdx.x / static_cast<unsigned>(p.R)), r = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.R));
  const int b = bh / p.Hkv, kvh = bh % p.Hkv;
  const int nblk = line_blocks<KB>(line_len(p, b));
  const long long per = static_cast<long long>(p.Hkv) * p.row_tiles;
  const long long T = p.lens ? line_blocks_before<KB>(p, p.B, lane) : p.B * per * nblk;
  const long long first = (p.lens ? line_blocks_before<KB>(p, b, lane) : b * per * nblk) +
                          static_cast<long long>(kvh * p.row_tiles + r / tile_rows) * nblk;
  const int P = line_pieces_used(p, T);
  const int p0 = line_piece_of(T, P, first), p1 = line_piece_of(T, P, first + nblk - 1);
  // Every CTA waits, so that what follows this kernel in the stream follows the pieces too.
  wait_for_primary();
  if (p0 == p1) return;  // written by its piece
  // The piece in which the segment begins holds it in slot 1, later ones in slot 0.
  auto slot = [&](int i) {
    return p.part + ((static_cast<long long>(i) * 2 + (i == p0 ? 1 : 0)) * tile_rows + r % tile_rows) * (D + 2);
  };
  float m = -INFINITY;
  for (int i = p0 + lane; i <= p1; i += 32) m = fmaxf(m, slot(i)[D]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float mu = m == -INFINITY ? 0.f : m;
  float l = 0.f, acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int i = p0 + warp; i <= p1; i += 4) {
    const float *src = slot(i);
    const float f = ex2_approx(src[D] - mu);
    l = fmaf(f, src[D + 1], l);
#pragma unroll
    for (int e = 0; e < kPer; e += 2) {
      const float2 o = *reinterpret_cast<const float2 *>(src + lane * kPer + e);
      acc[e] = fmaf(f, o.x, acc[e]);
      acc[e + 1] = fmaf(f, o.y, acc[e + 1]);
    }
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) sm_acc[warp][lane * kPer + e] = acc[e];
  if (lane == 0) sm_l[warp] = l;
  __syncthreads();
  l = (sm_l[0] + sm_l[1]) + (sm_l[2] + sm_l[3]);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  for (int ch = 2 * threadIdx.x; ch < D; ch += 256) {
    const float o0 = (sm_acc[0][ch] + sm_acc[1][ch]) + (sm_acc[2][ch] + sm_acc[3][ch]);
    const float o1 = (sm_acc[0][ch + 1] + sm_acc[1][ch + 1]) + (sm_acc[2][ch + 1] + sm_acc[3][ch + 1]);
    *reinterpret_cast<uint32_t *>(p.o + row * D + ch) = pack_bf16x2(o0 * inv, o1 * inv);
  }
  if (threadIdx.x == 0) p.lse[row] = l == 0.f ? -INFINITY : (mu + log2f(l)) * kLn2;
}

}  // namespace fa
