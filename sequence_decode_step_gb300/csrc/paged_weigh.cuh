// What the kernels of qw_paged_weigh share: a sequence's rows and keys, shares of the work, fragments of mma.sync, strips.
#pragma once
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "paged.h"
#include "qw_ptx.cuh"

namespace qw {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kStrip = 16;               // keys of a warp at a time
constexpr int kTile = kStrip * kWarps;   // keys of a CTA at a time
constexpr int kRows = 128;               // query rows of an item: more take further passes over the keys
constexpr int kTileCost = 56;  // of a pass over a tile's keys, in tiles of 8 rows: 16 rows take 0.8 of the time of 128

__device__ __forceinline__ float exp2_approx(float x) {  // 2^-inf = 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {  // a in the low half
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
// (a, b) as up to three pairs of bf16 whose sums are a and b.
template <int T>
__device__ __forceinline__ void split(float a, float b, uint32_t (&t)[T]) {
#pragma unroll
  for (int i = 0; i < T; ++i) {
    t[i] = pack_bf16(a, b);
    if (i + 1 < T) {
      a -= __uint_as_float(t[i] << 16);
      b -= __uint_as_float(t[i] & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ------------------------------------------------------------------ the line
struct WSeq {     // a sequence's part of it
  int lo, rows;   // first token that counts, query rows of a KV head
  int base, len;  // keys before the first such token; all keys
  int fresh;      // first key of the call's own tokens
  int nkt;        // key tiles
};

// PRE: the shared prefix, one sequence with the batch's tokens, all of which see all its keys.
template <bool PRE>
__device__ __forceinline__ WSeq weigh_seq(const WeighArgs& a, int b) {
  WSeq s;
  if (PRE) {
    const int end = min(max(__ldg(a.c.q_start + a.c.n_seqs), 0), a.n_tokens);
    s.lo = min(max(__ldg(a.c.q_start), 0), end);
    s.rows = (end - s.lo) * a.gq;
    s.len = s.base = s.fresh = a.c.prefix_len;
  } else {
    s.lo = min(max(__ldg(a.c.q_start + b), 0), a.n_tokens);
    // the sequence may go on behind the call's rows: its last token still has its last key
    const int end = max(__ldg(a.c.q_start + b + 1), s.lo);
    const long long cap = (long long)a.c.max_pages << a.c.page_shift;
    s.len = (int)min((long long)max(__ldg(a.c.kv_len + b), 0), cap);
    s.base = s.len - (end - s.lo);
    s.fresh = max(s.base, 0);
    const int skip = a.window > 0 ? max(end - s.lo - a.window, 0) : 0;
    const bool any = min(end, a.n_tokens) > s.lo;
    s.lo += skip;
    s.base += skip;
    s.rows = max(min(end, a.n_tokens) - s.lo, 0) * a.gq;
    if (!any) s.len = 0;  // a sequence without tokens is left as it is
  }
  s.nkt = (s.len + kTile - 1) / kTile;
  return s;
}

// The first launch's line: items of kRows query rows for each KV head, each its key tiles and, before them, `head` tiles
// that stand for what comes before the keys: q, page entries, one after another. Shares of few tiles go without, as
// every CTA has that to do once there: they would mostly lie idle (9 chunks of 61 tokens 98 us, with head tiles 104).
constexpr int kHeadTiles = 3;
__device__ __forceinline__ int head_tiles(int tiles, int grid) { return tiles >= 8 * grid ? kHeadTiles : 0; }
__device__ __forceinline__ int row_blocks(const WSeq& s) { return (int)((unsigned)(s.rows + kRows - 1) / kRows); }
__device__ __forceinline__ int lse_units(const WeighArgs& a, const WSeq& s, int head) {
  return s.nkt ? a.c.nkv * row_blocks(s) * (s.nkt + head) : 0;
}
// Key tiles kt0 .. kt1 - 1 of an item that units u .. u1 - 1 of a line hold; moves u behind them.
struct LseTiles {
  int kvh, r0, kt0, kt1;
};
__device__ __forceinline__ LseTiles lse_tiles(const WSeq& s, int head, int unit, int u1, int* u) {
  const int nrb = row_blocks(s), n = s.nkt + head, item = (*u - unit) / n;
  const int in = *u - unit - item * n, to = min(n, in + (u1 - *u));
  *u += to - in;
  return LseTiles{item / nrb, item % nrb * kRows, max(in - head, 0), max(to - head, 0)};
}
// How a line is shared: units of a share, and its head tiles.
struct Line {
  int per, head;
};
__device__ __forceinline__ int share_of(int total, int grid) {
  return max((int)(((unsigned)total + grid - 1) / (unsigned)grid), 1);
}

// ------------------------------------------------------------------ fragments
// A k-step of 16 dimensions takes from a thread (row g = lane / 4, t = lane % 4) the dimensions of its four slots:
// bf16 pages two k-steps per load of 8 dimensions at 32 i + 8 t, f32 pages one per load of 4 at 16 i + 4 t.
template <int HD, bool KB, int QT>
struct Frag {
  static constexpr int L = KB ? HD / 32 : HD / 16;  // loads of 16 bytes per row
  static constexpr int S = HD / 16;         // k-steps
  static constexpr int kRow = HD * (KB ? 2 : 4);  // bytes
  uint4 lo[L], hi[L];                       // keys g and g + 8

  __device__ __forceinline__ void load(const void* pages, long long row, int lane) {
    constexpr int D = KB ? 32 : 16;
    const int esz = KB ? 2 : 4, g = lane >> 2, t = lane & 3;
    const char* p = static_cast<const char*>(pages) + ((row + g) * HD + t * (D / 4)) * esz;
#pragma unroll
    for (int i = 0; i < L; ++i) {
      lo[i] = __ldg(reinterpret_cast<const uint4*>(p + i * D * esz));
      hi[i] = __ldg(reinterpret_cast<const uint4*>(p + (8 * HD + i * D) * esz));
    }
  }
  // the strip from shared memory as stage_strip() has laid it there
  __device__ __forceinline__ void take(const uint8_t* strip, int lane) {
    const int g = lane >> 2, t = lane & 3, flip = (g & 1) * 64;
#pragma unroll
    for (int i = 0; i < L; ++i) {
      lo[i] = *reinterpret_cast<const uint4*>(strip + g * kRow + ((i * 64 + t * 16) ^ flip));
      hi[i] = *reinterpret_cast<const uint4*>(strip + (g + 8) * kRow + ((i * 64 + t * 16) ^ flip));
    }
  }
  __device__ __forceinline__ void split_key(int s, uint32_t (&k)[4][3]) const {
    split<3>(__uint_as_float(lo[s].x), __uint_as_float(lo[s].y), k[0]);
    split<3>(__uint_as_float(hi[s].x), __uint_as_float(hi[s].y), k[1]);
    split<3>(__uint_as_float(lo[s].z), __uint_as_float(lo[s].w), k[2]);
    split<3>(__uint_as_float(hi[s].z), __uint_as_float(hi[s].w), k[3]);
  }
};
// One k-step of f32 keys: products of like size in one accumulator, so that chains stay short and small terms are
// added up before large ones.
template <int QT>
__device__ __forceinline__ void step_f32(const uint32_t (&k)[4][3], const uint2 (&q)[QT], float (&c)[3][4]) {
#pragma unroll
  for (int x = 0; x < QT; ++x)
#pragma unroll
    for (int y = 2 - x; y >= 0; --y) mma(c[x + y], k[0][y], k[1][y], k[2][y], k[3][y], q[x].x, q[x].y);
}
// Scores of 16 keys x 8 query rows; q[term][i]: this lane's fragments, k-steps 2 i and 2 i + 1.
template <int HD, bool KB, int QT>
__device__ __forceinline__ void scores(const Frag<HD, KB, QT>& f, const uint4 (&q)[QT][HD / 32], float (&s)[4]) {
  constexpr int H = HD / 32;
  if constexpr (KB) {
    s[0] = s[1] = s[2] = s[3] = 0.f;
#pragma unroll
    for (int x = QT - 1; x >= 0; --x)
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const uint4 &a = f.lo[i], &b = f.hi[i], &w = q[x][i];
        mma(s, a.x, b.x, a.y, b.y, w.x, w.y);
        mma(s, a.z, b.z, a.w, b.w, w.z, w.w);
      }
  } else {
    float c[3][4] = {};
#pragma unroll
    for (int i = 0; i < H; ++i) {
      uint2 w0[QT], w1[QT];
#pragma unroll
      for (int x = 0; x < QT; ++x) w0[x] = make_uint2(q[x][i].x, q[x][i].y), w1[x] = make_uint2(q[x][i].z, q[x][i].w);
      uint32_t k[4][3];
      f.split_key(2 * i, k);
      step_f32<QT>(k, w0, c);
      f.split_key(2 * i + 1, k);
      step_f32<QT>(k, w1, c);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = c[0][i] + (c[1][i] + c[2][i]);
  }
}
// A strip of 16 rows into shared memory, by its warp; rows alternate in which half of 128 bytes they begin, so that
// eight lanes of a fragment meet all banks.
template <int ROW>
__device__ __forceinline__ void stage_strip(uint8_t* to, const void* pages, long long row, int lane) {
  constexpr int C = ROW / 16;
  const char* from = static_cast<const char*>(pages) + row * ROW;
#pragma unroll
  for (int i = 0; i < kStrip * C / 32; ++i) {
    const int e = i * 32 + lane, r = e / C, c = e % C;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to + r * ROW + ((c * 16) ^ ((r & 1) * 64)))),
                 "l"(from + e * 16)
                 : "memory");
  }
}
__device__ __forceinline__ void stage_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void stage_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
  __syncwarp();
}

// Page-table entry of key `key`, and its first pool row under KV head kvh once it has come: a page outside the pool is
// reported and read as page 0. (Apart, so that a loop can fetch the next entry without waiting for it.)
template <bool PRE>
__device__ __forceinline__ int strip_page(const WeighArgs& a, int b, int key) {
  const int at = key >> a.c.page_shift;
  return PRE ? __ldg(a.c.prefix_pages + at) : __ldg(a.c.page_table + (size_t)b * a.c.max_pages + at);
}
__device__ __forceinline__ int row_in(const WeighArgs& a, int page, int kvh, int key, bool* ok) {
  *ok = (unsigned)page < (unsigned)a.c.n_pages;
  if (!*ok) {
    if (a.c.status && (threadIdx.x & 31) == 0) atomicOr(a.c.status, PG_BAD_PAGE);
    page = 0;
  }
  return ((page * a.c.nkv + kvh) << a.c.page_shift) + (key & ((1 << a.c.page_shift) - 1));  // (below 2^31)
}
template <bool PRE>
__device__ __forceinline__ int strip_row(const WeighArgs& a, int b, int kvh, int key, bool* ok) {
  return row_in(a, strip_page<PRE>(a, b, key), kvh, key, ok);
}

// Joins two (maximum, sum) of base 2.
__device__ __forceinline__ float2 join(float2 x, float2 y) {
  const float m = fmaxf(x.x, y.x);
  if (m == -INFINITY) return make_float2(m, 0.f);
  return make_float2(m, x.y * exp2_approx(x.x - m) + y.y * exp2_approx(y.x - m));
}

// Keys that query row `row` of the sequence sees.
template <bool PRE>
__device__ __forceinline__ int row_sees(const WeighArgs& a, const WSeq& s, int row) {
  return row >= s.rows ? 0 : PRE ? s.len : min(max(s.base + row / a.gq + 1, 0), s.len);
}

// Reports a sequence whose rows decrease or leave the call's, or whose length is out of range.
__device__ __forceinline__ void report_length(const WeighArgs& a, int b) {
  const int lo = __ldg(a.c.q_start + b), hi = __ldg(a.c.q_start + b + 1), len = __ldg(a.c.kv_len + b);
  if (a.c.status && (lo < 0 || hi < lo || hi > a.n_tokens || len < hi - lo || len < 0 ||
                     len > (long long)a.c.max_pages << a.c.page_shift))
    atomicOr(a.c.status, PG_BAD_LENGTH);
}

// (maximum, sum) of a query row over all CTAs of the first launch that had part of its item. unit: the first unit
// of its sequence.
__device__ __forceinline__ float2 row_stats(const WeighArgs& a, const WeighStats& st, const WSeq& s, int unit,
                                            Line line, int kvh, int row, int lane, int lanes) {
  const int rb = (int)((unsigned)row / kRows);
  float2 x = make_float2(-INFINITY, 0.f);
  if (s.nkt == 0) return x;
  const int u = unit + (kvh * row_blocks(s) + rb) * (s.nkt + line.head) + line.head;  // (of the first tile)
  const int c0 = u / line.per, c1 = (u + s.nkt - 1) / line.per;
  if (c0 == c1) {
    const int token = row / a.gq;
    if (lane == 0) x = __ldcg(st.whole + (size_t)(s.lo + token) * a.nq + kvh * a.gq + row - token * a.gq);
  } else {
    for (int c = c0 + lane; c <= c1; c += 8 * lanes) {  // eight records on their way at a time
      float2 y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = c + i * lanes;
        y[i] = make_float2(-INFINITY, 0.f);
        if (at <= c1) y[i] = __ldcg(st.slots + ((size_t)at * 2 + (at == c0)) * kRows + (row - rb * kRows));
      }
#pragma unroll
      for (int i = 4; i > 0; i >>= 1)
#pragma unroll
        for (int j = 0; j < i; ++j) y[j] = join(y[j], y[j + i]);
      x = join(x, y[0]);
    }
  }
  return x;
}
// ------------------------------------------------------------------ shares of key tiles
// The second launch's line: a key tile takes as long as it has tiles of 8 rows, and for each pass over its keys as long
// as kTileCost more. Each KV head begins as the first launch's items do (without that, and with a lower cost of the keys,
// the slowest CTA of 16 ragged windows took 73 us where others took 47), always: a share of a tile and a half that reaches into the next
// head does the start twice (64 rows over 8192 keys of 8 heads: 25 us, without 31).
__device__ __forceinline__ int key_cost(const WSeq& s) {
  return kTileCost * max(row_blocks(s), 1) + (int)((unsigned)(s.rows + 7) / 8);
}
__device__ __forceinline__ int sum_units(const WeighArgs& a, const WSeq& s, int head) {
  return s.nkt ? a.c.nkv * (s.nkt + head) * key_cost(s) : 0;
}
// The tiles (of keys) that begin in units u .. u1 - 1 of a sequence's line, which begins at `unit`; moves u to their end.
struct SumTiles {
  int kvh, kt0, kt1;
};
__device__ __forceinline__ SumTiles sum_tiles(const WSeq& s, int head, int unit, int u1, int* u) {
  const int cost = key_cost(s), n = s.nkt + head, all = n * cost, kvh = (*u - unit) / all;
  const int in = *u - unit - kvh * all, t0 = (in + cost - 1) / cost, t1 = min(n, (in + (u1 - *u) + cost - 1) / cost);
  *u = unit + kvh * all + (t0 < n ? max(t0, t1) * cost : all);
  return SumTiles{kvh, max(t0 - head, 0), max(t1 - head, 0)};
}
struct Share {            // in shared memory: where a CTA's share begins
  int u0, u1;             // its units
  int head;               // head tiles here
  Line lse_line;          // the first launch's shares
  int unit, lse;          // first unit of sequence b, here and in the first launch
  int b;                  // n_seqs: nothing to do
};

// Block-wide. SUM: the second launch. Reports lengths out of range (the second launch does).
template <bool PRE, bool SUM>
__device__ void find_share(const WeighArgs& a, Share* sh, int (*warp_sums)[kWarps]) {
  const int n = PRE ? 1 : a.c.n_seqs, spt = (n + kThreads - 1) / kThreads;
  const int b0 = min((int)threadIdx.x * spt, n), b1 = min(b0 + spt, n);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // units without head tiles and per head tile, first launch and here
  constexpr int N = SUM ? 4 : 2;
  int mine[4] = {0, 0, 0, 0};
  bool back = false;
  for (int b = b0; b < b1; ++b) {
    const WSeq s = weigh_seq<PRE>(a, b);
    const int whole = lse_units(a, s, 0);
    mine[0] += whole;
    mine[1] += lse_units(a, s, 1) - whole;
    if (SUM) {
      const int keys = sum_units(a, s, 0);
      mine[2] += keys;
      mine[3] += sum_units(a, s, 1) - keys;
    }
    if (!PRE) {
      back |= __ldg(a.c.q_start + b + 1) < __ldg(a.c.q_start + b);
      if (SUM && blockIdx.x == 0) report_length(a, b);
    }
  }
  int sum[N], total[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    sum[i] = mine[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, sum[i], o);
      if (lane >= o) sum[i] += x;
    }
    if (lane == 31) warp_sums[i][warp] = sum[i];
    sum[i] -= mine[i];
    total[i] = 0;
  }
  if (threadIdx.x == 0) sh->b = n;
  if (__syncthreads_or(back)) return;  // a q_start that decreases: nothing is done
#pragma unroll
  for (int w = 0; w < kWarps; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (w < warp) sum[i] += warp_sums[i][w];
      total[i] += warp_sums[i][w];
    }
  const int grid = PRE ? a.pre_grid : a.grid, head_lse = head_tiles(total[0], grid);
  const int head = SUM ? kHeadTiles : head_lse;
  constexpr int H = SUM ? 2 : 0;
  const int all = total[H] + head * total[H + 1], per = share_of(all, grid);
  int unit = sum[H] + head * sum[H + 1], lse = sum[0] + head_lse * sum[1];
  const int u0 = (int)min((long long)per * blockIdx.x, (long long)all);
  if (u0 < all && u0 >= unit && u0 < unit + mine[H] + head * mine[H + 1]) {
    for (int b = b0; b < b1; ++b) {
      const WSeq s = weigh_seq<PRE>(a, b);
      const int l = lse_units(a, s, head_lse), u = SUM ? sum_units(a, s, head) : l;
      if (u0 < unit + u) {
        sh->u0 = u0, sh->u1 = min(u0 + per, all);
        sh->head = head;
        sh->lse_line = Line{share_of(total[0] + head_lse * total[1], grid), head_lse};
        sh->unit = unit, sh->lse = lse;
        sh->b = b;
        break;
      }
      unit += u, lse += l;
    }
  }
  __syncthreads();
}

// How the prefix's launch has shared its line.
__device__ __forceinline__ Line prefix_line(const WeighArgs& a, const WSeq& pre) {
  const int head = head_tiles(lse_units(a, pre, 0), a.pre_grid);
  return Line{share_of(lse_units(a, pre, head), a.pre_grid), head};
}
struct SumItem {  // in shared memory: tiles kt0 .. kt1 - 1 of a sequence and KV head
  WSeq s;
  int b, kvh, kt0, kt1;
  int lse;           // first unit of the sequence, first launch
  Line line;         // its shares
};
// L and the keys seen of `n` query rows from row r0 on, into shared memory: the CTA's threads share a row's records.
__device__ __forceinline__ void stage_stats(const WeighArgs& a, const SumItem& it, int r0, int n, float* big_l, int* see) {
  const int lanes = n <= 64 ? 4 : 2;  // a power of two, within a warp
  const WSeq pre = weigh_seq<true>(a, 0);
  const Line pre_line = prefix_line(a, pre);
  for (int i0 = 0; i0 < n; i0 += kThreads / lanes) {
    const int i = i0 + (int)threadIdx.x / lanes, lane = (int)threadIdx.x % lanes, row = r0 + i;
    float2 x = make_float2(-INFINITY, 0.f);
    if (i < n && row < it.s.rows) {
      x = row_stats(a, a.own, it.s, it.lse, it.line, it.kvh, row, lane, lanes);
      if (pre.nkt)
        x = join(x, row_stats(a, a.pre, pre, 0, pre_line, it.kvh, row + (it.s.lo - pre.lo) * a.gq, lane, lanes));
    }
    for (int o = 1; o < lanes; o <<= 1)
      x = join(x, make_float2(__shfl_xor_sync(0xffffffffu, x.x, o), __shfl_xor_sync(0xffffffffu, x.y, o)));
    if (lane == 0 && i < n) {
      big_l[i] = x.y > 0.f || x.y != x.y ? x.x + log2f(x.y) : INFINITY;  // (no key: weighs nothing)
      see[i] = row_sees<false>(a, it.s, row);
    }
  }
}

}  // namespace
}  // namespace qw
