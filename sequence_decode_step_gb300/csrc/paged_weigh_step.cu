// qw_paged_weigh for up to 8 query rows of a sequence and KV head (a decode step, or a few tokens): the keys' bytes
// are the bound, and with short sequences the latency of many small items.
//
// An item is 8 query rows of one sequence and KV head over its strips of 16 keys. All items' strips laid end to end
// (an item is one unit longer, for its q, its statistics and its records) form one line, cut into equal shares for
// the warps: no warp waits for another, and a sequence of any length is read by as many as its bytes deserve. The
// first launch keeps every score (base 2), by place in the pool: 4 to 32 bytes a key beside its 128 to 512, so that
// the second launch, with the same shares, reads these and not the keys. Keys go from memory by asynchronous copies into
// a warp's own part of shared memory, 16 ahead of the 16 at work, and from there into mma.sync fragments (m16n8k16: keys on
// the 16-row side, query rows on the 8-column side, so that a thread sums its keys' weights by itself); a 128-row
// tcgen05 tile would be empty.
// 256 sequences of up to 8K bf16 keys, 8 heads of 128 dimensions: 2.2 GB in 391 us (5.6 TB/s) and the scores in 48.
// (Sums over whole CTAs with barriers between items took 146 us for that second launch.) 64 ragged sequences: 32 us
// (39 from cold caches), a chain of dependent reads per launch: lengths, page entries, keys, records. One sequence of 4K
// keys: 13 us.

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "paged.h"
#include "paged_plan.h"
#include "paged_weigh.cuh"

namespace qw {
namespace {

constexpr int kLeastStrips = 2;  // least units of a share: fewer records of a short line to join (1: a sequence of 16K
                                 // keys 17.2 us, 15.2 with 2 and 15.8 with 3; 64 of 64 keys 11.6, 13.3 and 21)

__device__ __forceinline__ int strips_of(const WSeq& s) { return (s.len + kStrip - 1) / kStrip; }
__device__ __forceinline__ int blocks_of(const WSeq& s) { return max((s.rows + 7) / 8, 1); }
__device__ __forceinline__ int step_units(const WeighArgs& a, const WSeq& s) {
  return s.len ? a.c.nkv * blocks_of(s) * (strips_of(s) + 1) : 0;
}

// A CTA's warps take every eighth strip of its share, so that 32 KB of neighbours are read at a time (each warp on
// its own piece of the share: 5.0 TB/s, 446 us for the keys of 256 sequences; so 5.6). Their parts of an item's
// statistics are joined for kGroup items at once.
// An item of fewer than kAlone strips goes to one warp, so that the latencies of eight items are passed at once, if the
// share is long enough for several of its size: n^2 < 4 S for n strips in a share of S, as an item's start takes about as
// long as four strips. Else, and for pieces of longer items, all warps work on one (all items of up to 15 strips by one
// warp: 8 sequences of 4K keys 21 us, 14 so; all by eight: 64 ragged sequences 48 us, 32 so). Pieces of longer items by one
// warp too: 45 drawn steps 2 % slower in the mean, a few long sequences among many short ones 8 % faster from cold caches.
constexpr int kGroup = 8, kAlone = 16;
struct StepParts {           // in shared memory
  float2 x[kGroup][kWarps][8];
  bool alone[kGroup];        // by warp i alone
  int to[kGroup][8];         // where a row's statistics go: a place in WeighStats::whole, in the CTA's slots (-1 - slot) or
};                           // nowhere (kNowhere)
constexpr int kNowhere = -17;

struct StepShares {          // in shared memory
  int b[kWarps];             // first sequence of a warp's share, n_seqs: nothing to do
  int unit[kWarps];          // that sequence's first unit
  int per, total;
  int warp_sums[kWarps];
};

// Block-wide.
__device__ __forceinline__ void find_shares(const WeighArgs& a, StepShares* sh, bool report) {
  const int n = a.c.n_seqs, spt = (n + kThreads - 1) / kThreads;
  const int b0 = min((int)threadIdx.x * spt, n), b1 = min(b0 + spt, n);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int mine = 0;
  bool back = false;
  for (int b = b0; b < b1; ++b) {
    mine += step_units(a, weigh_seq<false>(a, b));
    const int lo = __ldg(a.c.q_start + b), hi = __ldg(a.c.q_start + b + 1);
    back |= hi < lo;
    if (report && blockIdx.x == 0) report_length(a, b);
  }
  int sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += x;
  }
  if (lane == 31) sh->warp_sums[warp] = sum;
  if (threadIdx.x < kWarps) sh->b[threadIdx.x] = n;
  if (__syncthreads_or(back)) return;  // a q_start that decreases: nothing is done
  sum -= mine;
  int total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) sum += sh->warp_sums[w];
    total += sh->warp_sums[w];
  }
  const int warps = (int)gridDim.x * kWarps, per = max((int)(((unsigned)total + warps - 1) / (unsigned)warps), kLeastStrips);
  if (threadIdx.x == 0) sh->per = per, sh->total = total;
  const long long u0 = (long long)per * (blockIdx.x * kWarps);
  if (mine && u0 < sum + mine && u0 + (long long)per * kWarps > sum) {
    int unit = sum;
    for (int b = b0; b < b1; ++b) {
      const int u = step_units(a, weigh_seq<false>(a, b));
      for (int w = 0; w < kWarps; ++w) {
        const long long at = u0 + (long long)per * w;
        if (at >= unit && at < unit + u) sh->b[w] = b, sh->unit[w] = unit;
      }
      unit += u;
    }
  }
  __syncthreads();
}

// A place on the line: of a warp's share, or (CTA) of those of all its warps.
struct StepCursor {
  WSeq s;
  int b, unit, u, u1;
  int kvh, rb, k0, k1, nks;  // the item's KV head and row block; this share's strips of it, and all
  __device__ __forceinline__ StepCursor(const WeighArgs& a, const StepShares& sh, int warp, int warps) {
    b = sh.b[warp];
    unit = sh.unit[warp];
    const long long at = (long long)sh.per * (blockIdx.x * kWarps + warp);
    u = (int)min(at, (long long)sh.total), u1 = (int)min(at + (long long)sh.per * warps, (long long)sh.total);
    if (b >= a.c.n_seqs) u = u1;
    else s = weigh_seq<false>(a, b);
  }
  // To the next item of which the share has a strip.
  __device__ __forceinline__ bool next(const WeighArgs& a) {
    while (u < u1) {
      for (int n; u - unit >= (n = step_units(a, s)); s = weigh_seq<false>(a, ++b)) unit += n;
      nks = strips_of(s);
      const int item = (u - unit) / (nks + 1), first = unit + item * (nks + 1) + 1, blocks = blocks_of(s);
      kvh = item / blocks, rb = item - kvh * blocks;
      k0 = max(u - first, 0), k1 = min(nks, u1 - first);
      u = first + nks;
      if (k0 < k1) return true;
    }
    return false;
  }
};

// Query rows 8 rb .. 8 rb + 7 as fragments in registers.
template <int HD, bool KB, int QT>
struct QFrag {
  uint4 w[QT][HD / 32];
  __device__ __forceinline__ void load(const WeighArgs& a, const WSeq& s, int kvh, int rb, int lane) {
    const int row = rb * 8 + (lane >> 2), t = lane & 3, token = row / a.gq, head = kvh * a.gq + row - token * a.gq;
    const long long at = (long long)(s.lo + token) * a.ldq + head * HD;
#pragma unroll
    for (int i = 0; i < HD / 32; ++i) {
      // dimensions of k-steps 2 i and 2 i + 1
      const int d0 = KB ? 32 * i + 8 * t : 32 * i + 4 * t, d1 = KB ? d0 + 4 : d0 + 16;
#pragma unroll
      for (int x = 0; x < QT; ++x) w[x][i] = make_uint4(0u, 0u, 0u, 0u);
      if (row >= s.rows) continue;
      if (QT == 1) {
        const uint16_t* p = static_cast<const uint16_t*>(a.q) + at;
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(p + d0)), v = __ldg(reinterpret_cast<const uint2*>(p + d1));
        w[0][i] = make_uint4(u.x, u.y, v.x, v.y);
      } else {
        const float* p = static_cast<const float*>(a.q) + at;
        const float4 u = __ldg(reinterpret_cast<const float4*>(p + d0)), v = __ldg(reinterpret_cast<const float4*>(p + d1));
        uint32_t y[4][QT];
        split<QT>(u.x, u.y, y[0]);
        split<QT>(u.z, u.w, y[1]);
        split<QT>(v.x, v.y, y[2]);
        split<QT>(v.z, v.w, y[3]);
#pragma unroll
        for (int x = 0; x < QT; ++x) w[x][i] = make_uint4(y[0][x], y[1][x], y[2][x], y[3][x]);
      }
    }
  }
};

// CTAs per SM of the first launch: as many as the strips' shared memory and the fragments' registers leave room for.
constexpr int step_ctas(int hd, bool kv_bf16, int q_terms) {
  return hd == 128 ? (kv_bf16 ? (q_terms == 1 ? 3 : 2) : 1) : kv_bf16 ? (q_terms == 1 ? 4 : 3) : 2;
}

template <int HD, bool KB, int QT>
__global__ void __launch_bounds__(kThreads, step_ctas(HD, KB, QT)) step_scores_kernel(const __grid_constant__ WeighArgs a) {
  using F = Frag<HD, KB, QT>;
  constexpr int kBytes = kStrip * F::kRow;
  __shared__ StepShares sh;
  __shared__ StepParts parts;
  extern __shared__ __align__(16) uint8_t ring[];  // two strips of every warp
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = lane & 3, g = lane >> 2;
  pdl_wait();
  pdl_launch_dependents();
  find_shares(a, &sh, false);
  uint8_t* mine = ring + warp * 2 * kBytes;
  float2* slots = a.own.slots + (size_t)blockIdx.x * 16;
  auto join_parts = [&](int items) {
    __syncthreads();
    const int i = threadIdx.x >> 3, r = threadIdx.x & 7;
    if (i < items) {
      float2 x = parts.x[i][parts.alone[i] ? i : 0][r];
      if (!parts.alone[i]) {
#pragma unroll
        for (int w = 1; w < kWarps; ++w) x = join(x, parts.x[i][w][r]);
      }
      const int to = parts.to[i][r];
      if (to >= 0) a.own.whole[to] = x;
      else if (to != kNowhere) slots[-1 - to] = x;
    }
    __syncthreads();
  };
  StepCursor c(a, sh, 0, kWarps);
  int items = 0;
  while (c.next(a)) {
    const int r0 = c.rb * 8, limit = row_sees<false>(a, c.s, min(r0 + 8, c.s.rows) - 1);
    const bool alone = c.nks < kAlone && c.nks * c.nks < 4 * kWarps * sh.per;
    if (alone && items != warp) {
      if (++items == kGroup) join_parts(items), items = 0;
      continue;
    }
    const int step = alone ? kStrip : kTile;
    const int first = (c.k0 + (alone ? 0 : warp)) * kStrip, end = min(c.k1 * kStrip, limit);
    // the strip's place in the pool (-1 behind a bad page: page 0, which is read for it, keeps its owner's scores), and
    // the next one's page
    int row = 0, page = 0;
    auto fetch = [&](int entry, int key, uint8_t* to) {
      bool ok;
      row = row_in(a, entry, c.kvh, key, &ok);
      stage_strip<F::kRow>(to, a.c.k_pages, row, lane);
      if (!ok) row = -1;
    };
    if (first < end) fetch(strip_page<false>(a, c.b, first), first, mine);
    stage_commit();
    if (first + step < end) page = strip_page<false>(a, c.b, first + step);
    QFrag<HD, KB, QT> q;
    q.load(a, c.s, c.kvh, c.rb, lane);
    // of the thread's query rows 2 t and 2 t + 1: keys seen; maximum (before the factor), its product with it, sum
    int see[2];
    float m[2], base[2], l[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      see[e] = row_sees<false>(a, c.s, r0 + 2 * t + e);
      m[e] = -INFINITY, base[e] = 0.f, l[e] = 0.f;
    }
    int at = 0;
    for (int key = first; key < end; key += step, at ^= 1) {
      const int here = row;
      if (key + step < end) {
        fetch(page, key + step, mine + (at ^ 1) * kBytes);
        if (key + 2 * step < end) page = strip_page<false>(a, c.b, key + 2 * step);
      }
      stage_commit();
      stage_wait<1>();
      F f;
      f.take(mine + at * kBytes, lane);
      float x[4];
      scores<HD, KB, QT>(f, q.w, x);
      if (here >= 0 && 2 * t < a.keep) {
        float* to = a.kept + (long long)(here + g) * a.keep + 2 * t;
        *reinterpret_cast<float2*>(to) = make_float2(x[0] * a.scale_log2, x[1] * a.scale_log2);
        *reinterpret_cast<float2*>(to + 8 * a.keep) = make_float2(x[2] * a.scale_log2, x[3] * a.scale_log2);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float x0 = key + g < see[e] ? x[e] : -INFINITY, x1 = key + g + 8 < see[e] ? x[2 + e] : -INFINITY;
        const float top = fmaxf(x0, x1);
        if (top > m[e]) {
          l[e] *= exp2_approx((m[e] - top) * a.scale_log2);
          m[e] = top, base[e] = -top * a.scale_log2;
        }
        l[e] += exp2_approx(fmaf(x0, a.scale_log2, base[e])) + exp2_approx(fmaf(x1, a.scale_log2, base[e]));
      }
      __syncwarp();  // all lanes have read the buffer that is filled next
    }
    stage_wait<0>();
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float2 x = make_float2(m[e] * a.scale_log2, l[e]);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1)
        x = join(x, make_float2(__shfl_xor_sync(0xffffffffu, x.x, o), __shfl_xor_sync(0xffffffffu, x.y, o)));
      if (lane < 4) parts.x[items][warp][2 * t + e] = x;
    }
    if (alone ? lane < 8 : threadIdx.x < 8) {
      const int q_row = r0 + lane, token = q_row / a.gq;
      parts.alone[items] = alone;
      parts.to[items][lane] = q_row >= c.s.rows                  ? kNowhere
                                     : c.k0 == 0 && c.k1 == c.nks ? (c.s.lo + token) * a.nq + c.kvh * a.gq + q_row - token * a.gq
                                                                   : -1 - ((c.k0 == 0 ? 8 : 0) + lane);
    }
    if (++items == kGroup) {
      join_parts(items);
      items = 0;
    }
  }
  if (items) join_parts(items);
}

// L of query rows r0 .. r0 + 7 in the lanes 4 r .. 4 r + 3, by a warp: four lanes share a row's records.
__device__ __forceinline__ float step_stats(const WeighArgs& a, const WSeq& s, int unit, int per, int kvh, int r0) {
  const int per_cta = per * kWarps;
  const int lane = threadIdx.x & 31, row = r0 + (lane >> 2), sub = lane & 3;
  float2 x = make_float2(-INFINITY, 0.f);
  if (row < s.rows) {
    const int nks = strips_of(s), u = unit + (kvh * blocks_of(s) + r0 / 8) * (nks + 1) + 1;
    const int w0 = u / (per_cta), w1 = (u + nks - 1) / (per_cta), token = row / a.gq;  // CTAs
    if (w0 == w1) {
      if (sub == 0) x = __ldcg(a.own.whole + (size_t)(s.lo + token) * a.nq + kvh * a.gq + row - token * a.gq);
    } else {
#pragma unroll 4
      for (int w = w0 + sub; w <= w1; w += 4) x = join(x, __ldcg(a.own.slots + ((size_t)w * 2 + (w == w0)) * 8 + (row - r0)));
    }
    if (a.c.prefix_len > 0) {
      const WSeq pre = weigh_seq<true>(a, 0);
      x = join(x, row_stats(a, a.pre, pre, 0, prefix_line(a, pre), kvh, row + (s.lo - pre.lo) * a.gq, sub, 4));
    }
  }
  x = join(x, make_float2(__shfl_xor_sync(0xffffffffu, x.x, 1), __shfl_xor_sync(0xffffffffu, x.y, 1)));
  x = join(x, make_float2(__shfl_xor_sync(0xffffffffu, x.x, 2), __shfl_xor_sync(0xffffffffu, x.y, 2)));
  return x.y > 0.f || x.y != x.y ? x.x + log2f(x.y) : INFINITY;  // (no key: weighs nothing)
}

// A sequence of more query rows than the call's hints promise: its scores are formed again, 8 rows at a time.
template <int HD, bool KB, int QT>
__device__ __noinline__ void step_again(const WeighArgs& a, int b, int unit, int per, int kvh, int k0, int k1) {
  const int lane = threadIdx.x & 31, t = lane & 3, g = lane >> 2;
  const WSeq s = weigh_seq<false>(a, b);
  for (int r0 = 0; r0 < s.rows; r0 += 8) {
    const float mine = step_stats(a, s, unit, per, kvh, r0);
    const float big[2] = {__shfl_sync(0xffffffffu, mine, 8 * t), __shfl_sync(0xffffffffu, mine, 8 * t + 4)};
    const int see[2] = {row_sees<false>(a, s, r0 + 2 * t), row_sees<false>(a, s, r0 + 2 * t + 1)};
    QFrag<HD, KB, QT> q;
    q.load(a, s, kvh, r0 / 8, lane);
    for (int k = k0; k < k1; ++k) {
      const int key = k * kStrip + g;
      bool ok;
      const int row = strip_row<false>(a, b, kvh, k * kStrip, &ok);
      Frag<HD, KB, QT> f;
      f.load(a.c.k_pages, row, lane);
      float x[4], w[2] = {0.f, 0.f};
      scores<HD, KB, QT>(f, q.w, x);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (key < see[e]) w[0] += exp2_approx(fmaf(x[e], a.scale_log2, -big[e]));
        if (key + 8 < see[e]) w[1] += exp2_approx(fmaf(x[2 + e], a.scale_log2, -big[e]));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        w[i] += __shfl_xor_sync(0xffffffffu, w[i], 1);
        w[i] += __shfl_xor_sync(0xffffffffu, w[i], 2);
        const int at = key + 8 * i;
        float* to = a.scores + row + g + 8 * i;
        if (t == 0 && ok && at < s.len) *to = w[i] + (r0 ? *to : at < s.fresh ? *to * a.decay : 0.f);
      }
    }
  }
}

template <int HD, bool KB, int QT>
__global__ void __launch_bounds__(kThreads, 3) step_sum_kernel(const __grid_constant__ WeighArgs a) {
  __shared__ StepShares sh;
  __shared__ float big_l[kWarps][8];
  __shared__ int see[kWarps][8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  find_shares(a, &sh, true);
  // the first keys' places and old scores are fetched before the first launch is waited for: it writes neither
  bool waited = false;
  auto wait = [&] {
    if (waited) return;
    pdl_wait();
    pdl_launch_dependents();
    waited = true;
  };
  StepCursor c(a, sh, warp, 1);
  while (c.next(a)) {
    if (c.rb > 0) continue;  // (of the first row block's item)
    if (c.s.rows > a.keep) {
      wait();
      step_again<HD, KB, QT>(a, c.b, c.unit, sh.per, c.kvh, c.k0, c.k1);
      continue;
    }
    // a lane per key, four at a time
    constexpr int N = 4;
    const int end = min(c.k1 * kStrip, c.s.len);
    bool staged = false;
    for (int k0 = c.k0 * kStrip + lane; k0 - lane < end; k0 += N * 32) {
      int row[N];  // -1: none
      float w[N];
      float2 x[N];
#pragma unroll
      for (int i = 0; i < N; ++i) row[i] = k0 + i * 32 < end ? strip_page<false>(a, c.b, k0 + i * 32) : 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        bool ok = false;
        const int key = k0 + i * 32, at = key < end ? row_in(a, row[i], c.kvh, key, &ok) : 0;
        row[i] = ok ? at : -1;
      }
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = row[i] >= 0 && k0 + i * 32 < c.s.fresh ? a.scores[row[i]] : 0.f;
      wait();
      auto kept = [&](int i, int r) {
        return row[i] >= 0 ? __ldcg(reinterpret_cast<const float2*>(a.kept + (long long)row[i] * a.keep + r))
                           : make_float2(0.f, 0.f);
      };
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = kept(i, 0);
      if (!staged) {
        const float l = step_stats(a, c.s, c.unit, sh.per, c.kvh, 0);
        __syncwarp();
        if ((lane & 3) == 0) big_l[warp][lane >> 2] = l, see[warp][lane >> 2] = row_sees<false>(a, c.s, lane >> 2);
        __syncwarp();
        staged = true;
      }
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] *= a.decay;
#pragma unroll 1
      for (int r = 0; r < a.keep; r += 2) {
        const float2 big = *reinterpret_cast<const float2*>(&big_l[warp][r]);
        const int2 n = *reinterpret_cast<const int2*>(&see[warp][r]);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int key = k0 + i * 32;
          w[i] += (key < n.x ? exp2_approx(x[i].x - big.x) : 0.f) + (key < n.y ? exp2_approx(x[i].y - big.y) : 0.f);
        }
        if (r + 2 < a.keep) {
#pragma unroll
          for (int i = 0; i < N; ++i) x[i] = kept(i, r + 2);
        }
      }
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (row[i] >= 0) a.scores[row[i]] = w[i];
    }
  }
  wait();
}

template <int HD, bool KB, int QT>
struct Step {
  static constexpr uint32_t kRing = kWarps * 2 * kStrip * Frag<HD, KB, QT>::kRow;
  static cudaError_t attributes() {
    cudaError_t e = cudaFuncSetAttribute(step_scores_kernel<HD, KB, QT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(step_scores_kernel<HD, KB, QT>, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
    return e;
  }
  static cudaError_t run(const WeighArgs& a, int sms, cudaStream_t s) {
    // (the second launch walks the same shares, so its grid is the first one's)
    const dim3 grid(step_ctas(HD, KB, QT) * sms);
    const cudaError_t e = launch_pdl(step_scores_kernel<HD, KB, QT>, grid, kThreads, kRing, s, a);
    return e == cudaSuccess ? launch_pdl(step_sum_kernel<HD, KB, QT>, grid, kThreads, 0, s, a) : e;
  }
};

template <class Use>
cudaError_t with_types(int hd, bool kv_bf16, bool act_bf16, Use use) {
  if (hd == 64) {
    if (kv_bf16) return act_bf16 ? use(Step<64, true, 1>()) : use(Step<64, true, 3>());
    return act_bf16 ? use(Step<64, false, 1>()) : use(Step<64, false, 3>());
  }
  if (kv_bf16) return act_bf16 ? use(Step<128, true, 1>()) : use(Step<128, true, 3>());
  return act_bf16 ? use(Step<128, false, 1>()) : use(Step<128, false, 3>());
}

}  // namespace

cudaError_t set_weigh_step_attributes() {
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < 8 && e == cudaSuccess; ++i)
    e = with_types(i & 1 ? 64 : 128, i & 2, i & 4, [](auto s) { return s.attributes(); });
  return e;
}
cudaError_t launch_weigh_step(const WeighArgs& a, int hd, int sms, cudaStream_t s) {
  return with_types(hd, a.c.kv_bf16, a.act_bf16, [&](auto x) { return x.run(a, sms, s); });
}

}  // namespace qw
