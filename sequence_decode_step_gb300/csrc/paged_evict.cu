// qw_paged_evict: every sequence above a budget keeps its newest keys and the best-scored others, per KV
// head, moved together inside the pages it has.
//
// With n keys, budget b and r newest ones: of rows [0, n - r) the b - r of the largest scores stay (ties: the
// lowest row; a NaN is below all). Those in rows below b - r stay where they are, those behind fill the
// others' places, both in ascending order, and the r newest move behind them in order. So a sequence that is
// a few keys over its budget moves these few and its newest, not half of its rows, as an order kept
// throughout would; attention over the cache does not depend on the order of its rows.
//
// A cluster of CTAs serves one sequence and KV head. Each of its CTAs finds the least score that stays by
// histograms over the scores' bits (2048 bins between the least and the largest: two rounds, or three), then
// the places and their fillers by running counts in row order: cheaper than sharing them, and the moves are
// dealt to the CTAs. Bytes bound the moves: 128 sequences of 4K f32 keys cut to 3333, 1.14 GB in 200 us (5.7
// TB/s). 24 prompts of up to 16K keys take 57 us, half of them for the longest one's histograms and counts; one step's
// eviction of 64 sequences 17 us, a chain of barriers and dependent reads.

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "cluster.cuh"
#include "paged.h"

namespace qw {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kCtasPerSm = 2;
constexpr int kPairs = 1024;  // of a place and its filler in shared memory

// Place in the order: a larger score has a larger key; NaN below all, both zeros alike.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0u;
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

struct EvictShared {
  uint32_t hist[kBins];
  uint32_t warp[kWarps], warp2[kWarps];
  uint4 counts[kWarps];
  uint32_t bin, above, in;
  int2 moves[kThreads];  // pool rows: from, to
  int2 pairs[kPairs];    // rows: a place, and its filler
};

struct Rows {  // a sequence's rows under one KV head
  const int* table;
  int head, stride;
  int shift;
  __device__ __forceinline__ int at(int r) const {  // (below 2^31)
    return ((__ldg(table + (r >> shift)) * stride + head) << shift) + (r & ((1 << shift) - 1));
  }
};

// The key of the `want`-th largest of [0, m) in *key, and how many equal to it are among these; lo and hi are the
// least and the largest of this thread's keys.
template <class Key>
__device__ __forceinline__ uint32_t nth_key(EvictShared& s, Key key_of, int m, uint32_t want, uint32_t lo, uint32_t hi,
                                            uint32_t* key) {
  lo = __reduce_min_sync(0xffffffffu, lo), hi = __reduce_max_sync(0xffffffffu, hi);
  if ((threadIdx.x & 31) == 0) s.warp[threadIdx.x >> 5] = lo, s.warp2[threadIdx.x >> 5] = hi;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) lo = min(lo, s.warp[w]), hi = max(hi, s.warp2[w]);
  while (lo < hi) {
    const int sh = max(0, 32 - __clz((int)(hi - lo)) - 11);
    for (int i = threadIdx.x; i < kBins; i += kThreads) s.hist[i] = 0;
    __syncthreads();
    for (int r = threadIdx.x; r < m; r += kThreads) {
      const uint32_t k = key_of(r);
      if (k >= lo && k <= hi) atomicAdd(&s.hist[(k - lo) >> sh], 1u);
    }
    __syncthreads();
    // running counts from the largest bin on, kBins / kThreads bins per thread
    constexpr int C = kBins / kThreads;
    const int first = kBins - 1 - threadIdx.x * C;
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) mine += s.hist[first - i];
    uint32_t sum = mine;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) s.warp[warp] = sum;
    __syncthreads();
    uint32_t above = sum - mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) above += w < warp ? s.warp[w] : 0u;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const uint32_t n = s.hist[first - i];
      if (above < want && above + n >= want) s.bin = first - i, s.above = above, s.in = n;
      above += n;
    }
    __syncthreads();
    const uint32_t bin = s.bin, in = s.in;
    want -= s.above;
    const uint64_t a = (uint64_t)lo + ((uint64_t)bin << sh);
    hi = (uint32_t)min((uint64_t)hi, a + ((uint64_t)1 << sh) - 1);
    lo = (uint32_t)a;
    __syncthreads();
    if (in == want) break;  // all of the bin stay
  }
  *key = lo;
  return want;
}

// Moves the n rows of s.moves, 1 << shift 16-byte columns of keys and values from column col0 on, by the whole block.
__device__ __forceinline__ void move_rows(const EvictShared& s, uint4* k, uint4* v, int row16, int col0, int shift, int n,
                                          bool in_order) {
  constexpr int U = 8;
  const int total = n << shift, mask = (1 << shift) - 1;
  for (int e0 = 0; e0 < total; e0 += U * kThreads) {
    uint4 x[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int e = e0 + i * kThreads + (int)threadIdx.x;
      if (e < total) {
        const int c = col0 + (e & mask);
        x[i] = __ldcg((c < row16 ? k + c : v + (c - row16)) + (long long)s.moves[e >> shift].x * row16);
      }
    }
    if (in_order) __syncthreads();  // rows go down: behind this, nobody reads what is written here
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int e = e0 + i * kThreads + (int)threadIdx.x;
      if (e < total) {
        const int c = col0 + (e & mask);
        (c < row16 ? k + c : v + (c - row16))[(long long)s.moves[e >> shift].y * row16] = x[i];
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads, kCtasPerSm) paged_evict_kernel(EvictArgs a) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ EvictShared s;
  const uint32_t rank = cluster_rank(), ranks = cluster_size();
  const int item = (int)(blockIdx.x / ranks), b = item / a.c.nkv, h = item - b * a.c.nkv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = __ldcg(a.c.kv_len + b);
  const long long cap = (long long)a.c.max_pages << a.c.page_shift;
  const Rows rows{a.c.page_table + (size_t)b * a.c.max_pages, h, a.c.nkv, a.c.page_shift};
  const int row16 = a.row16;

  int bad = n < 0 || n > cap ? PG_BAD_LENGTH : 0;
  bool out = false;
  if (!bad) {
    const int pages = (int)(((long long)n + (1 << a.c.page_shift) - 1) >> a.c.page_shift);
    for (int i = threadIdx.x; i < pages; i += kThreads)
      out |= (unsigned)__ldg(rows.table + i) >= (unsigned)a.c.n_pages;
  }
  if (__syncthreads_or(out)) bad = PG_BAD_PAGE;
  const bool over = !bad && n > a.budget;
  if (bad && threadIdx.x == 0 && rank == 0 && a.c.status) atomicOr(a.c.status, bad);

  if (!bad && !over && a.scores_out != a.scores)
    for (int r = (int)(rank * kThreads + threadIdx.x); r < n; r += (int)(ranks * kThreads)) {
      const int at = rows.at(r);
      a.scores_out[at] = a.scores[at];
    }
  if (over) {
    const int m = n - a.recent, keep = a.budget - a.recent;
    // which rows stay
    const bool kept_here = m <= a.max_keys;
    auto key_at = [&](int r) { return score_key(__ldcg(a.scores + rows.at(r))); };
    uint32_t lo = 0xffffffffu, hi = 0;
    if (kept_here) {  // four rows of a page at a time
      const int groups = (m + 3) / 4;
#pragma unroll 4
      for (int i = threadIdx.x; i < groups; i += kThreads) {
        const float4 x = __ldcg(reinterpret_cast<const float4*>(a.scores + rows.at(4 * i)));
        const uint4 k = make_uint4(score_key(x.x), score_key(x.y), score_key(x.z), score_key(x.w));
        reinterpret_cast<uint4*>(keys)[i] = k;
        lo = min(lo, k.x), hi = max(hi, k.x);
        if (4 * i + 1 < m) lo = min(lo, k.y), hi = max(hi, k.y);
        if (4 * i + 2 < m) lo = min(lo, k.z), hi = max(hi, k.z);
        if (4 * i + 3 < m) lo = min(lo, k.w), hi = max(hi, k.w);
      }
    } else {
      for (int r = threadIdx.x; r < m; r += kThreads) {
        const uint32_t k = key_at(r);
        lo = min(lo, k), hi = max(hi, k);
      }
    }
    __syncthreads();
    auto key_of = [&](int r) { return kept_here ? keys[r] : key_at(r); };
    uint32_t least = 0xffffffffu, ties = 0;
    if (keep > 0) ties = nth_key(s, key_of, m, (uint32_t)keep, lo, hi, &least);
    // A warp takes adjacent rows: running counts, of rows above and at the least key, before and behind
    // the kept ones' places. (With keep == 0 no row stays: `least` is a key that no score has.)
    const int seg = ((m + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int r0 = min(warp * seg, m), r1 = min(r0 + seg, m);
    uint4 mine4 = make_uint4(0, 0, 0, 0);
#pragma unroll 4
    for (int r = r0 + lane; r < r1; r += 32) {
      const uint32_t k = key_of(r);
      const uint32_t more = k > least, same = k == least, front = r < keep;
      mine4.x += more & front, mine4.y += more & (front ^ 1), mine4.z += same & front, mine4.w += same & (front ^ 1);
    }
    mine4.x = __reduce_add_sync(0xffffffffu, mine4.x), mine4.y = __reduce_add_sync(0xffffffffu, mine4.y);
    mine4.z = __reduce_add_sync(0xffffffffu, mine4.z), mine4.w = __reduce_add_sync(0xffffffffu, mine4.w);
    if (lane == 0) s.counts[warp] = mine4;
    __syncthreads();
    // of the warps before this one, and of all: ties, places to fill, and their fillers
    uint32_t eq = 0, eq0 = 0, hole0 = 0, fill0 = 0, pairs = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) eq0 = eq, hole0 = pairs;
      const uint4 n4 = s.counts[w];
      const int w0 = min(w * seg, m), w1 = min(w0 + seg, m), fronts = max(min(w1, keep) - w0, 0);
      const uint32_t left = ties - min(eq, ties), front_ties = min(n4.z, left), back_ties = min(n4.w, left - front_ties);
      pairs += (uint32_t)fronts - n4.x - front_ties;
      if (w < warp) fill0 += n4.y + back_ties;
      eq += n4.z + n4.w;
    }
    // this CTA's pairs of a place and its filler: in shared memory, or (many) in the workspace beside the sequence's
    // first rows
    const uint32_t p0 = (uint32_t)((uint64_t)pairs * rank / ranks), p1 = (uint32_t)((uint64_t)pairs * (rank + 1) / ranks);
    const bool pairs_here = p1 - p0 <= kPairs;
    cluster_sync();  // nobody reads scores any more, if they are in shared memory (they may change in place)
    // HERE: keys and pairs are in shared memory. Four times 32 rows at once and no branches, as a row's steps are a chain
    // of some hundred clocks (24 prompts of up to 16K keys 61 us row by row).
    auto walk = [&](auto here) {
      constexpr bool HERE = decltype(here)::value;
      constexpr int U = HERE ? 4 : 1;
      const uint32_t before = (1u << lane) - 1, mine = p1 - p0;
      int* const to = reinterpret_cast<int*>(s.pairs);
      eq = eq0;
      for (int r = r0; r < r1; r += 32 * U) {
        uint32_t k[U], same[U], hole[U], fill[U];
        bool stays[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int at = r + 32 * i + lane;
          k[i] = at < r1 ? (HERE ? keys[at] : key_of(at)) : 0u;
        }
#pragma unroll
        for (int i = 0; i < U; ++i) same[i] = __ballot_sync(0xffffffffu, r + 32 * i + lane < r1 && k[i] == least);
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int at = r + 32 * i + lane;
          stays[i] = at < r1 && (k[i] > least || (k[i] == least && eq + __popc(same[i] & before) < ties));
          eq += __popc(same[i]);
          hole[i] = __ballot_sync(0xffffffffu, at < r1 && at < keep && !stays[i]);
          fill[i] = __ballot_sync(0xffffffffu, at >= keep && stays[i]);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int at = r + 32 * i + lane;
          const uint32_t j = (stays[i] ? fill0 : hole0) + __popc((stays[i] ? fill[i] : hole[i]) & before) - p0;
          const bool moves = at < r1 && (at < keep) != stays[i] && j < mine;  // (or has its place taken)
          hole0 += __popc(hole[i]), fill0 += __popc(fill[i]);
          if (HERE) {
            if (moves) to[2 * j + stays[i]] = at;
            // (a row that stays is marked by its key: the scores that do not move are copied below)
            if (at < r1) keys[at] = stays[i];
          } else {
            if (moves) {
              if (pairs_here) to[2 * j + stays[i]] = at;
              else reinterpret_cast<int*>(a.pairs + rows.at((int)(p0 + j)))[stays[i]] = at;
            }
            if (kept_here && at < r1) keys[at] = stays[i];
            else if (!kept_here && a.scores_out != a.scores && stays[i] && at < keep && ((at >> 5) & (ranks - 1)) == rank)
              a.scores_out[rows.at(at)] = a.scores[rows.at(at)];
          }
        }
      }
    };
    if (kept_here && pairs_here) walk(std::true_type());
    else walk(std::false_type());
    if (kept_here) __syncthreads();
    else cluster_sync();  // nor have the others scores to read (which may change in place) from here on
    if (kept_here && a.scores_out != a.scores) {
#pragma unroll 4
      for (int r = (int)(rank * kThreads + threadIdx.x); r < keep; r += (int)(ranks * kThreads))
        if (keys[r]) {
          const int at = rows.at(r);
          a.scores_out[at] = __ldcg(a.scores + at);
        }
    }
    uint4* kp = static_cast<uint4*>(a.c.k_pages);
    uint4* vp = static_cast<uint4*>(a.c.v_pages);
    const int mine = (int)(p1 - p0), all_cols = 31 - __clz(2 * row16);
    for (int j0 = 0; j0 < mine; j0 += kThreads) {
      const int j = j0 + (int)threadIdx.x;
      if (j < mine) {
        // (were a page in two places of the table, another item could have written here: stay in the table)
        const int2 x = pairs_here ? s.pairs[j] : __ldcg(&a.pairs[rows.at((int)p0 + j)]);
        const int2 r = make_int2(rows.at((int)min((uint32_t)x.y, (uint32_t)n - 1)),
                                 rows.at((int)min((uint32_t)x.x, (uint32_t)n - 1)));
        s.moves[threadIdx.x] = r;
        a.scores_out[r.y] = __ldcg(a.scores + r.x);
      }
      __syncthreads();
      move_rows(s, kp, vp, row16, 0, all_cols, min(mine - j0, kThreads), false);
      __syncthreads();
    }
    cluster_sync();  // the fillers have been read: their rows may be written
    // the newest rows move down, each CTA with its columns
    const int cols = 2 * row16 / (int)ranks, shift = 31 - __clz(cols);
    for (int j0 = 0; j0 < a.recent; j0 += kThreads) {
      const int j = j0 + (int)threadIdx.x;
      float x = 0.f;
      if (j < a.recent) {
        s.moves[threadIdx.x] = make_int2(rows.at(m + j), rows.at(keep + j));
        if (rank == ranks - 1) x = __ldcg(a.scores + s.moves[threadIdx.x].x);
      }
      __syncthreads();
      if (j < a.recent && rank == ranks - 1) a.scores_out[s.moves[threadIdx.x].y] = x;
      move_rows(s, kp, vp, row16, (int)rank * cols, shift, min(a.recent - j0, kThreads), n - a.budget < a.recent);
      __syncthreads();
    }
  }
  if (h == 0 && threadIdx.x == 0 && rank == 0) a.new_len[b] = over ? a.budget : n;
}

// The new lengths into kv_len itself, once every KV head has read the old ones.
__global__ void __launch_bounds__(256) evict_lengths_kernel(const int* from, int* to, int n) {
  pdl_wait();
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < n) to[i] = __ldcg(from + i);
}

// Most scores of a sequence in shared memory: 160 KB, or 64 KB where there are CTAs enough for two on an SM (each has 20 KB
// of EvictShared besides, of 228).
constexpr int kMostKeys = 40960, kManyKeys = 16384;

}  // namespace

cudaError_t set_evict_attributes() {
  return cudaFuncSetAttribute(paged_evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostKeys * 4);
}

cudaError_t launch_paged_evict(const EvictArgs& base, int sms, cudaStream_t s) {
  EvictArgs a = base;
  const long long items = (long long)a.c.n_seqs * a.c.nkv, cap = (long long)a.c.max_pages << a.c.page_shift;
  int ranks = 1;
  while (ranks < 8 && items * ranks * 2 <= kCtasPerSm * sms) ranks *= 2;
  a.max_keys = (int)std::min<long long>((cap + 3) / 4 * 4, items * ranks > sms ? kManyKeys : kMostKeys);
  const bool in_place = a.kv_len_out == a.c.kv_len;
  a.new_len = in_place ? a.kept_len : a.kv_len_out;
  cudaError_t e = launch_cluster(paged_evict_kernel, (unsigned)(items * ranks), ranks, kThreads,
                                 (size_t)a.max_keys * 4, s, a);
  if (e == cudaSuccess && in_place)
    e = launch_pdl(evict_lengths_kernel, dim3((a.c.n_seqs + 255) / 256), 256, 0, s, (const int*)a.kept_len,
                   a.kv_len_out, a.c.n_seqs);
  return e;
}

}  // namespace qw
