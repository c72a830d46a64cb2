// qw_paged_attention for few query rows per sequence: the decode step of a ragged batch, with the keys
// read once from their pages where the rows fit one row tile. More rows run as several row tiles that
// each stream the sequence's keys (9 to 16 over bf16 pages always, two or three times; more where the plan finds it
// the shorter way).
//
//   o = sum_j p_j v_j / sum_j p_j,   p_j = 2^(s_j - m),   s_j = log2(e) / sqrt(hd) q . k_j
//
// kept per row as (m, l = sum p, o = sum p v) while the keys stream by; two records of the same
// row join as m' = max, weights 2^(m - m').
//
// One producer warp walks the CTA's units (paged_sched.cuh), looks the pages up one unit ahead and
// streams key and value tiles of 32 KB into a ring with TMA, across item boundaries, so that short
// sequences do not drain the stream; three CTAs per SM (rings of 64 KB) keep 192 KB in flight and fill
// each other's gaps between items. Four consumer warps share every tile by keys, each with its own
// (m, l, o) in registers: no barrier per tile, one join in shared memory per item.
//
// bf16 pages, tiles of up to 8 query rows (kernel _mma): 64-key tiles, products on the tensor cores with mma.sync,
// keys and head columns as the 16-row side and the query rows as the 8-column side. So few rows meet a
// key that a tcgen05 tile of 128 rows would be empty and HBM is the bound: the 64 (NT = 1) or 192 (NT = 3)
// mma of a tile take about 200-600 cycles of an SM whose HBM share delivers its 32 KB in ~1400. f32
// activations keep f32 results: q and P enter as three bf16 terms (24 bits). Measured: 256 sequences of
// up to 8K keys 654 us bf16, 651 f32 (6.8 TB/s, the copy's rate); 256 x 128 keys 35 and 40 us (20 of HBM).
// f32 pages, up to 4 query rows (kernel _fma): 32-key tiles and f32 FMAs, lanes splitting the head
// dimension (512 contiguous bytes of a row per load), scores summed by a transposing butterfly. 256
// sequences of up to 8K keys: 1 256 us (6.9 TB/s).
// f32 pages, up to 8 rows (kernel _mma8): as _mma, with all four operands in three bf16 terms. FMAs for 8
// rows take 1.2 times the HBM time; these products about half of it.
// f32 pages, more rows and few keys (kernel _mma32): tiles of 32 query rows x 32 keys on mma.sync with q, K, P and V
// in three bf16 terms each and the six products above 2^-24. A warp takes 16 rows x 16 keys and splits
// the keys and values in its registers: ~1000 instructions for 256 (row, key) pairs, where the FMA
// kernel needs ~950 for 64. The bound is mma.sync itself, at 3.1 cycles per instruction and SM.

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "paged.h"
#include "paged_sched.cuh"
#include "qw_internal.h"
#include "qw_ptx.cuh"

namespace qw {
namespace {

constexpr int kConsumers = 4;                       // consumer warps
constexpr int kThreads = (kConsumers + 1) * 32;     // and one producer warp

// Shared memory: tile ring, two partial records of the join, then barriers and small words.
template <int HD, int KT, int ES, int R, int RING = 96 * 1024>
struct PgLayout {
  static constexpr uint32_t kRing = RING;
  static constexpr uint32_t kTile = (uint32_t)KT * HD * ES;     // K or V of one stage
  static constexpr int kStages = kRing / (2 * kTile);
  static constexpr uint32_t off_join = kRing;
  static constexpr uint32_t off_ml = off_join + 2u * R * HD * 4 + R * 4;  // [warps][R] (m, l)
  static constexpr uint32_t off_row = off_ml + kConsumers * R * 8;  // [R] joined (m, l)
  static constexpr uint32_t off_start = off_row + R * 8;
  static constexpr uint32_t off_bar = off_start + 96 + 48;
  static constexpr uint32_t bytes = off_bar + 2u * kStages * 8;
  static_assert(sizeof(PagedStart) <= 96, "start words");
};

__device__ __forceinline__ void consumer_sync() {
  asm volatile("bar.sync 1, %0;" ::"r"(kConsumers * 32) : "memory");
}

// ------------------------------------------------------------------ producer
// Lane l of the producer copies one piece of a tile: pieces of a page's rows (and of 128 bytes of
// columns for the swizzled tensor copies), K and V.
template <class LY, int HD, int KT, int ES, bool TENSOR>
__device__ __forceinline__ void produce(const PagedAttnArgs& a, const CUtensorMap* tk,
                                        const CUtensorMap* tv, const PagedStart* st, uint8_t* sm,
                                        uint64_t* full, uint64_t* empty) {
  constexpr int NS = LY::kStages;
  constexpr int COLS = TENSOR ? HD * ES / 128 : 1;  // column blocks of a row
  const int lane = threadIdx.x & 31;
  const int prow = min(KT, 1 << a.c.page_shift);  // rows of a piece
  const int np = KT / prow;                       // pieces of KT keys
  const int piece = lane % np, rest = lane / np;  // piece, then (K or V, column block)
  const bool mine = rest < 2 * COLS;
  const int kv = rest & 1, cb = rest >> 1;
  const uint32_t dst = kv * LY::kTile + (TENSOR ? cb * (KT * 128) + piece * prow * 128
                                                : piece * prow * HD * ES);
  PagedCursor c = paged_cursor<KT>(a, st);
  int issued = 0;
  bool ok = true, more = true;
  auto page_of = [&](const PagedCursor& x) {
    const int key = x.kt * KT + piece * prow;
    return key < x.limit ? paged_page(a, x.b, key) : -1;
  };
  // the item's q rows (gq heads of a token lie together) into L1 for the consumers
  auto fetch_q = [&](const PagedCursor& x) {
    const int bytes = a.gq * HD * (a.act_bf16 ? 2 : 4), tok0 = x.rt * a.tpt;
    const int lines = (bytes + 127) / 128, n = min(a.tpt, x.s.nb - tok0);
    for (int i = lane; i < n * lines; i += 32) {
      const char* p = static_cast<const char*>(a.q) +
                      ((size_t)(x.s.lo + tok0 + i / lines) * a.ldq + (size_t)x.kvh * a.gq * HD) *
                          (a.act_bf16 ? 2 : 4) + i % lines * 128;
      asm volatile("prefetch.global.L1 [%0];" ::"l"(p));
    }
  };
  int page = page_of(c);
  while (more) {
    const int stage = issued % NS;
    const int key = c.kt * KT + piece * prow, kvh = c.kvh, now = page;
    const int pieces = min(np, (max(c.limit - c.kt * KT, 0) + prow - 1) / prow);
    // the next unit's pages, before waiting for this unit's stage
    if (++c.kt == c.kend) {
      more = c.next<KT>(a);
      if (more) fetch_q(c);
    }
    if (more) page = page_of(c);
    // (the lanes vote: one that gives up alone would miss the barriers of the others)
    if (issued >= NS &&
        !__all_sync(0xffffffffu, mbar_wait(&empty[stage], (uint32_t)((issued / NS - 1) & 1), a.wait_ns))) {
      ok = false;
      break;
    }
    if (lane == 0)  // arrives, with 0 bytes for a tile without keys
      mbar_expect_tx(&full[stage], (uint32_t)pieces * prow * HD * ES * 2);
    __syncwarp();
    if (mine && now >= 0) {
      const long long row = paged_row(a, now, kvh, key);
      uint8_t* to = sm + (uint32_t)stage * 2 * LY::kTile + dst;
      if constexpr (TENSOR)
        tma_load_2d(to, kv ? tv : tk, cb * (128 / ES), (int)row, &full[stage]);
      else
        bulk_load(to, static_cast<const float*>(kv ? a.c.v_pages : a.c.k_pages) + row * HD,
                  (uint32_t)prow * HD * ES, &full[stage]);
    }
    ++issued;
  }
  if (!ok && lane == 0 && a.c.status) atomicOr(a.c.status, PG_TIMEOUT);
  // leave only once the copies issued into this CTA's shared memory have landed
  for (int i = max(0, issued - NS); i < issued; ++i)
    mbar_wait(&full[i % NS], (uint32_t)((i / NS) & 1), kDrainNs);
}

// Place of column d of row r in a join record: 8-column groups exchanged by the row, so that the
// rows of an mma fragment do not meet in the same banks.
template <int HD>
__device__ __forceinline__ int join_at(int r, int d) {
  return r * HD + (d ^ ((r >> 1 & 3) << 3));
}

// ------------------------------------------------------------------ end of an item's segment
// The four warps' records are in join[0] + join[1] (o) and row_ml (m, l). A whole item is emitted;
// a split one goes to this CTA's slot and the last CTA to arrive joins all of them in order.
template <int HD, int R>
__device__ __forceinline__ void finish_segment(const PagedAttnArgs& a, const PagedCursor& c,
                                               uint32_t gmul, const float* join, const float2* row_ml,
                                               int* flag) {
  const int tid = threadIdx.x;
  constexpr int V4 = HD / 4;
  const int tok0 = c.rt * a.tpt, rows = min(a.tpt, c.s.nb - tok0) * a.gq;
  const int c0 = c.first_cta(), c1 = c.last_cta();
  const bool whole = c.whole();
  const size_t slot = (size_t)(2 * blockIdx.x + (c.first() ? 1 : 0)) * R;
  if (a.pre.o && !a.prefix_pass) pdl_wait();  // the prefix's records, before any is read
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
    for (int i = tid; i < rows * V4; i += kConsumers * 32) {
      const int r = i / V4, d = (i % V4) * 4;
      PagedAcc acc;
      if (pass == 0) {
        const float4 x = *reinterpret_cast<const float4*>(join + join_at<HD>(r, d));
        const float4 y = *reinterpret_cast<const float4*>(join + R * HD + join_at<HD>(r, d));
        acc.o = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
        acc.m = row_ml[r].x;
        acc.l = row_ml[r].y;
        if (!whole) {
          __stcg(reinterpret_cast<float4*>(a.slots.o + slot * HD) + i, acc.o);
          if (d == 0) __stcg(a.slots.ml + slot + r, make_float2(acc.m, acc.l));
          continue;
        }
      }
      const int t = paged_token(r, gmul), token = c.s.lo + tok0 + t, hg = r - t * a.gq;
      // records to join: this item's, if it was split, then the prefix's
#pragma unroll 1
      for (int src = pass == 1 ? 0 : 1; src < 2; ++src) {
        const float* so = a.slots.o;
        const float2* sml = a.slots.ml;
        size_t row = r, rows_of = R;  // record of CTA z: row (2 z + (z == first)) rows_of + row
        int z0 = c0, z1 = c1;
        if (src == 1) {
          if (!a.pre.o || a.prefix_pass) break;
          const PagedShare p = paged_prefix_share(a, token, c.kvh, hg);
          z0 = p.c0, z1 = p.c1;
          row = p.row, rows_of = a.pre.slots.rows;
          so = a.pre.slots.o, sml = a.pre.slots.ml;
          if (z0 == z1) {  // done whole by one CTA
            row = (size_t)token * a.nq + c.kvh * a.gq + hg, rows_of = 0;
            so = a.pre.o, sml = a.pre.ml;
          }
        }
        constexpr int NB = 8;  // records per round of loads
#pragma unroll 1
        for (int x = z0; x <= z1; x += NB) {
          float2 ml[NB];
          float4 o[NB];
          float top = acc.m;
#pragma unroll
          for (int y = 0; y < NB; ++y) {
            const int z = min(x + y, z1);
            const size_t at = (size_t)(2 * z + (z == z0)) * rows_of + row;
            ml[y] = __ldcg(sml + at);
            o[y] = __ldcg(reinterpret_cast<const float4*>(so + at * HD + d));
          }
#pragma unroll
          for (int y = 0; y < NB; ++y) {
            if (x + y > z1) ml[y].x = -INFINITY;
            top = fmaxf(top, ml[y].x);
          }
          const float mu = top == -INFINITY ? 0.f : top;
          const float f = paged_exp2(acc.m - mu);
          acc.m = top;
          acc.l *= f, acc.o.x *= f, acc.o.y *= f, acc.o.z *= f, acc.o.w *= f;
#pragma unroll
          for (int y = 0; y < NB; ++y) acc.add(paged_exp2(ml[y].x - mu), ml[y].y, o[y]);
        }
      }
      paged_emit<false>(a, HD, token, c.kvh * a.gq + hg, d, acc);
    }
    if (whole || pass == 1) break;
    if (a.prefix_pass) {  // joined by the next launch
      if (c.first() && tid == 0)
        a.splits[blockIdx.x] = PagedSplit{c1, c.s.lo + tok0, rows, c.kvh * a.gq};
      break;
    }
    __threadfence();
    consumer_sync();
    if (tid == 0) {
      const int last = atomicAdd(a.counters + c0, 1) == c1 - c0;
      if (last) a.counters[c0] = 0;  // ready for the next launch
      *flag = last;
    }
    consumer_sync();
    if (!*flag) break;
    __threadfence();
  }
}

// Barriers, the CTA's start; false when there is nothing to do. Every thread of a launch waits for
// the launch before it (pdl_wait) before it leaves, so that stream order holds for what follows.
template <int KT, class LY>
__device__ __forceinline__ bool open_cta(const PagedAttnArgs& a, uint8_t* sm) {
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + LY::off_bar);
  uint64_t* empty = full + LY::kStages;
  PagedStart* st = reinterpret_cast<PagedStart*>(sm + LY::off_start);
  if (threadIdx.x == 0) {
    for (int i = 0; i < LY::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kConsumers);
    }
    fence_barrier_init();
  }
  paged_pdl_open(a);
  if (a.prefix_pass && threadIdx.x == 0) a.splits[blockIdx.x].c1 = -1;
  paged_find_start<KT, kThreads>(a, st, reinterpret_cast<int*>(sm + LY::off_start + 96));
  return st->any;
}

// Gives a tile's stage back once this warp has read it. The fence is needed: with __syncwarp and the arrival
// alone, a tile's last reads came behind the next copy into its stage about once in 10^5 tiles.
__device__ __forceinline__ void release_tile(uint64_t* empty, int lane) {
  __threadfence_block();
  __syncwarp();
  if (lane == 0) mbar_arrive_cta(empty);
}

// Join of the NW records' (m, l) in ml_s [record][R] (a warp's keys each): the rows' (m, l) into
// row_ml, and in ml_s[..].x the factor of each record's o.
template <int R, int NW = kConsumers>
__device__ __forceinline__ void join_rows(float2* ml_s, float2* row_ml) {
  consumer_sync();
  if (threadIdx.x < R) {
    float M = -INFINITY, den = 0.f;
#pragma unroll
    for (int x = 0; x < NW; ++x) M = fmaxf(M, ml_s[x * R + threadIdx.x].x);
    const float mu = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int x = 0; x < NW; ++x) {
      const float w = paged_exp2(ml_s[x * R + threadIdx.x].x - mu);
      den = fmaf(w, ml_s[x * R + threadIdx.x].y, den);
      ml_s[x * R + threadIdx.x].x = w;
    }
    row_ml[threadIdx.x] = make_float2(M, den);
  }
  consumer_sync();
}

// ------------------------------------------------------------------ bf16 pages: mma.sync
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Two floats as three bf16 pairs whose sums carry 24 bits.
__device__ __forceinline__ void split3(float a, float b, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  hi = paged_pack(a, b);
  const float ra = a - __uint_as_float(hi << 16), rb = b - __uint_as_float(hi & 0xffff0000u);
  mid = paged_pack(ra, rb);
  lo = paged_pack(ra - __uint_as_float(mid << 16), rb - __uint_as_float(mid & 0xffff0000u));
}

// 8x8 matrix of 16-bit elements across the warp, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// R = 8 query rows as the n side of the products, keys (16 per warp and tile) and head columns as
// the m side:  S^T = K q^T,  O^T += V^T P^T.  NT = 1: bf16 q and P; NT = 3: three bf16 terms of each, added
// into the same accumulators. P^T comes from S^T's fragment by one 8x8 transpose per 8 keys.
template <int HD>
using MmaLayout = PgLayout<HD, 64, 2, 8, 64 * 1024>;
template <int HD, int NT>
__global__ void __launch_bounds__(kThreads, 3)
    paged_attn_mma_kernel(const __grid_constant__ PagedAttnArgs a,
                          const __grid_constant__ CUtensorMap tk,
                          const __grid_constant__ CUtensorMap tv) {
  constexpr int KT = 64, R = 8, KS = HD / 16, HT = HD / 16;
  using LY = MmaLayout<HD>;
  constexpr int NS = LY::kStages;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + LY::off_bar);
  uint64_t* empty = full + NS;
  PagedStart* st = reinterpret_cast<PagedStart*>(sm + LY::off_start);
  if (!open_cta<KT, LY>(a, sm)) return pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == kConsumers) {
    produce<LY, HD, KT, 2, true>(a, &tk, &tv, st, sm, full, empty);
    return pdl_wait();
  }
  float* join = reinterpret_cast<float*>(sm + LY::off_join);
  float2* ml_s = reinterpret_cast<float2*>(sm + LY::off_ml);
  float2* row_ml = reinterpret_cast<float2*>(sm + LY::off_row);
  int* flag = reinterpret_cast<int*>(sm + LY::off_start + 96 + 40);

  const int g = lane >> 2, q2 = (lane & 3) * 2;  // this thread's keys g, g + 8 and rows q2, q2 + 1
  // ldmatrix rows of this lane: matrices of keys 0-7 / 8-15 and 16-byte chunks of the row.
  // K (plain): keys 8 (matrix % 2), chunk matrix / 2; V (transposed): keys 8 (matrix / 2), chunk matrix % 2
  const int mat = lane >> 3, mr = lane & 7;
  const int krow = 16 * warp + (mat & 1) * 8 + mr, kch = mat >> 1;
  const int vrow = 16 * warp + (mat >> 1) * 8 + mr, vch = mat & 1;
  const uint32_t ring = smem_addr(sm);

  const uint32_t gmul = 65536u / a.gq + 1;
  PagedCursor c = paged_cursor<KT>(a, st);
  int seen = 0;      // tiles taken from the ring
  // A wait gave up: no more tiles, and their stages are not given back (a stage armed again before its copy
  // has come would spoil its barrier), so that the producer gives up too; the block's barriers and the
  // arrivals of split items are still kept.
  bool bad = false;
  do {
    const int n = c.kend - c.kt;
    const int tok0 = c.rt * a.tpt, rows = min(a.tpt, c.s.nb - tok0) * a.gq;
    // q through shared memory (where the join works at the item's end) as B fragments, a plane of
    // [8 rows][HD] per term
    constexpr uint32_t kPlane = 8 * HD * 2;
    {
      uint8_t* to = reinterpret_cast<uint8_t*>(join);
#pragma unroll 1
      for (int i = threadIdx.x; i < R * HD / 8; i += kConsumers * 32) {
        const int r = i / (HD / 8), u = i % (HD / 8), t = paged_token(r, gmul);
        const size_t at = (size_t)(c.s.lo + tok0 + t) * a.ldq + (size_t)(c.kvh * a.gq + r - t * a.gq) * HD + u * 8;
        const uint32_t off = r * (HD * 2) + ((u ^ (r & 7)) << 4);
        uint4 x = make_uint4(0, 0, 0, 0);
        if constexpr (NT == 1) {
          if (r < rows) x = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at));
          *reinterpret_cast<uint4*>(to + off) = x;
        } else {
          uint4 y = x;
          if (r < rows) {
            const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(a.q) + at);
            x = __ldg(q);
            y = __ldg(q + 1);
          }
          uint4 h, m, l;
          split3(__uint_as_float(x.x), __uint_as_float(x.y), h.x, m.x, l.x);
          split3(__uint_as_float(x.z), __uint_as_float(x.w), h.y, m.y, l.y);
          split3(__uint_as_float(y.x), __uint_as_float(y.y), h.z, m.z, l.z);
          split3(__uint_as_float(y.z), __uint_as_float(y.w), h.w, m.w, l.w);
          *reinterpret_cast<uint4*>(to + off) = h;
          *reinterpret_cast<uint4*>(to + kPlane + off) = m;
          *reinterpret_cast<uint4*>(to + 2 * kPlane + off) = l;
        }
      }
    }
    consumer_sync();
    uint32_t qb[NT][KS][2];
    {
      const uint32_t from = smem_addr(join) + mr * (HD * 2);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int ks = 0; ks < KS; ks += 2) {
          uint32_t x[4];
          ldsm4(from + t * kPlane + (((ks * 2 + mat) ^ mr) << 4), x);
          qb[t][ks][0] = x[0], qb[t][ks][1] = x[1], qb[t][ks + 1][0] = x[2], qb[t][ks + 1][1] = x[3];
        }
    }
    int lim[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = q2 + i, t = tok0 + paged_token(r, gmul);
      lim[i] = r >= rows ? 0 : a.prefix_pass ? c.limit : min(max(c.s.base + t + 1, 0), c.s.len);
    }
    float o[HT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int d = 0; d < HT; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;

    for (int x = 0; x < n; ++x, ++seen) {
      const int stage = seen % NS;
      bad = bad || !__all_sync(0xffffffffu, mbar_wait(&full[stage], (uint32_t)((seen / NS) & 1), a.wait_ns));
      if (bad) break;
      const uint32_t kb = ring + (uint32_t)stage * 2 * LY::kTile, vb = kb + LY::kTile;
      float s[4], s2[4];  // even and odd k-steps; with NT = 3 the first terms' and the others' products
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = s2[i] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int ch = ks * 2 + kch;  // 16-byte chunk of the row; 8 of them per column block
        uint32_t kf[4];
        ldsm4(kb + (ch >> 3) * (KT * 128) + krow * 128 + (((ch & 7) ^ (krow & 7)) << 4), kf);
        if constexpr (NT == 1) {
          mma16816(ks & 1 ? s2 : s, kf[0], kf[1], kf[2], kf[3], qb[0][ks][0], qb[0][ks][1]);
        } else {
          mma16816(s, kf[0], kf[1], kf[2], kf[3], qb[0][ks][0], qb[0][ks][1]);
          mma16816(s2, kf[0], kf[1], kf[2], kf[3], qb[2][ks][0], qb[2][ks][1]);
          mma16816(s2, kf[0], kf[1], kf[2], kf[3], qb[1][ks][0], qb[1][ks][1]);
        }
      }
      const int k0 = (c.kt + x) * KT + 16 * warp;  // this warp's first key
      const bool edge = k0 + 16 > c.limit - a.tpt;  // keys some row does not see
      float p[4], alpha[2];  // p[0], p[1]: key g, rows q2 and q2 + 1; p[2], p[3]: key g + 8
      bool moved = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float u = (s[i] + s2[i]) * a.scale_log2, v = (s[2 + i] + s2[2 + i]) * a.scale_log2;
        if (edge || rows < R) {
          if (k0 + g >= lim[i]) u = -INFINITY;
          if (k0 + 8 + g >= lim[i]) v = -INFINITY;
        }
        float mx = fmaxf(u, v);
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const float mn = fmaxf(m[i], mx);
        const float mu = mn == -INFINITY ? 0.f : mn;
        alpha[i] = paged_exp2(m[i] - mu);
        moved = moved || mn != m[i];
        m[i] = mn;
        p[i] = paged_exp2(u - mu);
        p[2 + i] = paged_exp2(v - mu);
        l[i] = l[i] * alpha[i] + (p[i] + p[2 + i]);  // this thread's keys; the lanes are added at the end
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int d = 0; d < HT; ++d)
          o[d][0] *= alpha[0], o[d][1] *= alpha[1], o[d][2] *= alpha[0], o[d][3] *= alpha[1];
      }
      // P^T as B fragments. NT = 1: rounded to bf16, as q, keys and values are, for one product per value
      // instead of two; the sum l takes the unrounded weights. Error against 64 bits 1.9e-3 (256
      // sequences of up to 8K keys), of which the output's own rounding is 1.7e-3. f32 activations keep three terms.
      uint32_t pb[NT][2];
      if constexpr (NT == 1) {
        pb[0][0] = transpose8(paged_pack(p[0], p[1]));
        pb[0][1] = transpose8(paged_pack(p[2], p[3]));
      } else {
        split3(p[0], p[1], pb[0][0], pb[1][0], pb[2][0]);
        split3(p[2], p[3], pb[0][1], pb[1][1], pb[2][1]);
#pragma unroll
        for (int t = 0; t < 3; ++t) pb[t][0] = transpose8(pb[t][0]), pb[t][1] = transpose8(pb[t][1]);
      }
      // values behind the last key are whatever the page held: cleared, since 0 * NaN is NaN
      const int left = c.limit - k0;  // keys of this warp's 16 that exist
      uint32_t vm0 = 0xffffffffu, vm1 = 0xffffffffu;
      if (left < 16) {
        vm0 = (q2 < left ? 0xffffu : 0u) | (q2 + 1 < left ? 0xffff0000u : 0u);
        vm1 = (q2 + 8 < left ? 0xffffu : 0u) | (q2 + 9 < left ? 0xffff0000u : 0u);
      }
#pragma unroll
      for (int d = 0; d < HT; ++d) {
        const int ch = d * 2 + vch;
        uint32_t vf[4];  // head columns 16 d + g (+ 8), keys q2, q2 + 1 (+ 8)
        ldsm4t(vb + (ch >> 3) * (KT * 128) + vrow * 128 + (((ch & 7) ^ (vrow & 7)) << 4), vf);
        if (left < 16) vf[0] &= vm0, vf[1] &= vm0, vf[2] &= vm1, vf[3] &= vm1;
        if constexpr (NT == 1) {
          mma16816(o[d], vf[0], vf[1], vf[2], vf[3], pb[0][0], pb[0][1]);
        } else {  // (mma adds with rounding towards zero: a tile's sum is formed apart)
          float t[4] = {0.f, 0.f, 0.f, 0.f};
          mma16816(t, vf[0], vf[1], vf[2], vf[3], pb[2][0], pb[2][1]);
          mma16816(t, vf[0], vf[1], vf[2], vf[3], pb[1][0], pb[1][1]);
          mma16816(t, vf[0], vf[1], vf[2], vf[3], pb[0][0], pb[0][1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[d][e] += t[e];
        }
      }
      release_tile(&empty[stage], lane);
    }
    // join the warps
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
      if (g == 0) ml_s[warp * R + q2 + i] = make_float2(m[i], l[i]);
    }
    join_rows<R>(ml_s, row_ml);
    const float w0 = ml_s[warp * R + q2].x, w1 = ml_s[warp * R + q2 + 1].x;
    // warps 2 and 3 put their o down, warps 0 and 1 add theirs
#pragma unroll 1
    for (int step = 0; step < 2; ++step) {
      if ((warp < 2) == (step == 1)) {
        float* at = join + (warp & 1) * (R * HD);
#pragma unroll
        for (int d = 0; d < HT; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float& to = at[join_at<HD>(q2 + (e & 1), 16 * d + g + 8 * (e >> 1))];
            to = fmaf(o[d][e], e & 1 ? w1 : w0, step ? to : 0.f);
          }
      }
      consumer_sync();
    }
    finish_segment<HD, R>(a, c, gmul, join, row_ml, flag);
    consumer_sync();  // join and row_ml are free again
  } while (c.next<KT>(a));
  if (bad && lane == 0 && a.c.status) atomicOr(a.c.status, PG_TIMEOUT);
}

// ------------------------------------------------------------------ f32 pages, many rows: mma.sync
// The item's q rows as three bf16 planes [R][HD] in shared memory (where the join works at its end):
// 16-byte units of a row exchanged by the row, columns 4q + e (4q + 2 + e) of a 16-column k-step at its
// positions 2q + e (8 + 2q + e).
template <int HD, int R>
__device__ __forceinline__ void stage_q_terms(const PagedAttnArgs& a, const PagedCursor& c, uint32_t gmul,
                                              int tok0, int rows, uint8_t* to) {
  constexpr uint32_t kPlane = R * HD * 2;
#pragma unroll 1
  for (int i = threadIdx.x; i < R * HD / 8; i += kConsumers * 32) {
    const int r = i / (HD / 8), u = i % (HD / 8), t = paged_token(r, gmul);
    const size_t at = (size_t)(c.s.lo + tok0 + t) * a.ldq + (size_t)(c.kvh * a.gq + r - t * a.gq) * HD + u * 8;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
    if (r < rows) {
      if (a.act_bf16) {
        x = KvElem<true>::load4(static_cast<const uint16_t*>(a.q) + at);
        y = KvElem<true>::load4(static_cast<const uint16_t*>(a.q) + at + 4);
      } else {
        x = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at));
        y = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at + 4));
      }
    }
    uint32_t t0[3], t1[3], t2[3], t3[3];  // terms of columns (0, 1), (2, 3), (4, 5), (6, 7)
    split3(x.x, x.y, t0[0], t0[1], t0[2]);
    split3(x.z, x.w, t1[0], t1[1], t1[2]);
    split3(y.x, y.y, t2[0], t2[1], t2[2]);
    split3(y.z, y.w, t3[0], t3[1], t3[2]);
    uint8_t* row = to + r * (HD * 2) + (u & 1) * 8;
    const int ch = u & ~1;
#pragma unroll
    for (int e = 0; e < 3; ++e) {
      *reinterpret_cast<uint2*>(row + e * kPlane + ((ch ^ (r & 7)) << 4)) = make_uint2(t0[e], t2[e]);
      *reinterpret_cast<uint2*>(row + e * kPlane + (((ch + 1) ^ (r & 7)) << 4)) = make_uint2(t1[e], t3[e]);
    }
  }
}

// Warp (kh, rh) = (warp & 1, warp >> 1) takes keys 16 kh .. and rows 16 rh .. of every 32 x 32 tile.
// Which of a fragment's k and n positions a column or a key takes is free as long as both operands
// agree; the places below let every thread read 16 bytes at once without bank conflicts:
//   scores:  k position 2q + e (8 + 2q + e) of a k-step is column 4q + e (4q + 2 + e); the staged q
//            has its columns in that order; n position n is key n for even n, ((n - 1) ^ 4) + 1 for odd
//   outputs: k positions are the scores' keys; n position n of tile 4 blk + j is column 32 blk + 4n + j
template <int HD>
using Mma32Layout = PgLayout<HD, 32, 4, 32, 64 * 1024>;
template <int HD>
__global__ void __launch_bounds__(kThreads, 2)
    paged_attn_mma32_kernel(const __grid_constant__ PagedAttnArgs a,
                            const __grid_constant__ CUtensorMap tk,
                            const __grid_constant__ CUtensorMap tv) {
  constexpr int KT = 32, R = 32, KS = HD / 16, NB = HD / 32;
  using LY = Mma32Layout<HD>;
  constexpr int NS = LY::kStages;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + LY::off_bar);
  uint64_t* empty = full + NS;
  PagedStart* st = reinterpret_cast<PagedStart*>(sm + LY::off_start);
  if (!open_cta<KT, LY>(a, sm)) return pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == kConsumers) {
    produce<LY, HD, KT, 4, true>(a, &tk, &tv, st, sm, full, empty);
    return pdl_wait();
  }
  float* join = reinterpret_cast<float*>(sm + LY::off_join);
  float2* ml_s = reinterpret_cast<float2*>(sm + LY::off_ml);
  float2* row_ml = reinterpret_cast<float2*>(sm + LY::off_row);
  int* flag = reinterpret_cast<int*>(sm + LY::off_start + 96 + 40);

  const int g = lane >> 2, q = lane & 3, mat = lane >> 3, mr = lane & 7;
  const int kh = warp & 1, rh = warp >> 1;
  const int key_n = g & 1 ? ((g - 1) ^ 4) + 1 : g;         // key of n position g
  const int key_a = 2 * q, key_b = ((2 * q) ^ 4) + 1;      // of n (and k) positions 2q, 2q + 1
  constexpr uint32_t kPlane = R * HD * 2;                  // a term of q
  const uint32_t gmul = 65536u / a.gq + 1;
  PagedCursor c = paged_cursor<KT>(a, st);
  int seen = 0;
  bool bad = false;
  do {
    const int n = c.kend - c.kt;
    const int tok0 = c.rt * a.tpt, rows = min(a.tpt, c.s.nb - tok0) * a.gq;
    stage_q_terms<HD, R>(a, c, gmul, tok0, rows, reinterpret_cast<uint8_t*>(join));
    consumer_sync();
    const uint32_t qrow = smem_addr(join) + (16 * rh + (mat & 1) * 8 + mr) * (HD * 2);
    int lim[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 16 * rh + g + 8 * i, t = tok0 + paged_token(r, gmul);
      lim[i] = r >= rows ? 0 : a.prefix_pass ? c.limit : min(max(c.s.base + t + 1, 0), c.s.len);
    }
    float o[4 * NB][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int d = 0; d < 4 * NB; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;

    for (int x = 0; x < n; ++x, ++seen) {
      const int stage = seen % NS;
      bad = bad || !__all_sync(0xffffffffu, mbar_wait(&full[stage], (uint32_t)((seen / NS) & 1), a.wait_ns));
      if (bad) break;
      const uint8_t* kb = sm + (uint32_t)stage * 2 * LY::kTile;
      const uint8_t* vb = kb + LY::kTile;
      // products of weight 1, 2^-8 and 2^-16 apart: six chains of mma with the two key groups
      float s[2][4], s2[2][4], s3[2][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        s[0][i] = s[1][i] = s2[0][i] = s2[1][i] = s3[0][i] = s3[1][i] = 0.f;
#pragma unroll 2
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t q0[4], q1[4], q2[4];
        const uint32_t ch = ((ks * 2 + (mat >> 1)) ^ mr) << 4;
        ldsm4(qrow + ch, q0);
        ldsm4(qrow + kPlane + ch, q1);
        ldsm4(qrow + 2 * kPlane + ch, q2);
        uint32_t b[2][3], d[2][3];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const int row = 16 * kh + 8 * nt + key_n;
          const float4 k = *reinterpret_cast<const float4*>(
              kb + (ks >> 1) * (KT * 128) + row * 128 + ((((ks & 1) * 4 + q) ^ (row & 7)) << 4));
          split3(k.x, k.y, b[nt][0], b[nt][1], b[nt][2]);
          split3(k.z, k.w, d[nt][0], d[nt][1], d[nt][2]);
        }
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) mma16816(s[nt], q0[0], q0[1], q0[2], q0[3], b[nt][0], d[nt][0]);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) mma16816(s2[nt], q1[0], q1[1], q1[2], q1[3], b[nt][0], d[nt][0]);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) mma16816(s3[nt], q2[0], q2[1], q2[2], q2[3], b[nt][0], d[nt][0]);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) mma16816(s2[nt], q0[0], q0[1], q0[2], q0[3], b[nt][1], d[nt][1]);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) mma16816(s3[nt], q1[0], q1[1], q1[2], q1[3], b[nt][1], d[nt][1]);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) mma16816(s3[nt], q0[0], q0[1], q0[2], q0[3], b[nt][2], d[nt][2]);
      }
      const int k0 = (c.kt + x) * KT + 16 * kh;  // this warp's first key
      const bool edge = k0 + 16 > c.limit - a.tpt;
      float p[2][4], alpha[2];
      bool moved = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mx = -INFINITY;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int nt = e >> 1;
          const int f = 2 * i + (e & 1);
          float v = (s[nt][f] + (s2[nt][f] + s3[nt][f])) * a.scale_log2;
          if ((edge || rows < R) && k0 + nt * 8 + (e & 1 ? key_b : key_a) >= lim[i]) v = -INFINITY;
          p[i][e] = v;
          mx = fmaxf(mx, v);
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[i], mx);
        const float mu = mn == -INFINITY ? 0.f : mn;
        alpha[i] = paged_exp2(m[i] - mu);
        moved = moved || mn != m[i];
        m[i] = mn;
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[i][e] = paged_exp2(p[i][e] - mu);
          sum += p[i][e];
        }
        l[i] = l[i] * alpha[i] + sum;
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int d = 0; d < 4 * NB; ++d)
          o[d][0] *= alpha[0], o[d][1] *= alpha[0], o[d][2] *= alpha[1], o[d][3] *= alpha[1];
      }
      uint32_t pt[3][4];  // P's terms as A fragments
      split3(p[0][0], p[0][1], pt[0][0], pt[1][0], pt[2][0]);
      split3(p[1][0], p[1][1], pt[0][1], pt[1][1], pt[2][1]);
      split3(p[0][2], p[0][3], pt[0][2], pt[1][2], pt[2][2]);
      split3(p[1][2], p[1][3], pt[0][3], pt[1][3], pt[2][3]);
      const int left = c.limit - k0;  // behind the last key lies whatever the page held
#pragma unroll
      for (int blk = 0; blk < NB; ++blk) {
        float v[4][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = (e & 1 ? key_b : key_a) + (e & 2 ? 8 : 0), row = 16 * kh + key;
          const float4 f = *reinterpret_cast<const float4*>(vb + blk * (KT * 128) + row * 128 +
                                                            ((g ^ (row & 7)) << 4));
          const bool in = key < left;
          v[e][0] = in ? f.x : 0.f, v[e][1] = in ? f.y : 0.f, v[e][2] = in ? f.z : 0.f, v[e][3] = in ? f.w : 0.f;
        }
        uint32_t b[4][3], d[4][3];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          split3(v[0][j], v[1][j], b[j][0], b[j][1], b[j][2]);
          split3(v[2][j], v[3][j], d[j][0], d[j][1], d[j][2]);
        }
        float t[4][4];  // (mma adds with rounding towards zero: a tile's sum is formed apart)
#pragma unroll
        for (int j = 0; j < 4; ++j) t[j][0] = t[j][1] = t[j][2] = t[j][3] = 0.f;
        auto add = [&](int pe, int ve) {  // four independent outputs per product
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma16816(t[j], pt[pe][0], pt[pe][1], pt[pe][2], pt[pe][3], b[j][ve], d[j][ve]);
        };
        add(2, 0);
        add(1, 1);
        add(0, 2);
        add(1, 0);
        add(0, 1);
        add(0, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[4 * blk + j][e] += t[j][e];
      }
      release_tile(&empty[stage], lane);
    }
    // the two key halves are the join's two records
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if (q == 0) ml_s[kh * R + 16 * rh + g + 8 * i] = make_float2(m[i], l[i]);
    }
    join_rows<R, 2>(ml_s, row_ml);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 16 * rh + g + 8 * i;
      const float w = ml_s[kh * R + r].x;
      float* at = join + kh * (R * HD);
#pragma unroll
      for (int blk = 0; blk < NB; ++blk)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<float4*>(at + join_at<HD>(r, 32 * blk + 8 * q + 4 * e)) =
              make_float4(o[4 * blk][2 * i + e] * w, o[4 * blk + 1][2 * i + e] * w,
                          o[4 * blk + 2][2 * i + e] * w, o[4 * blk + 3][2 * i + e] * w);
    }
    consumer_sync();
    finish_segment<HD, R>(a, c, gmul, join, row_ml, flag);
    consumer_sync();
  } while (c.next<KT>(a));
  if (bad && lane == 0 && a.c.status) atomicOr(a.c.status, PG_TIMEOUT);
}

// ------------------------------------------------------------------ f32 pages, 5 to 8 rows: mma.sync
// As paged_attn_mma_kernel, with keys and values split into three bf16 terms in registers and six
// products. Two warps take a 32-key tile by halves, the other two the next one. Fragment places as in
// paged_attn_mma32_kernel: a thread reads 16 bytes at once without bank conflicts; output rows g and
// g + 8 of m-tile (blk, t) are columns 32 blk + 4 g + 2 t and the one after it.
// 256 sequences up to 4K keys, 16 heads over 2: 68 us, with FMAs 88; 64 up to 4K, 40 over 8: 83 and 108;
// one of 8K, 16 over 2: 26.8 and 28.7. Two CTAs per SM: the fragments take 168 registers.
template <int HD>
using Mma8Layout = PgLayout<HD, 32, 4, 8, 96 * 1024>;
template <int HD>
__global__ void __launch_bounds__(kThreads, 2)
    paged_attn_mma8_kernel(const __grid_constant__ PagedAttnArgs a,
                           const __grid_constant__ CUtensorMap tk,
                           const __grid_constant__ CUtensorMap tv) {
  constexpr int KT = 32, R = 8, KS = HD / 16, NB = HD / 32;
  using LY = Mma8Layout<HD>;
  constexpr int NS = LY::kStages;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + LY::off_bar);
  uint64_t* empty = full + NS;
  PagedStart* st = reinterpret_cast<PagedStart*>(sm + LY::off_start);
  if (!open_cta<KT, LY>(a, sm)) return pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == kConsumers) {
    produce<LY, HD, KT, 4, true>(a, &tk, &tv, st, sm, full, empty);
    return pdl_wait();
  }
  float* join = reinterpret_cast<float*>(sm + LY::off_join);
  float2* ml_s = reinterpret_cast<float2*>(sm + LY::off_ml);
  float2* row_ml = reinterpret_cast<float2*>(sm + LY::off_row);
  int* flag = reinterpret_cast<int*>(sm + LY::off_start + 96 + 40);

  const int g = lane >> 2, q = lane & 3, mat = lane >> 3, mr = lane & 7;
  const int kh = warp & 1, pair = warp >> 1;
  const int key_m = g & 1 ? ((g - 1) ^ 4) + 1 : g;     // key of m position g
  const int key_a = 2 * q, key_b = ((2 * q) ^ 4) + 1;  // of k positions 2q, 2q + 1 of the outputs
  constexpr uint32_t kPlane = R * HD * 2;
  const uint32_t gmul = 65536u / a.gq + 1;
  PagedCursor c = paged_cursor<KT>(a, st);
  int seen = 0;
  bool bad = false;
  do {
    const int n = c.kend - c.kt;
    const int tok0 = c.rt * a.tpt, rows = min(a.tpt, c.s.nb - tok0) * a.gq;
    stage_q_terms<HD, R>(a, c, gmul, tok0, rows, reinterpret_cast<uint8_t*>(join));
    consumer_sync();
    uint32_t qb[3][KS][2];
    {
      const uint32_t from = smem_addr(join) + mr * (HD * 2);
#pragma unroll
      for (int t = 0; t < 3; ++t)
#pragma unroll
        for (int ks = 0; ks < KS; ks += 2) {
          uint32_t x[4];
          ldsm4(from + t * kPlane + (((ks * 2 + mat) ^ mr) << 4), x);
          qb[t][ks][0] = x[0], qb[t][ks][1] = x[1], qb[t][ks + 1][0] = x[2], qb[t][ks + 1][1] = x[3];
        }
    }
    int lim[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 2 * q + i, t = tok0 + paged_token(r, gmul);
      lim[i] = r >= rows ? 0 : a.prefix_pass ? c.limit : min(max(c.s.base + t + 1, 0), c.s.len);
    }
    float o[2 * NB][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int d = 0; d < 2 * NB; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;

    for (int x = 0; x < n; ++x, ++seen) {
      const int stage = seen % NS;
      bad = bad || !__all_sync(0xffffffffu, mbar_wait(&full[stage], (uint32_t)((seen / NS) & 1), a.wait_ns));
      if (bad) break;
      if ((seen & 1) != pair) {  // the other pair's; a warp that left its phase out would mistake the next
        if (lane == 0) mbar_arrive_cta(&empty[stage]);
        continue;
      }
      const uint8_t* kb = sm + (uint32_t)stage * 2 * LY::kTile;
      const uint8_t* vb = kb + LY::kTile;
      float s[4], s2[4], s3[4];  // products of weight 1, 2^-8 and 2^-16 apart
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = s2[i] = s3[i] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t k[3][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = 16 * kh + 8 * h + key_m;
          const float4 f = *reinterpret_cast<const float4*>(
              kb + (ks >> 1) * (KT * 128) + row * 128 + ((((ks & 1) * 4 + q) ^ (row & 7)) << 4));
          split3(f.x, f.y, k[0][h], k[1][h], k[2][h]);
          split3(f.z, f.w, k[0][2 + h], k[1][2 + h], k[2][2 + h]);
        }
        auto add = [&](float (&d)[4], int ke, int qe) {
          mma16816(d, k[ke][0], k[ke][1], k[ke][2], k[ke][3], qb[qe][ks][0], qb[qe][ks][1]);
        };
        add(s, 0, 0);
        add(s2, 0, 1);
        add(s3, 0, 2);
        add(s2, 1, 0);
        add(s3, 1, 1);
        add(s3, 2, 0);
      }
      const int k0 = (c.kt + x) * KT + 16 * kh;  // this warp's first key
      const bool edge = k0 + 16 > c.limit - a.tpt;
      float p[4], alpha[2];
      bool moved = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float u = (s[i] + (s2[i] + s3[i])) * a.scale_log2;
        float v = (s[2 + i] + (s2[2 + i] + s3[2 + i])) * a.scale_log2;
        if (edge || rows < R) {
          if (k0 + key_m >= lim[i]) u = -INFINITY;
          if (k0 + 8 + key_m >= lim[i]) v = -INFINITY;
        }
        float mx = fmaxf(u, v);
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const float mn = fmaxf(m[i], mx);
        const float mu = mn == -INFINITY ? 0.f : mn;
        alpha[i] = paged_exp2(m[i] - mu);
        moved = moved || mn != m[i];
        m[i] = mn;
        p[i] = paged_exp2(u - mu);
        p[2 + i] = paged_exp2(v - mu);
        l[i] = l[i] * alpha[i] + (p[i] + p[2 + i]);
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int d = 0; d < 2 * NB; ++d)
          o[d][0] *= alpha[0], o[d][1] *= alpha[1], o[d][2] *= alpha[0], o[d][3] *= alpha[1];
      }
      uint32_t pb[3][2];
      split3(p[0], p[1], pb[0][0], pb[1][0], pb[2][0]);
      split3(p[2], p[3], pb[0][1], pb[1][1], pb[2][1]);
#pragma unroll
      for (int t = 0; t < 3; ++t) pb[t][0] = transpose8(pb[t][0]), pb[t][1] = transpose8(pb[t][1]);
      const int left = c.limit - k0;  // behind the last key lies whatever the page held
#pragma unroll
      for (int blk = 0; blk < NB; ++blk) {
        float v[4][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = (e & 1 ? key_b : key_a) + (e & 2 ? 8 : 0), row = 16 * kh + key;
          const float4 f = *reinterpret_cast<const float4*>(vb + blk * (KT * 128) + row * 128 +
                                                            ((g ^ (row & 7)) << 4));
          const bool in = key < left;
          v[e][0] = in ? f.x : 0.f, v[e][1] = in ? f.y : 0.f, v[e][2] = in ? f.z : 0.f, v[e][3] = in ? f.w : 0.f;
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          uint32_t w[3][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            split3(v[0][2 * t + h], v[1][2 * t + h], w[0][h], w[1][h], w[2][h]);
            split3(v[2][2 * t + h], v[3][2 * t + h], w[0][2 + h], w[1][2 + h], w[2][2 + h]);
          }
          // (mma adds with rounding towards zero: a tile's sum is formed apart)
          float d[4] = {0.f, 0.f, 0.f, 0.f}, d2[4] = {0.f, 0.f, 0.f, 0.f};
          auto add = [&](float (&x2)[4], int ve, int pe) {
            mma16816(x2, w[ve][0], w[ve][1], w[ve][2], w[ve][3], pb[pe][0], pb[pe][1]);
          };
          add(d2, 0, 2);
          add(d, 0, 0);
          add(d2, 1, 1);
          add(d2, 2, 0);
          add(d2, 0, 1);
          add(d2, 1, 0);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[2 * blk + t][e] += d[e] + d2[e];
        }
      }
      release_tile(&empty[stage], lane);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
      if (g == 0) ml_s[warp * R + 2 * q + i] = make_float2(m[i], l[i]);
    }
    join_rows<R>(ml_s, row_ml);
#pragma unroll 1
    for (int step = 0; step < 2; ++step) {
      if ((warp < 2) == (step == 1)) {
        float* at = join + (warp & 1) * (R * HD);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float w = ml_s[warp * R + 2 * q + e].x;
#pragma unroll
          for (int blk = 0; blk < NB; ++blk) {
            float4& to = *reinterpret_cast<float4*>(at + join_at<HD>(2 * q + e, 32 * blk + 4 * g));
            const float4 old = step ? to : make_float4(0.f, 0.f, 0.f, 0.f);
            to = make_float4(fmaf(o[2 * blk][e], w, old.x), fmaf(o[2 * blk][2 + e], w, old.y),
                             fmaf(o[2 * blk + 1][e], w, old.z), fmaf(o[2 * blk + 1][2 + e], w, old.w));
          }
        }
      }
      consumer_sync();
    }
    finish_segment<HD, R>(a, c, gmul, join, row_ml, flag);
    consumer_sync();
  } while (c.next<KT>(a));
  if (bad && lane == 0 && a.c.status) atomicOr(a.c.status, PG_TIMEOUT);
}

// ------------------------------------------------------------------ f32 pages: FMAs
template <int E>
struct Lane;  // E consecutive floats of a lane
template <>
struct Lane<4> {
  static __device__ __forceinline__ void load(const float* p, float (&x)[4]) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  }
};
template <>
struct Lane<2> {
  static __device__ __forceinline__ void load(const float* p, float (&x)[2]) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    x[0] = v.x, x[1] = v.y;
  }
};

// R query rows (2 or 4), q and o in registers.
template <int HD, int R>
using FmaLayout = PgLayout<HD, 32, 4, R, 64 * 1024>;
template <int HD, int R>
__global__ void __launch_bounds__(kThreads, 3)
    paged_attn_fma_kernel(const __grid_constant__ PagedAttnArgs a) {
  constexpr int KT = 32, E = HD / 32, KW = KT / kConsumers;  // 8 keys of a tile per warp
  using LY = FmaLayout<HD, R>;
  constexpr int NS = LY::kStages;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + LY::off_bar);
  uint64_t* empty = full + NS;
  PagedStart* st = reinterpret_cast<PagedStart*>(sm + LY::off_start);
  if (!open_cta<KT, LY>(a, sm)) return pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == kConsumers) {
    produce<LY, HD, KT, 4, false>(a, nullptr, nullptr, st, sm, full, empty);
    return pdl_wait();
  }
  float* join = reinterpret_cast<float*>(sm + LY::off_join);
  float2* ml_s = reinterpret_cast<float2*>(sm + LY::off_ml);
  float2* row_ml = reinterpret_cast<float2*>(sm + LY::off_row);
  int* flag = reinterpret_cast<int*>(sm + LY::off_start + 96 + 40);

  const uint32_t gmul = 65536u / a.gq + 1;
  PagedCursor c = paged_cursor<KT>(a, st);
  int seen = 0;
  bool bad = false;
  do {
    const int n = c.kend - c.kt;
    const int tok0 = c.rt * a.tpt, rows = min(a.tpt, c.s.nb - tok0) * a.gq;
    // q, scaled, through shared memory (where the join works at the item's end) into registers
#pragma unroll 1
    for (int i = threadIdx.x; i < R * HD / 4; i += kConsumers * 32) {
      const int r = i / (HD / 4), u = i % (HD / 4), t = paged_token(r, gmul);
      const size_t at = (size_t)(c.s.lo + tok0 + t) * a.ldq + (size_t)(c.kvh * a.gq + r - t * a.gq) * HD + u * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows) {
        if (a.act_bf16)
          x = KvElem<true>::load4(static_cast<const uint16_t*>(a.q) + at);
        else
          x = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at));
      }
      const float k = a.scale_log2;
      *reinterpret_cast<float4*>(join + i * 4) = make_float4(x.x * k, x.y * k, x.z * k, x.w * k);
    }
    consumer_sync();
    float q[R][E], o[R][E], m[R], l[R];
    int lim[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int t = tok0 + paged_token(r, gmul);
      lim[r] = r >= rows ? 0 : a.prefix_pass ? c.limit : min(max(c.s.base + t + 1, 0), c.s.len);
      m[r] = -INFINITY;
      l[r] = 0.f;
      Lane<E>::load(join + r * HD + lane * E, q[r]);
#pragma unroll
      for (int e = 0; e < E; ++e) o[r][e] = 0.f;
    }
    for (int x = 0; x < n; ++x, ++seen) {
      const int stage = seen % NS;
      bad = bad || !__all_sync(0xffffffffu, mbar_wait(&full[stage], (uint32_t)((seen / NS) & 1), a.wait_ns));
      if (bad) break;
      const float* kb = reinterpret_cast<const float*>(sm + (uint32_t)stage * 2 * LY::kTile) +
                        warp * KW * HD + lane * E;
      const float* vb = kb + KT * HD;
      const int k0 = (c.kt + x) * KT + warp * KW;
      float part[R][KW];
#pragma unroll
      for (int k = 0; k < KW; ++k) {
        float kx[E];
        Lane<E>::load(kb + k * HD, kx);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          part[r][k] = q[r][0] * kx[0];
#pragma unroll
          for (int e = 1; e < E; ++e) part[r][k] = fmaf(q[r][e], kx[e], part[r][k]);
        }
      }
      // lanes 4k .. 4k+3 hold key k's score and weight
      float p[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float s = rows_reduce<KW>(part[r], lane);
        if (k0 + (lane >> 2) >= lim[r]) s = -INFINITY;
        float mx = s;
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const float mn = fmaxf(m[r], mx);
        const float mu = mn == -INFINITY ? 0.f : mn;
        if (mn != m[r]) {  // the same on every lane
          const float alpha = paged_exp2(m[r] - mu);
          l[r] *= alpha;
#pragma unroll
          for (int e = 0; e < E; ++e) o[r][e] *= alpha;
          m[r] = mn;
        }
        p[r] = paged_exp2(s - mu);
        l[r] += p[r];  // this lane's key; the eight keys are added at the end
      }
      const int kn = min(KW, c.limit - k0);  // behind the last key lies whatever the page held
#pragma unroll 4
      for (int k = 0; k < kn; ++k) {
        float vx[E];
        Lane<E>::load(vb + k * HD, vx);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float pk = __shfl_sync(0xffffffffu, p[r], 4 * k);
#pragma unroll
          for (int e = 0; e < E; ++e) o[r][e] = fmaf(pk, vx[e], o[r][e]);
        }
      }
      release_tile(&empty[stage], lane);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], d);
      if (lane == 0) ml_s[warp * R + r] = make_float2(m[r], l[r]);
    }
    join_rows<R>(ml_s, row_ml);
#pragma unroll 1
    for (int step = 0; step < 2; ++step) {
      if ((warp < 2) == (step == 1)) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float w = ml_s[warp * R + r].x;
          float* at = join + (warp & 1) * (R * HD) + join_at<HD>(r, lane * E);
#pragma unroll
          for (int e = 0; e < E; ++e) at[e] = fmaf(o[r][e], w, step ? at[e] : 0.f);
        }
      }
      consumer_sync();
    }
    finish_segment<HD, R>(a, c, gmul, join, row_ml, flag);
    consumer_sync();
  } while (c.next<KT>(a));
  if (bad && lane == 0 && a.c.status) atomicOr(a.c.status, PG_TIMEOUT);
}

template <int HD, int NT>
cudaError_t launch_mma(const PagedAttnArgs& a, int grid, cudaStream_t s) {
  CUtensorMap tk, tv;
  const uint64_t rows = (uint64_t)a.c.n_pages * a.c.nkv << a.c.page_shift;
  const uint32_t box = std::min(64, 1 << a.c.page_shift);
  if (!make_tmap_bf16_2d(&tk, a.c.k_pages, rows, HD, box) ||
      !make_tmap_bf16_2d(&tv, a.c.v_pages, rows, HD, box))
    return cudaErrorInvalidValue;
  return launch_pdl(paged_attn_mma_kernel<HD, NT>, dim3(grid), kThreads, MmaLayout<HD>::bytes, s, a,
                    tk, tv);
}
template <int HD, int R>
cudaError_t launch_mma_f32(const PagedAttnArgs& a, int grid, cudaStream_t s) {
  CUtensorMap tk, tv;
  const uint64_t rows = (uint64_t)a.c.n_pages * a.c.nkv << a.c.page_shift;
  const uint32_t box = std::min(32, 1 << a.c.page_shift);
  if (!make_tmap_f32_2d(&tk, a.c.k_pages, rows, HD, box) ||
      !make_tmap_f32_2d(&tv, a.c.v_pages, rows, HD, box))
    return cudaErrorInvalidValue;
  if constexpr (R == 8)
    return launch_pdl(paged_attn_mma8_kernel<HD>, dim3(grid), kThreads, Mma8Layout<HD>::bytes, s, a, tk, tv);
  else
    return launch_pdl(paged_attn_mma32_kernel<HD>, dim3(grid), kThreads, Mma32Layout<HD>::bytes, s, a, tk, tv);
}
template <int HD, int R>
cudaError_t launch_fma(const PagedAttnArgs& a, int grid, cudaStream_t s) {
  return launch_pdl(paged_attn_fma_kernel<HD, R>, dim3(grid), kThreads, FmaLayout<HD, R>::bytes, s, a);
}
template <int HD>
cudaError_t launch_pass(const PagedAttnArgs& a, const PagedPlan& p, cudaStream_t s) {
  if (p.tc) return launch_paged_tc(a, HD, p.grid, s);
  if (a.c.kv_bf16)
    return a.act_bf16 ? launch_mma<HD, 1>(a, p.grid, s) : launch_mma<HD, 3>(a, p.grid, s);
  if (p.rows == 32) return launch_mma_f32<HD, 32>(a, p.grid, s);
  if (p.rows == 8) return launch_mma_f32<HD, 8>(a, p.grid, s);
  if (p.rows == 2) return launch_fma<HD, 2>(a, p.grid, s);
  return launch_fma<HD, 4>(a, p.grid, s);
}

template <class K>
cudaError_t allow_smem(K kernel, uint32_t bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}
template <int HD>
cudaError_t set_attributes_hd() {
  cudaError_t e = allow_smem(paged_attn_mma_kernel<HD, 1>, MmaLayout<HD>::bytes);
  if (e == cudaSuccess) e = allow_smem(paged_attn_mma_kernel<HD, 3>, MmaLayout<HD>::bytes);
  if (e == cudaSuccess) e = allow_smem(paged_attn_mma32_kernel<HD>, Mma32Layout<HD>::bytes);
  if (e == cudaSuccess) e = allow_smem(paged_attn_mma8_kernel<HD>, Mma8Layout<HD>::bytes);
  if (e == cudaSuccess) e = allow_smem(paged_attn_fma_kernel<HD, 2>, FmaLayout<HD, 2>::bytes);
  if (e == cudaSuccess) e = allow_smem(paged_attn_fma_kernel<HD, 4>, FmaLayout<HD, 4>::bytes);
  return e;
}

// Workspace of a call: counters (of the launch over own keys), then split descriptors, O records and
// slots, a copy for each of the two launches, which may overlap; the prefix's whole records. A slot
// holds as many rows as an item can have: at most kMaxRows and at most 8 query heads of every token.
constexpr int kMaxSms = kPagedMaxSms;
constexpr int kMaxCtas = 3 * kMaxSms;  // of a launch
constexpr int kMaxRows = 256;
constexpr size_t align256(size_t v) { return (v + 255) / 256 * 256; }
int slot_rows(int n_tokens) {
  return std::max(16, (int)std::min<long long>(kMaxRows, (8LL * n_tokens + 15) / 16 * 16));
}
struct Workspace {
  size_t counters = 0, splits[2], flush[2], ml[2], o[2], whole_ml, whole_o, total;
  size_t rows;  // of a launch's slots
  Workspace(int n_tokens, int nq, int hd, bool prefix) {
    // tensor-core tiles have one CTA per SM, tiles of 32 rows (from 9 rows on: two tokens) two, smaller three
    rows = (size_t)2 * std::max({kMaxSms * slot_rows(n_tokens),
                                 2 * kMaxSms * (n_tokens > 1 ? 32 : 8), 3 * kMaxSms * 8});
    splits[0] = align256(kMaxCtas * 4);
    splits[1] = splits[0] + align256(kMaxCtas * sizeof(PagedSplit));
    size_t at = splits[1] + align256(kMaxCtas * sizeof(PagedSplit));
    for (int i = 0; i < (prefix ? 2 : 1); ++i) {
      flush[i] = at;
      // (tensor-core tiles have more than 16 rows: three tokens at least)
      ml[i] = at + (n_tokens > 2 ? (size_t)kMaxSms * 128 * 128 * 4 : 0);
      o[i] = ml[i] + align256(rows * 8);
      at = o[i] + align256(rows * hd * 4);
    }
    whole_ml = at;
    whole_o = at + (prefix ? align256((size_t)n_tokens * nq * 8) : 0);
    total = whole_o + (prefix ? (size_t)n_tokens * nq * hd * 4 : 0);
  }
};

}  // namespace

size_t paged_attn_workspace_bytes(int n_tokens, int nq, int hd, bool prefix) {
  return Workspace(n_tokens, nq, hd, prefix).total;
}

cudaError_t set_paged_attributes() {
  cudaError_t e = set_attributes_hd<64>();
  if (e == cudaSuccess) e = set_attributes_hd<128>();
  return e == cudaSuccess ? set_paged_tc_attributes() : e;
}

cudaError_t launch_paged_attention(const PagedAttnArgs& base, int hd, int max_new, void* workspace,
                                   int sms, cudaStream_t s) {
  PagedAttnArgs a = base;
  const bool prefix = a.c.prefix_len > 0;
  const Workspace w(a.n_tokens, a.nq, hd, prefix);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.counters = reinterpret_cast<int*>(ws);
  auto tile_tokens = [&](const PagedPlan& p) { return p.rows > 128 ? 2 * (128 / a.gq) : p.rows / a.gq; };
  auto run = [&](const PagedPlan& p, int i) {
    a.item_units = p.item_units;
    a.least_units = p.least_units;
    a.tpt = tile_tokens(p);
    a.splits = reinterpret_cast<PagedSplit*>(ws + w.splits[i]);
    a.flush = reinterpret_cast<float*>(ws + w.flush[i]);
    a.slots.ml = reinterpret_cast<float2*>(ws + w.ml[i]);
    a.slots.o = reinterpret_cast<float*>(ws + w.o[i]);
    a.slots.rows = p.tc ? slot_rows(a.n_tokens) : p.rows;
    if ((size_t)2 * p.grid * a.slots.rows > w.rows || p.grid > kMaxCtas) return cudaErrorInvalidValue;
    return hd == 64 ? launch_pass<64>(a, p, s) : launch_pass<128>(a, p, s);
  };
  // the line of a launch is counted in 32 bits
  auto too_long = [&](const PagedPlan& p, long long tiles, long long seqs) {
    const long long items = a.n_tokens / tile_tokens(p) + seqs;
    return tiles / p.kt + 8 > INT32_MAX / 2 / a.c.nkv / items;
  };
  const long long cap = (long long)a.c.max_pages << a.c.page_shift;
  // (the lengths are on the device: the longest that the table can hold stands for them)
  auto plan = [&](int seqs, int new_tokens, long long keys) {
    return plan_paged_pass(a.c.kv_bf16, a.act_bf16, a.c.nkv, a.gq, a.n_tokens, seqs, new_tokens, keys, sms);
  };
  const PagedPlan own = plan(a.c.n_seqs, max_new, cap);
  if (too_long(own, cap, a.c.n_seqs)) return cudaErrorInvalidValue;
  if (prefix) {
    a.pre.ml = reinterpret_cast<float2*>(ws + w.whole_ml);
    a.pre.o = reinterpret_cast<float*>(ws + w.whole_o);
    a.prefix_pass = 1;
    const PagedPlan p = plan(1, a.n_tokens, a.c.prefix_len);
    if (too_long(p, a.c.prefix_len, 1)) return cudaErrorInvalidValue;
    cudaError_t e = run(p, 1);
    if (e == cudaSuccess && own.tc) e = launch_paged_join(a, hd, p.grid, p.rows, s);
    if (e != cudaSuccess) return e;
    a.prefix_pass = 0;
    a.pre.slots = a.slots;
    a.pre.tpt = a.tpt;
    a.pre.kt = p.kt;
    a.pre.grid = p.grid;
    a.pre.item_units = p.item_units;
    a.pre.least_units = p.least_units;
  }
  return run(own, 0);
}

}  // namespace qw
