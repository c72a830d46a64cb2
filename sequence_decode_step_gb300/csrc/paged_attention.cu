// qw_paged_attention for few query rows per sequence: the decode step of a ragged batch (and, in
// row tiles, anything else), with the keys read once from their pages.
//
//   o = sum_j p_j v_j / sum_j p_j,   p_j = 2^(s_j - m),   s_j = log2(e) / sqrt(hd) q . k_j
//
// kept per row as (m, l = sum p, o = sum p v) while the keys stream by; two records of the same
// row join as m' = max, weights 2^(m - m').
//
// One producer warp walks the CTA's units (paged_sched.cuh), looks the pages up one unit ahead and
// streams key and value tiles into a ring of 96 KB with TMA, across item boundaries, so that short
// sequences do not drain the stream; two CTAs per SM keep 192 KB in flight. Four consumer warps
// share every tile by keys, each with its own (m, l, o) in registers: no barrier per tile, one
// join in shared memory per item.
//
// bf16 pages (kernel _mma): 64-key tiles, products on the tensor cores with mma.sync. At most 16
// query rows meet a key here, so a tcgen05 tile of 128 rows would be empty and HBM is the bound:
// 128 (NT = 1) or 256 (NT = 3) mma of 64 keys take ~250-500 cycles of an SM whose HBM share
// delivers the tile's 32 KB in ~1400. f32 activations keep f32 results: q and P enter as three
// bf16 terms (24 bits), rows 0-7 of a fragment carrying the first and rows 8-15 the second term,
// the third in a second mma, so R = 8 rows cost two mma instead of three.
// f32 pages (kernel _fma): 32-key tiles and f32 FMAs, lanes splitting the head dimension (512
// contiguous bytes of a row per load), scores summed by a transposing butterfly.

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "paged.h"
#include "paged_sched.cuh"
#include "qw_internal.h"
#include "qw_ptx.cuh"

namespace qw {
namespace {

constexpr int kConsumers = 4;                       // consumer warps
constexpr int kThreads = (kConsumers + 1) * 32;     // and one producer warp
constexpr uint32_t kRing = 96 * 1024;               // bytes of the tile ring

// Shared memory: ring, two partial records of the join, then barriers and small words.
template <int HD, int KT, int ES, int R>
struct PgLayout {
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
// Lane l of the producer copies one piece of a tile: pieces of a page's rows (and of 64 columns
// for the swizzled tensor copies), K and V.
template <int HD, int KT, bool BF>
__device__ __forceinline__ void produce(const PagedAttnArgs& a, const CUtensorMap* tk,
                                        const CUtensorMap* tv, const PagedStart* st, uint8_t* sm,
                                        uint64_t* full, uint64_t* empty) {
  constexpr int ES = BF ? 2 : 4;
  using LY = PgLayout<HD, KT, ES, 8>;  // ring part only: the same for every R
  constexpr int NS = LY::kStages;
  constexpr int COLS = BF ? HD / 64 : 1;  // column blocks of a row
  const int lane = threadIdx.x & 31;
  const int prow = min(KT, 1 << a.c.page_shift);  // rows of a piece
  const int np = KT / prow;                       // pieces of KT keys
  const int piece = lane % np, rest = lane / np;  // piece, then (K or V, column block)
  const bool mine = rest < 2 * COLS;
  const int kv = rest & 1, cb = rest >> 1;
  const uint32_t dst = kv * LY::kTile + (BF ? cb * (KT * 128) + piece * prow * 128
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
    if (issued >= NS && !mbar_wait(&empty[stage], (uint32_t)((issued / NS - 1) & 1), a.wait_ns)) {
      ok = false;
      break;
    }
    if (lane == 0)  // arrives, with 0 bytes for a tile without keys
      mbar_expect_tx(&full[stage], (uint32_t)pieces * prow * HD * ES * 2);
    __syncwarp();
    if (mine && now >= 0) {
      const long long row = paged_row(a, now, kvh, key);
      uint8_t* to = sm + (uint32_t)stage * 2 * LY::kTile + dst;
      if constexpr (BF)
        tma_load_2d(to, kv ? tv : tk, cb * 64, (int)row, &full[stage]);
      else
        bulk_load(to, static_cast<const float*>(kv ? a.c.v_pages : a.c.k_pages) + row * HD,
                  (uint32_t)prow * HD * ES, &full[stage]);
    }
    ++issued;
  }
  if (!__all_sync(0xffffffffu, ok) && lane == 0 && a.c.status) atomicOr(a.c.status, PG_TIMEOUT);
  // leave only once the copies issued into this CTA's shared memory have landed
  for (int i = max(0, issued - NS); i < issued; ++i)
    mbar_wait(&full[i % NS], (uint32_t)((i / NS) & 1), kDrainNs);
}

// ------------------------------------------------------------------ end of an item's segment
// A load that stays in front of what follows it (the compiler moves plain ones down to their uses,
// one round trip each).
__device__ __forceinline__ float4 ld_first(const float4* p) {
  float4 v;
  asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(p));
  return v;
}
// The four warps' records are in join[0] + join[1] (o) and row_ml (m, l). A whole item is emitted;
// a split one goes to this CTA's slot and the last CTA to arrive joins all of them in order.
template <int HD, int R>
__device__ __forceinline__ void finish_segment(const PagedAttnArgs& a, const PagedCursor& c,
                                               float* join, float2* row_ml, int* flag) {
  const int tid = threadIdx.x;
  constexpr int V4 = HD / 4, N = R * V4;
  const int tok0 = c.rt * a.tpt, ntok = min(a.tpt, c.s.nb - tok0), rows = ntok * a.gq;
  auto local = [&](int i) {
    const float4 x = *reinterpret_cast<const float4*>(join + i * 4);
    const float4 y = *reinterpret_cast<const float4*>(join + R * HD + i * 4);
    return make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
  };
  if (a.pre.o && !a.prefix_pass) pdl_wait();  // the prefix's records, before any is read
  if (c.whole()) {
    for (int i = tid; i < N; i += kConsumers * 32) {
      const int r = i / V4;
      if (r >= rows) break;
      PagedAcc acc;
      acc.m = row_ml[r].x;
      acc.l = row_ml[r].y;
      acc.o = local(i);
      paged_emit(a, HD, c.s.lo + tok0 + r / a.gq, c.kvh * a.gq + r % a.gq, (i % V4) * 4, acc);
    }
    return;
  }
  const int c0 = c.first_cta(), c1 = c.last_cta();
  const size_t slot = (size_t)(2 * blockIdx.x + (c.first() ? 1 : 0)) * a.slots.rows;
  for (int i = tid; i < rows * V4; i += kConsumers * 32)
    __stcg(reinterpret_cast<float4*>(a.slots.o + slot * HD) + i, local(i));
  if (tid < rows) __stcg(a.slots.ml + slot + tid, row_ml[tid]);
  if (a.prefix_pass) {  // joined by the next launch
    if (c.first() && tid == 0)
      a.splits[blockIdx.x] = PagedSplit{c1, c.s.lo + tok0, rows, c.kvh * a.gq};
    return;
  }
  __threadfence();
  consumer_sync();
  if (tid == 0) {
    const int last = atomicAdd(a.counters + c0, 1) == c1 - c0;
    if (last) a.counters[c0] = 0;  // ready for the next launch
    *flag = last;
  }
  consumer_sync();
  if (!*flag) return;
  __threadfence();
  // The last CTA: weights of a batch of records in shared memory (a warp per row), then every
  // thread sums its columns over the batch with 16 loads in flight.
  constexpr int NB = 2 * HD, WR = R < kConsumers ? 1 : R / kConsumers, NI = (N + 127) / 128;
  const int warp = tid >> 5, lane = tid & 31;
  float* wgt = join;  // [records][R]
  PagedAcc acc[NI];
  for (int x0 = c0; x0 <= c1; x0 += NB) {
    const int nb = min(NB, c1 + 1 - x0);
    if (x0 > c0) consumer_sync();
#pragma unroll
    for (int j = 0; j < WR; ++j) {
      const int r = warp + j * kConsumers;
      if (r >= R) break;
      float2 ml[NB / 32];
      float top = x0 > c0 ? row_ml[r].x : -INFINITY;
      const float old = top;
#pragma unroll
      for (int k = 0; k < NB / 32; ++k) {
        const int x = x0 + 32 * k + lane;
        ml[k] = make_float2(-INFINITY, 0.f);
        if (32 * k + lane < nb && r < rows) ml[k] = __ldcg(a.slots.ml + (size_t)(2 * x + (x == c0)) * R + r);
        top = fmaxf(top, ml[k].x);
      }
      top = warp_max(top);
      const float mu = top == -INFINITY ? 0.f : top;
      float den = 0.f;
#pragma unroll
      for (int k = 0; k < NB / 32; ++k) {
        if (32 * k >= nb) break;
        const float w = paged_exp2(ml[k].x - mu);
        if (32 * k + lane < nb) wgt[(32 * k + lane) * R + r] = w;
        den = fmaf(w, ml[k].y, den);
      }
      den = warp_sum(den);
      __syncwarp();
      if (lane == 0) {  // y: the sum; the batches before are scaled by 2^(old - top)
        if (x0 > c0) den = fmaf(row_ml[r].y, paged_exp2(old - mu), den);
        row_ml[r] = make_float2(top, den);
      }
      if (x0 > c0 && lane == 0) wgt[nb * R + r] = paged_exp2(old - mu);
    }
    consumer_sync();
#pragma unroll
    for (int k = 0; k < NI; ++k) {
      const int i = tid + 128 * k, r = i / V4;
      if (x0 > c0 && i < rows * V4) {
        const float f = wgt[nb * R + r];
        acc[k].o.x *= f, acc[k].o.y *= f, acc[k].o.z *= f, acc[k].o.w *= f;
      }
    }
    constexpr int NL = 16 / NI;  // records per round of loads
    const float4* o = reinterpret_cast<const float4*>(a.slots.o + (size_t)2 * x0 * R * HD);
    for (int x = 0; x < nb; x += NL) {
      float4 v[NL][NI];
#pragma unroll
      for (int y = 0; y < NL; ++y) {
        const int xx = min(x + y, nb - 1);  // (no branch between the loads)
        const float4* rec = o + (size_t)(2 * xx + (x0 + xx == c0)) * (R * V4);
#pragma unroll
        for (int k = 0; k < NI; ++k) v[y][k] = ld_first(rec + min(tid + 128 * k, N - 1));
      }
#pragma unroll
      for (int y = 0; y < NL; ++y) {
        if (x + y >= nb) break;
#pragma unroll
        for (int k = 0; k < NI; ++k)
          acc[k].add(wgt[(x + y) * R + min((tid + 128 * k) / V4, R - 1)], 0.f, v[y][k]);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < NI; ++k) {
    const int i = tid + 128 * k, r = i / V4;
    if (i >= rows * V4) break;
    acc[k].m = row_ml[r].x;
    acc[k].l = row_ml[r].y;
    paged_emit(a, HD, c.s.lo + tok0 + r / a.gq, c.kvh * a.gq + r % a.gq, (i % V4) * 4, acc[k]);
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
  paged_find_start<KT, kThreads>(a, st, reinterpret_cast<long long*>(sm + LY::off_start + 96));
  return st->any;
}

// Join of the four warps: common maximum per row, then the weights every warp scales its o with.
// Returns through `w` this thread's rows' weights. Rows of this thread: `NRW` of them at `rows`.
template <int R, int NRW>
__device__ __forceinline__ void join_rows(const float (&m)[NRW], const float (&l)[NRW],
                                          const int (&row)[NRW], bool writer, int warp,
                                          float2* ml_s, float2* row_ml, float (&w)[NRW]) {
  if (writer)
#pragma unroll
    for (int i = 0; i < NRW; ++i) ml_s[warp * R + row[i]] = make_float2(m[i], l[i]);
  consumer_sync();
#pragma unroll
  for (int i = 0; i < NRW; ++i) {
    float M = -INFINITY;
#pragma unroll
    for (int x = 0; x < kConsumers; ++x) M = fmaxf(M, ml_s[x * R + row[i]].x);
    const float mu = M == -INFINITY ? 0.f : M;
    w[i] = paged_exp2(m[i] - mu);
    float den = 0.f;
#pragma unroll
    for (int x = 0; x < kConsumers; ++x) {
      const float2 v = ml_s[x * R + row[i]];
      den = fmaf(paged_exp2(v.x - mu), v.y, den);
    }
    if (warp == 0 && writer) row_ml[row[i]] = make_float2(M, den);
  }
}

// ------------------------------------------------------------------ bf16 pages: mma.sync
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
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

// NT = 1: R = 16 rows, bf16 q and P. NT = 3: R = 8 rows, q and P in three bf16 terms.
template <int HD, int NT>
__global__ void __launch_bounds__(kThreads, 2)
    paged_attn_mma_kernel(const __grid_constant__ PagedAttnArgs a,
                          const __grid_constant__ CUtensorMap tk,
                          const __grid_constant__ CUtensorMap tv) {
  constexpr int KT = 64, R = NT == 1 ? 16 : 8, NRW = R / 8, KS = HD / 16, DT = HD / 8;
  using LY = PgLayout<HD, KT, 2, R>;
  constexpr int NS = LY::kStages;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + LY::off_bar);
  uint64_t* empty = full + NS;
  PagedStart* st = reinterpret_cast<PagedStart*>(sm + LY::off_start);
  if (!open_cta<KT, LY>(a, sm)) return pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == kConsumers) {
    produce<HD, KT, true>(a, &tk, &tv, st, sm, full, empty);
    return pdl_wait();
  }
  float* join = reinterpret_cast<float*>(sm + LY::off_join);
  float2* ml_s = reinterpret_cast<float2*>(sm + LY::off_ml);
  float2* row_ml = reinterpret_cast<float2*>(sm + LY::off_row);
  int* flag = reinterpret_cast<int*>(sm + LY::off_start + 96 + 40);

  const int g = lane >> 2, q2 = (lane & 3) * 2;
  // ldmatrix rows of this lane. K (plain): keys 16 warp + (matrix / 2) * 8 + row, chunk matrix % 2.
  // V (transposed): keys 16 warp + (matrix % 2) * 8 + row, chunk matrix / 2.
  const int mat = lane >> 3, mr = lane & 7;
  const int krow = 16 * warp + (mat >> 1) * 8 + mr, kch = mat & 1;
  const int vrow = 16 * warp + (mat & 1) * 8 + mr, vch = mat >> 1;
  const uint32_t ring = smem_addr(sm);

  PagedCursor c = paged_cursor<KT>(a, st);
  int seen = 0;      // tiles taken from the ring
  bool bad = false;  // a wait gave up: no more waits, the barriers are still kept
  do {
    const int n = c.kend - c.kt;
    const int tok0 = c.rt * a.tpt, rows = min(a.tpt, c.s.nb - tok0) * a.gq;
    // q as A fragments: rows g (and g + 8), columns 16 ks + q2 + {0, 1} (and + 8)
    uint32_t qa[KS][4], ql[NT == 3 ? KS : 1][2];
    int lim[NRW];
#pragma unroll
    for (int i = 0; i < NRW; ++i) {
      const int r = g + 8 * i, t = tok0 + r / a.gq;
      lim[i] = a.prefix_pass ? c.limit : min(max(c.s.base + t + 1, 0), c.s.len);
      const bool live = r < rows;
      if (!live) lim[i] = 0;
      const size_t at = (size_t)(c.s.lo + t) * a.ldq + (size_t)(c.kvh * a.gq + r % a.gq) * HD + q2;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const size_t e = at + ks * 16 + hf * 8;
          if constexpr (NT == 1) {
            qa[ks][2 * hf + i] =
                live ? __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) + e))
                     : 0u;
          } else {
            const float2 x = live ? __ldg(reinterpret_cast<const float2*>(
                                        static_cast<const float*>(a.q) + e))
                                  : make_float2(0.f, 0.f);
            split3(x.x, x.y, qa[ks][2 * hf], qa[ks][2 * hf + 1], ql[ks][hf]);
          }
        }
    }
    float o[DT][4], m[NRW], l[NRW];
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
#pragma unroll
    for (int i = 0; i < NRW; ++i) m[i] = -INFINITY, l[i] = 0.f;

    for (int x = 0; x < n; ++x, ++seen) {
      const int stage = seen % NS;
      if (!bad)
        bad = !__all_sync(0xffffffffu, mbar_wait(&full[stage], (uint32_t)((seen / NS) & 1), a.wait_ns));
      const uint32_t kb = ring + (uint32_t)stage * 2 * LY::kTile, vb = kb + LY::kTile;
      float s[2][4], s2[2][4];  // even and odd k-steps: two chains of mma
#pragma unroll
      for (int i = 0; i < 4; ++i) s[0][i] = s[1][i] = s2[0][i] = s2[1][i] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int ch = ks * 2 + kch;  // 16-byte chunk of the row; 8 of them per column block
        uint32_t kf[4];
        ldsm4(kb + (ch >> 3) * (KT * 128) + krow * 128 + (((ch & 7) ^ (krow & 7)) << 4), kf);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          float(&d)[4] = ks & 1 ? s2[nt] : s[nt];
          mma16816(d, qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], kf[2 * nt], kf[2 * nt + 1]);
        }
        if constexpr (NT == 3) {
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
            mma16816(ks & 1 ? s[nt] : s2[nt], ql[ks][0], 0u, ql[ks][1], 0u, kf[2 * nt], kf[2 * nt + 1]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) s[0][i] += s2[0][i], s[1][i] += s2[1][i];
      const int k0 = (c.kt + x) * KT + 16 * warp;  // this warp's first key
      const bool edge = k0 + 16 > c.limit - a.tpt;  // keys some row does not see
      float p[NRW][4];
      bool moved = false;
      float alpha[NRW];
#pragma unroll
      for (int i = 0; i < NRW; ++i) {
        float mx = -INFINITY;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int nt = e >> 1, j = e & 1;
          float v = NT == 3 ? s[nt][j] + s[nt][2 + j] : s[nt][2 * i + j];
          v *= a.scale_log2;
          if ((edge || rows < R) && k0 + nt * 8 + q2 + j >= lim[i]) v = -INFINITY;
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
        l[i] = l[i] * alpha[i] + sum;  // this thread's keys; the four lanes are added at the end
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          o[d][0] *= alpha[0], o[d][1] *= alpha[0];
          o[d][2] *= alpha[NRW - 1], o[d][3] *= alpha[NRW - 1];
        }
      }
      // P as A fragments over this warp's 16 keys
      uint32_t pa[4], pl[2];
      if constexpr (NT == 1) {
        pa[0] = paged_pack(p[0][0], p[0][1]);
        pa[2] = paged_pack(p[0][2], p[0][3]);
        pa[1] = paged_pack(p[NRW - 1][0], p[NRW - 1][1]);
        pa[3] = paged_pack(p[NRW - 1][2], p[NRW - 1][3]);
      } else {
        split3(p[0][0], p[0][1], pa[0], pa[1], pl[0]);
        split3(p[0][2], p[0][3], pa[2], pa[3], pl[1]);
      }
      // values behind the last key are whatever the page held: cleared, since 0 * NaN is NaN
      const int left = c.limit - k0;  // keys of this warp's 16 that exist
      uint32_t vm0 = 0xffffffffu, vm1 = 0xffffffffu;
      if (left < 16) {
        vm0 = (q2 < left ? 0xffffu : 0u) | (q2 + 1 < left ? 0xffff0000u : 0u);
        vm1 = (q2 + 8 < left ? 0xffffu : 0u) | (q2 + 9 < left ? 0xffff0000u : 0u);
      }
#pragma unroll
      for (int d2 = 0; d2 < DT / 2; ++d2) {
        const int ch = d2 * 2 + vch;
        uint32_t vf[4];
        ldsm4t(vb + (ch >> 3) * (KT * 128) + vrow * 128 + (((ch & 7) ^ (vrow & 7)) << 4), vf);
        if (left < 16) vf[0] &= vm0, vf[1] &= vm1, vf[2] &= vm0, vf[3] &= vm1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float(&od)[4] = o[2 * d2 + h];
          mma16816(od, pa[0], pa[1], pa[2], pa[3], vf[2 * h], vf[2 * h + 1]);
          if constexpr (NT == 3) mma16816(od, pl[0], 0u, pl[1], 0u, vf[2 * h], vf[2 * h + 1]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(&empty[stage]);
    }
    // join the warps
#pragma unroll
    for (int i = 0; i < NRW; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    }
    int row[NRW];
    float w[NRW];
#pragma unroll
    for (int i = 0; i < NRW; ++i) row[i] = g + 8 * i;
    join_rows<R, NRW>(m, l, row, (lane & 3) == 0, warp, ml_s, row_ml, w);
    float* mine = join + (warp & 1) * (R * HD);
    auto put = [&](bool add) {
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < NRW; ++i) {
          float2* at = reinterpret_cast<float2*>(mine + (g + 8 * i) * HD + d * 8 + q2);
          float2 v = NT == 3 ? make_float2(o[d][0] + o[d][2], o[d][1] + o[d][3])
                             : make_float2(o[d][2 * i], o[d][2 * i + 1]);
          v.x *= w[i], v.y *= w[i];
          if (add) {
            const float2 b = *at;
            v.x += b.x, v.y += b.y;
          }
          *at = v;
        }
    };
    if (warp >= 2) put(false);
    consumer_sync();
    if (warp < 2) put(true);
    consumer_sync();
    finish_segment<HD, R>(a, c, join, row_ml, flag);
    consumer_sync();  // join and row_ml are free again
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

// R query rows (2, 4 or 8, the least power of two that holds a tile), q and o in registers.
template <int HD, int R>
__global__ void __launch_bounds__(kThreads, 2)
    paged_attn_fma_kernel(const __grid_constant__ PagedAttnArgs a) {
  constexpr int KT = 32, E = HD / 32, KW = KT / kConsumers;  // 8 keys of a tile per warp
  using LY = PgLayout<HD, KT, 4, R>;
  constexpr int NS = LY::kStages;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + LY::off_bar);
  uint64_t* empty = full + NS;
  PagedStart* st = reinterpret_cast<PagedStart*>(sm + LY::off_start);
  if (!open_cta<KT, LY>(a, sm)) return pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == kConsumers) {
    produce<HD, KT, false>(a, nullptr, nullptr, st, sm, full, empty);
    return pdl_wait();
  }
  float* join = reinterpret_cast<float*>(sm + LY::off_join);
  float2* ml_s = reinterpret_cast<float2*>(sm + LY::off_ml);
  float2* row_ml = reinterpret_cast<float2*>(sm + LY::off_row);
  int* flag = reinterpret_cast<int*>(sm + LY::off_start + 96 + 40);

  PagedCursor c = paged_cursor<KT>(a, st);
  int seen = 0;
  bool bad = false;
  do {
    const int n = c.kend - c.kt;
    const int tok0 = c.rt * a.tpt, rows = min(a.tpt, c.s.nb - tok0) * a.gq;
    float q[R][E], o[R][E], m[R], l[R];
    int lim[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int t = tok0 + r / a.gq;
      lim[r] = r >= rows ? 0 : a.prefix_pass ? c.limit : min(max(c.s.base + t + 1, 0), c.s.len);
      m[r] = -INFINITY;
      l[r] = 0.f;
      const size_t at = (size_t)(c.s.lo + t) * a.ldq + (size_t)(c.kvh * a.gq + r % a.gq) * HD + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        o[r][e] = 0.f;
        q[r][e] = r >= rows       ? 0.f
                  : a.act_bf16 ? bf16f(__ldg(static_cast<const uint16_t*>(a.q) + at + e))
                               : __ldg(static_cast<const float*>(a.q) + at + e);
        q[r][e] *= a.scale_log2;
      }
    }
    for (int x = 0; x < n; ++x, ++seen) {
      const int stage = seen % NS;
      if (!bad)
        bad = !__all_sync(0xffffffffu, mbar_wait(&full[stage], (uint32_t)((seen / NS) & 1), a.wait_ns));
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
#pragma unroll
      for (int k = 0; k < KW; ++k) {
        if (k0 + k >= c.limit) break;  // behind the last key lies whatever the page held
        float vx[E];
        Lane<E>::load(vb + k * HD, vx);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float pk = __shfl_sync(0xffffffffu, p[r], 4 * k);
#pragma unroll
          for (int e = 0; e < E; ++e) o[r][e] = fmaf(pk, vx[e], o[r][e]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(&empty[stage]);
    }
    int row[R];
    float w[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      row[r] = r;
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], d);
    }
    join_rows<R, R>(m, l, row, lane == 0, warp, ml_s, row_ml, w);
    float* mine = join + (warp & 1) * (R * HD) + lane * E;
    auto put = [&](bool add) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          float* at = mine + r * HD + e;
          const float v = o[r][e] * w[r];
          *at = add ? *at + v : v;
        }
    };
    if (warp >= 2) put(false);
    consumer_sync();
    if (warp < 2) put(true);
    consumer_sync();
    finish_segment<HD, R>(a, c, join, row_ml, flag);
    consumer_sync();
  } while (c.next<KT>(a));
  if (bad && lane == 0 && a.c.status) atomicOr(a.c.status, PG_TIMEOUT);
}

template <int HD, int NT>
cudaError_t launch_mma(const PagedAttnArgs& a, int grid, cudaStream_t s) {
  constexpr int R = NT == 1 ? 16 : 8;
  CUtensorMap tk, tv;
  const uint64_t rows = (uint64_t)a.c.n_pages * a.c.nkv << a.c.page_shift;
  const uint32_t box = std::min(64, 1 << a.c.page_shift);
  if (!make_tmap_bf16_2d(&tk, a.c.k_pages, rows, HD, box) ||
      !make_tmap_bf16_2d(&tv, a.c.v_pages, rows, HD, box))
    return cudaErrorInvalidValue;
  return launch_pdl(paged_attn_mma_kernel<HD, NT>, dim3(grid), kThreads, PgLayout<HD, 64, 2, R>::bytes, s,
                    a, tk, tv);
}
template <int HD, int R>
cudaError_t launch_fma(const PagedAttnArgs& a, int grid, cudaStream_t s) {
  return launch_pdl(paged_attn_fma_kernel<HD, R>, dim3(grid), kThreads, PgLayout<HD, 32, 4, R>::bytes, s, a);
}
template <int HD>
cudaError_t launch_pass(const PagedAttnArgs& a, const PagedPlan& p, cudaStream_t s) {
  if (p.tc) return launch_paged_tc(a, HD, p.grid, s);
  if (a.c.kv_bf16)
    return a.act_bf16 ? launch_mma<HD, 1>(a, p.grid, s) : launch_mma<HD, 3>(a, p.grid, s);
  if (p.rows == 2) return launch_fma<HD, 2>(a, p.grid, s);
  if (p.rows == 4) return launch_fma<HD, 4>(a, p.grid, s);
  return launch_fma<HD, 8>(a, p.grid, s);
}

template <class K>
cudaError_t allow_smem(K kernel, uint32_t bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}
template <int HD>
cudaError_t set_attributes_hd() {
  cudaError_t e = allow_smem(paged_attn_mma_kernel<HD, 1>, PgLayout<HD, 64, 2, 16>::bytes);
  if (e == cudaSuccess) e = allow_smem(paged_attn_mma_kernel<HD, 3>, PgLayout<HD, 64, 2, 8>::bytes);
  if (e == cudaSuccess) e = allow_smem(paged_attn_fma_kernel<HD, 2>, PgLayout<HD, 32, 4, 2>::bytes);
  if (e == cudaSuccess) e = allow_smem(paged_attn_fma_kernel<HD, 4>, PgLayout<HD, 32, 4, 4>::bytes);
  if (e == cudaSuccess) e = allow_smem(paged_attn_fma_kernel<HD, 8>, PgLayout<HD, 32, 4, 8>::bytes);
  return e;
}

// Workspace of a call: counters and split descriptors, the slots of the two launches, the
// prefix's whole records. A slot holds as many rows as an item can have: at most kMaxRows and at
// most 8 query heads of every token.
constexpr int kMaxSms = 192;         // CTAs per launch: at most two per SM
constexpr int kMaxRows = 256;
constexpr size_t align256(size_t v) { return (v + 255) / 256 * 256; }
int slot_rows(int n_tokens) {
  return std::max(16, (int)std::min<long long>(kMaxRows, (8LL * n_tokens + 15) / 16 * 16));
}
struct Workspace {
  size_t counters = 0, splits[2], ml[2], o[2], whole_ml, whole_o, total;
  Workspace(int n_tokens, int nq, int hd, bool prefix) {
    // an item of more than 16 rows belongs to one CTA per SM, smaller ones to two
    const size_t rows = (size_t)2 * std::max(kMaxSms * slot_rows(n_tokens), 2 * kMaxSms * 16);
    splits[0] = align256(2 * kMaxSms * 4);
    splits[1] = splits[0] + align256(2 * kMaxSms * sizeof(PagedSplit));
    size_t at = splits[1] + align256(2 * kMaxSms * sizeof(PagedSplit));
    for (int i = 0; i < (prefix ? 2 : 1); ++i) {
      ml[i] = at;
      o[i] = at + align256(rows * 8);
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

// max_rows: the most query rows (tokens x heads of a KV head) that meet one key.
PagedPlan plan_paged_pass(const PagedAttnArgs& a, int hd, int max_rows, int sms) {
  sms = std::min(sms, kMaxSms);
  PagedPlan p{};
  if (a.c.kv_bf16) {
    p.tc = max_rows > 16;
    p.kt = p.tc ? kPagedTcKeys : 64;
    p.rows = p.tc ? paged_tc_rows(a.act_bf16) : a.act_bf16 ? 16 : 8;
    p.grid = p.tc ? sms : 2 * sms;
  } else {
    p.kt = 32;
    p.rows = max_rows <= 2 ? 2 : max_rows <= 4 ? 4 : 8;  // the smallest tile that holds them
    p.grid = 2 * sms;
  }
  return p;
}

cudaError_t launch_paged_attention(const PagedAttnArgs& base, int hd, int max_new, void* workspace,
                                   int sms, cudaStream_t s) {
  PagedAttnArgs a = base;
  const bool prefix = a.c.prefix_len > 0;
  const Workspace w(a.n_tokens, a.nq, hd, prefix);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.counters = reinterpret_cast<int*>(ws);
  auto run = [&](const PagedPlan& p, int i) {
    a.tpt = p.rows > 128 ? 2 * (128 / a.gq) : p.rows / a.gq;
    a.splits = reinterpret_cast<PagedSplit*>(ws + w.splits[i]);
    a.slots.ml = reinterpret_cast<float2*>(ws + w.ml[i]);
    a.slots.o = reinterpret_cast<float*>(ws + w.o[i]);
    a.slots.rows = p.tc ? slot_rows(a.n_tokens) : p.rows;
    return hd == 64 ? launch_pass<64>(a, p, s) : launch_pass<128>(a, p, s);
  };
  const long long cap = 1 << 20;  // row counts only choose a kernel
  if (prefix) {
    a.pre.ml = reinterpret_cast<float2*>(ws + w.whole_ml);
    a.pre.o = reinterpret_cast<float*>(ws + w.whole_o);
    a.prefix_pass = 1;
    const PagedPlan p = plan_paged_pass(a, hd, (int)std::min(cap, (long long)a.n_tokens * a.gq), sms);
    cudaError_t e = run(p, 1);
    if (e == cudaSuccess) e = launch_paged_join(a, hd, p.grid, p.rows, s);
    if (e != cudaSuccess) return e;
    a.prefix_pass = 0;
  }
  const int rows = (int)std::min(cap, (long long)std::min(max_new, a.n_tokens) * a.gq);
  return run(plan_paged_pass(a, hd, rows, sms), 0);
}

}  // namespace qw
