// qw_paged_attention for many query rows per key: a prefix that a batch shares, and chunks of
// prompts. tcgen05 tiles of 128 query rows x 128 keys (bf16 pages) or 64 keys (f32 pages).
//
//   S = Q K^T (TMEM, f32),  P = 2^(s scale - m) as bf16 back into TMEM,  O += P V (TMEM, f32)
//
// with the running maximum m and sum of a row in the registers of the one thread that owns the
// row. P as bf16 (NT = 1) is the A operand's type beside bf16 values: two terms would double P V for an error
// of 2.3e-3 against 64 bits (chunks of 512, 32K prefix), 1.7e-3 of it the output's own rounding; l takes the
// unrounded weights.
// m only moves when a row's maximum rises by more than 8 (P stays below 2^8, l and O in f32),
// so the rescaling of O in TMEM is rare. K tiles are K-major and V tiles MN-major as their pages
// hold them (rows of head_dim): nothing is transposed.
//
// bf16 activations (NT = 1): two row tiles (streams) of 128 rows per CTA share the key tiles, which
// halves their L2 traffic, and the tensor core works on one stream's products while the other
// stream's warps form their exponentials. A stream's P overwrites its S. Per stream and tile the
// products take 2 x 128^3 MACs = 1024 cycles at the dense bf16 rate and the 128 x 128 exponentials
// and packing about as long, so two streams keep the tensor core busy.
// f32 activations (NT = 3): q and P as three bf16 terms each (24 bits, f32 results), six products
// per tile, one stream with two S buffers; the tensor core is the bound by itself. Its accumulators
// round every addition towards zero, about 1.2e-8 of the value per product: 1.8e-5 over 64 tiles when
// they ran into one O. So the small terms go first into S, and every kFlush tiles O moves into a record
// in L2 that is added to in f32 (round to nearest): below 1e-6 at any length, at 414 TFLOP/s of the formula's
// products (32K keys, 4096 rows); every 4 tiles it would be 1.8e-6 at 494.
//
// f32 pages (F; NT = 3): keys and values as three bf16 terms as well, six products each for S and O. Eight
// warps of their own load the pages into registers, a tile ahead, and write the terms as three swizzled
// planes (four warps with 16 keys each were the bound at 3.4 us a tile, eight take 2.5). Three q and six
// key and value planes leave room for one tile of 64 keys: its keys are split while P V of the tile before
// runs, its values during the next tile's scores. A product q . k reads 4 KB of q and 2 KB of k from shared
// memory, 48 cycles where the tensor core needs 32, so q's first term, half of the products, lies in TMEM.
// The small products of P V have an accumulator of their own, so that O takes 4 additions a tile at full
// size and moves to the record every 8 tiles. 238 TFLOP/s (32K keys, 4096 rows); mma.sync tiles: 61.
//
// Warps: 0 page look-up and TMA, 1 MMA issue, 2-5 softmax, 6-9 softmax (NT = 1), 6-13 the planes (f32
// pages); TMEM is S/P and O:
//   NT = 1: S_A, S_B (128 columns each), O_A, O_B
//   NT = 3: S_0, S_1, O, X_0, X_1 (64 each); P's first two terms overwrite S_i, the third is in X_i
//   f32 pages: S_0, S_1 (64 each), X_0, X_1 (32 each), q's first term (64), O, O's small products
// Work is shared as in paged_sched.cuh with one CTA per SM (its tiles fill the shared memory).

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


// mbar_wait inlined: a call in the softmax loop would have to save the row of scores around it. A limit
// of 0 is not looked at here: a warp whose waits give up at once begins as one that has given up.
__device__ __forceinline__ bool wait_for(uint64_t* bar, int phase, uint64_t limit_ns) {
  uint64_t t0 = 0;
  for (uint32_t n = 1;; ++n) {
    if (mbar_try_wait(bar, (uint32_t)(phase & 1))) return true;
    if ((n & 15u) != 0) continue;
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    else if (now - t0 > limit_ns) return false;
  }
}

// Two f32 operations in one instruction.
__device__ __forceinline__ float2 fma2(const float2& a, const float2& b, const float2& c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)),
        "l"(*reinterpret_cast<const uint64_t*>(&c)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 add2(const float2& a, const float2& b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}

// TMEM columns of O, of X_i (NT = 3), of O's small products and q's first term (f32 pages)
constexpr uint32_t kO = 256, kO2 = 384, kQ0 = 192;
template <bool F>
constexpr uint32_t kX = F ? 128 : 384;

// F: f32 pages (NT = 3).
template <int HD, int NT, bool F>
struct TcLayout {
  static constexpr int KT = paged_tc_keys(!F);
  static constexpr int kStreams = NT == 1 ? 2 : 1;
  static constexpr int kThreads = 64 + 128 * kStreams + (F ? 256 : 0);
  static constexpr uint32_t kQ1 = 128 * HD * 2;            // one term of a stream's q tile
  static constexpr uint32_t kQ = kQ1 * (NT == 1 ? 2 : 3);
  static constexpr uint32_t kPlane = KT * HD * 2;
  static constexpr uint32_t kTile = kPlane * (F ? 3 : 1);  // a K or V tile
  static constexpr int kFit = (224 * 1024 - kQ) / kTile;
  static constexpr int kSlots = F ? kFit / 2 * 2 : kFit > 10 ? 10 : kFit;
  // Tile g's keys are use 2g of the ring, its values use 2g + 1. With f32 pages the two take turns out of
  // this order and have a ring each.
  static __device__ __forceinline__ int slot(int use) {
    return F ? (use & 1) * (kSlots / 2) + (use >> 1) % (kSlots / 2) : use % kSlots;
  }
  static __device__ __forceinline__ int phase(int use) {
    return F ? (use >> 1) / (kSlots / 2) : use / kSlots;
  }
  static constexpr uint32_t off_ring = kQ;
  static constexpr uint32_t off_start = off_ring + kSlots * kTile;
  static constexpr uint32_t off_bar = off_start + 96 + 128;
  static constexpr int kBars = 2 * kSlots + 11;
  static constexpr uint32_t off_tmem = off_bar + kBars * 8;
  static constexpr uint32_t bytes = off_tmem + 16;
  static constexpr uint32_t t_s = F ? 64 : 128;            // TMEM columns between S buffers or streams
  static constexpr int kFlush = F ? 8 : 2;                 // tiles of one O (NT = 3)
  static_assert(sizeof(PagedStart) <= 96, "start words");
  static_assert(bytes <= 227 * 1024, "tiles fit one CTA's shared memory");
};

__device__ __forceinline__ void split3(float a, float b, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  hi = paged_pack(a, b);
  const float ra = a - __uint_as_float(hi << 16), rb = b - __uint_as_float(hi & 0xffff0000u);
  mid = paged_pack(ra, rb);
  lo = paged_pack(ra - __uint_as_float(mid << 16), rb - __uint_as_float(mid & 0xffff0000u));
}

// O of this thread's row into its column of the CTA's record [HD][128 rows], whose earlier
// contents are scaled by f (nothing before the first time). ready() waits for O, under the first loads.
template <int HD, bool F, class Ready>
__device__ __forceinline__ void add_record(float* rec, uint32_t to, bool first, float f, Ready ready) {
  if (!F) ready();
#pragma unroll 1
  for (int d = 0; d < HD; d += 64) {
    float old[64];
#pragma unroll
    for (int e = 0; e < 64; ++e) old[e] = first ? 0.f : __ldcg(rec + (d + e) * 128);
    if (F && d == 0) ready();
    constexpr int C = F ? 1 : 4;  // 16 columns each
#pragma unroll
    for (int i0 = 0; i0 < 4; i0 += C) {
      uint32_t o[C][16], o2[16];
#pragma unroll
      for (int i = 0; i < C; ++i) tmem_ld16(to + d + 16 * (i0 + i), o[i]);
      if constexpr (F) tmem_ld16(to + (kO2 - kO) + d + 16 * i0, o2);
      tmem_ld_wait();
      if constexpr (F) tmem_regs_ready(o2);
#pragma unroll
      for (int i = 0; i < C; ++i) {
        tmem_regs_ready(o[i]);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float x = __uint_as_float(o[i][e]) + (F ? __uint_as_float(o2[e]) : 0.f);
          __stcg(rec + (d + 16 * (i0 + i) + e) * 128, fmaf(old[16 * (i0 + i) + e], f, x));
        }
      }
    }
  }
}

__device__ __forceinline__ float4 load_once(const float* p) {  // 16 bytes that this SM does not read again
  float4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(p));
  return v;
}

// f32 pages: one of eight warps' 8 keys of a tile, split into the three bf16 planes [KT][HD] of a K or V
// tile (rows of 128 bytes with 128-byte swizzling, as TMA writes them for bf16 pages). A load takes 512
// bytes of a page; keys behind the last one are zeros.
template <int HD>
struct TcRows {
  static constexpr int kKeys = 8, RPI = 128 / HD, N = kKeys / RPI;  // rows per load, loads
  float4 v[N];
  __device__ __forceinline__ void load(const float* pages, long long row, int keys, int lane) {
    const int sub = lane / (HD / 4), col = lane % (HD / 4) * 4;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i * RPI + sub < keys) v[i] = load_once(pages + (row + i * RPI + sub) * HD + col);
    }
  }
  template <uint32_t PLANE>
  __device__ __forceinline__ void store(uint8_t* tile, int w, int lane) const {
    const int sub = lane / (HD / 4), u = lane % (HD / 4);
    uint8_t* to = tile + (u >> 4) * (64 * 128) + (u & 1) * 8;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int row = kKeys * w + i * RPI + sub;
      uint2 t[3];
      split3(v[i].x, v[i].y, t[0].x, t[1].x, t[2].x);
      split3(v[i].z, v[i].w, t[0].y, t[1].y, t[2].y);
#pragma unroll
      for (int e = 0; e < 3; ++e)
        *reinterpret_cast<uint2*>(to + e * PLANE + row * 128 + ((((u >> 1) & 7) ^ (row & 7)) << 4)) = t[e];
    }
  }
};

template <int HD, int NT, bool F>
__global__ void __launch_bounds__(TcLayout<HD, NT, F>::kThreads, 1)
    paged_attn_tc_kernel(const __grid_constant__ PagedAttnArgs a, const __grid_constant__ CUtensorMap tk,
                         const __grid_constant__ CUtensorMap tv) {
  using LY = TcLayout<HD, NT, F>;
  constexpr int KT = LY::KT, NS = LY::kSlots, QA = HD / 64, kFlush = LY::kFlush;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(sm + LY::off_bar);
  uint64_t* kv_empty = kv_full + NS;
  uint64_t* q_full = kv_empty + NS;
  uint64_t* s_full = q_full + 2;   // NT = 1: of each stream; NT = 3: of each S buffer
  uint64_t* p_full = s_full + 2;   // NT = 1: of each stream; NT = 3: p_full[0]
  uint64_t* p_half = p_full + 2;   // NT = 1: the first 64 keys' weights of each stream
  uint64_t* o_full = p_half + 2;   // NT = 1: the end of an item, of each stream; NT = 3: every tile
  uint64_t* done = o_full + 2;     // every MMA of this CTA has finished
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + LY::off_tmem);
  PagedStart* st = reinterpret_cast<PagedStart*>(sm + LY::off_start);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&kv_full[i], F ? 8 : 1);          // the converting warps, or the tensor copies
      mbar_init(&kv_empty[i], NT == 1 ? 2 : 1);  // the streams' softmax warps, or a commit
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 4);  // one arrival per softmax warp
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&p_half[i], 4);
      mbar_init(&o_full[i], 1);
    }
    mbar_init(done, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tslot, 512);
    tmem_relinquish();
  }
  paged_pdl_open(a);
  if (threadIdx.x == 0) a.splits[blockIdx.x].c1 = -1;
  tc_fence_before();
  paged_find_start<KT, LY::kThreads>(a, st, reinterpret_cast<int*>(sm + LY::off_start + 96));
  tc_fence_after();
  const uint32_t tb = *tslot;
  const int half = 128 / a.gq;  // tokens of a row tile
  const bool idle = !st->any;

  if (idle) {
  } else if (F && warp == 0) {
  } else if (F && warp >= 6) {
    // ---- f32 pages into the planes. The tensor core's order is S_0, then S_(g+1), P V_g: the keys of tile
    // g + 1 are split during P V_(g-1), the values of tile g during S_(g+1). A thread's next rows of
    // both are in flight meanwhile.
    const int w = warp - 6;
    PagedCursor c = paged_cursor<KT>(a, st);
    TcRows<HD> k, v;
    struct Place {
      long long row;
      int keys;
    };
    bool ok = a.wait_ns != 0, more = true;
    int page = 0;  // of the cursor's tile, not yet checked, so that nothing waits for it before it is used
    auto find = [&] {
      const int key = c.kt * KT + TcRows<HD>::kKeys * w;
      if (key < c.limit) page = paged_page_entry(a, c.b, key);
    };
    auto take = [&] {  // the cursor's place; on to the next tile
      const int key = c.kt * KT + TcRows<HD>::kKeys * w, keys = c.limit - key;
      const Place x{keys > 0 ? paged_row(a, paged_page_checked(a, page), c.kvh, key) : 0, keys};
      if (++c.kt == c.kend) more = c.next<KT>(a);
      if (more) find();
      return x;
    };
    auto load = [&](TcRows<HD>& x, const void* pages, const Place& at) {
      x.load(static_cast<const float*>(pages), at.row, at.keys, lane);
    };
    auto put = [&](const TcRows<HD>& x, int use) {
      const int slot = LY::slot(use), n = LY::phase(use);
      if (ok && n > 0) ok = __all_sync(0xffffffffu, wait_for(&kv_empty[slot], n - 1, a.wait_ns));
      if (!ok) return;
      x.template store<LY::kPlane>(sm + LY::off_ring + slot * LY::kTile, w, lane);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(&kv_full[slot]);
    };
    find();
    Place at = take();
    load(k, a.c.k_pages, at);
    load(v, a.c.v_pages, at);
    put(k, 0);
    bool ahead = more;  // k holds tile g + 1, v tile g
    if (more) {
      at = take();
      load(k, a.c.k_pages, at);
    }
#pragma unroll 1
    for (int g = 0; ok; ++g) {
      const Place now = at;
      const bool was = ahead;
      if (was) put(k, 2 * g + 2);
      ahead = more;
      if (more) {
        at = take();
        load(k, a.c.k_pages, at);
      }
      put(v, 2 * g + 1);
      if (!was) break;
      load(v, a.c.v_pages, now);
    }
    if (!ok && lane == 0 && a.c.status) atomicOr(a.c.status, PG_TIMEOUT);
  } else if (warp == 0) {
    // ---- producer: lane = (K or V) x column block x piece of a page's rows
    const int prow = min(KT, 1 << a.c.page_shift), np = KT / prow;
    const int piece = lane % np, cb = (lane / np) % QA, kv = lane / (np * QA);
    const bool mine = kv < 2;
    PagedCursor c = paged_cursor<KT>(a, st);
    auto page_of = [&](const PagedCursor& x) {
      const int key = x.kt * KT + piece * prow;
      return key < x.limit ? paged_page(a, x.b, key) : -1;
    };
    int page = page_of(c), issued = 0;
    bool ok = a.wait_ns != 0, more = true;
    while (ok && more) {
      const int key = c.kt * KT + piece * prow, kvh = c.kvh, now = page;
      const int pieces = min(np, (max(c.limit - c.kt * KT, 0) + prow - 1) / prow);
      if (++c.kt == c.kend) {
        more = c.next<KT>(a);
        if (more) {  // its q rows (gq heads of a token lie together) into L2
          const int bytes = a.gq * HD * (NT == 1 ? 2 : 4), lines = bytes / 128;
          const int n = min(a.tpt, c.s.nb - c.rt * a.tpt);
          for (int i = lane; i < n * lines; i += 32) {
            const char* q = static_cast<const char*>(a.q) +
                            ((size_t)(c.s.lo + c.rt * a.tpt + i / lines) * a.ldq + (size_t)c.kvh * a.gq * HD) *
                                (NT == 1 ? 2 : 4) + i % lines * 128;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
          }
        }
      }
      if (more) page = page_of(c);
#pragma unroll 1
      for (int t = 0; t < 2; ++t) {
        const int slot = issued % NS;
        if (issued >= NS &&
            !__all_sync(0xffffffffu,
                        wait_for(&kv_empty[slot], issued / NS - 1, a.wait_ns))) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_expect_tx(&kv_full[slot], (uint32_t)pieces * prow * HD * 2);
        __syncwarp();
        if (mine && kv == t && now >= 0)
          tma_load_2d(sm + LY::off_ring + slot * LY::kTile + cb * (KT * 128) + piece * prow * 128,
                      t ? &tv : &tk, cb * 64, (int)paged_row(a, now, kvh, key), &kv_full[slot]);
        ++issued;
      }
    }
    if (!ok && lane == 0 && a.c.status) atomicOr(a.c.status, PG_TIMEOUT);
    for (int i = max(0, issued - NS); i < issued; ++i)  // the copies have landed
      wait_for(&kv_full[i % NS], i / NS, kDrainNs);
  } else if (warp == 1) {
    // ---- MMA issue: the whole warp walks in step, so that addresses and descriptors live in uniform
    // registers, and one elected lane issues. The queue behind it is short, so every wait, fence and
    // commit between two groups of MMAs costs the tensor core 50-100 cycles: a stream's turn has
    // few of them, and the tiles' slots are given back by the softmax warps. The MMAs of a group are
    // unrolled: a rolled loop takes 82 cycles for each, the tensor core 64
    constexpr uint32_t id_s = idesc_bf16_f32(128, KT);
    constexpr uint32_t id_o = idesc_bf16_f32(128, HD) | kIdescBMnMajor;
    const uint32_t tm = __shfl_sync(0xffffffffu, tb, 0);
    const bool lead = elect_one();
    // operand descriptors of the first k-step; a step adds to the address field (16-byte units)
    const uint64_t dq = sw128_kmajor_desc(smem_addr(sm));
    const uint64_t dk = sw128_kmajor_desc(smem_addr(sm + LY::off_ring));
    const uint64_t dv = sw128_mnmajor_desc(smem_addr(sm + LY::off_ring), KT * 128);
    auto slot_at = [&](int use) { return (uint64_t)((uint32_t)LY::slot(use) * (LY::kTile >> 4)); };
    auto issue_s = [&](uint64_t q, uint64_t k, uint32_t d) {  // d = q . k^T, the smallest term of q first
      if (lead) {
        auto product = [&](int tq, int tkey, bool zero) {
#pragma unroll
          for (int i = 0; i < HD / 16; ++i) {
            const int in = (i & 3) * 32, cb = i >> 2;  // k-step i: place in the column block
            const uint64_t kd = k + ((tkey * LY::kPlane + cb * (KT * 128) + in) >> 4);
            if (F && tq == 0)
              tc_mma_bf16_ta(d, tm + kQ0 + 8 * i, kd, id_s, !zero || i != 0);
            else
              tc_mma_bf16(d, q + ((tq * LY::kQ1 + cb * (128 * 128) + in) >> 4), kd, id_s, !zero || i != 0);
          }
        };
        if constexpr (F) {
          product(2, 0, true);
          product(1, 1, false);
          product(0, 2, false);
          product(1, 0, false);
          product(0, 1, false);
          product(0, 0, false);
        } else {
#pragma unroll
          for (int t = NT - 1; t >= 0; --t) product(t, 0, t == NT - 1);
        }
      }
      __syncwarp();
    };
    auto commit = [&](uint64_t* bar) {
      if (lead) tc_commit(bar);
      __syncwarp();
    };
    PagedCursor c = paged_cursor<KT>(a, st);
    int items = 0, tiles = 0;  // of this CTA so far; tile g uses slots 2g (K), 2g + 1 (V)
    int turns[2] = {0, 0};     // tiles of each stream (NT = 1)
    int pairs = 0;             // items with two streams
    auto wait = [&](uint64_t* bar, int n) {
      return __all_sync(0xffffffffu, wait_for(bar, n, a.wait_ns)) != 0;
    };
    auto kv_wait = [&](int use) { return wait(&kv_full[LY::slot(use)], LY::phase(use)); };
    bool ok = a.wait_ns != 0;
    if (ok) do {
      const int n = __shfl_sync(0xffffffffu, c.kend - c.kt, 0);
      const int streams =  // the second stream may have no rows in this item
          __shfl_sync(0xffffffffu, NT == 1 && c.s.nb - c.rt * a.tpt > half ? 2 : 1, 0);
      ok = wait(&q_full[0], items) && (streams == 1 || wait(&q_full[1], pairs++)) && kv_wait(2 * tiles);
      if (!ok) break;
      tc_fence_after();
      if constexpr (NT == 1) {
#pragma unroll 1
        for (int s = 0; s < streams; ++s) {
          issue_s(dq + s * (LY::kQ1 >> 4), dk + slot_at(2 * tiles), tm + 128 * s);
          commit(&s_full[s]);
        }
        ok = kv_wait(2 * tiles + 1);
#pragma unroll 1
        for (int x = 0; ok && x < n; ++x) {
          const int g = tiles + x;
          const uint64_t v = dv + slot_at(2 * g + 1), k = dk + slot_at(2 * g + 2);
          const bool last = x + 1 == n;
#pragma unroll 1
          for (int s = 0; ok && s < streams; ++s) {
            const uint32_t p = tm + 128 * s;
            auto issue_pv = [&](int i0) {  // half of the tile's keys
              tc_fence_after();
              if (lead) {
#pragma unroll
                for (int i = 0; i < KT / 32; ++i)
                  tc_mma_bf16_ta(p + kO, p + 8 * (i0 + i), v + ((i0 + i) * 2048 >> 4), id_o,
                                 (x | i0 | i) != 0);
              }
              __syncwarp();
            };
            ok = wait(&p_half[s], turns[s]);
            if (!ok) break;
            issue_pv(0);
            ok = wait(&p_full[s], turns[s]++);
            if (!ok) break;
            issue_pv(KT / 32);
            if (!last) {
              if (s == 0) ok = kv_wait(2 * g + 2);
              if (!ok) break;
              issue_s(dq + s * (LY::kQ1 >> 4), k, p);  // into the columns P leaves
            }
            commit(last ? &o_full[s] : &s_full[s]);
            // the next turn's values, while the queue still holds this turn's products
            if (s == 0 && !last) ok = kv_wait(2 * g + 3);
          }
        }
      } else {
        issue_s(dq, dk + slot_at(2 * tiles), tm + LY::t_s * (tiles & 1));
        commit(&s_full[tiles & 1]);
        commit(&kv_empty[LY::slot(2 * tiles)]);
        for (int x = 0; x < n; ++x) {
          const int g = tiles + x;
          if (x + 1 < n) {  // the next tile's scores while this one's weights are formed
            ok = kv_wait(2 * g + 2);
            if (!ok) break;
            tc_fence_after();
            issue_s(dq, dk + slot_at(2 * g + 2), tm + LY::t_s * ((g + 1) & 1));
            commit(&s_full[(g + 1) & 1]);
            commit(&kv_empty[LY::slot(2 * g + 2)]);
          }
          ok = kv_wait(2 * g + 1) && wait(&p_full[0], g);
          if (!ok) break;
          tc_fence_after();
          const uint64_t v = dv + slot_at(2 * g + 1);
          const uint32_t p = tm + LY::t_s * (g & 1), px = tm + kX<F> + KT / 2 * (g & 1);
          const bool fresh = x % kFlush == 0;  // (O has been taken away before p_full)
          if (lead) {
            auto product = [&](uint32_t d, int tp, int tval, bool zero) {
#pragma unroll
              for (int i = 0; i < KT / 16; ++i)
                tc_mma_bf16_ta(d, (tp == 2 ? px : p + KT / 2 * tp) + 8 * i,
                               v + ((tval * LY::kPlane + i * 2048) >> 4), id_o, !zero || i != 0);
            };
            if constexpr (F) {
              product(tm + kO2, 2, 0, fresh);
              product(tm + kO2, 1, 1, false);
              product(tm + kO2, 0, 2, false);
              product(tm + kO2, 1, 0, false);
              product(tm + kO2, 0, 1, false);
              product(tm + kO, 0, 0, fresh);
            } else {
#pragma unroll
              for (int t = 2; t >= 0; --t) product(tm + kO, t, 0, fresh && t == 2);
            }
          }
          __syncwarp();
          commit(&o_full[0]);
          commit(&kv_empty[LY::slot(2 * g + 1)]);
        }
      }
      tiles += n;
      ++items;
    } while (ok && c.next<KT>(a));
    if (!ok && lead && a.c.status) atomicOr(a.c.status, PG_TIMEOUT);
    // TMEM is released only after every MMA issued here has finished
    commit(done);
    wait_for(done, 0, kDrainNs);
  } else {
    // ---- softmax of a stream: thread = query row
    const int s = (warp - 2) >> 2, r = (warp & 3) * 32 + lane;  // a warp reaches 32 lanes of TMEM
    const uint32_t lrow = (uint32_t)((warp & 3) * 32) << 16;
    // row / gq for rows below 256 and gq <= 8
    float* const rec = a.flush + (size_t)blockIdx.x * (128 * 128) + r;  // NT = 3: [HD][128 rows]
    const uint32_t gmul = 65536u / a.gq + 1;
    auto token_of = [&](int row) { return (int)((uint32_t)row * gmul >> 16); };
    PagedCursor c = paged_cursor<KT>(a, st);
    int tiles = 0, mine = 0;  // of the CTA; of this stream
    int ends = 0;             // items whose end this stream has waited for
    // A wait gave up: this warp leaves, without another arrival (a slot given back before its copy has
    // come would be armed twice), so that the warps behind these barriers give up as well.
    bool bad = a.wait_ns == 0;
    auto wait = [&](uint64_t* bar, int n) {
      if (!bad) bad = !__all_sync(0xffffffffu, wait_for(bar, n, a.wait_ns));
    };
    do {
      const int n = c.kend - c.kt;
      const bool first = c.first(), whole = c.whole();
      const int tok0 = c.rt * a.tpt + s * half;              // of this stream's row tile
      const int ntok = min(max(c.s.nb - tok0, 0), half), rows = ntok * a.gq;
      const bool live = r < rows;
      const int lim = !live           ? 0
                      : a.prefix_pass ? c.limit
                                      : min(max(c.s.base + tok0 + token_of(r) + 1, 0), c.s.len);
      // This thread's row as others of its warp move it (whole rows at a time): token and head
      const int rtok = token_of(r), rhead = c.kvh * a.gq + r - rtok * a.gq;
      // q into shared memory, K-major with 128-byte swizzling, in 16-byte units of 8 columns
      {
        constexpr int RU = HD / 8, RPI = 32 / RU;  // units of a row, rows per step
        const int u = lane % RU, sub = lane / RU;
        uint8_t* base = sm + (NT == 1 ? s * LY::kQ1 : 0) + (u >> 3) * (128 * 128) + (warp & 3) * 4096;
        auto place = [&](int i) {  // of row i of the warp
          return base + (i >> 3) * 1024 + (i & 7) * 128 + (((u & 7) ^ (i & 7)) << 4);
        };
        auto source = [&](int i) {
          const int t = __shfl_sync(0xffffffffu, rtok, i), h = __shfl_sync(0xffffffffu, rhead, i);
          return (size_t)(c.s.lo + tok0 + t) * a.ldq + (size_t)h * HD + u * 8;
        };
        const int live_rows = rows - (warp & 3) * 32;
        if constexpr (NT == 1) {
#pragma unroll 4
          for (int i0 = 0; i0 < 32; i0 += RPI) {
            const int i = i0 + sub;
            const size_t at = source(i);
            const bool in = i < live_rows;  // (a row that is not there: zeros)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(place(i))),
                         "l"(static_cast<const uint16_t*>(a.q) + (in ? at : 0)), "r"(in ? 16 : 0)
                         : "memory");
          }
          asm volatile("cp.async.wait_all;" ::: "memory");
        } else {
          constexpr int NB = 4;
#pragma unroll 1
          for (int i0 = 0; i0 < 32; i0 += NB * RPI) {
            float4 v[NB][2];
#pragma unroll
            for (int k = 0; k < NB; ++k) {
              const int i = i0 + k * RPI + sub;
              const size_t at = source(i);
              v[k][0] = v[k][1] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (F && a.act_bf16) {
                if (i >= live_rows) continue;
                const uint4 x = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at));
                v[k][0] = make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u),
                                      __uint_as_float(x.y << 16), __uint_as_float(x.y & 0xffff0000u));
                v[k][1] = make_float4(__uint_as_float(x.z << 16), __uint_as_float(x.z & 0xffff0000u),
                                      __uint_as_float(x.w << 16), __uint_as_float(x.w & 0xffff0000u));
              } else if (i < live_rows) {
                const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at);
                v[k][0] = __ldg(p);
                v[k][1] = __ldg(p + 1);
              }
            }
#pragma unroll
            for (int k = 0; k < NB; ++k) {
              uint4 t[3];
              split3(v[k][0].x, v[k][0].y, t[0].x, t[1].x, t[2].x);
              split3(v[k][0].z, v[k][0].w, t[0].y, t[1].y, t[2].y);
              split3(v[k][1].x, v[k][1].y, t[0].z, t[1].z, t[2].z);
              split3(v[k][1].z, v[k][1].w, t[0].w, t[1].w, t[2].w);
              uint8_t* to = place(i0 + k * RPI + sub);
#pragma unroll
              for (int e = 0; e < 3; ++e) *reinterpret_cast<uint4*>(to + e * LY::kQ1) = t[e];
            }
          }
        }
        if constexpr (F) {  // q's first term into TMEM too
          __syncwarp();
          const uint8_t* from = sm + (warp & 3) * 4096 + (lane >> 3) * 1024 + (lane & 7) * 128;
#pragma unroll
          for (int i = 0; i < HD / 32; ++i) {
            uint32_t x[16];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<uint4*>(x + 4 * e) = *reinterpret_cast<const uint4*>(
                  from + (i >> 1) * (128 * 128) + ((((i & 1) * 4 + e) ^ (lane & 7)) << 4));
            tmem_st16(tb + kQ0 + lrow + 16 * i, x);
          }
          tmem_st_wait();
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && rows > 0) mbar_arrive_cta(&q_full[s]);  // (without rows it may run items ahead)
      }
      float m = -INFINITY, l = 0.f, rec_m = -INFINITY;
      const uint32_t to = tb + kO + 128 * s + lrow;
      for (int x = 0; x < (rows > 0 ? n : 0); ++x, ++mine) {
        const int g = tiles + x, buf = NT == 1 ? s : g & 1;
        const uint32_t ts = tb + LY::t_s * buf + lrow;
        wait(&s_full[buf], NT == 1 ? mine : g >> 1);
        if (bad) break;
        tc_fence_after();
        if (NT == 1 && (warp & 3) == 0 && lane == 0) {  // S_g and P V of tile g - 1 have finished
          mbar_arrive_cta(&kv_empty[(2 * g) % NS]);
          if (x > 0) mbar_arrive_cta(&kv_empty[(2 * g - 1) % NS]);
        }
        const int k0 = (c.kt + x) * KT;
        if (!F && k0 + KT > c.limit) {
          // values behind the last key are whatever the page held: cleared (0 * NaN is NaN), by both
          // streams alike, each before its own products
          wait(&kv_full[(2 * g + 1) % NS], (2 * g + 1) / NS);
          if (bad) break;
          if (k0 + r >= c.limit) {
            uint4* v = reinterpret_cast<uint4*>(sm + LY::off_ring + ((2 * g + 1) % NS) * LY::kTile + r * 128);
#pragma unroll
            for (int cb = 0; cb < QA; ++cb)
#pragma unroll
              for (int i = 0; i < 8; ++i) v[cb * (KT * 8) + i] = make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        uint32_t sv[KT];  // the row's scores; keys it does not see are -inf
#pragma unroll
        for (int i = 0; i < KT / 16; ++i)
          tmem_ld16(ts + 16 * i, *reinterpret_cast<uint32_t(*)[16]>(sv + 16 * i));
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < KT / 16; ++i) tmem_regs_ready(*reinterpret_cast<uint32_t(*)[16]>(sv + 16 * i));
        if (k0 + KT > c.limit - a.tpt) {
#pragma unroll
          for (int j = 0; j < KT; ++j)
            if (k0 + j >= lim) sv[j] = 0xff800000u;
        }
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < KT; j += 2)
          mx4[j / 2 & 3] = fmaxf(fmaxf(mx4[j / 2 & 3], __uint_as_float(sv[j])), __uint_as_float(sv[j + 1]));
        const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * a.scale_log2;
        const float mn = mx > m + 8.f ? mx : m;  // a row without a key yet keeps -inf
        const float mu = mn == -INFINITY ? 0.f : mn;
        const float alpha = paged_exp2(m - mu);
        const bool take = NT == 3 && x > 0 && x % kFlush == 0;  // O goes into the record below
        const float m_old = m;
        if (x > 0 && !take && __any_sync(0xffffffffu, mn != m)) {  // O moves to the new reference
          if (NT == 3) {  // (NT = 1: P V of the last tile was done before s_full of this one)
            wait(&o_full[0], g - 1);
            if (bad) break;
            tc_fence_after();
          }
#pragma unroll 1
          for (int d = 0; d < HD; d += 16) {
            uint32_t o[16];
            tmem_ld16(to + d, o);
            tmem_ld_wait();
            tmem_regs_ready(o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st16(to + d, o);
            if constexpr (F) {
              tmem_ld16(to + (kO2 - kO) + d, o);
              tmem_ld_wait();
              tmem_regs_ready(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st16(to + (kO2 - kO) + d, o);
            }
          }
        }
        m = mn;
        // the weights, 32 keys at a time, into TMEM over columns of S, which is in registers
        const float2 sc2 = make_float2(a.scale_log2, a.scale_log2), mu2 = make_float2(-mu, -mu);
        float2 ps[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int i = 0; i < KT / 32; ++i) {
          float2 p[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 z = fma2(make_float2(__uint_as_float(sv[32 * i + 2 * e]),
                                              __uint_as_float(sv[32 * i + 2 * e + 1])), sc2, mu2);
            p[e] = make_float2(paged_exp2(z.x), paged_exp2(z.y));
            ps[e & 1] = add2(ps[e & 1], p[e]);
          }
          uint32_t ph[16];
          if constexpr (NT == 1) {
#pragma unroll
            for (int e = 0; e < 16; ++e) ph[e] = paged_pack(p[e].x, p[e].y);
            tmem_st16(ts + 16 * i, ph);
            if (i == KT / 64 - 1) {  // half of P V starts while the other half's weights are formed
              tmem_st_wait();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_cta(&p_half[s]);
            }
          } else {
            uint32_t pm[16], pl[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) split3(p[e].x, p[e].y, ph[e], pm[e], pl[e]);
            tmem_st16(ts + 16 * i, ph);
            tmem_st16(ts + KT / 2 + 16 * i, pm);
            tmem_st16(tb + kX<F> + KT / 2 * buf + lrow + 16 * i, pl);
          }
        }
        l = l * alpha + ((ps[0].x + ps[0].y) + (ps[1].x + ps[1].y));
        // every phase of o_full is waited for before the next can end: a parity skipped could be
        // taken for the one before it
        if (NT == 3 && x > 0) {
          auto ready = [&] {
            wait(&o_full[0], g - 1);
            tc_fence_after();
          };
          if (take) {
            add_record<HD, F>(rec, to, x == kFlush, paged_exp2(rec_m - (m_old == -INFINITY ? 0.f : m_old)), ready);
            rec_m = m_old;
          } else {
            ready();
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (NT == 3 && bad) break;
        if (lane == 0) mbar_arrive_cta(&p_full[NT == 1 ? s : 0]);
      }
      if (NT == 1 && rows == 0 && (warp & 3) == 0) {  // a stream without rows lets the tiles pass
        for (int u = 2 * tiles; u < 2 * (tiles + n); ++u) {
          wait(&kv_full[u % NS], u / NS);
          if (bad) break;
          if (lane == 0) mbar_arrive_cta(&kv_empty[u % NS]);
        }
      }
      if (rows > 0) {
        wait(&o_full[NT == 1 ? s : 0], NT == 1 ? ends++ : tiles + n - 1);
        if (bad) break;
        if (NT == 1 && (warp & 3) == 0 && lane == 0) mbar_arrive_cta(&kv_empty[(2 * (tiles + n) - 1) % NS]);
        tc_fence_after();
        if (whole && a.pre.o && !a.prefix_pass) pdl_wait();  // the prefix's records
        // O out through shared memory (the q tile's, which no MMA reads any more), 32 columns of the
        // warp's 32 rows at a time, so that whole 128-byte lines leave. The row's own thread forms its
        // factors and place: out = o wa + (the prefix's o) wb
        const size_t slot = (size_t)(2 * blockIdx.x + (first ? 1 : 0)) * a.slots.rows + s * half * a.gq;
        float* stage = reinterpret_cast<float*>(sm + s * LY::kQ1 + (warp & 3) * 4096);
        const bool raw = !whole || a.prefix_pass, joins = whole && a.pre.o && !a.prefix_pass;
        const size_t row = whole ? (size_t)(c.s.lo + tok0 + rtok) * a.nq + rhead : slot + r;
        const int place = live ? (int)row : -1;  // (rows of a call fit: the host checks)
        float wa = 1.f, wb = 0.f;
        if (!raw) {
          float2 ml = make_float2(-INFINITY, 0.f);
          if (joins && live) ml = __ldcg(a.pre.ml + row);
          const float top = fmaxf(m, ml.x), f = top == -INFINITY ? 0.f : paged_exp2(m - top);
          const float g = top == -INFINITY ? 0.f : paged_exp2(ml.x - top), den = fmaf(l, f, ml.y * g);
          const float inv = den > 0.f || den != den ? __frcp_rn(den) : 0.f;
          wa = f * inv;
          wb = g * inv;
        } else if (live) {
          __stcg((whole ? a.pre.ml : a.slots.ml) + row, make_float2(m, l));
        }
        const float rec_f = paged_exp2(rec_m - (m == -INFINITY ? 0.f : m));
        float* const to_f = !whole ? a.slots.o : a.prefix_pass ? a.pre.o : static_cast<float*>(a.out);
        const int lr = lane >> 3, lc = lane & 7;  // rows of 8 lanes
#pragma unroll 1
        for (int d = 0; d < HD; d += 32) {
          uint32_t o[2][16];
          tmem_ld16(to + d, o[0]);
          tmem_ld16(to + d + 16, o[1]);
          tmem_ld_wait();
          tmem_regs_ready(o[0]);
          tmem_regs_ready(o[1]);
          if constexpr (F) {
            uint32_t o2[2][16];
            tmem_ld16(to + (kO2 - kO) + d, o2[0]);
            tmem_ld16(to + (kO2 - kO) + d + 16, o2[1]);
            tmem_ld_wait();
            tmem_regs_ready(o2[0]);
            tmem_regs_ready(o2[1]);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o[e >> 4][e & 15] = __float_as_uint(__uint_as_float(o[e >> 4][e & 15]) + __uint_as_float(o2[e >> 4][e & 15]));
          }
          if (NT == 3 && n > kFlush) {  // and the record of the tiles before
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              uint32_t& x = o[e >> 4][e & 15];
              x = __float_as_uint(fmaf(__ldcg(rec + (d + e) * 128), rec_f, __uint_as_float(x)));
            }
          }
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<uint4*>(stage + lane * 32 + ((e ^ (lane & 7)) << 2)) =
                make_uint4(o[e >> 2][4 * (e & 3)], o[e >> 2][4 * (e & 3) + 1], o[e >> 2][4 * (e & 3) + 2],
                           o[e >> 2][4 * (e & 3) + 3]);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int q = 4 * i + lr;
            const int to_row = __shfl_sync(0xffffffffu, place, q);
            const float fa = __shfl_sync(0xffffffffu, wa, q), fb = __shfl_sync(0xffffffffu, wb, q);
            float4 x = *reinterpret_cast<const float4*>(stage + q * 32 + ((lc ^ (q & 7)) << 2));
            x.x *= fa, x.y *= fa, x.z *= fa, x.w *= fa;
            if (to_row < 0) continue;
            const size_t at = (size_t)to_row * HD + d + 4 * lc;
            if (joins) {
              const float4 y = __ldcg(reinterpret_cast<const float4*>(a.pre.o + at));
              x.x = fmaf(fb, y.x, x.x), x.y = fmaf(fb, y.y, x.y);
              x.z = fmaf(fb, y.z, x.z), x.w = fmaf(fb, y.w, x.w);
            }
            if (!raw && (NT == 1 || (F && a.act_bf16)))
              *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
                  make_uint2(paged_pack(x.x, x.y), paged_pack(x.z, x.w));
            else
              *reinterpret_cast<float4*>(to_f + at) = x;
          }
          __syncwarp();
        }
        tc_fence_before();
      }
      if (bad) break;
      if (!whole && first && s == 0 && r == 0)  // the joining kernel's work
        a.splits[blockIdx.x] = PagedSplit{c.last_cta(), c.s.lo + c.rt * a.tpt,
                                          min(a.tpt, c.s.nb - c.rt * a.tpt) * a.gq, c.kvh * a.gq};
      tiles += n;
    } while (c.next<KT>(a));
    if (bad && lane == 0 && a.c.status) atomicOr(a.c.status, PG_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tb, 512);
  }
  pdl_wait();
}

// Joins the records of the items that a launch split: CTA (x, y) takes the 8 rows from 8 y on (16
// with head_dim 64) of the item that begins in CTA x, a row by hd/4 lanes.
constexpr int kJoinThreads = 256;
template <int HD>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ PagedAttnArgs a) {
  constexpr int V4 = HD / 4, RB = kJoinThreads / V4;
  pdl_launch_dependents();
  pdl_wait();
  const PagedSplit sp = a.splits[blockIdx.x];
  const int r = blockIdx.y * RB + threadIdx.x / V4, d = threadIdx.x % V4 * 4;
  if (sp.c1 < 0 || r >= sp.rows) return;
  PagedAcc acc;
  paged_join_slots<HD>(a.slots, blockIdx.x, sp.c1, r, d, acc);
  paged_emit<true>(a, HD, sp.token + r / a.gq, sp.head + r % a.gq, d, acc);
}

template <int HD, int NT, bool F>
cudaError_t launch_tc(const PagedAttnArgs& a, int grid, cudaStream_t s) {
  using LY = TcLayout<HD, NT, F>;
  CUtensorMap tk{}, tv{};
  const uint64_t rows = (uint64_t)a.c.n_pages * a.c.nkv << a.c.page_shift;
  const uint32_t box = std::min(LY::KT, 1 << a.c.page_shift);
  if (!F && (!make_tmap_bf16_2d(&tk, a.c.k_pages, rows, HD, box) ||
             !make_tmap_bf16_2d(&tv, a.c.v_pages, rows, HD, box)))
    return cudaErrorInvalidValue;
  cudaError_t e = launch_pdl(paged_attn_tc_kernel<HD, NT, F>, dim3(grid), LY::kThreads, LY::bytes, s, a, tk, tv);
  if (e == cudaSuccess && !a.prefix_pass) e = launch_paged_join(a, HD, grid, 128 * LY::kStreams, s);
  return e;
}
template <int HD>
cudaError_t launch_hd(const PagedAttnArgs& a, int grid, cudaStream_t s) {
  if (!a.c.kv_bf16) return launch_tc<HD, 3, true>(a, grid, s);
  return a.act_bf16 ? launch_tc<HD, 1, false>(a, grid, s) : launch_tc<HD, 3, false>(a, grid, s);
}
template <int HD, int NT, bool F>
cudaError_t allow_smem() {
  return cudaFuncSetAttribute(paged_attn_tc_kernel<HD, NT, F>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)TcLayout<HD, NT, F>::bytes);
}
template <int HD>
cudaError_t set_attributes_hd() {
  cudaError_t e = allow_smem<HD, 1, false>();
  if (e == cudaSuccess) e = allow_smem<HD, 3, false>();
  return e == cudaSuccess ? allow_smem<HD, 3, true>() : e;
}

}  // namespace

cudaError_t launch_paged_tc(const PagedAttnArgs& a, int hd, int grid, cudaStream_t s) {
  return hd == 64 ? launch_hd<64>(a, grid, s) : launch_hd<128>(a, grid, s);
}

cudaError_t launch_paged_join(const PagedAttnArgs& a, int hd, int grid, int item_rows, cudaStream_t s) {
  const int rb = kJoinThreads * 4 / hd;  // rows of a CTA
  const dim3 g(grid, (std::min(item_rows, a.slots.rows) + rb - 1) / rb);
  return hd == 64 ? launch_pdl(paged_join_kernel<64>, g, kJoinThreads, 0, s, a)
                  : launch_pdl(paged_join_kernel<128>, g, kJoinThreads, 0, s, a);
}

cudaError_t set_paged_tc_attributes() {
  cudaError_t e = set_attributes_hd<64>();
  return e == cudaSuccess ? set_attributes_hd<128>() : e;
}

}  // namespace qw
