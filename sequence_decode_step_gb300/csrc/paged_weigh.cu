// qw_paged_weigh: adds to every key's score the softmax weight that the call's queries give it, summed over
// the tokens and the heads of its KV head.
//
//   score[r] = decay score[r] + sum over query rows i of 2^(s_ir - L_i),  L_i = m_i + log2 sum_r 2^(s_ir - m_i)
//
// Two launches: one forms L of every query row (the running maximum and sum of a row, as attention does without
// its values), one sums the weights of every key. Up to 8 query rows of a KV head (a decode step): paged_weigh_step.cu.
// More, and the shared prefix's part of L: here, in tiles of 128 query rows x 128 keys on tcgen05.
//
// First launch: S = Q K^T with a query row per TMEM lane, so that a thread forms the running maximum and sum of half
// a row's tile by itself. Second launch: S^T = K Q^T with a key per lane and the query rows along the columns (32 to 128
// of them, as many as there are), so that a thread sums its key's weights by itself. Neither needs a shuffle per
// score; per score the threads do a multiply-add, an exponential and an addition (and a comparison in the first
// launch), in pairs where the instructions take two. For a tile of each of an SM's two CTAs the exponentials (32 a clock
// and SM) take 0.5 us, the products 0.3, the keys' bytes 1.4 at HBM's rate (64 KB): the bytes bound both launches where
// a KV head has up to 128 rows, the scores' instructions beyond. Measured 1.2 to 1.7 us a tile in the first launch, 1.3 to
// 1.5 in the second, and 5 in each before the first tile. 16 windows of 32 tokens over up to 8K keys: 68 us, for 160
// MB in 33 us and again in 36. The scores are formed twice because kept ones would be more bytes than the keys.
// Tried without gain: the second launch backwards, for what L2 still holds, and the copies of the next tile behind the
// products instead of before them.
//
// f32 q and f32 keys are three bf16 planes each (24 bits); the products of planes whose size reaches 2^-24 are formed,
// small ones first: for f32 on both sides six products, 0.8 us a tile at 128 dimensions, where the planes leave room
// for one CTA on an SM (two at 64 dimensions).
// bf16 keys come by asynchronous 16-byte copies into K-major tiles with 128-byte swizzling, one tile ahead; f32 keys
// through registers, one tile ahead. The products of a tile run while the scores of the one before it are worked on, from
// two S buffers of 128 TMEM columns. All eight warps copy and work on scores; a barrier per tile hands the tile to
// the thread that issues the products. mma.sync in place of this took 137 us for 16 windows of 32 tokens over bf16
// pages (68 here), 99 for 9 chunks of 61 tokens over f32 pages (48 here); it was up to a third faster only with 9 to 32
// rows over f32 pages of 128 dimensions (16 rows x 16 sequences of up to 8K keys 134 us, 198 here; 128 rows 360, 208 here).
//
// Work is shared as in attention: every sequence's tiles of 128 keys, for each KV head (and, in the first launch,
// each block of query rows), laid end to end form one line that is cut into equal shares. Items at a share's ends
// are split: their statistics go to a record per CTA and are joined by who needs them, in CTA order.

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "paged.h"
#include "paged_plan.h"
#include "paged_weigh.cuh"
#include "qw_internal.h"

namespace qw {
namespace {

static_assert(kTile == 128, "keys of a tile are lanes or columns of S");

// QT and KT: bf16 planes that hold q and the keys (three for f32)
template <int HD, int QT, int KT>
struct TcLayout {
  static constexpr uint32_t kHalf = 128 * 128;          // 128 rows of 64 dimensions
  static constexpr uint32_t kPlane = kHalf * (HD / 64);  // 128 rows, as a K-major operand
  static constexpr uint32_t off_q = 0;
  static constexpr uint32_t off_k = QT * kPlane;         // two tiles of bf16 keys, or one of f32 keys' planes
  static constexpr uint32_t off_l = off_k + (KT == 1 ? 2 : KT) * kPlane;  // per query row: L and keys seen, or halves to be joined
  static constexpr uint32_t bytes = off_l + 3 * kRows * 8 + 1024;  // (its start is rounded up to 1024)
  static constexpr int kCtas = 2 * (bytes + 2048) <= 227 * 1024 ? 2 : 1;
};

// Place of 16 bytes (8 dimensions from 8 c on) of row r in a K-major tile of 128 rows with 128-byte swizzling.
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
  return (uint32_t)(c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Each warp copies its strip of a tile (nothing, if that begins at `end` or behind it). The page's entry is fetched a
// tile ahead.
template <bool PRE>
__device__ __forceinline__ int page_of_strip(const WeighArgs& a, int b, int key, int end) {
  key += ((int)threadIdx.x >> 5) * kStrip;
  return key < end ? strip_page<PRE>(a, b, key) : 0;
}
template <int HD>
__device__ __forceinline__ void stage_keys(const WeighArgs& a, int page, int kvh, int key, int end, uint8_t* to) {
  constexpr int C = HD / 8, RPI = 32 / C;  // 16-byte pieces of a row; rows at a time
  const int lane = threadIdx.x & 31, first = ((int)threadIdx.x >> 5) * kStrip;
  if (key + first >= end) return;
  bool ok;
  const int r = lane / C, c = lane % C;
  const char* from = static_cast<const char*>(a.c.k_pages) +
                     ((long long)row_in(a, page, kvh, key + first, &ok) * HD + lane * 8) * 2;
  const uint32_t at = smem_addr(to + swizzled(first + r, c));
#pragma unroll
  for (int i = 0; i < kStrip / RPI; ++i)  // (rows RPI i + r: r has the low bits)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((at ^ (((i * RPI) & 7) << 4)) + i * RPI * 128),
                 "l"(from + i * 512)
                 : "memory");
}

// f32 keys: a warp's strip of a tile on its way in registers, and from there into shared memory as three planes.
template <int HD>
struct KeyRegs {
  static constexpr int C = HD / 8, RPI = 32 / C, N = kStrip / RPI;
  float4 v[N][2];
  __device__ __forceinline__ void load(const WeighArgs& a, int page, int kvh, int key, int end) {
    const int lane = threadIdx.x & 31, first = ((int)threadIdx.x >> 5) * kStrip;
    if (key + first >= end) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i][0] = v[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
      return;
    }
    bool ok;
    const float4* from = reinterpret_cast<const float4*>(
        static_cast<const float*>(a.c.k_pages) + (long long)row_in(a, page, kvh, key + first, &ok) * HD + lane * 8);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)  // (volatile: these loads are to start here)
        asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v[i][j].x), "=f"(v[i][j].y), "=f"(v[i][j].z), "=f"(v[i][j].w)
                     : "l"(from + i * 64 + j));
  }
  __device__ __forceinline__ void store(uint8_t* to) const {
    constexpr int P = 128 * HD * 2;
    const int lane = threadIdx.x & 31, first = ((int)threadIdx.x >> 5) * kStrip;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      uint32_t y[4][3];
      split<3>(v[i][0].x, v[i][0].y, y[0]);
      split<3>(v[i][0].z, v[i][0].w, y[1]);
      split<3>(v[i][1].x, v[i][1].y, y[2]);
      split<3>(v[i][1].z, v[i][1].w, y[3]);
      const uint32_t at = swizzled(first + i * RPI + lane / C, lane % C);
#pragma unroll
      for (int x = 0; x < 3; ++x) *reinterpret_cast<uint4*>(to + x * P + at) = make_uint4(y[0][x], y[1][x], y[2][x], y[3][x]);
    }
  }
};

// Query rows r0 .. r0 + n - 1 of the item as QT planes (n up to 128; rows that are not there are zeros). bf16 rows are
// copied asynchronously.
template <int HD, int QT>
__device__ __forceinline__ void stage_rows(const WeighArgs& a, const WSeq& s, int kvh, int r0, int n, uint8_t* to) {
  constexpr int C = HD / 8;
#pragma unroll 4
  for (int e = threadIdx.x; e < n * C; e += kThreads) {
    const int r = e / C, c = e % C, row = r0 + r;
    const bool there = row < s.rows;
    const int token = row / a.gq, head = kvh * a.gq + row - token * a.gq;
    const long long at = there ? (long long)(s.lo + token) * a.ldq + head * HD + c * 8 : 0;
    if (QT == 1) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(to + swizzled(r, c))),
                   "l"(static_cast<const uint16_t*>(a.q) + at), "r"(there ? 16 : 0)
                   : "memory");
    } else {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at);
      const float4 none = make_float4(0.f, 0.f, 0.f, 0.f), u = there ? __ldg(p) : none, v = there ? __ldg(p + 1) : none;
      uint32_t y[4][QT];
      split<QT>(u.x, u.y, y[0]);
      split<QT>(u.z, u.w, y[1]);
      split<QT>(v.x, v.y, y[2]);
      split<QT>(v.z, v.w, y[3]);
#pragma unroll
      for (int x = 0; x < QT; ++x)
        *reinterpret_cast<uint4*>(to + x * 128 * HD * 2 + swizzled(r, c)) =
            make_uint4(y[0][x], y[1][x], y[2][x], y[3][x]);
    }
  }
}

// The pipeline of both launches over tiles kt0 .. kt1 - 1: use(tile) with the tile's S complete in TMEM buffer
// (tile - kt0) & 1. q and all that use() reads of shared memory is in place.
struct TcState {
  uint64_t* bars;     // [2]: S of a buffer is complete
  uint32_t tmem;
  uint32_t phase[2];
  bool dead;          // a wait gave up: no more are made and no more products issued
  int dead_buf;
};
// Where the first tile's keys are on their way: behind the item's first barrier, before its copies' commit.
template <int HD, int KT, bool PRE>
struct KeyPipe {
  int page;  // of the warp's strip in the tile to be fetched next
  KeyRegs<HD> regs;  // (f32 keys)
  __device__ __forceinline__ void next(const WeighArgs& a, int b, int kvh, int kt, int kt1, int end, uint8_t* to) {
    if (kt < kt1) {
      if (KT == 1) stage_keys<HD>(a, page, kvh, kt * kTile, end, to);
      else regs.load(a, page, kvh, kt * kTile, end);
    }
    if (kt + 1 < kt1) page = page_of_strip<PRE>(a, b, (kt + 1) * kTile, end);
  }
};
template <int HD, int QT, int KT, bool PRE, bool SUM, class Use>
__device__ __forceinline__ void tc_tiles(const WeighArgs& a, TcState& st, uint8_t* sm, int b, int kvh, int kt0, int kt1,
                                         int end, int n_cols, KeyPipe<HD, KT, PRE>& keys, Use use) {
  using LY = TcLayout<HD, QT, KT>;
  auto wait = [&](int buf) {
    if (st.dead) return;
    if (mbar_wait(st.bars + buf, st.phase[buf], a.wait_ns)) {
      st.phase[buf] ^= 1;
      return;
    }
    st.dead = true, st.dead_buf = buf;
    if (a.c.status) atomicOr(a.c.status, PG_TIMEOUT);
  };
  for (int kt = kt0; kt < kt1; ++kt) {
    const int i = kt - kt0, buf = i & 1;
    // the products of the tile before are done: its keys' place is free, its scores are complete
    if (i > 0) wait(buf ^ 1);
    uint8_t* k = sm + LY::off_k + (KT == 1 ? buf * LY::kPlane : 0);
    if (KT == 1) {
      keys.next(a, b, kvh, kt + 1, kt1, end, sm + LY::off_k + (buf ^ 1) * LY::kPlane);
      stage_commit();
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      keys.regs.store(k);
      asm volatile("cp.async.wait_group 0;" ::: "memory");  // (q)
    }
    fence_async();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && !st.dead) {
      tc_fence_after();
      const uint64_t dq = sw128_kmajor_desc(smem_addr(sm + LY::off_q));
      const uint64_t dk = sw128_kmajor_desc(smem_addr(k));
      const uint32_t id = idesc_bf16_f32(128, n_cols), d = st.tmem + buf * 128;
      bool first = true;
      // products of like size one after another, the smallest first
#pragma unroll
      for (int o = KT == 1 ? QT - 1 : 2; o >= 0; --o)
#pragma unroll
        for (int x = 0; x < QT; ++x) {
          if (o - x < 0 || o - x >= KT) continue;
#pragma unroll
          for (int s = 0; s < HD / 16; ++s) {
            const uint64_t in = (uint64_t)((((s >> 2) * LY::kHalf) + (s & 3) * 32) >> 4);
            const uint64_t q = dq + ((x * LY::kPlane) >> 4) + in, kk = dk + (((o - x) * LY::kPlane) >> 4) + in;
            tc_mma_bf16(d, SUM ? kk : q, SUM ? q : kk, id, !first);
            first = false;
          }
        }
      tc_commit(st.bars + buf);
    }
    if (KT != 1) keys.next(a, b, kvh, kt + 1, kt1, end, nullptr);
    if (i > 0) use(kt - 1, buf ^ 1);
  }
  if (kt1 > kt0) {
    const int buf = (kt1 - 1 - kt0) & 1;
    wait(buf);
    use(kt1 - 1, buf);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Sets up barriers and TMEM: behind the launch before (pdl_wait), and before the next one may start, as its CTAs
// would otherwise hold TMEM that this launch's wait for.
__device__ __forceinline__ void tc_open(TcState& st, uint64_t* bars, uint32_t* slot) {
  if (threadIdx.x == 0) {
    mbar_init(bars, 1);
    mbar_init(bars + 1, 1);
    fence_barrier_init();
  }
  if (threadIdx.x < 32) {
    tmem_alloc(slot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  st.bars = bars;
  st.tmem = *slot;
  st.phase[0] = st.phase[1] = 0;
  st.dead = false;
}
__device__ __forceinline__ void tc_close(const WeighArgs& a, TcState& st) {
  // the products that a wait has given up on may still run (those before them are done, and after them came none):
  // they are awaited before their memory goes
  if (threadIdx.x == 0 && st.dead) mbar_wait(st.bars + st.dead_buf, st.phase[st.dead_buf], kDrainNs);
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x < 32) {
    tc_fence_after();
    tmem_dealloc(st.tmem, 256);
  }
}

// a b + c and a + b of two floats at once; the largest of three.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return reinterpret_cast<float2&>(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return reinterpret_cast<float2&>(r);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 16 columns of the warp's lanes of S, from column `col` on.
__device__ __forceinline__ void load_scores(const TcState& st, int buf, int col, uint32_t (&x)[16]) {
  tmem_ld16(st.tmem + buf * 128 + (((threadIdx.x >> 5) & 3) * 32 << 16) + col, x);
}

// ------------------------------------------------------------------ first launch
template <int HD, int QT, int KT, bool PRE>
__global__ void __launch_bounds__(kThreads, TcLayout<HD, QT, KT>::kCtas) weigh_lse_kernel(const __grid_constant__ WeighArgs a) {
  using LY = TcLayout<HD, QT, KT>;
  extern __shared__ __align__(1024) uint8_t raw[];
  uint8_t* sm = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  __shared__ Share sh;
  __shared__ int warp_sums[4][kWarps];
  __shared__ uint64_t bars[2];
  __shared__ uint32_t slot;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = warp >> 2, mine = (warp & 3) * 32 + lane;
  float2* other = reinterpret_cast<float2*>(sm + LY::off_l);  // [128]: the second half's statistics
  pdl_wait();
  TcState st;
  tc_open(st, bars, &slot);
  pdl_launch_dependents();
  find_share<PRE, false>(a, &sh, warp_sums);
  if (sh.b < (PRE ? 1 : a.c.n_seqs)) {
    const WeighStats& out = PRE ? a.pre : a.own;
    float2* slots = out.slots + (size_t)blockIdx.x * 2 * kRows;
    int u = sh.u0, unit = sh.unit, b = sh.b;
    WSeq s = weigh_seq<PRE>(a, b);
    while (u < sh.u1) {
      for (int n; u - unit >= (n = lse_units(a, s, sh.head)); s = weigh_seq<PRE>(a, ++b)) unit += n;
      const LseTiles part_of = lse_tiles(s, sh.head, unit, sh.u1, &u);
      const int kvh = part_of.kvh, r0 = part_of.r0, kt0 = part_of.kt0, kt1 = part_of.kt1, rows = min(kRows, s.rows - r0);
      if (kt0 >= kt1) continue;
      const int limit = row_sees<PRE>(a, s, r0 + rows - 1);
      const int see = row_sees<PRE>(a, s, r0 + mine), last = min(kt1, (limit + kTile - 1) / kTile);
      KeyPipe<HD, KT, PRE> keys;
      keys.page = page_of_strip<PRE>(a, b, kt0 * kTile, limit);
      __syncthreads();  // the item before has left shared memory
      keys.next(a, b, kvh, kt0, last, limit, sm + LY::off_k);
      stage_rows<HD, QT>(a, s, kvh, r0, (rows + 31) / 32 * 32, sm + LY::off_q);
      stage_commit();
      // maximum (before the factor), its product with the factor, and sum over this half of the row's keys
      float m = -INFINITY, base = 0.f, l = 0.f;
      tc_tiles<HD, QT, KT, PRE, false>(a, st, sm, b, kvh, kt0, last, limit, kTile, keys, [&](int kt, int buf) {
        tc_fence_after();
        if ((warp & 3) * 32 >= rows) return;  // (of the whole warp)
        uint32_t x[4][16];
#pragma unroll
        for (int i = 0; i < 4; ++i) load_scores(st, buf, half * 64 + 16 * i, x[i]);
        tmem_ld_wait();
        float c[64], top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          tmem_regs_ready(x[i]);
#pragma unroll
          for (int e = 0; e < 16; ++e) c[16 * i + e] = __uint_as_float(x[i][e]);
        }
        const int seen = see - kt * kTile - half * 64;  // of these 64 keys
        if (__any_sync(0xffffffffu, seen < 64)) {
#pragma unroll
          for (int e = 0; e < 64; ++e) c[e] = e < seen ? c[e] : -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 64; e += 2) top[(e >> 1) & 3] = max3(top[(e >> 1) & 3], c[e], c[e + 1]);
        const float t = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        if (t > m) {
          l *= exp2_approx((m - t) * a.scale_log2);
          m = t, base = -t * a.scale_log2;
        }
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const float2 scale = make_float2(a.scale_log2, a.scale_log2), from = make_float2(base, base);
#pragma unroll
        for (int e = 0; e < 64; e += 2) {
          const float2 y = fma2(make_float2(c[e], c[e + 1]), scale, from);
          sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], make_float2(exp2_approx(y.x), exp2_approx(y.y)));
        }
        const float2 both = add2(sum[0], sum[1]);
        l += both.x + both.y;
      });
      const float2 part = make_float2(m * a.scale_log2, l);
      if (half) other[mine] = part;
      __syncthreads();
      if (!half && mine < rows) {
        const float2 x = join(part, other[mine]);
        if (kt0 == 0 && kt1 == s.nkt) {
          const int row = r0 + mine, token = row / a.gq;
          out.whole[(size_t)(s.lo + token) * a.nq + kvh * a.gq + row - token * a.gq] = x;
        } else {
          slots[(kt0 == 0 ? kRows : 0) + mine] = x;
        }
      }
    }
  }
  tc_close(a, st);
}

// ------------------------------------------------------------------ second launch
// Adds the weights of a key (a lane) in query rows c0 .. c0 + n - 1 (columns; n a multiple of 16). AHEAD: the next 16
// scores are on their way while 16 are worked on.
template <bool AHEAD, bool MASK>
__device__ __forceinline__ void sum_columns(const TcState& st, int buf, int c0, int n, int key, float scale,
                                            const float* big_l, const int* see, float (&w)[4]) {
  uint32_t x[AHEAD ? 2 : 1][16];
  if (AHEAD) load_scores(st, buf, c0, x[0]);
#pragma unroll
  for (int i = 0; i < kRows / 32; ++i) {
    if (16 * i >= n) break;
    if (!AHEAD) load_scores(st, buf, c0 + 16 * i, x[0]);
    uint32_t(&y16)[16] = x[AHEAD ? i & 1 : 0];
    tmem_ld_wait();
    tmem_regs_ready(y16);
    if (AHEAD && 16 * (i + 1) < n) load_scores(st, buf, c0 + 16 * (i + 1), x[AHEAD ? (i + 1) & 1 : 0]);
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
      const int at = c0 + 16 * i + e;
      const float4 big = *reinterpret_cast<const float4*>(big_l + at);
      float y[4] = {fmaf(__uint_as_float(y16[e]), scale, -big.x), fmaf(__uint_as_float(y16[e + 1]), scale, -big.y),
                    fmaf(__uint_as_float(y16[e + 2]), scale, -big.z),
                    fmaf(__uint_as_float(y16[e + 3]), scale, -big.w)};
      if (MASK) {
        const int4 seen = *reinterpret_cast<const int4*>(see + at);
        y[0] = key < seen.x ? y[0] : -INFINITY;
        y[1] = key < seen.y ? y[1] : -INFINITY;
        y[2] = key < seen.z ? y[2] : -INFINITY;
        y[3] = key < seen.w ? y[3] : -INFINITY;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] += exp2_approx(y[j]);
    }
  }
}

template <int HD, int QT, int KT>
__global__ void __launch_bounds__(kThreads, TcLayout<HD, QT, KT>::kCtas) weigh_sum_kernel(const __grid_constant__ WeighArgs a) {
  using LY = TcLayout<HD, QT, KT>;
  extern __shared__ __align__(1024) uint8_t raw[];
  uint8_t* sm = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  __shared__ Share sh;
  __shared__ int warp_sums[4][kWarps];
  __shared__ SumItem item;
  __shared__ uint64_t bars[2];
  __shared__ uint32_t slot;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = warp >> 2, mine = (warp & 3) * 32 + lane;
  float* big_l = reinterpret_cast<float*>(sm + LY::off_l);  // [128]
  int* see = reinterpret_cast<int*>(big_l + kRows);         // [128]
  float* other = reinterpret_cast<float*>(see + kRows);     // [2][128]: the second half's sums of a tile's keys
  find_share<false, true>(a, &sh, warp_sums);
  pdl_wait();
  TcState st;
  tc_open(st, bars, &slot);
  pdl_launch_dependents();
  if (sh.b < a.c.n_seqs) {
    int u = sh.u0, unit = sh.unit, lse = sh.lse, b = sh.b;
    WSeq s = weigh_seq<false>(a, b);
    while (u < sh.u1) {
      for (int n; u - unit >= (n = sum_units(a, s, sh.head)); s = weigh_seq<false>(a, ++b))
        unit += n, lse += lse_units(a, s, sh.lse_line.head);
      const SumTiles part = sum_tiles(s, sh.head, unit, sh.u1, &u);
      const int kvh = part.kvh, kt0 = part.kt0, kt1 = part.kt1;
      if (kt0 >= kt1) continue;
      for (int r0 = 0; r0 == 0 || r0 < s.rows; r0 += kRows) {
        const int rows = max(min(kRows, s.rows - r0), 0), cols = max((rows + 31) / 32 * 32, 32);
        // a thread's own key: its page two tiles ahead, its score so far one tile ahead
        auto page_of = [&](int key) { return !half && key < s.len ? strip_page<false>(a, b, key) : 0; };
        // and its new score written a tile late: a proxy fence waits for the stores before it
        bool ok_next, due = false;
        int row_next, row_due = 0;
        float old_next, value_due = 0.f;
        auto score_of = [&](int key, int own_page) {
          ok_next = false, row_next = 0, old_next = 0.f;
          if (half || key >= s.len) return;
          row_next = row_in(a, own_page, kvh, key, &ok_next);
          if (r0 || key < s.fresh) old_next = a.scores[row_next];
        };
        KeyPipe<HD, KT, false> keys;
        keys.page = page_of_strip<false>(a, b, kt0 * kTile, s.len);
        int own_page = page_of(kt0 * kTile + mine);
        __syncthreads();  // the item before has left shared memory
        if (threadIdx.x == 0) item = SumItem{s, b, kvh, kt0, kt1, lse, sh.lse_line};
        keys.next(a, b, kvh, kt0, kt1, s.len, sm + LY::off_k);
        if (QT == 1) stage_rows<HD, QT>(a, s, kvh, r0, cols, sm + LY::off_q);
        stage_commit();
        score_of(kt0 * kTile + mine, own_page);
        if (kt0 + 1 < kt1) own_page = page_of((kt0 + 1) * kTile + mine);
        if (QT != 1) stage_rows<HD, QT>(a, s, kvh, r0, cols, sm + LY::off_q);
        __syncthreads();
        stage_stats(a, item, r0, cols, big_l, see);
        const int all_see = rows ? row_sees<false>(a, s, r0) : 0;
        __syncthreads();
        tc_tiles<HD, QT, KT, false, true>(a, st, sm, b, kvh, kt0, kt1, s.len, cols, keys, [&](int kt, int buf) {
          const int key = kt * kTile + mine, row = row_next;
          const bool ok = ok_next;
          const float old = r0 ? old_next : old_next * a.decay;
          if (due) a.scores[row_due] = value_due;
          if (kt + 1 < kt1) score_of(key + kTile, own_page);
          if (kt + 2 < kt1) own_page = page_of(key + 2 * kTile);
          tc_fence_after();
          // this half of the query rows, 16 at a time
          const int c0 = half * (cols / 2), n = cols / 2;
          float w[4] = {0.f, 0.f, 0.f, 0.f};
          if ((kt + 1) * kTile > all_see)
            sum_columns<KT == 1, true>(st, buf, c0, n, key, a.scale_log2, big_l, see, w);
          else
            sum_columns<KT == 1, false>(st, buf, c0, n, key, a.scale_log2, big_l, see, w);
          const float sum = (w[0] + w[1]) + (w[2] + w[3]);
          float* halves = other + buf * kRows;
          if (half) halves[mine] = sum;
          asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp & 3)) : "memory");  // the two warps of these keys
          due = ok, row_due = row, value_due = old + (sum + halves[mine]);
        });
        if (due) a.scores[row_due] = value_due;
      }
    }
  }
  tc_close(a, st);
}

template <int HD, int QT, int KT>
struct Tc {
  using LY = TcLayout<HD, QT, KT>;
  static cudaError_t attributes() {
    cudaError_t e = cudaSuccess;
    for (const void* f : {(const void*)weigh_lse_kernel<HD, QT, KT, false>, (const void*)weigh_lse_kernel<HD, QT, KT, true>,
                          (const void*)weigh_sum_kernel<HD, QT, KT>}) {
      if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)LY::bytes);
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(f, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    }
    return e;
  }
  static cudaError_t prefix(WeighArgs& a, int sms, cudaStream_t s) {
    a.pre_grid = LY::kCtas * sms;
    return launch_pdl(weigh_lse_kernel<HD, QT, KT, true>, dim3(a.pre_grid), kThreads, LY::bytes, s, a);
  }
  static cudaError_t run(WeighArgs a, int sms, cudaStream_t s) {
    a.grid = LY::kCtas * sms;
    const cudaError_t e = launch_pdl(weigh_lse_kernel<HD, QT, KT, false>, dim3(a.grid), kThreads, LY::bytes, s, a);
    return e == cudaSuccess ? launch_pdl(weigh_sum_kernel<HD, QT, KT>, dim3(a.grid), kThreads, LY::bytes, s, a) : e;
  }
};
template <int HD, class Use>
cudaError_t with_types(bool act_bf16, bool kv_bf16, Use use) {
  if (kv_bf16) return act_bf16 ? use(Tc<HD, 1, 1>()) : use(Tc<HD, 3, 1>());
  return act_bf16 ? use(Tc<HD, 1, 3>()) : use(Tc<HD, 3, 3>());
}
template <class Use>
cudaError_t with_types(int hd, bool act_bf16, bool kv_bf16, Use use) {
  return hd == 64 ? with_types<64>(act_bf16, kv_bf16, use) : with_types<128>(act_bf16, kv_bf16, use);
}

constexpr int kMostGrid = 2 * kPagedMaxSms;  // CTAs of a launch that leave records
constexpr size_t kSlotBytes = (size_t)kMostGrid * 2 * kRows * sizeof(float2);

// Query rows of a KV head that a call's hints promise for one sequence.
long long hinted_rows(int n_tokens, int gq, int max_new, int window) {
  int tokens = std::min(max_new, n_tokens);
  if (window > 0) tokens = std::min(tokens, window);
  return (long long)tokens * gq;
}
// Scores kept for a key, of up to 8 rows.
int kept_rows(long long rows) { return rows <= 8 ? (int)(rows + 1) / 2 * 2 : 0; }

size_t stats_bytes(int n_tokens, int nq) {
  return kSlotBytes + ((size_t)n_tokens * nq * sizeof(float2) + 255) / 256 * 256;
}

}  // namespace

size_t paged_weigh_workspace_bytes(size_t pool_rows, int n_tokens, int nq, int gq, int max_new, int window, bool prefix) {
  return (prefix ? 2 : 1) * stats_bytes(n_tokens, nq) +
         pool_rows * kept_rows(hinted_rows(n_tokens, gq, max_new, window)) * sizeof(float);
}

cudaError_t set_weigh_attributes() {
  cudaError_t e = set_weigh_step_attributes();
  for (int i = 0; i < 8 && e == cudaSuccess; ++i)
    e = with_types(i & 1 ? 64 : 128, i & 2, i & 4, [](auto t) { return t.attributes(); });
  return e;
}

cudaError_t launch_paged_weigh(const WeighArgs& base, int hd, int max_new, void* workspace, int sms, cudaStream_t s) {
  WeighArgs a = base;
  // units of the longest possible lines are counted in 32 bits: of the counted tokens' rows over the sequences' own keys
  // (key_cost() is at most 58 and a unit for every row), and of blocks of all tokens' rows over the prefix
  auto units = [&](long long keys, double of_a_tile) {
    return a.c.nkv * (double)((keys + kTile - 1) / kTile + kHeadTiles) * of_a_tile;
  };
  const double tokens = a.n_tokens, counted = a.window > 0 ? std::min(tokens, (double)a.c.n_seqs * a.window) : tokens;
  if (units((long long)a.c.max_pages << a.c.page_shift, 58.0 * a.c.n_seqs + counted * a.gq + 2) >= 1073741824.0 ||
      units(a.c.prefix_len, tokens * a.gq / kRows + 2) >= 1073741824.0)
    return cudaErrorInvalidValue;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  auto stats = [&] {
    WeighStats st{reinterpret_cast<float2*>(w), reinterpret_cast<float2*>(w + kSlotBytes)};
    w += stats_bytes(a.n_tokens, a.nq);
    return st;
  };
  a.own = a.pre = stats();
  if (a.c.prefix_len > 0) a.pre = stats();
  const long long rows = hinted_rows(a.n_tokens, a.gq, max_new, a.window);
  a.keep = kept_rows(rows);
  a.kept = reinterpret_cast<float*>(w);
  sms = std::min(sms, kPagedMaxSms);
  if (a.c.prefix_len > 0) {
    const cudaError_t e = with_types(hd, a.act_bf16, a.c.kv_bf16, [&](auto t) { return t.prefix(a, sms, s); });
    if (e != cudaSuccess) return e;
  }
  if (a.keep > 0) return launch_weigh_step(a, hd, sms, s);
  return with_types(hd, a.act_bf16, a.c.kv_bf16, [&](auto t) { return t.run(a, sms, s); });
}

}  // namespace qw
