// Work of a paged-attention launch and how its CTAs share it.
//
// An item is one row tile (up to R query rows: tpt tokens x gq heads of one KV head) of one
// sequence; its work is its key tiles of KT keys. Items in the order (sequence, KV head, row
// tile) laid end to end form one line of units, and CTA c takes units [c per, (c + 1) per): the
// lengths live on the device, so every CTA forms the same prefix sums of the sequences' units
// and finds its own start. The load is even to one key tile whatever the lengths are, and only the
// items at a CTA's ends are split: at most two partial records per CTA, slot 2c for an item that
// began in an earlier CTA and slot 2c + 1 for one that goes on in the next. Records are joined in
// CTA order, so results do not depend on which CTA is last: small ones by the last CTA to arrive
// (counters[first CTA]), 128-row ones by a kernel of their own.
//
// The shared prefix is the same line with one pseudo-sequence: all the batch's tokens, every one
// of which sees all prefix_len keys. Its records are not joined by its own launch: the launch over
// the sequences' own keys adds them, row by row, to the rows it writes.
#pragma once
#include "paged.h"
#include "qw_ptx.cuh"

namespace qw {

struct PagedSeq {  // one sequence's share of the line
  int lo, nb;      // first token row and tokens
  int base, len;   // keys before the first new token, all keys
  int nrt;         // row tiles per KV head
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedAttnArgs& a, int b) {
  PagedSeq s;
  if (a.prefix_pass) {
    const int end = min(max(__ldg(a.c.q_start + a.c.n_seqs), 0), a.n_tokens);
    s.lo = min(max(__ldg(a.c.q_start), 0), end);
    s.nb = end - s.lo;
    s.len = a.c.prefix_len;
    s.base = s.len;
  } else {
    s.lo = min(max(__ldg(a.c.q_start + b), 0), a.n_tokens);
    s.nb = min(max(__ldg(a.c.q_start + b + 1), s.lo), a.n_tokens) - s.lo;
    const long long cap = (long long)a.c.max_pages << a.c.page_shift;
    const int len = __ldg(a.c.kv_len + b);
    s.len = (int)min((long long)max(len, 0), cap);
    if (len != s.len && a.c.status) atomicOr(a.c.status, PG_BAD_LENGTH);
    s.base = s.len - s.nb;
  }
  s.nrt = (s.nb + a.tpt - 1) / a.tpt;
  return s;
}
// Keys that the last token of row tile rt sees.
__device__ __forceinline__ int paged_limit(const PagedAttnArgs& a, const PagedSeq& s, int rt) {
  const int l = s.base + min(s.nb, (rt + 1) * a.tpt);
  return a.prefix_pass ? s.len : min(max(l, 0), s.len);
}
// Key tiles of an item: one at least, so that every row is written.
template <int KT>
__device__ __forceinline__ int paged_tiles(int limit) {
  return max(1, (limit + KT - 1) / KT);
}
template <int KT>
__device__ __forceinline__ long long paged_head_units(const PagedAttnArgs& a, const PagedSeq& s) {
  long long n = 0;
  for (int rt = 0; rt < s.nrt; ++rt) n += paged_tiles<KT>(paged_limit(a, s, rt));
  return n;
}

struct PagedCursor {  // a place on the line
  long long u, u1, per;
  int b, kvh, rt, kt;  // current item and key tile
  int nkt, limit;      // of the current item
  PagedSeq s;

  template <int KT>
  __device__ __forceinline__ void enter(const PagedAttnArgs& a) {
    limit = paged_limit(a, s, rt);
    nkt = paged_tiles<KT>(limit);
  }
  // To the next item (only called while u < u1, so there is one).
  template <int KT>
  __device__ __forceinline__ void next_item(const PagedAttnArgs& a) {
    kt = 0;
    if (++rt == s.nrt) {
      rt = 0;
      if (++kvh == a.c.nkv) {
        kvh = 0;
        do s = paged_seq(a, ++b);
        while (s.nb == 0);
      }
    }
    enter<KT>(a);
  }
};

struct PagedStart {  // in shared memory: where this CTA starts
  long long u, u1, per;
  int b, kvh, rt, kt;
};

// Block-wide: fills *st (st->u >= st->u1: nothing to do). warp_sums: one long long per warp.
template <int KT, int THREADS>
__device__ void paged_find_start(const PagedAttnArgs& a, PagedStart* st, long long* warp_sums) {
  constexpr int W = THREADS / 32;
  const int n = a.prefix_pass ? 1 : a.c.n_seqs;
  const int spt = (n + THREADS - 1) / THREADS;
  const int b0 = min((int)threadIdx.x * spt, n), b1 = min(b0 + spt, n);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const PagedSeq s = paged_seq(a, b);
    mine += paged_head_units<KT>(a, s) * a.c.nkv;
  }
  long long scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += v;
  }
  if (lane == 31) warp_sums[warp] = scan;
  if (threadIdx.x == 0) st->u = 0, st->u1 = 0;
  __syncthreads();
  long long before = scan - mine, total = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < warp) before += warp_sums[w];
    total += warp_sums[w];
  }
  const long long per = (total + gridDim.x - 1) / gridDim.x;
  const long long u0 = per * blockIdx.x;
  if (u0 < total && before <= u0 && u0 < before + mine) {
    long long r = u0 - before;
    int b = b0;
    PagedSeq s = paged_seq(a, b);
    long long hu = paged_head_units<KT>(a, s);
    while (r >= hu * a.c.nkv) {
      r -= hu * a.c.nkv;
      s = paged_seq(a, ++b);
      hu = paged_head_units<KT>(a, s);
    }
    const int kvh = (int)(r / hu);
    r -= hu * kvh;
    int rt = 0;
    for (;; ++rt) {
      const int t = paged_tiles<KT>(paged_limit(a, s, rt));
      if (r < t) break;
      r -= t;
    }
    st->u = u0;
    st->u1 = min(u0 + per, total);
    st->per = per;
    st->b = b;
    st->kvh = kvh;
    st->rt = rt;
    st->kt = (int)r;
  }
  __syncthreads();
}

template <int KT>
__device__ __forceinline__ PagedCursor paged_cursor(const PagedAttnArgs& a, const PagedStart* st) {
  PagedCursor c;
  c.u = st->u;
  c.u1 = st->u1;
  if (c.u < c.u1) {
    c.per = st->per;
    c.b = st->b;
    c.kvh = st->kvh;
    c.rt = st->rt;
    c.kt = st->kt;
    c.s = paged_seq(a, c.b);
    c.enter<KT>(a);
  }
  return c;
}

// Page of key tile row `key` of the cursor's item; a page id outside the pool is reported and
// read as page 0, so that no read leaves the pool.
__device__ __forceinline__ int paged_page(const PagedAttnArgs& a, int b, int key) {
  const int at = key >> a.c.page_shift;
  int pg = a.prefix_pass ? __ldg(a.c.prefix_pages + at)
                         : __ldg(a.c.page_table + (size_t)b * a.c.max_pages + at);
  if ((unsigned)pg >= (unsigned)a.c.n_pages) {
    if (a.c.status) atomicOr(a.c.status, PG_BAD_PAGE);
    pg = 0;
  }
  return pg;
}
// First row (of hd elements) in the pool of key `key` under KV head kvh.
__device__ __forceinline__ long long paged_row(const PagedAttnArgs& a, int page, int kvh, int key) {
  return (((long long)page * a.c.nkv + kvh) << a.c.page_shift) + (key & ((1 << a.c.page_shift) - 1));
}

__device__ __forceinline__ float paged_exp2(float x) {  // 2^x, 2^-inf = 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Sums of one float4 of a row over the records that share it.
struct PagedAcc {
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  __device__ __forceinline__ void add(float w, float l2, const float4& v) {
    l = fmaf(w, l2, l);
    o.x = fmaf(w, v.x, o.x);
    o.y = fmaf(w, v.y, o.y);
    o.z = fmaf(w, v.z, o.z);
    o.w = fmaf(w, v.w, o.w);
  }
  // another record (m2, l2, v) of the same row
  __device__ __forceinline__ void join(float m2, float l2, const float4& v) {
    const float mn = fmaxf(m, m2);
    if (mn == -INFINITY) return;
    const float f = paged_exp2(m - mn);
    l *= f, o.x *= f, o.y *= f, o.z *= f, o.w *= f;
    m = mn;
    add(paged_exp2(m2 - mn), l2, v);
  }
};

__device__ __forceinline__ uint32_t paged_pack(float a, float b) {  // bf16, a in the low half
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// Adds records of slots c0 .. c1 (row r, columns 4 i4 ..) to acc, in CTA order.
__device__ __forceinline__ void paged_join_slots(const PagedSlots& sl, int hd, int c0, int c1, int r,
                                                 int d, PagedAcc& acc) {
  float top = acc.m;
  for (int x = c0; x <= c1; ++x)
    top = fmaxf(top, __ldcg(sl.ml + (size_t)(2 * x + (x == c0)) * sl.rows + r).x);
  const float mu = top == -INFINITY ? 0.f : top;
  const float f = paged_exp2(acc.m - mu);
  acc.m = top;
  acc.l *= f, acc.o.x *= f, acc.o.y *= f, acc.o.z *= f, acc.o.w *= f;
#pragma unroll 4
  for (int x = c0; x <= c1; ++x) {
    const size_t row = (size_t)(2 * x + (x == c0)) * sl.rows + r;
    const float2 ml = __ldcg(sl.ml + row);
    acc.add(paged_exp2(ml.x - mu), ml.y, __ldcg(reinterpret_cast<const float4*>(sl.o + row * hd + d)));
  }
}

// Adds the prefix's record(s) of (token, head) to acc.
__device__ __forceinline__ void paged_join_prefix(const PagedAttnArgs& a, int hd, int token, int head,
                                                  int d, PagedAcc& acc) {
  const PagedPrefix& p = a.pre;
  const int end = min(max(__ldg(a.c.q_start + a.c.n_seqs), 0), a.n_tokens);
  const int lo = min(max(__ldg(a.c.q_start), 0), end);
  const int t = token - lo, nrt = (end - lo + p.tpt - 1) / p.tpt;
  const int nkt = (a.c.prefix_len + p.kt - 1) / p.kt;
  const int kvh = head / a.gq, rt = t / p.tpt;
  const long long units = (long long)a.c.nkv * nrt * nkt;
  const long long per = (units + p.grid - 1) / p.grid;
  const long long begin = ((long long)kvh * nrt + rt) * nkt;
  const int c0 = (int)(begin / per), c1 = (int)((begin + nkt - 1) / per);
  if (c0 == c1) {
    const size_t row = (size_t)token * a.nq + head;
    const float2 ml = __ldcg(p.whole_ml + row);
    acc.join(ml.x, ml.y, __ldcg(reinterpret_cast<const float4*>(p.whole_o + row * hd + d)));
  } else {
    paged_join_slots(p.slots, hd, c0, c1, (t - rt * p.tpt) * a.gq + (head - kvh * a.gq), d, acc);
  }
}

// Writes one float4 (columns d..d+3) of query row (token, head): in the prefix pass the record of an
// item that was not split, else the output after the prefix's records are joined; a row without
// a key is 0.
__device__ __forceinline__ void paged_emit(const PagedAttnArgs& a, int hd, int token, int head, int d,
                                           PagedAcc& acc) {
  const size_t row = (size_t)token * a.nq + head;
  if (a.prefix_pass) {
    *reinterpret_cast<float4*>(a.pre.whole_o + row * hd + d) = acc.o;
    if (d == 0) a.pre.whole_ml[row] = make_float2(acc.m, acc.l);
    return;
  }
  if (a.pre.whole_o) paged_join_prefix(a, hd, token, head, d, acc);
  const float inv = acc.l > 0.f || acc.l != acc.l ? 1.f / acc.l : 0.f;
  const float4 o = make_float4(acc.o.x * inv, acc.o.y * inv, acc.o.z * inv, acc.o.w * inv);
  if (a.act_bf16)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * hd + d) =
        make_uint2(paged_pack(o.x, o.y), paged_pack(o.z, o.w));
  else
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * hd + d) = o;
}

}  // namespace qw
