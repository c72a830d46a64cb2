// Work of a paged-attention launch and how its CTAs share it.
//
// An item is one row tile (up to R query rows: tpt tokens x gq heads of one KV head) of one
// sequence; its work is its key tiles of KT keys. Items in the order (sequence, KV head, row
// tile) laid end to end form one line of units, and CTA c takes units [c per, (c + 1) per): the
// lengths live on the device, so every CTA forms the same prefix sums of the sequences' units
// and finds its own start. The load is even to one key tile whatever the lengths are, and only the
// items at a CTA's ends are split: at most two partial records per CTA, slot 2c for an item that
// began in an earlier CTA and slot 2c + 1 for one that goes on in the next. Records are joined in
// CTA order, so results do not depend on which CTA is last: those of a decode step's launch by the
// last CTA to arrive (counters[first CTA]), those of a prefix or of tensor-core tiles by a kernel
// of their own (many rows: one CTA would read them for 5-10 us).
//
// An item costs a CTA some tiles beside its keys (q, the join, the output), so on the line it is
// that much longer (item_units); the units before its first tile are empty.
//
// The shared prefix is the same line with one pseudo-sequence: all the batch's tokens, every one
// of which sees all prefix_len keys.
#pragma once
#include "paged.h"
#include "qw_ptx.cuh"

namespace qw {

// Units are counted in 32 bits: the host refuses calls whose line could be longer, as long as no row counts
// twice. A q_start that decreases is reported and its line not walked, so neither that nor a row that the
// prefix's launch did not take can lead out of the workspace. The code of
// these kernels is kept short on purpose: a decode step's weights sweep the instructions out of the
// caches between two calls, and code that runs once then waits for its own lines (16 KB of joining
// code took 9 us, 70 ns per line of 128 bytes).

// Programmatic launches: every kernel here may start while the one before it still runs, and waits
// for its end (griddepcontrol.wait) before it touches memory. The launch over the sequences' own keys
// behind a prefix waits only before it reads the prefix's records: the prefix's launch lets it start
// after its own wait, so everything older is done by then. Until that wait it may run beside the
// prefix's launch, from which it shares nothing that either writes: split descriptors, slots and O
// records have a copy per launch, counters belong to it alone, and outputs are written behind the wait.
__device__ __forceinline__ void paged_pdl_open(const PagedAttnArgs& a) {
  if (a.prefix_pass || !a.pre.o) pdl_wait();
  pdl_launch_dependents();
}

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
    // the sequence may go on behind the call's rows: its last token still has its last key
    const int end = max(__ldg(a.c.q_start + b + 1), s.lo);
    s.nb = min(end, a.n_tokens) - s.lo;
    const long long cap = (long long)a.c.max_pages << a.c.page_shift;
    const int len = __ldg(a.c.kv_len + b);
    s.len = (int)min((long long)max(len, 0), cap);
    s.base = s.len - (end - s.lo);
  }
  s.nrt = (s.nb + a.tpt - 1) / a.tpt;
  return s;
}
// Rows of sequence b that decrease or leave the call's.
__device__ __forceinline__ bool paged_bad_start(const PagedAttnArgs& a, int b) {
  const int lo = __ldg(a.c.q_start + b), hi = __ldg(a.c.q_start + b + 1);
  return lo < 0 || hi < lo || hi > a.n_tokens;
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
__device__ __forceinline__ int paged_head_units(const PagedAttnArgs& a, const PagedSeq& s) {
  int n = 0;
#pragma unroll 1
  for (int rt = 0; rt < s.nrt; ++rt) n += a.item_units + paged_tiles<KT>(paged_limit(a, s, rt));
  return n;
}

struct PagedCursor {  // a place on the line
  int item, u1, per;        // the current item's first unit; end of the CTA's share
  int lead;                 // units of an item before its first tile
  int b, kvh, rt;           // current item
  int kt, kend;             // this CTA's tiles of it
  int nkt, limit;           // all its tiles; its keys
  PagedSeq s;

  __device__ __forceinline__ bool first() const { return kt == 0; }
  __device__ __forceinline__ bool whole() const { return kt == 0 && kend == nkt; }
  // CTAs that share the item's tiles
  __device__ __forceinline__ int first_cta() const { return (item + lead) / per; }
  __device__ __forceinline__ int last_cta() const {
    return (item + lead + nkt - 1) / per;
  }
  template <int KT>
  __device__ __forceinline__ void enter(const PagedAttnArgs& a) {
    limit = paged_limit(a, s, rt);
    nkt = paged_tiles<KT>(limit);
    kend = min(nkt, u1 - item - lead);
  }
  // To the CTA's next item; false when its share ends before that item's first tile.
  template <int KT>
  __device__ __forceinline__ bool next(const PagedAttnArgs& a) {
    item += lead + nkt;
    if (item + lead >= u1) return false;
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
    return true;
  }
};

struct PagedStart {  // in shared memory: where this CTA starts
  int item, u1, per;
  int b, kvh, rt, kt;
  int any;           // 0: nothing to do
  PagedSeq s;
};

// Block-wide: fills *st. warp_sums: an int per warp.
template <int KT, int THREADS>
__device__ __forceinline__ void paged_find_start(const PagedAttnArgs& a, PagedStart* st, int* warp_sums) {
  constexpr int W = THREADS / 32;
  const int n = a.prefix_pass ? 1 : a.c.n_seqs;
  const int spt = (n + THREADS - 1) / THREADS;
  const int b0 = min((int)threadIdx.x * spt, n), b1 = min(b0 + spt, n);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // the thread's sequences, twice: their units, then (in the one that holds the CTA's start) the place
  int mine = 0, before = 0, r = -1, per = 0, total = 0, back = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      const PagedSeq s = paged_seq(a, b);
      const int hu = paged_head_units<KT>(a, s), units = hu * a.c.nkv;
      if (pass == 0) {
        if (blockIdx.x == 0 && !a.prefix_pass && a.c.status &&
            (s.base < 0 || s.len != __ldg(a.c.kv_len + b) || paged_bad_start(a, b)))
          atomicOr(a.c.status, PG_BAD_LENGTH);
        mine += units;
        back |= !a.prefix_pass && __ldg(a.c.q_start + b + 1) < __ldg(a.c.q_start + b);
        continue;
      }
      if (r >= units) {
        r -= units;
        continue;
      }
      const int kvh = r / hu;
      r -= hu * kvh;
      int rt = 0;
#pragma unroll 1
      for (;; ++rt) {
        const int t = a.item_units + paged_tiles<KT>(paged_limit(a, s, rt));
        if (r < t) break;
        r -= t;
      }
      const int u0 = per * blockIdx.x;
      st->item = u0 - r;
      st->u1 = min(u0 + per, total);
      st->per = per;
      st->b = b;
      st->kvh = kvh;
      st->rt = rt;
      st->s = s;
      st->kt = max(r - a.item_units, 0);
      st->any = u0 - r + a.item_units < st->u1;  // the share has a tile
      break;
    }
    if (pass == 1) break;
    int scan = mine;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += v;
    }
    if (lane == 31) warp_sums[warp] = scan;
    if (threadIdx.x == 0) st->any = 0;
    if (__syncthreads_or(back)) break;
    before = scan - mine;
#pragma unroll 1
    for (int w = 0; w < W; ++w) {
      if (w < warp) before += warp_sums[w];
      total += warp_sums[w];
    }
    per = max((total + (int)gridDim.x - 1) / (int)gridDim.x, a.least_units);
    r = per * (int)blockIdx.x - before;
    if (per * (int)blockIdx.x >= total || r < 0 || r >= mine) break;
  }
  __syncthreads();
}

template <int KT>
__device__ __forceinline__ PagedCursor paged_cursor(const PagedAttnArgs& a, const PagedStart* st) {
  PagedCursor c;
  c.lead = a.item_units;
  c.item = st->item;
  c.u1 = st->u1;
  c.per = st->per;
  c.b = st->b;
  c.kvh = st->kvh;
  c.rt = st->rt;
  c.kt = st->kt;
  c.s = st->s;
  c.enter<KT>(a);
  return c;
}

// Page of key tile row `key` of the cursor's item; a page id outside the pool is reported and read
// as page 0, so that no read leaves the pool.
__device__ __forceinline__ int paged_page_entry(const PagedAttnArgs& a, int b, int key) {
  const int at = key >> a.c.page_shift;
  return a.prefix_pass ? __ldg(a.c.prefix_pages + at)
                       : __ldg(a.c.page_table + (size_t)b * a.c.max_pages + at);
}
__device__ __forceinline__ int paged_page_checked(const PagedAttnArgs& a, int pg) {
  if ((unsigned)pg >= (unsigned)a.c.n_pages) {
    if (a.c.status) atomicOr(a.c.status, PG_BAD_PAGE);
    pg = 0;
  }
  return pg;
}
__device__ __forceinline__ int paged_page(const PagedAttnArgs& a, int b, int key) {
  return paged_page_checked(a, paged_page_entry(a, b, key));
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

// Adds records c0 .. c1 of row r to acc (columns d .. d+3 of hd), in CTA order. The hd/4 lanes of a
// row call it together: each loads the statistics of some records, the weights go round by
// shuffles, and the records' loads are independent.
template <int HD>
__device__ __forceinline__ void paged_join_slots(const PagedSlots& sl, int c0, int c1, int r, int d,
                                                 PagedAcc& acc) {
  constexpr int W = HD / 4;  // lanes of a row: a warp or half of one
  const int lane = threadIdx.x & 31, sub = lane % W;
  const unsigned mask = W == 32 ? 0xffffffffu : 0xffffu << (lane / W * W);
  for (int x0 = c0; x0 <= c1; x0 += W) {
    const int x = x0 + sub, n = min(W, c1 + 1 - x0);
    float2 ml = make_float2(-INFINITY, 0.f);
    if (sub < n) ml = __ldcg(sl.ml + (size_t)(2 * x + (x == c0)) * sl.rows + r);
    float top = ml.x;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(mask, top, o));
    top = fmaxf(top, acc.m);
    const float mu = top == -INFINITY ? 0.f : top;
    const float f = paged_exp2(acc.m - mu);
    acc.m = top;
    acc.l *= f, acc.o.x *= f, acc.o.y *= f, acc.o.z *= f, acc.o.w *= f;
    const float w = paged_exp2(ml.x - mu), wl = ml.y;
    const float4* o = reinterpret_cast<const float4*>(sl.o + ((size_t)2 * x0 * sl.rows + r) * HD + d);
    const size_t step = (size_t)2 * sl.rows * (HD / 4);
    const size_t skip = (size_t)sl.rows * (HD / 4);  // the first record is in its CTA's other slot
#pragma unroll 4
    for (int i = 0; i < n; ++i)
      acc.add(__shfl_sync(mask, w, i, W), __shfl_sync(mask, wl, i, W),
              __ldcg(o + i * step + (x0 + i == c0 ? skip : 0)));
  }
}

// The CTAs c0 .. c1 of the prefix launch that share the item of (token, KV head), and the query
// head's row in it.
struct PagedShare {
  int c0, c1, row;
};
__device__ __forceinline__ PagedShare paged_prefix_share(const PagedAttnArgs& a, int token, int kvh,
                                                         int head_in_group) {
  const PagedPrefix& p = a.pre;
  const int end = min(max(__ldg(a.c.q_start + a.c.n_seqs), 0), a.n_tokens);
  const int lo = min(max(__ldg(a.c.q_start), 0), end);
  const int nrt = (end - lo + p.tpt - 1) / p.tpt, nkt = (a.c.prefix_len + p.kt - 1) / p.kt;
  const int rt = (token - lo) / p.tpt, units = p.item_units + nkt;
  const int per = max((a.c.nkv * nrt * units + p.grid - 1) / p.grid, p.least_units);
  const int first = (kvh * nrt + rt) * units + p.item_units;
  return PagedShare{first / per, (first + nkt - 1) / per, (token - lo - rt * p.tpt) * a.gq + head_in_group};
}

// row / gq for rows below 256 and gq <= 8, with gmul = 65536 / gq + 1.
__device__ __forceinline__ int paged_token(int row, uint32_t gmul) {
  return (int)((uint32_t)row * gmul >> 16);
}

// Writes one float4 (columns d..d+3) of query row (token, head): the prefix's record in its
// launches, else the output (JOIN: after the prefix's record is joined); a row without a key is 0.
template <bool JOIN>
__device__ __forceinline__ void paged_emit(const PagedAttnArgs& a, int hd, int token, int head, int d,
                                           PagedAcc acc) {
  const size_t row = (size_t)token * a.nq + head, at = row * hd + d;
  float* to = static_cast<float*>(a.out);
  if (a.prefix_pass) {
    to = a.pre.o;
    if (d == 0) a.pre.ml[row] = make_float2(acc.m, acc.l);
  } else {
    if (JOIN && a.pre.o) {
      const float2 ml = __ldcg(a.pre.ml + row);
      acc.join(ml.x, ml.y, __ldcg(reinterpret_cast<const float4*>(a.pre.o + at)));
    }
    const float inv = acc.l > 0.f || acc.l != acc.l ? __frcp_rn(acc.l) : 0.f;
    acc.o.x *= inv, acc.o.y *= inv, acc.o.z *= inv, acc.o.w *= inv;
    if (a.act_bf16) {
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
          make_uint2(paged_pack(acc.o.x, acc.o.y), paged_pack(acc.o.z, acc.o.w));
      return;
    }
  }
  *reinterpret_cast<float4*>(to + at) = acc.o;
}

}  // namespace qw
