// qw_paged_append: the raw projections of a ragged batch's new tokens -> rotated queries, and keys
// and values in their pages, in one pass.
//
//   x^ = g * x / sqrt(mean(x^2) + eps)                  (q and k heads, when gains are given)
//   y_j        = x^_j cos a_j - x^_{j+hd/2} sin a_j
//   y_{j+hd/2} = x^_{j+hd/2} cos a_j + x^_j sin a_j,     a_j = p * theta^(-2j/hd)
//
// with p the token's position, or the position on axis 0, 1 or 2 for the pairs below sec0, below
// sec1 and above (time, height, width). Every element is read once and written once with ~10
// flops between, so HBM bounds long calls and the chain of dependent loads (q_start, the page
// table, the store) bounds short ones.
//
// Angles. p * f reaches 10^5 rad and more, where an f32 product has lost the fraction of a turn
// that matters. f / 2 pi comes from the host in two f32 terms (h + l, 48 bits); p is cut into two
// 16-bit halves, exact in f32, and for each half t = p h is reduced by rint(t) with the product's
// rounding error recovered by one fma: the turn's fraction is good to ~1e-7 while |p| <= 2^24 (the
// 2^-49 of f that two terms lose reach it then), and sincospif does the rest. No f64 arithmetic runs on the device (this card has two f64 lanes per
// SM and clock).
//
// Layout. A thread owns 16 bytes of a head's first half and the 16 bytes hd/2 further on, the
// pairs that rotate together, so a head is hd/8 threads of f32 (hd/16 of bf16), loads and stores
// are 16 bytes wide, and the norm is a shuffle over those threads. A CTA takes `tb` whole tokens:
// the cosines of a token are formed once in shared memory for all its heads (24 of them in the
// 16/8-head models), and so is the token's place in the cache. Few tokens get a CTA each, so that
// the chain is all there is; many go 8 to a CTA, which shares the chain and its barriers among them,
// and every thread has the next head's loads in flight while it works on one.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include <algorithm>

#include "paged.h"
#include "qw_ptx.cuh"

namespace qw {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTb = 16;  // most tokens of a CTA

__device__ __forceinline__ float turn_part(float x, float h, float l) {
  const float t = x * h;
  return (t - rintf(t)) + fmaf(x, l, fmaf(x, h, -t));
}
// Fraction of a turn (within a few ulp of one) of position p times the frequency h + l.
__device__ __forceinline__ float turns(int p, float h, float l) {
  const float hi = (float)(p >> 16) * 65536.f, lo = (float)(p & 0xffff);
  const float r = turn_part(hi, h, l) + turn_part(lo, h, l);
  return r - rintf(r);
}

template <bool BF>
struct Act;
template <>
struct Act<false> {
  static constexpr int V = 4;  // elements per 16 bytes
  static __device__ __forceinline__ uint4 load(const void* base, size_t i) {
    return __ldcs(reinterpret_cast<const uint4*>(static_cast<const float*>(base) + i));
  }
  static __device__ __forceinline__ void widen(const uint4& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
};
template <>
struct Act<true> {
  static constexpr int V = 8;
  static __device__ __forceinline__ uint4 load(const void* base, size_t i) {
    return __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i));
  }
  static __device__ __forceinline__ void widen(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(w[e] << 16);
      x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  }
};

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {  // a in the low half
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// V (4 or 8) consecutive elements, rounded once to the stored type.
template <int V>
__device__ __forceinline__ void store_bf16(uint16_t* p, const float (&x)[V]) {
  if constexpr (V == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                              pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
}
template <int V>
__device__ __forceinline__ void store_f32(float* p, const float (&x)[V]) {
#pragma unroll
  for (int e = 0; e < V; e += 4)
    *reinterpret_cast<float4*>(p + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
}
template <int V>
__device__ __forceinline__ void store_any(void* base, size_t i, bool bf, const float (&x)[V]) {
  if (bf)
    store_bf16<V>(static_cast<uint16_t*>(base) + i, x);
  else
    store_f32<V>(static_cast<float*>(base) + i, x);
}

template <int HD, bool BF>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const __grid_constant__ AppendArgs a,
                                                                int tb) {
  constexpr int V = Act<BF>::V, HALF = HD / 2, LPH = HALF / V;  // lanes per head
  constexpr int HPP = kThreads / LPH;                          // heads per pass of the CTA
  __shared__ __align__(16) float2 cs[kMaxTb][HALF];
  __shared__ int row_s[kMaxTb];        // cache row, or INT_MIN: the token belongs to no sequence
  __shared__ long long place_s[kMaxTb];  // first row of the token's slot in the pool, or -1
  __shared__ int seq_s[kMaxTb];
  const int t0 = blockIdx.x * tb, nt = min(tb, a.n_tokens - t0);
  const int heads = a.nq + 2 * a.c.nkv, units = nt * heads;
  const int sub = threadIdx.x % LPH, j0 = sub * V;
  const int page = 1 << a.c.page_shift;

  pdl_wait();
  pdl_launch_dependents();
  // the first unit's loads leave before the lookups below
  int u = threadIdx.x / LPH;
  uint4 n0, n1;
  auto load = [&](int unit) {
    const int t = unit / heads, h = unit - t * heads;
    const size_t i = (size_t)(t0 + t) * a.ld + (size_t)h * HD + j0;
    n0 = Act<BF>::load(a.qkv, i);
    n1 = Act<BF>::load(a.qkv, i + HALF);
  };
  if (u < units) load(u);
  // this thread's gains, as bf16 pairs: of q, then of k, first and second half
  uint32_t g[2][2][V / 2];
  if (a.q_norm) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const int j = j0 / 2 + i;
      g[0][0][i] = __ldg(reinterpret_cast<const uint32_t*>(a.q_norm) + j);
      g[0][1][i] = __ldg(reinterpret_cast<const uint32_t*>(a.q_norm) + HALF / 2 + j);
      g[1][0][i] = __ldg(reinterpret_cast<const uint32_t*>(a.k_norm) + j);
      g[1][1][i] = __ldg(reinterpret_cast<const uint32_t*>(a.k_norm) + HALF / 2 + j);
    }
  }

  if (threadIdx.x < kMaxTb) row_s[threadIdx.x] = INT_MIN;
  __syncthreads();
  bool bad = false;
  // each token's sequence: every thread looks at some sequences' ranges
  for (int b = threadIdx.x; b < a.c.n_seqs; b += kThreads) {
    const int lo = __ldg(a.c.q_start + b), hi = __ldg(a.c.q_start + b + 1);
    const int len = __ldg(a.c.kv_len + b);
    bad |= lo < 0 || hi < lo || hi > a.n_tokens;
    const int first = max(lo, t0), last = min(hi, t0 + nt);
    if (first < last) {
      for (int t = first; t < last; ++t) {
        row_s[t - t0] = len - (hi - t);
        seq_s[t - t0] = b;
      }
    }
  }
  if (bad && a.c.status) atomicOr(a.c.status, PG_BAD_LENGTH);
  __syncthreads();
  if (threadIdx.x < nt) {
    const int row = row_s[threadIdx.x];
    long long place = -1;
    if (row != INT_MIN) {
      if (row < 0 || (row >> a.c.page_shift) >= a.c.max_pages) {
        if (a.c.status) atomicOr(a.c.status, PG_BAD_LENGTH);
      } else {
        const int pg = __ldg(a.c.page_table + (size_t)seq_s[threadIdx.x] * a.c.max_pages +
                             (row >> a.c.page_shift));
        if ((unsigned)pg >= (unsigned)a.c.n_pages) {
          if (a.c.status) atomicOr(a.c.status, PG_BAD_PAGE);
        } else {
          place = ((long long)pg * a.c.nkv << a.c.page_shift) + (row & (page - 1));
        }
      }
    }
    place_s[threadIdx.x] = place;
  }
  for (int i = threadIdx.x; i < nt * HALF; i += kThreads) {
    const int t = i / HALF, j = i % HALF;
    int p = 0;
    if (a.positions) {
      const int axis = (j >= a.sec0) + (j >= a.sec1);
      p = __ldg(a.positions + (size_t)(t0 + t) * a.n_axes + axis);
    } else if (row_s[t] != INT_MIN) {
      p = a.c.prefix_len + row_s[t];
    }
    float sn, cn;
    sincospif(2.f * turns(p, a.inv_hi[j], a.inv_lo[j]), &sn, &cn);
    cs[t][j] = make_float2(cn, sn);
  }
  __syncthreads();

  for (; u < units;) {
    const int t = u / heads, h = u - t * heads;
    const bool is_q = h < a.nq, is_v = h >= a.nq + a.c.nkv;
    float x0[V], x1[V];
    Act<BF>::widen(n0, x0);
    Act<BF>::widen(n1, x1);
    if (u + HPP < units) load(u + HPP);
    if (!is_v) {
      if (a.q_norm) {  // both gains or neither
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) ss = fmaf(x0[e], x0[e], fmaf(x1[e], x1[e], ss));
        // the lanes of a head are active together: units of a pass differ by whole heads
        const unsigned mask = LPH == 32 ? 0xffffffffu
                                        : ((1u << LPH) - 1u) << (threadIdx.x % 32 / LPH * LPH);
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
        const float r = rsqrtf(ss * (1.f / HD) + a.eps);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          const uint32_t w0 = is_q ? g[0][0][i] : g[1][0][i], w1 = is_q ? g[0][1][i] : g[1][1][i];
          x0[2 * i] *= r * __uint_as_float(w0 << 16);
          x0[2 * i + 1] *= r * __uint_as_float(w0 & 0xffff0000u);
          x1[2 * i] *= r * __uint_as_float(w1 << 16);
          x1[2 * i + 1] *= r * __uint_as_float(w1 & 0xffff0000u);
        }
      }
#pragma unroll
      for (int e = 0; e < V; e += 2) {
        const float4 w = *reinterpret_cast<const float4*>(&cs[t][j0 + e]);  // two pairs (cos, sin)
        const float y0 = x0[e] * w.x - x1[e] * w.y, y1 = x0[e + 1] * w.z - x1[e + 1] * w.w;
        x1[e] = x1[e] * w.x + x0[e] * w.y;
        x1[e + 1] = x1[e + 1] * w.z + x0[e + 1] * w.w;
        x0[e] = y0;
        x0[e + 1] = y1;
      }
    }
    if (row_s[t] != INT_MIN) {
      if (is_q) {
        const size_t o = ((size_t)(t0 + t) * a.nq + h) * HD + j0;
        store_any<V>(a.q_out, o, BF, x0);
        store_any<V>(a.q_out, o + HALF, BF, x1);
      } else if (place_s[t] >= 0) {
        const int kvh = h - a.nq - (is_v ? a.c.nkv : 0);
        const size_t o = ((size_t)place_s[t] + ((size_t)kvh << a.c.page_shift)) * HD + j0;
        void* pool = is_v ? a.c.v_pages : a.c.k_pages;
        store_any<V>(pool, o, a.c.kv_bf16, x0);
        store_any<V>(pool, o + HALF, a.c.kv_bf16, x1);
      }
    }
    u += HPP;
  }
}

}  // namespace

cudaError_t launch_paged_append(const AppendArgs& a, int hd, bool act_bf16, int sms, cudaStream_t s) {
  if (a.n_tokens <= 0) return cudaSuccess;
  const int heads = a.nq + 2 * a.c.nkv;
  const int hpp = kThreads / (hd / 2 / (act_bf16 ? 8 : 4));
  // a CTA of one token while each finds an SM for itself (4 or so fit one); at least a pass of heads
  const int narrow = std::max(1, hpp / heads), many = std::min(8, a.n_tokens / (4 * sms));
  const int tb = std::min(kMaxTb, std::max(narrow, many));
  const int grid = (a.n_tokens + tb - 1) / tb;
  if (hd == 64)
    return act_bf16 ? launch_pdl(paged_append_kernel<64, true>, dim3(grid), kThreads, 0, s, a, tb)
                    : launch_pdl(paged_append_kernel<64, false>, dim3(grid), kThreads, 0, s, a, tb);
  return act_bf16 ? launch_pdl(paged_append_kernel<128, true>, dim3(grid), kThreads, 0, s, a, tb)
                  : launch_pdl(paged_append_kernel<128, false>, dim3(grid), kThreads, 0, s, a, tb);
}

}  // namespace qw
