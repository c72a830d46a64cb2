// C entries of the paged-cache operators: argument checks on the host, then one launch each (two
// for attention behind a shared prefix).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "paged.h"
#include "qw.h"
#include "qw_internal.h"

namespace {

int fail(int code, const char* msg) {
  qw::set_op_error(msg);
  return code;
}

// Shape checks shared by both calls; *shift = log2(page_size). Returns an error text or nullptr.
const char* check_cache(const qw_paged_kv* c, int* shift) {
  if (c->kv_format != QW_KV_F32 && c->kv_format != QW_KV_BF16) return "unknown kv_format";
  if (c->head_dim != 64 && c->head_dim != 128) return "head_dim must be 64 or 128";
  if (c->n_kv_heads <= 0 || c->n_pages <= 0 || c->n_seqs <= 0 || c->max_pages <= 0)
    return "n_kv_heads, n_pages, n_seqs and max_pages must be positive";
  int sh = 4;
  while (sh < 8 && (1 << sh) != c->page_size) ++sh;
  if ((1 << sh) != c->page_size) return "page_size must be 16, 32, 64, 128 or 256";
  if (((int64_t)c->n_pages * c->n_kv_heads << sh) > INT32_MAX)
    return "n_pages * n_kv_heads * page_size must be below 2^31";
  if (c->prefix_len < 0) return "prefix_len must not be negative";
  // (places of keys, rounded up to a tile, are counted in 32 bits)
  if (c->prefix_len + ((int64_t)c->max_pages << sh) > INT32_MAX - 512)
    return "prefix_len + max_pages * page_size must be below 2^31 - 512";
  if (!c->k_pages || !c->v_pages || !c->page_table || !c->kv_len || !c->q_start)
    return "null buffer";
  if (c->prefix_len > 0 && !c->prefix_pages) return "prefix_len without prefix_pages";
  if (((uintptr_t)c->k_pages | (uintptr_t)c->v_pages) & 15) return "pages must be 16-byte aligned";
  *shift = sh;
  return nullptr;
}

qw::PagedView view(const qw_paged_kv* c, int shift) {
  qw::PagedView v{};
  v.k_pages = c->k_pages;
  v.v_pages = c->v_pages;
  v.page_table = c->page_table;
  v.kv_len = c->kv_len;
  v.q_start = c->q_start;
  v.prefix_pages = c->prefix_pages;
  v.status = c->status;
  v.n_pages = c->n_pages;
  v.page_shift = shift;
  v.nkv = c->n_kv_heads;
  v.n_seqs = c->n_seqs;
  v.max_pages = c->max_pages;
  v.prefix_len = c->prefix_len;
  v.kv_bf16 = c->kv_format == QW_KV_BF16;
  return v;
}

constexpr int kMaxDevices = 64;
std::atomic<int> g_sms[kMaxDevices];  // SM count of a device whose kernel attributes are set

// SM count of the current device; its kernels' attributes are set at the first call.
cudaError_t device_sms(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < kMaxDevices && (*sms = g_sms[dev].load()) > 0) return cudaSuccess;
  e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = qw::set_paged_attributes();
  if (e == cudaSuccess && dev >= 0 && dev < kMaxDevices) g_sms[dev].store(*sms);
  return e;
}

}  // namespace

extern "C" size_t qw_sizeof_paged_kv(void) { return sizeof(qw_paged_kv); }

extern "C" int qw_paged_append(const qw_paged_kv* c, const void* qkv, uint32_t act_format, int64_t ld,
                               int32_t n_tokens, int32_t n_q_heads, const uint16_t* q_norm,
                               const uint16_t* k_norm, float eps, float rope_theta,
                               const int32_t* positions, const int32_t* sections, void* q_out,
                               void* stream) {
  if (!c) return fail(QW_ERR_ARG, "qw_paged_append: null cache");
  if (c->struct_size != sizeof(qw_paged_kv))
    return fail(QW_ERR_ABI, "qw_paged_append: struct_size does not match this library's qw_paged_kv");
  int shift = 0;
  if (const char* why = check_cache(c, &shift)) return fail(QW_ERR_ARG, why);
  if (act_format != QW_ACT_F32 && act_format != QW_ACT_BF16)
    return fail(QW_ERR_ARG, "qw_paged_append: unknown act_format");
  if (n_tokens < 0 || n_q_heads <= 0 || n_q_heads > 4096 || c->n_kv_heads > 4096)
    return fail(QW_ERR_ARG, "qw_paged_append: n_tokens must not be negative, heads in [1, 4096]");
  if (n_tokens == 0) return QW_OK;
  if (!qkv || !q_out) return fail(QW_ERR_ARG, "qw_paged_append: null buffer");
  if (!q_norm != !k_norm)
    return fail(QW_ERR_ARG, "qw_paged_append: q_norm and k_norm come together or not at all");
  if (((uintptr_t)q_norm | (uintptr_t)k_norm) & 3)
    return fail(QW_ERR_ARG, "qw_paged_append: q_norm and k_norm must be 4-byte aligned");
  const int hd = c->head_dim, align = act_format == QW_ACT_BF16 ? 8 : 4;
  if (ld < (int64_t)(n_q_heads + 2 * (int64_t)c->n_kv_heads) * hd || ld % align)
    return fail(QW_ERR_ARG,
                "qw_paged_append: ld must hold a row of (n_q_heads + 2 n_kv_heads) * head_dim and be a "
                "multiple of 16 bytes");
  if (((uintptr_t)qkv | (uintptr_t)q_out) & 15)
    return fail(QW_ERR_ARG, "qw_paged_append: qkv and q_out must be 16-byte aligned");
  // (below 1 the frequencies grow along the head, past what two f32 terms carry: 9e-6 rad at 0.01 and
  // position 2^24, no digit at 1e-12)
  if (!(rope_theta >= 1.f) || !isfinite(rope_theta) || !(eps >= 0.f))
    return fail(QW_ERR_ARG, "qw_paged_append: rope_theta must be finite and at least 1, eps not negative");
  qw::AppendArgs a{};
  a.sec0 = a.sec1 = hd / 2;
  a.n_axes = 1;
  if (sections) {
    if (!positions) return fail(QW_ERR_ARG, "qw_paged_append: sections need positions [n_tokens][3]");
    if (sections[0] < 0 || sections[1] < 0 || sections[2] < 0 ||
        (int64_t)sections[0] + sections[1] + sections[2] != hd / 2)
      return fail(QW_ERR_ARG, "qw_paged_append: the three sections must add up to head_dim / 2 pairs");
    a.n_axes = 3;
    a.sec0 = sections[0];
    a.sec1 = sections[0] + sections[1];
  }
  a.c = view(c, shift);
  a.qkv = qkv;
  a.ld = ld;
  a.n_tokens = n_tokens;
  a.nq = n_q_heads;
  a.q_norm = q_norm;
  a.k_norm = k_norm;
  a.eps = eps;
  a.positions = positions;
  a.q_out = q_out;
  // frequencies in turns per position: theta^(-2j/hd) / 2 pi, a geometric row (its f64 rounding
  // stays below 64 * 2^-53 of the value)
  const double step = pow((double)rope_theta, -2.0 / hd);
  double f = 0.15915494309189533577;  // 1 / 2 pi
  for (int j = 0; j < hd / 2; ++j, f *= step) {
    a.inv_hi[j] = (float)f;
    a.inv_lo[j] = (float)(f - (double)a.inv_hi[j]);
  }
  int sms = 0;
  cudaError_t e = device_sms(&sms);
  if (e == cudaSuccess)
    e = qw::launch_paged_append(a, hd, act_format == QW_ACT_BF16, sms, (cudaStream_t)stream);
  if (e != cudaSuccess) return fail(QW_ERR_CUDA, cudaGetErrorString(e));
  return QW_OK;
}

extern "C" size_t qw_paged_attention_workspace_bytes(int32_t n_tokens, int32_t n_q_heads,
                                                     int32_t head_dim, int32_t prefix_len) {
  if (n_tokens < 0 || n_q_heads <= 0 || (head_dim != 64 && head_dim != 128) || prefix_len < 0) return 0;
  return qw::paged_attn_workspace_bytes(n_tokens, n_q_heads, head_dim, prefix_len > 0);
}

extern "C" int qw_paged_attention(const qw_paged_kv* c, const void* q, uint32_t act_format, int64_t ldq,
                                  int32_t n_tokens, int32_t n_q_heads, int32_t max_new, void* out,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  if (!c) return fail(QW_ERR_ARG, "qw_paged_attention: null cache");
  if (c->struct_size != sizeof(qw_paged_kv))
    return fail(QW_ERR_ABI, "qw_paged_attention: struct_size does not match this library's qw_paged_kv");
  int shift = 0;
  if (const char* why = check_cache(c, &shift)) return fail(QW_ERR_ARG, why);
  if (act_format != QW_ACT_F32 && act_format != QW_ACT_BF16)
    return fail(QW_ERR_ARG, "qw_paged_attention: unknown act_format");
  if (n_tokens < 0) return fail(QW_ERR_ARG, "qw_paged_attention: n_tokens must not be negative");
  if (n_q_heads <= 0 || n_q_heads % c->n_kv_heads || n_q_heads / c->n_kv_heads > 8)
    return fail(QW_ERR_ARG,
                "qw_paged_attention: n_q_heads must be a multiple of n_kv_heads, at most 8 times it");
  if (max_new < 1) return fail(QW_ERR_ARG, "qw_paged_attention: max_new must be at least 1");
  if ((int64_t)n_tokens * n_q_heads > INT32_MAX)
    return fail(QW_ERR_ARG, "qw_paged_attention: n_tokens * n_q_heads must be below 2^31");
  if (n_tokens == 0) return QW_OK;
  if (!q || !out || !workspace) return fail(QW_ERR_ARG, "qw_paged_attention: null buffer");
  const int hd = c->head_dim, align = act_format == QW_ACT_BF16 ? 8 : 4;
  if (ldq < (int64_t)n_q_heads * hd || ldq % align)
    return fail(QW_ERR_ARG,
                "qw_paged_attention: ldq must hold n_q_heads * head_dim elements and be a multiple of 16 "
                "bytes");
  if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)workspace) & 15)
    return fail(QW_ERR_ARG, "qw_paged_attention: q, out and workspace must be 16-byte aligned");
  if (workspace_bytes < qw_paged_attention_workspace_bytes(n_tokens, n_q_heads, hd, c->prefix_len))
    return fail(QW_ERR_ARG, "qw_paged_attention: workspace too small");
  int sms = 0;
  cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return fail(QW_ERR_CUDA, cudaGetErrorString(e));
  qw::PagedAttnArgs a{};
  a.c = view(c, shift);
  a.q = q;
  a.ldq = ldq;
  a.out = out;
  a.n_tokens = n_tokens;
  a.nq = n_q_heads;
  a.gq = n_q_heads / c->n_kv_heads;
  a.act_bf16 = act_format == QW_ACT_BF16;
  a.scale_log2 = (float)(1.4426950408889634 / sqrt((double)hd));
  a.wait_ns = c->wait_limit_us == 0                    ? 1000000000ull
              : c->wait_limit_us == QW_PAGED_WAIT_NONE ? 0ull
                                                       : 1000ull * c->wait_limit_us;
  e = qw::launch_paged_attention(a, hd, max_new, workspace, sms, (cudaStream_t)stream);
  if (e == cudaErrorInvalidValue)
    return fail(QW_ERR_ARG,
                "qw_paged_attention: tokens x keys beyond what one call counts (n_kv_heads x row tiles x "
                "key tiles of the longest possible sequences must stay below 2^30), or an unaligned pool");
  if (e != cudaSuccess) return fail(QW_ERR_CUDA, cudaGetErrorString(e));
  return QW_OK;
}
