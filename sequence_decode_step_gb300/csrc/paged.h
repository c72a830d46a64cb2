// Internal interface of the paged-cache operators (not part of the ABI).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace qw {

// Bits of the caller's status word (the QW_PAGED_* values of qw.h).
enum : int { PG_TIMEOUT = 1, PG_BAD_PAGE = 2, PG_BAD_LENGTH = 4 };

// The cache and the batch, as the kernels read them (qw_paged_kv after its checks).
struct PagedView {
  void* k_pages;            // [n_pages][nkv][page_size][hd]
  void* v_pages;
  const int* page_table;    // [n_seqs][max_pages]
  const int* kv_len;        // [n_seqs], the new tokens included
  const int* q_start;       // [n_seqs + 1]
  const int* prefix_pages;  // [ceil(prefix_len / page_size)] or nullptr
  int* status;              // or nullptr
  int n_pages, page_shift, nkv, n_seqs, max_pages, prefix_len;
  int kv_bf16;
};

// ---- append (paged_append.cu) ----
struct AppendArgs {
  PagedView c;
  const void* qkv;          // [n_tokens][ld]: q heads, k heads, v heads
  long long ld;             // elements
  int n_tokens, nq;
  const uint16_t* q_norm;   // bf16 [hd] or nullptr
  const uint16_t* k_norm;
  float eps;
  const int* positions;     // [n_tokens][n_axes] or nullptr: prefix_len + cache row
  int n_axes;
  int sec0, sec1;           // first pair of axis 1 and of axis 2
  void* q_out;              // [n_tokens][nq * hd]
  // theta^(-2j/hd) / 2 pi in two f32 terms
  float inv_hi[64], inv_lo[64];
};
cudaError_t launch_paged_append(const AppendArgs& a, int hd, bool act_bf16, cudaStream_t s);

// ---- attention (paged_attention.cu) ----
struct PagedAttnArgs {
  PagedView c;
  const void* q;            // [n_tokens][ldq]
  long long ldq;            // elements
  void* out;                // [n_tokens][nq * hd]
  int n_tokens, nq, gq;     // gq = nq / nkv
  int act_bf16;
  int tpt;                  // tokens per row tile
  float scale_log2;         // log2(e) / sqrt(hd)
  // split items (see PagedSched): slot records of [rows][hd] unnormalised outputs and their
  // (reference maximum, sum) in base 2, two slots per CTA, and an arrival counter per CTA
  float* part_o;
  float2* part_ml;
  int* counters;
  // the shared prefix's record per (token, query head): written by the prefix launch
  // (prefix_pass = 1), merged by the launch over the sequences' own keys (or nullptr)
  float* pre_o;             // [n_tokens][nq][hd]
  float2* pre_ml;           // [n_tokens][nq]
  int prefix_pass;
  int n_ctas;               // grid size
  uint64_t wait_ns;
};
constexpr int kPagedMaxCtas = 512;  // most CTAs of one attention launch (workspace slots)
size_t paged_attn_workspace_bytes(int n_tokens, int nq, int hd, bool prefix);
cudaError_t launch_paged_attention(const PagedAttnArgs& base, int hd, int max_new, void* workspace,
                                   int sms, cudaStream_t s);
cudaError_t set_paged_attributes();

}  // namespace qw
