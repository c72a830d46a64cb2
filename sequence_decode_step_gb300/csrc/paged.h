// Internal interface of the paged-cache operators (not part of the ABI).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "paged_plan.h"

namespace qw {

// A launch that may start while the kernel before it in the stream still runs; the kernel waits for
// that one's end itself (griddepcontrol.wait).
template <class... P, class... Args>
cudaError_t launch_pdl(void (*kernel)(P...), dim3 grid, int threads, uint32_t smem, cudaStream_t s,
                       const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

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
cudaError_t launch_paged_append(const AppendArgs& a, int hd, bool act_bf16, int sms, cudaStream_t s);

// ---- attention ----
// Partial records of query rows: [rows][hd] unnormalised outputs and their (reference maximum,
// sum) in base 2. A launch has two slots of `rows` rows per CTA for the items it splits.
struct PagedSlots {
  float* o;
  float2* ml;
  int rows;
};
// The prefix's record of every (token, query head): in (o, ml) for items that one CTA of the prefix
// launch did whole. Split items: behind tensor-core tiles over the sequences' own keys a kernel joins
// them into (o, ml) first; the decode kernels find the CTAs that share an item from the launch's shape
// and join their slots themselves, so that they can start under the prefix launch.
struct PagedPrefix {
  float* o;      // [n_tokens][nq][hd], nullptr without a prefix
  float2* ml;    // [n_tokens][nq]
  PagedSlots slots;
  int tpt, kt, grid, item_units, least_units;  // of the prefix launch
};
struct PagedSplit {    // a split item of a CTA, for the kernel that joins its records
  int c1;              // last CTA, -1: this CTA begins no split item
  int token, rows, head;  // first token row, query rows, first query head
};
struct PagedAttnArgs {
  PagedView c;
  const void* q;            // [n_tokens][ldq]
  long long ldq;            // elements
  void* out;                // [n_tokens][nq * hd]
  int n_tokens, nq, gq;     // gq = nq / nkv
  int act_bf16;
  int tpt;                  // tokens per row tile
  int item_units;           // tiles that an item costs beside its keys
  int least_units;          // least share of a CTA: fewer records of a short line to join
  float scale_log2;         // log2(e) / sqrt(hd)
  PagedSlots slots;         // of this launch
  int* counters;            // [grid] arrivals of split items, 0 between launches
  float* flush;             // [grid][128][128] of this launch (f32 sums on tensor-core tiles)
  PagedSplit* splits;       // [grid], for the joining kernel (prefix and tensor-core launches)
  int prefix_pass;          // 1: this launch reads the prefix's keys
  PagedPrefix pre;
  uint64_t wait_ns;
};
size_t paged_attn_workspace_bytes(int n_tokens, int nq, int hd, bool prefix);
cudaError_t launch_paged_attention(const PagedAttnArgs& base, int hd, int max_new, void* workspace,
                                   int sms, cudaStream_t s);
cudaError_t set_paged_attributes();

// ---- tensor-core tiles (paged_attention_tc.cu) ----
cudaError_t launch_paged_tc(const PagedAttnArgs& a, int hd, int grid, cudaStream_t s);
// Joins the records of the items that the launch before it (`grid` CTAs) has split.
cudaError_t launch_paged_join(const PagedAttnArgs& a, int hd, int grid, int item_rows, cudaStream_t s);
cudaError_t set_paged_tc_attributes();

// ---- scores by attention weight (paged_weigh.cu) ----
struct WeighStats {     // softmax statistics (maximum, sum; base 2) of query rows
  float2* slots;        // of split items: two slots of an item's rows per CTA
  float2* whole;        // [n_tokens][nq], of the others
};
struct WeighArgs {
  PagedView c;
  const void* q;        // [n_tokens][ldq]
  long long ldq;        // elements
  int n_tokens, nq, gq; // gq = nq / nkv
  int act_bf16;
  int window;           // tokens of a sequence that count, 0: all
  float decay, scale_log2;
  float* scores;        // [n_pages][nkv][page_size]
  WeighStats own, pre;  // over the sequences' own keys and over the prefix
  int grid, pre_grid;   // CTAs of these launches
  float* kept;          // [pool rows][keep] scores (base 2) of sequences with up to `keep` query rows
  int keep;             // even, or 0
  uint64_t wait_ns;     // bound of a wait for tensor-core products
};
size_t paged_weigh_workspace_bytes(size_t pool_rows, int n_tokens, int nq, int gq, int max_new, int window, bool prefix);
cudaError_t launch_paged_weigh(const WeighArgs& base, int hd, int max_new, void* workspace, int sms, cudaStream_t s);
cudaError_t set_weigh_attributes();
// Up to 8 query rows per sequence and KV head (paged_weigh_step.cu).
cudaError_t launch_weigh_step(const WeighArgs& a, int hd, int sms, cudaStream_t s);
cudaError_t set_weigh_step_attributes();

// ---- eviction (paged_evict.cu) ----
struct EvictArgs {
  PagedView c;
  const float* scores;  // [n_pages][nkv][page_size]
  float* scores_out;    // the same shape, or scores itself
  int* kv_len_out;      // [n_seqs], or kv_len itself
  int budget, recent;
  int row16;            // 16-byte columns of a row of keys
  int max_keys;         // scores of a sequence that fit shared memory
  int* kept_len;        // [n_seqs] in the workspace, for lengths that are written in place
  int* new_len;         // that, or kv_len_out
  int2* pairs;          // by place in the pool: a place to fill and the row that fills it
};
cudaError_t launch_paged_evict(const EvictArgs& a, int sms, cudaStream_t s);
cudaError_t set_evict_attributes();

}  // namespace qw
