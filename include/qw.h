/*
 * qw.h -- C ABI of the GB300 (sm_103a) batch-1 Qwen-style decode step.
 *
 * The operation: the autoregressive forward step of a Qwen3-style decoder
 * ("Failed Star / fs, M2" page, "One prefill, all shapes visible": gather ->
 * x L blocks of RMSNorm, QKV, QK-norm, RoPE, GQA causal attention, o_proj +
 * residual, RMSNorm, SwiGLU, down + residual -> final RMSNorm -> tied [V,H]
 * projection of the last row), with an f32-resident KV cache, RoPE applied on
 * the KV write and a greedy argmax taken on the device so that only the token
 * id crosses to the host ("flashmoon demo" page, Performance: decode-critical
 * invariants). Qwen2.5 variants add q/k/v biases, drop QK-norm, use an
 * untied lm_head, int4 group-128 weights and an optional LoRA on q_proj and
 * v_proj ("Emberglass" README, "Why it's hard"). The config and weight
 * structs follow the C structs of the "SuperKittens PR #7" page (sk_qwen_config
 * with eps and tie_word_embeddings; sk_qwen_weights with a nullable lm_head),
 * with a struct_size field so a caller whose struct is shorter than the
 * library's is rejected instead of read past (the bug that page's review found).
 *
 * Conventions for every call:
 *   - Return 0 (QW_OK) or a negative QW_ERR_* code; qw_last_error() gives text.
 *   - "device" pointers are CUDA device (or managed) addresses on the handle's
 *     device; "host" pointers are ordinary CPU memory.
 *   - All GPU work is queued on the handle's stream. Calls that return a host
 *     value (argmax_host, ids_host, qw_get_capture) synchronise that stream.
 *   - A handle is not thread-safe: one thread at a time per handle.
 *   - The library owns the memory it allocates and frees it in qw_destroy.
 */
#ifndef QW_H_
#define QW_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define QW_ABI_VERSION 2u

/* Status codes. */
enum {
  QW_OK = 0,
  QW_ERR_ABI = -1,            /* struct_size / abi_version mismatch */
  QW_ERR_ARG = -2,            /* null pointer, token out of [0,vocab), T <= 0, bad shape */
  QW_ERR_CTX = -3,            /* position would pass max_ctx (checked before any work) */
  QW_ERR_NOT_CAPTURED = -4,   /* checkpoint asked for before a forward that recorded it */
  QW_ERR_SIZE = -5,           /* caller's buffer is too small */
  QW_ERR_CUDA = -6,           /* a CUDA runtime call failed */
  QW_ERR_DEVICE_TIMEOUT = -7, /* a bounded device-side wait gave up */
  QW_ERR_STATE = -8,          /* call out of order (e.g. decode before weights) */
  QW_ERR_NUMERIC = -9         /* a logit was NaN, so there is no argmax */
};

/* qw_config.weight_format */
enum { QW_WEIGHTS_BF16 = 0, QW_WEIGHTS_INT4_G128 = 1, QW_WEIGHTS_Q8_0 = 2 };

/* qw_config.kv_format: how keys (after QK-norm and RoPE) and values are stored. bf16
 * halves the cache ("Emberglass" README, Context window & prefill sizes: the f32
 * cache could be quantised to roughly half); each value is rounded to the nearest
 * bf16 when stored, and attention reads the stored values, widened to f32. */
enum { QW_KV_F32 = 0, QW_KV_BF16 = 1 };

/* Element type of a batch's activations (raw projections, rotated queries, outputs, logits). */
enum { QW_ACT_F32 = 0, QW_ACT_BF16 = 1 };

/* qw_get_capture `which`: the four checkpoints of the "Failed Star / fs, M2"
 * page ("Four boundaries bisect the whole model"). */
enum {
  QW_CAPTURE_EMBEDDING = 0,  /* f32 [rows, hidden]: gathered embedding rows   */
  QW_CAPTURE_BLOCK0 = 1,     /* f32 [rows, hidden]: residual after block 0     */
  QW_CAPTURE_FINAL_NORM = 2, /* f32 [rows, hidden]: final RMSNorm output       */
  QW_CAPTURE_LOGITS = 3      /* f32 [vocab]: logits of the last row            */
};

typedef struct qw_handle qw_handle;

/* Model shape and options. Set struct_size = sizeof(qw_config) and
 * abi_version = QW_ABI_VERSION. head_dim must be 64 or 128; hidden,
 * n_q_heads*head_dim and intermediate must be multiples of 8 (of 128 for
 * int4, of 32 for Q8_0); n_q_heads must be a multiple of n_kv_heads with at
 * most 8 query heads per KV head. */
typedef struct qw_config {
  uint32_t struct_size;
  uint32_t abi_version;
  int32_t n_layers;
  int32_t hidden;
  int32_t n_q_heads;
  int32_t n_kv_heads;
  int32_t head_dim;
  int32_t intermediate;
  int32_t vocab;
  float eps;                    /* RMSNorm epsilon (inside the square root) */
  float rope_theta;             /* RoPE base */
  uint32_t tie_word_embeddings; /* 1: logits = embed . h ; 0: separate lm_head */
  uint32_t qk_norm;             /* 1: per-head RMSNorm of q and k before RoPE (Qwen3) */
  uint32_t qkv_bias;            /* 1: q/k/v projections carry a bias (Qwen2.5) */
  int32_t max_ctx;              /* KV-cache capacity in positions */
  int32_t max_prefill_t;        /* longest prompt taken by one batched prefill pass */
  uint32_t weight_format;       /* QW_WEIGHTS_BF16, QW_WEIGHTS_INT4_G128 or QW_WEIGHTS_Q8_0 */
  uint32_t kv_format;           /* QW_KV_F32 or QW_KV_BF16 */
} qw_config;

/* Weights, all DEVICE pointers owned by the caller; the per-layer members are
 * HOST arrays of n_layers DEVICE pointers. qw_load_weights copies (and repacks)
 * everything into library memory, so the caller may free all of it once the
 * call returns.
 *
 * bf16 tensors are raw bf16 bit patterns, row-major [out, in] as stored by
 * Hugging Face checkpoints ("Failed Star / fs, M2", Correct before fast).
 * int4 tensors (weight_format = QW_WEIGHTS_INT4_G128) are nibble-packed
 * [out, in/2] bytes (element 2i in the low nibble, value = nibble - 8) with
 * bf16 scales [out, in/128], one per 128 consecutive inputs of a row; see
 * qw_quantize_int4_g128. Q8_0 tensors (weight_format = QW_WEIGHTS_Q8_0) are
 * int8 [out, in] (two's complement) with fp16 scales [out, in/32], one per 32
 * consecutive inputs of a row, in the *_scales members; see qw_quantize_q8_0.
 * A Q8_0 model's LM head is Q8_0 too: the untied lm_head is passed quantised,
 * and a tied model's head is quantised from the embedding table at load (the
 * "SuperKittens PR #7" page, Q8_0 commit); the gather keeps the bf16 rows.
 * Embedding, norms and biases are always bf16. */
typedef struct qw_weights {
  uint32_t struct_size;
  uint32_t reserved0;
  const void* embed;          /* bf16 [vocab, hidden] */
  const void* final_norm;     /* bf16 [hidden] */
  const void* lm_head;        /* [vocab, hidden]; must be NULL iff tie_word_embeddings;
                               * int4 (with lm_head_scales) when weight_format is int4 */
  const void* lm_head_scales; /* scales of an int4 or Q8_0 untied lm_head, else NULL */
  const void* const* attn_norm; /* bf16 [hidden] */
  const void* const* q;         /* [n_q_heads*head_dim, hidden] */
  const void* const* k;         /* [n_kv_heads*head_dim, hidden] */
  const void* const* v;         /* [n_kv_heads*head_dim, hidden] */
  const void* const* o;         /* [hidden, n_q_heads*head_dim] */
  const void* const* mlp_norm;  /* bf16 [hidden] */
  const void* const* gate;      /* [intermediate, hidden] */
  const void* const* up;        /* [intermediate, hidden] */
  const void* const* down;      /* [hidden, intermediate] */
  const void* const* q_norm;    /* bf16 [head_dim]; qk_norm only, else NULL */
  const void* const* k_norm;    /* bf16 [head_dim]; qk_norm only, else NULL */
  const void* const* q_bias;    /* bf16 [n_q_heads*head_dim]; qkv_bias only, else NULL */
  const void* const* k_bias;    /* bf16 [n_kv_heads*head_dim] */
  const void* const* v_bias;    /* bf16 [n_kv_heads*head_dim] */
  const void* const* q_scales;  /* int4: bf16, Q8_0: fp16 scales of each linear, else NULL */
  const void* const* k_scales;
  const void* const* v_scales;
  const void* const* o_scales;
  const void* const* gate_scales;
  const void* const* up_scales;
  const void* const* down_scales;
} qw_weights;

/* Low-rank adapter on q_proj and v_proj: y += (alpha / rank) * B (A x)
 * ("Emberglass" README: LoRA hot-swap, perfect restore on clear). All members
 * are HOST arrays of n_layers DEVICE pointers to bf16 data. They are BORROWED:
 * the library keeps the pointers, so the tensors must stay alive until the
 * adapter is cleared with qw_set_lora(h, NULL) or the handle is destroyed. */
typedef struct qw_lora {
  uint32_t struct_size;
  int32_t rank;                 /* 1..64 */
  float alpha;
  uint32_t reserved0;
  const void* const* q_a;       /* [rank, hidden] */
  const void* const* q_b;       /* [n_q_heads*head_dim, rank] */
  const void* const* v_a;       /* [rank, hidden] */
  const void* const* v_b;       /* [n_kv_heads*head_dim, rank] */
} qw_lora;

/* ABI self-description, so a binding can check its struct layouts. */
uint32_t qw_abi_version(void);
size_t qw_sizeof_config(void);
size_t qw_sizeof_weights(void);
size_t qw_sizeof_lora(void);

/* Create a handle on the current CUDA device. cuda_stream is a cudaStream_t
 * the handle will use (borrowed), or NULL for a stream the handle creates and
 * owns. Allocates the KV cache (2 * n_layers * n_kv_heads * max_ctx * head_dim
 * elements of 4 bytes, or 2 with QW_KV_BF16) and work buffers. *out is set only
 * on success. */
int qw_create(const qw_config* cfg, void* cuda_stream, qw_handle** out);

/* Copy and repack the weights into library memory (fused [q;k;v] rows,
 * interleaved gate/up rows). May be called again to replace them; resets the
 * position to 0. */
int qw_load_weights(qw_handle* h, const qw_weights* w);

/* Process T prompt ids (HOST array) at positions pos..pos+T-1, appending their
 * keys and values to the cache; afterwards pos += T. Prompts of at most
 * max_prefill_t ids with no LoRA active run as one batched causal pass on the
 * tensor cores (int4 weights are dequantised exactly, layer by layer, into two
 * bf16 terms for it); longer prompts, any prompt while a LoRA is set, and every
 * prompt of a Q8_0 model run through the sequential decode path ("Emberglass"
 * README, Context window & prefill sizes: maxPrefillT). logits_dev (DEVICE, vocab
 * floats, nullable) receives the last row's logits; argmax_host (nullable)
 * receives its greedy token and makes the call synchronous.
 * Errors: QW_ERR_ARG (T <= 0, id out of range), QW_ERR_CTX (pos+T > max_ctx). */
int qw_prefill(qw_handle* h, const int32_t* ids_host, int32_t T, float* logits_dev,
               int32_t* argmax_host);

/* One decode step at position pos: token in [0, vocab), or token < 0 to feed
 * the previous step's device-resident argmax (no host round trip). Afterwards
 * pos += 1. logits_dev (DEVICE, vocab floats) and argmax_host are nullable as
 * in qw_prefill. Errors: QW_ERR_ARG, QW_ERR_CTX, QW_ERR_STATE (token < 0 with
 * no previous step), QW_ERR_DEVICE_TIMEOUT, QW_ERR_NUMERIC. */
int qw_decode_step(qw_handle* h, int32_t token, float* logits_dev, int32_t* argmax_host);

/* n_steps greedy steps on the device, the first fed `token` (or the previous
 * argmax if token < 0), each next one fed the previous argmax without leaving
 * the GPU ("Emberglass" README: GPU-resident batched decode loop, one sync per
 * batch). ids_host (HOST, n_steps ints, nullable) receives the n_steps greedy
 * tokens; the call synchronises once at the end. */
int qw_decode_greedy(qw_handle* h, int32_t token, int32_t n_steps, int32_t* ids_host);

/* pos = 0. Weights and LoRA are kept; cache contents are left as they are and
 * are overwritten as positions are reused. */
int qw_reset(qw_handle* h);

/* Set (lora != NULL) or clear (NULL) the adapter. Weights are never merged, so
 * clearing restores bit-identical outputs. */
int qw_set_lora(qw_handle* h, const qw_lora* lora);

/* Test hooks. qw_kv_cache returns DEVICE pointers to layer `layer`'s K and V
 * cache, each [n_kv_heads, max_ctx, head_dim] (keys stored after QK-norm and
 * RoPE) of f32, or of bf16 bits with QW_KV_BF16, owned by the handle.
 * qw_set_pos / qw_get_pos move or read the position (0 <= pos <= max_ctx). */
int qw_kv_cache(qw_handle* h, int32_t layer, void** k_dev, void** v_dev);
int qw_set_pos(qw_handle* h, int32_t pos);
int qw_get_pos(const qw_handle* h, int32_t* pos);

/* Checkpoints. qw_set_capture(h, 1) makes later forwards record the four
 * checkpoints (it costs extra writes, so it is off by default). After a
 * forward, qw_capture_size gives the floats of checkpoint `which` and
 * qw_get_capture copies them to out_host (HOST, n_floats >= that size).
 * Errors: QW_ERR_NOT_CAPTURED when capture was off for the last forward or
 * no forward ran since it was enabled; QW_ERR_SIZE when n_floats is short. */
int qw_set_capture(qw_handle* h, int32_t enable);
int qw_capture_size(qw_handle* h, int32_t which, size_t* n_floats);
int qw_get_capture(qw_handle* h, int32_t which, float* out_host, size_t n_floats);

/* Decode path (test and benchmarking hook). 0: one persistent cooperative kernel
 * per token, the default whenever the shape fits: head_dim 64 or 128, at most 8
 * query heads per KV head, hidden, intermediate and n_q_heads*head_dim <= 11264,
 * any weight format (int4 only with an untied lm_head) and either cache format,
 * and with a LoRA adapter when each CTA's share of the fused q/k/v rows is at
 * most 64 (every shape up to ~9.7K fused rows); 1: the graph of separate kernels (always
 * available). Asking for 0 on a shape that does not fit keeps 1. Both compute
 * the same step; results agree to f32 rounding. If the persistent
 * kernel cannot be recorded on this device (no cooperative launch), the handle
 * switches to 1 for the rest of its life: the step still succeeds, one line goes
 * to stderr, qw_last_error(h) holds a note saying why, and qw_get_decode_path
 * returns 1. The choice is kept across qw_set_lora. */
int qw_set_decode_path(qw_handle* h, int32_t path);
int qw_get_decode_path(const qw_handle* h, int32_t* path);

/* Bound, in nanoseconds, of every device-side wait (default 1e9). 0 makes
 * every wait give up at once, which tests the QW_ERR_DEVICE_TIMEOUT path. */
int qw_set_wait_limit_ns(qw_handle* h, uint64_t ns);

/* Text of the last error on this handle (or of the last failed handle-less
 * call when h is NULL), or the note of a decode-path switch (see
 * qw_set_decode_path). Valid until the next call. */
const char* qw_last_error(const qw_handle* h);

void qw_destroy(qw_handle* h);

/* ---------------------------------------------------------------------------
 * Stand-alone operations (no handle). They run the same kernels the decode
 * step uses, on caller-provided DEVICE buffers, for per-kernel checks
 * ("flashmoon demo" page, Verification: kernel unit checks against an f64
 * oracle). `stream` is a cudaStream_t or NULL for the legacy default stream.
 * ------------------------------------------------------------------------- */

/* int4 group-128 quantiser ("Emberglass" README: int4 group-128, quantised on
 * the way to the GPU). w: f32 [rows, cols] DEVICE, finite, cols % 128 == 0.
 * packed: u8 [rows, cols/2]; scales: bf16 bits [rows, cols/128]. Per group:
 * s = bf16_rne(f32(max|w| / 7)); q = clamp(rint(f32(w / s)), -7, 7) (0 if
 * s == 0); nibble = q + 8, element 2i in the low nibble. */
int qw_quantize_int4_g128(const float* w, int32_t rows, int32_t cols, uint8_t* packed,
                          uint16_t* scales, void* stream);

/* Decode attention for one layer at position pos: per-head QK-RMSNorm (if
 * q_norm/k_norm are non-NULL), RoPE at pos (rotate-half, cos/sin formed in
 * fp64), append of k and v at cache row pos, split-K flash attention of every
 * query head over keys 0..pos of its KV head, and the combine of the splits
 * ("Emberglass" README: split-K flash-style decode attention).
 *   qkv:       f32 [(nq + 2 nkv) * hd] DEVICE, raw projections (q heads, k heads, v heads)
 *   q_norm, k_norm: bf16 [hd] DEVICE or NULL
 *   k_cache, v_cache: f32 [nkv, cap, hd] DEVICE; row pos is written
 *   out:       f32 [nq * hd] DEVICE
 *   n_splits:  most key splits per KV head, with (nq / nkv) * (n_splits + 1) at most
 *              192 * hd (the combine keeps its weights in the kernel's tile buffers)
 *   workspace: DEVICE scratch of qw_attention_workspace_bytes(...) bytes,
 *              zero-filled before its first use and left zeroed by every call.
 * Errors: QW_ERR_ARG for unsupported shapes (nq or nkv <= 0 included), too many
 * splits, pos outside [0, cap), or a short workspace; all are found on the host
 * before any launch. A device-side wait that gives up is not reported by this
 * unit-check op (its outputs are then invalid); the decode step reports it. */
size_t qw_attention_workspace_bytes(int32_t nq, int32_t nkv, int32_t hd, int32_t n_splits);
int qw_attention_decode(const float* qkv, const uint16_t* q_norm, const uint16_t* k_norm,
                        float* k_cache, float* v_cache, int32_t nq, int32_t nkv, int32_t hd,
                        int32_t cap, int32_t pos, float eps, float rope_theta, int32_t n_splits,
                        float* out, void* workspace, size_t workspace_bytes, void* stream);

/* qw_attention_decode without a workspace argument, for callers that cannot
 * allocate device memory (code running while another thread captures a CUDA
 * graph, allocator-free real-time loops, embedders whose device memory belongs
 * to someone else's pool). The pages have no counterpart of this call; it is a
 * deployment convenience. Arguments and results are those of
 * qw_attention_decode. Its scratch is a fixed file-scope device array of
 * qw_attention_noalloc_max_bytes() bytes (1 MiB) that every GPU loading this
 * library keeps until the process exits; shapes whose scratch
 * (256 + nq*n_splits*(hd+2)*4 bytes, rounded) does not fit return QW_ERR_SIZE.
 * The first call on a device looks up that array's device address and sets the
 * kernel attributes, so make it before any stream capture on that device.
 * Every call shares the one array and clears its counters on `stream`: calls
 * that overlap on the GPU (different streams, or several host threads) race
 * and must be serialised by the caller. No call allocates memory. Failures set
 * qw_last_error(NULL) text like the other handle-less calls; a device-side wait
 * that gives up is not reported, as for qw_attention_decode. */
size_t qw_attention_noalloc_max_bytes(void);
int qw_attention_decode_noalloc(const float* qkv, const uint16_t* q_norm, const uint16_t* k_norm,
                                float* k_cache, float* v_cache, int32_t nq, int32_t nkv,
                                int32_t hd, int32_t cap, int32_t pos, float eps,
                                float rope_theta, int32_t n_splits, float* out, void* stream);

/* Final RMSNorm + LM head + greedy argmax over a bf16 [vocab, hidden] table
 * ("Failed Star / fs, M2": final norm, last row, tied [V,H] projection;
 * "flashmoon demo": argmax in the same submit):
 *   h = g * x / sqrt(mean(x^2) + eps); logits = table . h; argmax (ties -> lowest id).
 *   x: f32 [hidden] DEVICE; g: bf16 [hidden] DEVICE; table: bf16 [vocab, hidden] DEVICE;
 *   logits: f32 [vocab] DEVICE; argmax_dev: int32 [1] DEVICE (-1 if any logit is NaN);
 *   workspace: DEVICE scratch of qw_lm_head_workspace_bytes() bytes, zero-filled
 *   before its first use and left zeroed by every call. */
size_t qw_lm_head_workspace_bytes(void);
int qw_lm_head_argmax(const float* x, const uint16_t* g, const uint16_t* table, int32_t vocab,
                      int32_t hidden, float eps, float* logits, int32_t* argmax_dev,
                      void* workspace, size_t workspace_bytes, void* stream);

/* int4 group-128 matrix-vector product, the contraction the decode step runs for
 * int4 weights ("Emberglass" README, "Why it's hard": int4 group-128 weights,
 * dequantised inside the matvec):
 *   y[r] = sum_c W'[r][c] x[c],  W'[r][c] = (nibble(r, c) - 8) * scale[r][c / 128]
 *   packed: u8 [rows, cols/2] DEVICE, element 2i in the low nibble of byte i;
 *   scales: bf16 bits [rows, cols/128] DEVICE (the layout qw_quantize_int4_g128 writes);
 *   x: f32 [cols] DEVICE; y: f32 [rows] DEVICE; cols a multiple of 128, at most 16384;
 *   workspace: DEVICE scratch of qw_gemv_int4_workspace_bytes(rows, cols) bytes,
 *   16-byte aligned, no initialisation needed: the rows are repacked there (a row's
 *   nibbles, then its scales) and the decode step's int4 GEMV kernel runs on them.
 * The dequantisation is exact in f32 (a 4-bit integer times a bf16), so with
 * x = e_j the result is column j of W' bit for bit. Like the other stand-alone
 * ops it does not report a device-side wait that gave up (its outputs are then
 * invalid); QW_ERR_ARG for the argument errors above. */
size_t qw_gemv_int4_workspace_bytes(int32_t rows, int32_t cols);
int qw_gemv_int4_g128(const uint8_t* packed, const uint16_t* scales, int32_t rows, int32_t cols,
                      const float* x, float* y, void* workspace, size_t workspace_bytes,
                      void* stream);

/* Q8_0 quantiser ("SuperKittens PR #7" page, Q8_0 commit: GGUF type-8 weights, blocks
 * of 32 int8 values with one scale). w: f32 [rows, cols] DEVICE, finite, cols % 32 == 0.
 * q: int8 [rows, cols]; scales: fp16 bits [rows, cols/32]. Per block of 32 inputs:
 * s = fp16_rne(f32(max|w| / 127)); q = clamp(rint(f32(w / s)), -127, 127) (0 if s == 0). */
int qw_quantize_q8_0(const float* w, int32_t rows, int32_t cols, int8_t* q, uint16_t* scales,
                     void* stream);

/* Q8_0 matrix-vector product, the contraction the decode step runs for Q8_0 weights:
 *   y[r] = sum_c W'[r][c] x[c],  W'[r][c] = q[r][c] * scale[r][c / 32]
 *   q: int8 [rows, cols] DEVICE; scales: fp16 bits [rows, cols/32] DEVICE; x: f32 [cols];
 *   y: f32 [rows]; cols a multiple of 32, at most 16384; workspace: DEVICE scratch of
 *   qw_gemv_q8_0_workspace_bytes(rows, cols) bytes, 16-byte aligned, no initialisation
 *   needed (the rows are repacked there as the decode step streams them).
 * The dequantisation is exact in f32, so with x = e_j the result is column j of W' bit
 * for bit. A device-side wait that gives up is not reported (outputs invalid). */
size_t qw_gemv_q8_0_workspace_bytes(int32_t rows, int32_t cols);
int qw_gemv_q8_0(const int8_t* q, const uint16_t* scales, int32_t rows, int32_t cols,
                 const float* x, float* y, void* workspace, size_t workspace_bytes, void* stream);

/* Sampling on the device ("flashmoon demo" README: greedy plus temperature / top-k /
 * top-p sampling, temp = 0 meaning greedy; the demo reads every logits row back to
 * the host to sample, at about 2.7x the cost of the decode step). Here only the id
 * leaves the device. With the k largest logits ordered by (logit descending, index
 * ascending) and l_0 the largest:
 *   w_i = exp((l_i - l_0) / temperature)   (f64, i < k)
 *   the nucleus is the shortest prefix whose running sum of w reaches top_p times the
 *   sum over all k; the token is the first candidate of the nucleus whose running sum
 *   exceeds u times the nucleus sum.
 *   temperature <= 0 (or top_k == 1): the greedy argmax (ties -> lowest id).
 *   logits: f32 [vocab] DEVICE; vocab >= 1; top_k in [1, 256], larger than vocab is
 *   clamped to vocab; top_p in (0, 1] (>= 1: no nucleus cut); u in [0, 1), the
 *   uniform draw, supplied by the caller (the library draws no random numbers);
 *   token_dev: int32 [1] DEVICE, receives the id, or -1 when the row holds a NaN or
 *   no finite logit; workspace: DEVICE scratch of qw_sample_workspace_bytes(vocab,
 *   top_k) bytes, no initialisation needed. QW_ERR_ARG for arguments outside these
 *   ranges (also when vocab / 16384 * top_k > 4096, the final sort's capacity). */
size_t qw_sample_workspace_bytes(int32_t vocab, int32_t top_k);
int qw_sample(const float* logits, int32_t vocab, float temperature, int32_t top_k, float top_p,
              float u, int32_t* token_dev, void* workspace, size_t workspace_bytes, void* stream);

/* qw_sample over the handle's logits of its last step (qw_decode_step,
 * qw_decode_greedy or qw_prefill), on the handle's stream and with its own
 * workspace; writes the id to *token_host (synchronises). QW_ERR_STATE before any
 * step, QW_ERR_NUMERIC when the row holds a NaN or no finite logit. */
int qw_sample_last(qw_handle* h, float temperature, int32_t top_k, float top_p, float u,
                   int32_t* token_host);

/* Sampling for a batch: one token per row of logits, each row with its own settings. With a row's
 * logits ordered by (logit descending, index ascending), l_0 the largest and
 *   w_i = exp((l_i - l_0) / temperature)   (f64)
 * the row keeps the shortest of three prefixes: the top_k first; the nucleus, the shortest prefix whose
 * running sum of w reaches top_p times the sum over those top_k; and the w_i >= min_p. The token is the
 * first whose running sum exceeds u times the kept sum (as qw_sample, which this equals for one row with
 * min_p = 0, without its limit on top_k).
 *   temperature <= 0 or top_k == 1: the greedy argmax (ties -> lowest id), whatever the rest is;
 *   top_k <= 0 or >= vocab: no cut; top_p >= 1: no nucleus; min_p = 0: none.
 * A logit of -inf is never drawn. A row gets token -1 and probability 0 when it holds a NaN, +inf or
 * nothing above -inf, or when its settings lie outside their ranges (temperature NaN or infinite, top_p not
 * above 0, min_p outside [0, 1], u outside [0, 1)); one value for all rows outside its range is QW_ERR_ARG, for
 * greedy rows too. A running sum is right to 2^-27 of itself whatever the vocabulary is, so that the token is the
 * one of exact sums unless a border lies within 2^-26 of what is compared with it, and the same on every run.
 * Weights below e^-48 count as 0, a difference l_0 - l_i beyond f32's range as infinite, and a temperature between 0
 * and 3.2e-29 as 3.2e-29.
 *   params:    each setting as one value for all rows, or (its pointer not NULL) DEVICE [n_rows], which a
 *              captured graph may replay with new ones
 *   logits:    act_format [n_rows, ld] DEVICE, ld >= vocab elements, aligned to its type; vocab <= 2^20
 *   u:         f32 [n_rows] DEVICE, the uniform draws (the library draws no random numbers)
 *   tokens:    int32 [n_rows] DEVICE; probs: f32 [n_rows] DEVICE or NULL, w / kept sum of the token (1 for
 *              a greedy row)
 * No workspace. n_rows = 0 does nothing. */
typedef struct qw_sample_params {
  uint32_t struct_size;      /* sizeof(qw_sample_params) */
  float temperature;
  int32_t top_k;
  float top_p;
  float min_p;
  uint32_t reserved0;
  const float* temperatures;
  const int32_t* top_ks;
  const float* top_ps;
  const float* min_ps;
} qw_sample_params;
size_t qw_sizeof_sample_params(void);
int qw_sample_batch(const qw_sample_params* params, const void* logits, uint32_t act_format, int64_t ld,
                    int32_t n_rows, int32_t vocab, const float* u, int32_t* tokens, float* probs,
                    void* stream);

/* Prefill contraction on tcgen05 tensor cores: C[M,N] = (A_hi + A_lo)[M,K] . B[N,K]^T.
 * A_hi, A_lo (nullable), B: bf16 row-major DEVICE, 16-byte aligned, K % 8 == 0; C: f32
 * [M,N] DEVICE. The activation of a layer enters as its two-bf16 split (hi = bf16(x),
 * lo = bf16(x - hi)) against the exact bf16 weight rows ("Emberglass" README: batched
 * tiled-GEMM prefill). bn: output-tile width 64, 128 or 256 (0 picks one). */
int qw_gemm_bf16(const uint16_t* a_hi, const uint16_t* a_lo, const uint16_t* b, int32_t M,
                 int32_t N, int32_t K, float* c, int32_t bn, void* stream);

/* ---------------------------------------------------------------------------
 * A paged cache for a batch of sequences: the step around the projections when more
 * than one sequence is served. Keys and values of one layer lie in a pool of pages,
 * and every sequence owns a list of pages; qw_paged_append puts the new tokens of the
 * batch into them and qw_paged_attention reads them back for those tokens' queries.
 * Lengths and tables live on the device, so a captured CUDA graph replays with new
 * ones. All buffers are the caller's; calls queue on `stream` and return at once.
 * ------------------------------------------------------------------------- */

/* Bits that the kernels add (atomic OR) to qw_paged_kv.status. BAD_PAGE: a page id in
 * use lies outside [0, n_pages); append drops that row, attention reads page 0 instead
 * (that sequence's output is then meaningless). BAD_LENGTH: a kv_len outside
 * [0, max_pages * page_size], or smaller than the sequence's new tokens (append drops
 * rows that have no place, attention clamps), or a q_start that leaves [0, n_tokens]
 * (rows outside the call are left out; the others keep their places) or decreases
 * (attention then leaves its outputs as they were).
 * TIMEOUT: a device-side wait of attention or weigh gave up; its outputs are invalid. */
enum { QW_PAGED_TIMEOUT = 1, QW_PAGED_BAD_PAGE = 2, QW_PAGED_BAD_LENGTH = 4 };

/* qw_paged_kv.wait_limit_us: every wait of attention's and weigh's kernels gives up at once (to
 * test what follows: TIMEOUT is reported, the call ends, and its workspace is ready for the next one). */
#define QW_PAGED_WAIT_NONE 0xffffffffu

/* One layer's pages and the batch that uses them. Set struct_size =
 * sizeof(qw_paged_kv). All pointers are DEVICE addresses on the current device.
 *
 * The tokens of a call are rows 0 .. n_tokens-1; those of sequence b are rows
 * q_start[b] .. q_start[b+1]-1 (a sequence may have none), and they are the last
 * q_start[b+1] - q_start[b] of its kv_len[b] keys. Key r of sequence b is row
 * r % page_size of page page_table[b][r / page_size]; entries behind the last key's
 * page are not read. Rows of the call outside [q_start[0], q_start[n_seqs]) belong to
 * no sequence: their outputs are left as they were.
 *
 * A shared prefix (prefix_len > 0) is prefix_len keys in the pages prefix_pages that
 * every sequence sees before its own keys; kv_len and page_table count a sequence's own
 * keys only. Slots of a page behind a sequence's last key may hold anything (NaN too).
 * Two sequences may share pages that the call does not append to. */
typedef struct qw_paged_kv {
  uint32_t struct_size;
  uint32_t kv_format;          /* QW_KV_F32 or QW_KV_BF16 */
  int32_t n_pages;             /* pages of the pool; n_pages * n_kv_heads * page_size < 2^31 */
  int32_t page_size;           /* keys of a page: 16, 32, 64, 128 or 256 */
  int32_t n_kv_heads;
  int32_t head_dim;            /* 64 or 128 */
  int32_t n_seqs;
  int32_t max_pages;           /* columns of page_table; prefix_len + max_pages * page_size
                                  < 2^31 - 512 */
  int32_t prefix_len;          /* keys of the shared prefix, 0 for none */
  uint32_t wait_limit_us;      /* bound of a device-side wait of attention or weigh, in microseconds:
                                  0 for one second, QW_PAGED_WAIT_NONE to give up at once */
  void* k_pages;               /* [n_pages, n_kv_heads, page_size, head_dim], 16-byte aligned */
  void* v_pages;               /* the same shape */
  const int32_t* page_table;   /* [n_seqs, max_pages] */
  const int32_t* kv_len;       /* [n_seqs]: keys of each sequence, the call's tokens included */
  const int32_t* q_start;      /* [n_seqs + 1], not decreasing, within [0, n_tokens] */
  const int32_t* prefix_pages; /* [ceil(prefix_len / page_size)], or NULL */
  int32_t* status;             /* [1], QW_PAGED_* bits, or NULL */
} qw_paged_kv;
size_t qw_sizeof_paged_kv(void);

/* Per-head RMSNorm (with q_norm and k_norm), rotation, and append: of every token's raw
 * projections (q heads, k heads, v heads, biases added) the rotated queries go to q_out
 * and the keys (normed, rotated) and values (as they are) into the token's slot, each
 * rounded once to the type it is stored in.
 *   qkv:       act_format [n_tokens, ld] DEVICE, ld >= (n_q_heads + 2 n_kv_heads) * head_dim
 *              elements and a multiple of 16 bytes; 16-byte aligned
 *   q_norm, k_norm: bf16 [head_dim] DEVICE, 4-byte aligned, both or neither (NULL)
 *   rotation (rotate-half): pair (j, j + head_dim/2) turns by position * rope_theta^(-2j/head_dim),
 *              rope_theta >= 1; the angle keeps f32 accuracy for positions up to 2^24 in magnitude
 *   positions: without sections, int32 [n_tokens] DEVICE, or NULL for prefix_len + cache row;
 *              with sections, int32 [n_tokens, 3] DEVICE (time, height, width)
 *   sections:  HOST int32 [3] or NULL: how many of the head_dim/2 pairs turn by each axis, the
 *              first sections[0] by axis 0, the next sections[1] by axis 1, the rest by axis 2
 *   n_q_heads: any number up to 4096 (qw_paged_attention reads multiples of n_kv_heads up to 8 times it)
 *   q_out:     act_format [n_tokens, n_q_heads * head_dim] DEVICE, 16-byte aligned; must not
 *              overlap qkv
 * n_tokens = 0 does nothing. Two tokens must not name the same slot. */
int qw_paged_append(const qw_paged_kv* c, const void* qkv, uint32_t act_format, int64_t ld,
                    int32_t n_tokens, int32_t n_q_heads, const uint16_t* q_norm,
                    const uint16_t* k_norm, float eps, float rope_theta, const int32_t* positions,
                    const int32_t* sections, void* q_out, void* stream);

/* Causal attention of the call's tokens over their pages (append them first): token i of
 * sequence b sees the whole prefix and its own keys 0 .. kv_len[b] - (new tokens of b) + i.
 * Scores are scaled by 1/sqrt(head_dim); query head h reads KV head h / (n_q_heads /
 * n_kv_heads), at most 8 query heads per KV head. A token that sees no key gets zeros. The
 * prefix's keys are read once for the whole batch and joined with each sequence's own by
 * their softmax statistics. f32 activations give results of f32 accuracy from either cache
 * format; bf16 activations with a bf16 cache run one bf16 product with f32 sums (the softmax's
 * weights are rounded to bf16). Results do not depend on the order in which the CTAs finish: a call
 * repeated gives the same bits. Keys and values that a call's tokens may see are finite.
 *   q:         act_format [n_tokens, ldq] DEVICE, ldq >= n_q_heads * head_dim elements and a
 *              multiple of 16 bytes; 16-byte aligned (q_out of qw_paged_append, ldq = n_q_heads * head_dim)
 *   max_new:   the most new tokens of one sequence, which chooses the kernels together with
 *              n_tokens, n_seqs, the heads, the table's width (max_pages * page_size stands for
 *              the lengths, which are on the device) and prefix_len. Another kernel rounds
 *              elsewhere; a wrong value costs speed only
 *   limit:     n_kv_heads x row tiles (of the longest chunks that n_tokens and n_seqs allow) x key
 *              tiles (of the table's width, and of the prefix) must stay below 2^30, else
 *              QW_ERR_ARG: 256 sequences of 8 KV heads may have tables of 8M keys
 *   out:       act_format [n_tokens, n_q_heads * head_dim] DEVICE, 16-byte aligned; must not
 *              overlap q
 *   workspace: DEVICE scratch of qw_paged_attention_workspace_bytes(n_tokens, n_q_heads,
 *              head_dim, prefix_len) bytes, 16-byte aligned, zero-filled before its first use and
 *              left ready for the next call; calls that overlap on the GPU need one each */
size_t qw_paged_attention_workspace_bytes(int32_t n_tokens, int32_t n_q_heads, int32_t head_dim,
                                          int32_t prefix_len);
int qw_paged_attention(const qw_paged_kv* c, const void* q, uint32_t act_format, int64_t ldq,
                       int32_t n_tokens, int32_t n_q_heads, int32_t max_new, void* out,
                       void* workspace, size_t workspace_bytes, void* stream);

/* Scores of the cache's keys by the attention weight that they receive: for every sequence with tokens in the
 * call and each KV head,
 *   score[r] = (r is one of the call's own keys ? 0 : decay * score[r])
 *              + sum over the counted tokens i and the query heads h of the KV head of w[i][h][r]
 * with w the softmax weights that qw_paged_attention gives to the same q (prefix included: the prefix's keys
 * share the weight but have no score). Counted are the last `window` tokens of each sequence, or all of them.
 * Append first; scores need no initialisation (a key's score starts when it is new), and those of sequences
 * without tokens in the call, of rows behind kv_len and of pages that no sequence uses are left as they are.
 * Keys that the call's tokens see are finite, as for attention. Two sequences must not share pages outside the
 * prefix. Results are f32 whatever the types, and the same bits
 * on every run.
 *   q, act_format, ldq, n_tokens, n_q_heads, max_new: as for qw_paged_attention
 *   limit:     n_kv_heads x (tiles of 128 keys of the table's width + 3) x (58 n_seqs + counted tokens * n_q_heads /
 *              n_kv_heads + 2) must stay below 2^30, else QW_ERR_ARG; at most n_seqs * window tokens are counted.
 *              So must n_kv_heads x (tiles of the prefix + 3) x (n_tokens * n_q_heads / n_kv_heads / 128 + 2)
 *   window:    0 for all tokens
 *   decay:     in [0, 1], of what was there; 1 accumulates
 *   scores:    f32 [n_pages, n_kv_heads, page_size] DEVICE, one per key and KV head of the pools
 *   workspace: DEVICE scratch of qw_paged_weigh_workspace_bytes(c, n_tokens, n_q_heads, max_new, window) bytes,
 *              16-byte aligned, no initialisation needed; calls that overlap on the GPU need one each. With up to 8
 *              counted query rows per sequence and KV head it has room for their scores: 4 bytes for each row and
 *              key of the pool, so that a call of few tokens can need more than one of many
 * status: BAD_PAGE (the keys of that page count as page 0's, their scores are not written), BAD_LENGTH, TIMEOUT (a
 * tensor-core product, of more than 8 counted rows or of the prefix, was not done within the cache's wait_limit_us:
 * scores of the call's sequences are then undefined). */
size_t qw_paged_weigh_workspace_bytes(const qw_paged_kv* c, int32_t n_tokens, int32_t n_q_heads, int32_t max_new,
                                      int32_t window);
int qw_paged_weigh(const qw_paged_kv* c, const void* q, uint32_t act_format, int64_t ldq, int32_t n_tokens,
                   int32_t n_q_heads, int32_t max_new, int32_t window, float decay, float* scores,
                   void* workspace, size_t workspace_bytes, void* stream);

/* Eviction: every sequence with more than `budget` own keys goes down to `budget`, for each KV head apart. Of n
 * rows the `recent` last stay, and of the others the budget - recent of the largest scores (ties: the lowest
 * row; NaN is below everything). Those of them in rows below budget - recent stay where they are; the others
 * move, in ascending order, into the rows below budget - recent that became free, in ascending order; the
 * `recent` last move behind them in their order. Keys, values and scores move together inside the sequence's
 * pages; rows from budget on keep what they held, and pages that are no longer used may be given back. Shorter
 * sequences are left as they are.
 * A cache row is no longer its token's position afterwards: give qw_paged_append the positions of later tokens.
 * The rows at the end are the newest, so the call can be repeated as the cache grows.
 *   scores:     f32 [n_pages, n_kv_heads, page_size] DEVICE, 16-byte aligned
 *   scores_out: the same shape, where the rows' scores go (below the new length; of sequences that stay as they
 *               are all of them), or scores itself
 *   kv_len_out: int32 [n_seqs] DEVICE, the new lengths, or c->kv_len itself
 *   budget, recent: budget >= 1, recent in [0, budget]
 *   workspace:  DEVICE scratch of qw_paged_evict_workspace_bytes(c) bytes (8 for every row of the pool and KV
 *               head), 16-byte aligned, no initialisation needed; calls that overlap on the GPU need one each
 * q_start and the prefix are not read. Two sequences must not share pages. status: BAD_PAGE or BAD_LENGTH
 * (kv_len outside [0, max_pages * page_size]); that sequence is then left as it is. */
size_t qw_paged_evict_workspace_bytes(const qw_paged_kv* c);
int qw_paged_evict(const qw_paged_kv* c, const float* scores, float* scores_out, int32_t budget, int32_t recent,
                   int32_t* kv_len_out, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* QW_H_ */
