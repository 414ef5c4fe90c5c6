/*
 * palu_attn.h -- C ABI for Palu-style group-head low-rank (G-LRD) decode
 * attention over a latent KV cache, on one NVIDIA GB300 (sm_103a).
 *
 * The operation ("Palu: KV-Cache Compression With Low-Rank Projection", method
 * section "方法细节"):
 *   - The key/value projections of each group of s consecutive heads are
 *     factored offline, W_g ~= A_g B_g (truncated SVD, "背景知识"), and only the
 *     latents h_g = x A_g (r values per token and group) are cached.
 *   - RoPE models: each head's keys are rebuilt on chip from the cached latents,
 *     K = H_k,g B_k,g[:, head block], rotated by RoPE at every token's own
 *     position, and scored against the rotated query (RoPE paragraph and the
 *     online-rebuild kernel paragraph of "补充细节").
 *   - Non-RoPE models: the query is absorbed, q' = q B_k^T, and scored straight
 *     against H_k (key-fusion paragraph).
 *   - Softmax over all cached tokens, then p is applied to the value latents,
 *     o = p H_v, so the output stays in latent space: B_v is fused into W_o
 *     offline (value-fusion paragraph).
 *   - Optionally the latents are stored as per-token int4 codes with an fp16
 *     scale; a Walsh-Hadamard rotation folded into A and B beforehand needs no
 *     run-time work (Hadamard paragraph).
 *
 * Conventions fixed by this library (the pages leave them open):
 *   - Row vectors: h = x A, A in R^{d x r}. Head i is column block (i % s) of
 *     group (i / s).
 *   - Score scale 1/sqrt(d_h) on both paths.
 *   - RoPE is rotate-half: pairs (k, k + d_h/2) rotated by pos * theta^(-2k/d_h).
 *   - The query is passed UNROTATED; it is rotated at q_pos, which defaults to
 *     the position of the last cached token. No causal mask.
 *   - int4 codes: symmetric in [-7, 7], one fp16 scale per token and group,
 *     scale = fp16_rn(min(amax / 7, 65504)) with IEEE fp32 division,
 *     code = rint_half_even(h / scale) clamped to [-7, 7]; element 2j in the low
 *     nibble and 2j+1 in the high nibble of byte j (two's complement).
 *
 * Memory: every pointer argument that the comments call "device" is device
 * memory owned by the caller, and must stay valid until the work queued on the
 * given stream has finished. The library allocates no device memory: scratch
 * lives in the caller-provided workspace. A handle owns host memory only.
 *
 * Concurrency: the decode calls of one handle (palu_decode_attn, _hybrid, _paged)
 * share its workspace (split partials, the split-merge counters, the error word);
 * calls that may overlap on the GPU need one handle, with its own workspace, each.
 * Calls queued on one stream are ordered and safe.
 *
 * Errors: every call returns a palu_status_t; nothing aborts, prints or throws.
 * Argument checks happen on the host before anything is queued. Conditions only
 * the GPU can see (a position outside the RoPE table, a sequence longer than
 * the cache, a bounded wait that gave up) are recorded in an error word inside
 * the workspace; the kernels clamp the offending index and carry on, and
 * palu_attn_check reports (and clears) it. No other call synchronises.
 *
 * Threading: calls on one handle must not overlap (they share one workspace).
 * Different handles are independent.
 */
#ifndef PALU_ATTN_H
#define PALU_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define PALU_ABI_VERSION 1

/* A CUDA stream. Pass a cudaStream_t (or CUstream); NULL is the legacy default stream. */
typedef struct CUstream_st* palu_stream_t;

typedef enum palu_status_t {
  PALU_OK = 0,
  PALU_ERR_INVALID_ARG = 1,  /* null / misaligned pointer, bad size, inconsistent descriptor */
  PALU_ERR_UNSUPPORTED = 2,  /* a valid shape or dtype combination this build has no kernel for
                                (shapes the descriptor accepts but no fast kernel covers are not
                                refused: they run on the CUDA-core kernel, see palu_decode_plan) */
  PALU_ERR_CUDA = 3,         /* a CUDA runtime call or kernel launch failed */
  PALU_ERR_DEVICE = 4,       /* a kernel recorded an out-of-range index in the error word */
  PALU_ERR_TIMEOUT = 5,      /* a bounded device-side wait gave up (error word) */
  PALU_ERR_WORKSPACE = 6     /* workspace missing, too small or not 256-byte aligned */
} palu_status_t;

typedef enum palu_dtype_t {
  PALU_F32 = 0,
  PALU_F16 = 1,
  PALU_BF16 = 2,
  PALU_INT4 = 3   /* latents only: packed codes + fp16 per-token scales */
} palu_dtype_t;

typedef enum palu_mode_t {
  PALU_MODE_ROPE = 0,      /* rebuild K = H_k B_k on chip, rotate, score */
  PALU_MODE_ABSORBED = 1   /* score q B_k^T straight against H_k (no RoPE) */
} palu_mode_t;

typedef struct palu_attn_desc {
  int abi_version;        /* must be PALU_ABI_VERSION */
  int n_heads;            /* n */
  int head_dim;           /* d_h: 64 or 128 */
  int group_size;         /* s: 1, 2, 4 or 8 (M-LRD is s = 1); 16 or 32 (up to J-LRD, s = n) on the
                             RoPE path with head_dim 128, ranks 256 and F16/BF16/INT4 latents
                             ("方法细节", M-LRD / G-LRD / J-LRD paragraphs); n_heads % s == 0.
                             s = 1 or 2 with ranks 64 s, head_dim 128, F16/BF16 latents and
                             n_heads % 4 == 0 run packed four heads at a time with a block-diagonal
                             B_k (the workspace then holds 4 / s times the B_k bytes); the output
                             layout is unchanged ([batch][n_heads][rank_v]). On the absorbed path
                             s = 8, 16 or 32 at ranks 256 with F16/BF16 latents run as s / 4 groups
                             of four heads over the same cached latents */
  int rank_k;             /* r_k per group: 64, 128 or 256 */
  int rank_v;             /* r_v per group: 64, 128 or 256 */
  palu_dtype_t k_dtype;   /* key-latent storage */
  palu_dtype_t v_dtype;   /* value-latent storage: k_dtype, or PALU_INT4 under F16 / BF16 keys
                             (int4 values only, the Palu notes' 4-bit V setting, "实验结果") */
  palu_dtype_t bk_dtype;  /* B_k storage: equals k_dtype, or PALU_F16 when k_dtype is PALU_INT4 */
  palu_dtype_t q_dtype;   /* query storage: F32, F16 or BF16 */
  palu_mode_t mode;
  double rope_theta;      /* RoPE base (e.g. 10000); ignored by the absorbed mode */
  int max_batch;          /* largest batch any decode call will pass */
  int64_t max_tokens;     /* largest sequence length any decode call will see */
  int64_t max_position;   /* positions must lie in [0, max_position); 0 means max_tokens */
  uint32_t flags;         /* 0, PALU_FLAG_ALIBI, or PALU_FLAG_TEST_STALL (test builds of callers only) */
} palu_attn_desc;

/*
 * Failure-detection test hook; the pages have no counterpart. With this flag the
 * tensor-core RoPE kernel's H_v producer issues no loads, so the consumers' bounded
 * waits give up (after 50 ms instead of the normal 1 s), every CTA drains its copies,
 * frees its tensor memory and returns, and the next palu_attn_check reports
 * PALU_ERR_TIMEOUT. Outputs of such a call are undefined. The other kernels ignore it
 * (palu_decode_plan tells which kernel a call uses). Never set it in production.
 */
#define PALU_FLAG_TEST_STALL 0x80000000u

/*
 * ALiBi position bias on the absorbed path ("方法细节", key-fusion paragraph: a position
 * encoding that never touches the keys, ALiBi being the example, leaves the absorbed query
 * valid). Each score of head i gets -m_i (q_pos - pos_t) with the slopes m_i = 2^(-8 (i + 1) / n)
 * of the ALiBi paper the notes cite; pos_t comes from `positions` (default t) and q_pos from
 * `q_pos` (default the last cached token's position). Only with PALU_MODE_ABSORBED (else
 * PALU_ERR_INVALID_ARG); palu_decode_attn_noalloc and palu_decode_hybrid take no positions and
 * return PALU_ERR_UNSUPPORTED for it.
 */
#define PALU_FLAG_ALIBI 0x1u

/*
 * A latent cache, caller-owned device memory. With n_g = n_heads / group_size:
 *   hk       [max_rows][capacity][n_g][rank_k] elements of k_dtype
 *            (PALU_INT4: [max_rows][capacity][n_g][rank_k / 2] bytes)
 *   hv       [max_rows][capacity][n_g][rank_v] elements of v_dtype (same rule)
 *   k_scale  PALU_INT4 only: [max_rows][capacity][n_g] fp16 scales, else NULL
 *   v_scale  PALU_INT4 only: same for hv, else NULL
 * Batch element b of a call uses row b. hk and hv must be 16-byte aligned.
 */
typedef struct palu_cache {
  void* hk;
  void* hv;
  void* k_scale;
  void* v_scale;
  int64_t capacity;       /* tokens per row (the token stride) */
} palu_cache;

typedef struct palu_attn* palu_attn_t;

/* Bytes of device workspace palu_attn_create needs for this descriptor. */
palu_status_t palu_attn_workspace_size(const palu_attn_desc* desc, size_t* bytes);

/*
 * Create a handle. B_k is device memory [n_g][rank_k][group_size * head_dim]
 * row-major in desc->bk_dtype: the per-group reconstruction factor B_g of the
 * G-LRD factorisation ("方法细节", G-LRD paragraph), already Hadamard-folded if
 * the latents were rotated. It is copied (and re-laid out) into the workspace
 * on `stream`, together with a RoPE cos/sin table computed in float64, so B_k
 * may be freed once that stream has passed this call. `workspace` (device,
 * 256-byte aligned, at least palu_attn_workspace_size bytes) must outlive the
 * handle. The handle itself is host memory.
 */
palu_status_t palu_attn_create(const palu_attn_desc* desc, const void* B_k, void* workspace,
                               size_t workspace_bytes, palu_stream_t stream, palu_attn_t* out);

/*
 * Append n_new tokens per batch row to the cache ("方法细节": the latents h = x A
 * are what is stored). hk_new [batch][n_new][n_g][rank_k] and hv_new
 * [batch][n_new][n_g][rank_v] are device arrays of src_dtype (F32, F16 or BF16).
 * dst_slot (device, [batch] int32) gives the first token index written in each
 * row; tokens dst_slot[b] .. dst_slot[b] + n_new - 1 are overwritten. Float
 * caches store the values rounded to nearest; int4 caches quantise them per
 * token and group (convention in the file header). An index past the capacity
 * is recorded in the error word and the row is skipped.
 */
palu_status_t palu_append_latents(palu_attn_t h, const palu_cache* cache, const void* hk_new,
                                  const void* hv_new, palu_dtype_t src_dtype, const int32_t* dst_slot,
                                  int batch, int n_new, palu_stream_t stream);

/*
 * Decode attention for one new query per batch row.
 *   q          device [batch][n_heads][head_dim], desc->q_dtype, unrotated
 *   seq_lens   device [batch] int32: tokens 0 .. seq_lens[b]-1 of row b attend
 *   positions  device [batch][capacity] int32 RoPE positions, or NULL for
 *              position = token index (ignored by the absorbed mode)
 *   q_pos      device [batch] int32 query positions, or NULL for the position of
 *              the last cached token (ignored by the absorbed mode)
 *   max_seq_len host upper bound on every seq_lens[b] (<= desc->max_tokens and
 *              <= cache->capacity); it sizes the launch. A larger seq_lens[b] is
 *              clamped and recorded in the error word.
 *   out        device [batch][n_heads][rank_v] float32: o_i = p_i H_v,g
 *   lse        device [batch][n_heads] float32 natural log-sum-exp of the scaled
 *              scores, or NULL. An empty row (seq_lens[b] == 0) yields o = 0 and
 *              lse = -inf.
 * Asynchronous on `stream`. Kernel choice: RoPE mode with fp16/bf16/int4 latents,
 * head_dim 128, rank 256 and an even group size runs the tensor-core rebuild kernel;
 * absorbed mode with fp16/bf16 latents, group size 4 and rank 256 runs the TMA
 * streaming kernel; every other accepted descriptor (fp32 latents, int4 absorbed,
 * group size 1, head_dim 64, ranks 64/128) runs the CUDA-core kernel, which is
 * correct for all of them but not tuned. palu_decode_plan reports the choice.
 */
palu_status_t palu_decode_attn(palu_attn_t h, const void* q, const palu_cache* cache,
                               const int32_t* seq_lens, const int32_t* positions, const int32_t* q_pos,
                               int batch, int64_t max_seq_len, float* out, float* lse,
                               palu_stream_t stream);

/*
 * Which kernel palu_decode_attn would launch for this shape, and its split-T plan.
 * Host-only: reads no device memory and queues nothing. A convenience for tests and
 * benchmarks; the pages' statement of the problem has no such call.
 *   cache_capacity  tokens per batch row of the cache that would be passed
 *   batch, max_seq_len  as for palu_decode_attn (same limits)
 *   kernel    out: a palu_kernel_t
 *   n_splits  out: split-T ranges per (batch row, head group); 1 = no split
 *   launches  out: kernel launches the decode call makes (the query preparation
 *             of the CUDA-core and absorbed kernels counts as one)
 * PALU_ERR_INVALID_ARG on a NULL pointer or an argument outside the limits.
 */
typedef enum {
  PALU_KERNEL_TC_ROPE = 1,       /* tensor-core rebuild + RoPE (fp16, bf16, int4 latents) */
  PALU_KERNEL_TMA_ABSORBED = 2,  /* absorbed query, TMA-streamed latents (fp16, bf16) */
  PALU_KERNEL_SIMT = 3           /* CUDA-core kernel: every other supported combination */
} palu_kernel_t;
palu_status_t palu_decode_plan(palu_attn_t h, int64_t cache_capacity, int batch, int64_t max_seq_len,
                               int* kernel, int* n_splits, int* launches);

/*
 * Absorbed-mode decode for callers that cannot allocate device memory (a plugin
 * whose host owns every allocation, an engine with a fixed memory plan, code that
 * must not allocate once serving starts). The pages have no counterpart to it.
 * It takes no handle and no workspace: B_k (device, [n_g][rank_k][s * head_dim]
 * in desc->bk_dtype) and the query are read directly, and the scratch (error
 * word, absorbed queries, split partials) lives in one fixed 8 MiB device array
 * inside this library, which every GPU that loads the library holds until the
 * process exits. It calls no cudaMalloc, cudaFree or other allocating routine.
 *   - desc->mode must be PALU_MODE_ABSORBED (else PALU_ERR_UNSUPPORTED);
 *     arguments as for palu_decode_attn, without positions and q_pos.
 *   - A request whose scratch (4 bytes x batch x n_heads x (rank_k + rank_v) for
 *     one split, plus alignment) does not fit in 8 MiB returns PALU_ERR_WORKSPACE
 *     before anything is queued; larger T only lowers the split count.
 *   - The device is the calling thread's current device, and `stream` must belong
 *     to it (else PALU_ERR_INVALID_ARG). The first call on a device looks up the
 *     array's address on that device (cudaGetSymbolAddress), so make that first
 *     call before any stream capture.
 *   - int4 latents need k_scale / v_scale as for palu_decode_attn (non-NULL, 2-byte
 *     aligned, for each int4 side).
 *   - Every call shares the one array, and its contents persist between calls;
 *     the error word is cleared at the start of each call. Calls that overlap on
 *     the GPU (different streams, or host threads racing) race on the scratch:
 *     serialise them. Out-of-range sequence lengths are clamped; there is no
 *     handle through which to report them.
 */
palu_status_t palu_decode_attn_noalloc(const palu_attn_desc* desc, const void* B_k, const void* q,
                                       const palu_cache* cache, const int32_t* seq_lens, int batch,
                                       int64_t max_seq_len, float* out, float* lse, palu_stream_t stream);

/*
 * The layer's output projection from the latent decode outputs, with B_v fused into
 * W_o ("方法细节", value-fusion paragraph: head i's output p_i V_i = p_i H_v,g B_v^(i)
 * only meets its own rows W_o^(i), so V is never rebuilt):
 *   y[b] = sum_i o[b][i] W_f^(i),   W_f^(i) = B_v^(i) W_o^(i)   (rank_v x d_model).
 *
 * palu_fuse_value_output forms the fused weight once (an offline transform), on the
 * current device:
 *   B_v      device [n_g][rank_v][group_size * head_dim] in in_dtype (F32, F16, BF16),
 *            the per-group value factor; head i uses column block i % s of group i / s
 *   W_o      device [n_heads * head_dim][d_model] in in_dtype, row-major (the rows of
 *            head i are i * head_dim .. (i + 1) * head_dim - 1)
 *   W_fused  device [n_heads * rank_v][d_model] in out_dtype (F16 or BF16): head i's
 *            block is rows i * rank_v .. (i + 1) * rank_v - 1; fp32 accumulation over
 *            head_dim, rounded once to nearest
 *
 * palu_output_proj is the per-step GEMV y = o W_fused on the current device:
 *   W_fused  device [k_dim][d_model] F16/BF16, 16-byte aligned; k_dim = n_heads * rank_v
 *   o        device [batch][k_dim] float32 (palu_decode_attn's `out`, [batch][n][rank_v])
 *   y        device [batch][d_model] float32, overwritten
 *   workspace device, 256-byte aligned, palu_output_proj_workspace_size(k_dim, d_model,
 *            max_batch) bytes for any batch <= max_batch; it must be zero-filled before
 *            its first use, and every call leaves it ready for the next. Calls sharing a
 *            workspace must not overlap on the GPU.
 * d_model must be a multiple of 8 (else PALU_ERR_INVALID_ARG); k_dim <= 65536 and
 * batch <= 1024 (else PALU_ERR_UNSUPPORTED). The result is deterministic (fixed
 * summation order).
 * `stream` must belong to the calling thread's current device (else
 * PALU_ERR_INVALID_ARG). Asynchronous on `stream`.
 */
palu_status_t palu_fuse_value_output(const void* B_v, const void* W_o, palu_dtype_t in_dtype, int n_heads,
                                     int head_dim, int group_size, int rank_v, int64_t d_model, void* W_fused,
                                     palu_dtype_t out_dtype, palu_stream_t stream);
palu_status_t palu_output_proj_workspace_size(int64_t k_dim, int64_t d_model, int max_batch, size_t* bytes);
palu_status_t palu_output_proj(const void* W_fused, palu_dtype_t w_dtype, int64_t k_dim, int64_t d_model,
                               const float* o, int batch, float* y, void* workspace, size_t workspace_bytes,
                               palu_stream_t stream);

/*
 * Decode over a hybrid cache: dense attention-sink and recent-window tokens kept as a standard
 * KV cache next to the G-LRD latent middle ("PuzzleKV" section 3: the sink page and the local
 * window stay dense, the other pages are factorised, and each query attends over both kinds of
 * page, the partial results merged by online softmax; "Shard" section 7: four fp16 sink tokens
 * and a 64-token fp16 window around the compressed middle).
 *
 *   dense->k, dense->v  device [max_rows][capacity][n_heads][head_dim] in dense->dtype (F32, F16
 *                       or BF16), 8-byte aligned for F16 / BF16 and 4-byte for F32 (else
 *                       PALU_ERR_INVALID_ARG). On the RoPE path the keys are stored rotated at their
 *                       own positions (as a dense KV cache holds them); on the absorbed path unrotated.
 *   dense->n_tokens     device [batch] int32: tokens 0 .. n_tokens[b] - 1 of row b are attended
 *                       (their order does not matter); a count outside [0, capacity] is clamped
 *                       and recorded in the error word.
 *
 * The other arguments are palu_decode_attn's, for the latent middle only: seq_lens counts its
 * tokens and `positions` gives their positions (the middle usually starts after the sink tokens,
 * so the default t is rarely right). q_pos is required on the RoPE path (the position of the
 * decoded token). lse is required. One softmax spans both segments; the outputs are
 *   out       [batch][n_heads][rank_v]    sum over the middle of p h_v (latent space)
 *   out_dense [batch][n_heads][head_dim]  sum over the dense tokens of p v (value space)
 *   lse       [batch][n_heads]            natural log-sum-exp over all tokens
 * so head i's attention output is out_i B_v^(i) + out_dense_i (out feeds palu_output_proj with
 * the fused weight, out_dense the plain W_o). Supported head_dim: 32, 64, 96 or 128 (else
 * PALU_ERR_UNSUPPORTED). Two launches on `stream`: the latent decode, then the dense merge.
 */
typedef struct palu_dense_cache {
  const void* k;
  const void* v;
  const int32_t* n_tokens;
  int64_t capacity;
  palu_dtype_t dtype;
} palu_dense_cache;

palu_status_t palu_decode_hybrid(palu_attn_t h, const void* q, const palu_cache* cache, const int32_t* seq_lens,
                                 const int32_t* positions, const int32_t* q_pos, int batch, int64_t max_seq_len,
                                 const palu_dense_cache* dense, float* out, float* out_dense, float* lse,
                                 palu_stream_t stream);

/*
 * Decode over a page-factorised cache ("PuzzleKV" section 3.3, eq. 2 and step 4): every completed
 * page of P tokens of a head stores its keys and values as rank-r factors, K_p ~= L_K R_K and
 * V_p ~= L_V R_V (L: P x r with orthonormal columns from the page's truncated SVD, R: r x d_h).
 * A page is scored as s = (q R_K^T) L_K^T / sqrt(d_h) and its values are read as p L_V R_V,
 * without rebuilding the page. The dense sink and window tokens, when given, share the softmax.
 * This is the PuzzleKV alternative to the G-LRD latent middle of palu_decode_hybrid; the handle
 * supplies the heads, head_dim, q dtype, mode, RoPE table and workspace (its latent shape is not
 * used).
 *
 *   pages->pages     device, 16-byte aligned: [max_rows][capacity][n_heads] page records, each
 *                    L_K [P][r], R_K [r][head_dim], L_V [P][r], R_V [r][head_dim] row-major and
 *                    contiguous (640 r bytes for P = 32, head_dim 128), in pages->dtype (F16/BF16).
 *                    On the RoPE path the factorised keys are the stored, rotated keys.
 *   pages->n_pages   device [batch] int32: pages 0 .. n_pages[b] - 1 of row b are attended; a
 *                    count outside [0, max_pages] is clamped and recorded in the error word.
 *   max_pages        bound on n_pages for this call (<= capacity); it sizes the split plan.
 *   dense            NULL, or the sink / window tokens as for palu_decode_hybrid.
 *   q                [batch][n_heads][head_dim] in the handle's q dtype, unrotated; q_pos [batch]
 *                    is required on the RoPE path.
 *   out              [batch][n_heads][head_dim]: sum over the pages of p (L_V R_V) (value space)
 *   out_dense        [batch][n_heads][head_dim] when dense is given: sum over the dense tokens
 *   lse              [batch][n_heads], required: natural log-sum-exp over all attended tokens
 * so the attention output is out + out_dense. Supported: head_dim 128, P = 32, r in {8, 16, 32}
 * (else PALU_ERR_UNSUPPORTED); PALU_FLAG_ALIBI handles are refused (no positions). The split partials
 * live in the handle's workspace; a handle too small for one head_dim-wide partial per (row, head)
 * (rank_v below head_dim with max_tokens <= 16) gives PALU_ERR_WORKSPACE. One launch, two with the
 * dense segment, asynchronous on `stream`.
 */
typedef struct palu_page_cache {
  const void* pages;
  const int32_t* n_pages;
  int64_t capacity;
  int page_size;
  int rank;
  palu_dtype_t dtype;
} palu_page_cache;

palu_status_t palu_decode_paged(palu_attn_t h, const void* q, const palu_page_cache* pages, const int32_t* q_pos,
                                int batch, int64_t max_pages, const palu_dense_cache* dense, float* out,
                                float* out_dense, float* lse, palu_stream_t stream);

/*
 * Latent production: the step that fills the cache ("方法细节", SVD-rewrite paragraph: the
 * layer caches h = x A in place of k = x W and v = x W_v; G-LRD paragraph: one A_g per group;
 * "补充细节": per-token quantisation of the cached latents). For n_new new tokens of each
 * batch row, H_k = x A_k,g and H_v = x A_v,g are computed on the tensor cores (fp16 or bf16
 * operands, fp32 accumulation) and written into the cache at tokens dst_slot[b] ..
 * dst_slot[b] + n_new - 1 of row b, in the cache's dtype: F32 values as accumulated, F16/BF16
 * rounded to nearest, INT4 quantised per token and group exactly as palu_append_latents does
 * (the same codes and scales for the same fp32 values).
 *
 * palu_down_proj_size / palu_prepare_down_proj (once per layer, an offline transform): A_k and
 * A_v are device arrays [n_g][d_model][rank] in a_dtype (F32, F16, BF16), the Hadamard-folded
 * factors where the latents are rotated. W (device, 16-byte aligned, palu_down_proj_size
 * bytes) receives [2][n_g][rank][d_model] in w_dtype (F16 or BF16): each A_g transposed.
 *
 * palu_project_latents (per prefill or decode step): x device [batch][n_new][d_model] in
 * w_dtype, 16-byte aligned; W as prepared; cache and dst_slot as for palu_append_latents.
 * Supported: rank_k = rank_v in {128, 256}, key and value caches of one dtype, d_model a
 * multiple of 64, batch * n_new < 2^31 (else PALU_ERR_UNSUPPORTED). A slot past the capacity
 * is recorded in the error word and that token's rows are skipped. Asynchronous on `stream`.
 */
palu_status_t palu_down_proj_size(palu_attn_t h, int64_t d_model, size_t* bytes);
palu_status_t palu_prepare_down_proj(palu_attn_t h, const void* A_k, const void* A_v, palu_dtype_t a_dtype,
                                     int64_t d_model, palu_dtype_t w_dtype, void* W, size_t W_bytes,
                                     palu_stream_t stream);
palu_status_t palu_project_latents(palu_attn_t h, const void* W, palu_dtype_t w_dtype, int64_t d_model,
                                   const void* x, const palu_cache* cache, const int32_t* dst_slot, int batch,
                                   int n_new, palu_stream_t stream);

/*
 * Paged dense KV cache: rotation and norm of queries and keys, append, and attention of new tokens.
 *
 * Layers kept dense, and the dense sink and window tokens of palu_decode_hybrid, need a standard KV
 * cache filled with rotated keys ("PuzzleKV" section 3: the sink page and the window stay dense;
 * "Palu" method section, RoPE paragraph: keys are rotated at their own positions) and attention of
 * prompts, chunks and single tokens over it. The pages give no layout; this library's is
 *   k, v   [n_pages][page_size][n_kv_heads][head_dim] elements of desc->dtype
 * A batch row's token t lies in page page_table[row][t / page_size] at offset t % page_size. Without
 * a page table row b is page b, which is the layout of palu_dense_cache (capacity = page_size).
 *
 * A handle of its own (palu_kv_create) holds the shape, the rotation's frequencies and the workspace
 * (error word, split partials, counters), with the rules of palu_attn_t: host memory only, calls on
 * one handle share the workspace, so calls that may overlap on the GPU (two streams, two captured
 * graphs) need a handle each. No call but palu_kv_check synchronises; all can be captured into a
 * graph. The calls run on the workspace's device and leave the thread's current device as it was.
 * The workspace holds the partials of work that is cut along the cached tokens (61 MB for
 * head_dim 128); one handle serves all layers of a shape that run one after the other.
 */
typedef struct palu_kv_desc {
  int abi_version;        /* must be PALU_ABI_VERSION */
  int n_heads;            /* query heads */
  int n_kv_heads;         /* key/value heads; n_heads % n_kv_heads == 0, n_heads / n_kv_heads <= 64. Query
                             head i reads key/value head i / (n_heads / n_kv_heads) */
  int head_dim;           /* 64 or 128 */
  palu_dtype_t dtype;     /* pages, rotated queries and keys, attention output: F16 or BF16 (F32: palu_norm_rope
                             and palu_append_kv only) */
  palu_dtype_t x_dtype;   /* unrotated queries, keys, values and norm weights: F32, F16 or BF16 */
  double rope_theta;      /* RoPE base, 0 for no rotation (convention in the file header: rotate-half) */
  double norm_eps;        /* added to the mean square by the norm; >= 0 */
  int max_batch;          /* largest batch of a call, <= 65535 */
  int64_t max_tokens;     /* largest n_tokens of a call, < 2^31 */
  uint32_t flags;         /* 0, or PALU_FLAG_TEST_STALL (test builds of callers only): the tensor-core kernel's value
                             loader issues no loads, and its waits give up after 50 ms */
} palu_kv_desc;

typedef struct palu_kv* palu_kv_t;

palu_status_t palu_kv_workspace_size(const palu_kv_desc* desc, size_t* bytes);
palu_status_t palu_kv_create(const palu_kv_desc* desc, void* workspace, size_t workspace_bytes, palu_stream_t stream,
                             palu_kv_t* out);
/* As palu_destroy and palu_attn_check. */
palu_status_t palu_kv_destroy(palu_kv_t h);
palu_status_t palu_kv_check(palu_kv_t h, palu_stream_t stream);

/* The pages: caller-owned device memory, 16-byte aligned; n_pages * page_size < 2^31. */
typedef struct palu_kv_pages {
  void* k;
  void* v;
  int64_t n_pages;
  int page_size;          /* tokens of a page, any positive number */
} palu_kv_pages;

/*
 * The new tokens of a batch, packed: row b's are row_start[b] .. row_start[b + 1] - 1 of the token
 * arrays (row_start does not decrease). kv_len[b] counts the row's cached tokens with the new ones,
 * which are the last: new token i of n_b has slot kv_len[b] - n_b + i. Rows without new tokens are
 * fine. Output rows of tokens that belong to no batch row are left as they were.
 */
typedef struct palu_kv_rows {
  const int32_t* row_start;   /* device [batch + 1] */
  const int32_t* kv_len;      /* device [batch] */
  const int32_t* page_table;  /* device [batch][table_pages], or NULL (row b is page b; batch <= n_pages) */
  int64_t table_pages;        /* pages per row of the table */
  const int32_t* positions;   /* device [n_tokens] rotation positions for palu_append_kv, or NULL: the slots */
  int batch;
  int64_t n_tokens;           /* host: rows of the packed token arrays */
  int max_new;                /* host: bound on a row's new tokens */
  int64_t max_kv_len;         /* host: bound on kv_len; <= table_pages * page_size (page_size without a table) */
} palu_kv_rows;

/*
 * Norm and rotation of the queries and keys of n_tokens tokens in one pass:
 *   y = R(pos) (x * rsqrt(mean(x^2) + norm_eps) * w)  per head, R of the file header's convention.
 *   q, k            device [n_tokens][heads][head_dim] in x_dtype, heads and elements contiguous, tokens
 *                   q_stride / k_stride elements apart (a column block of a fused projection); 16-byte
 *                   aligned, strides in multiples of 16 bytes. k may be NULL
 *   q_norm, k_norm  device [head_dim] weights in x_dtype, 16-byte aligned, or NULL: no norm
 *   positions       device [n_tokens], any int32; may be NULL when the handle rotates nothing
 *   q_out, k_out    device, dtype, same layout and rules; may be q and k themselves where dtype = x_dtype and
 *                   the strides agree. Other overlaps are not allowed
 * fp32 arithmetic, one rounding to dtype at the end; before the fp32 sine and cosine an angle is right to
 * 2^-34 turns at any position (rope_theta >= 1).
 */
palu_status_t palu_norm_rope(palu_kv_t h, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                             const void* q_norm, const void* k_norm, const int32_t* positions, int64_t n_tokens,
                             void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                             palu_stream_t stream);

/*
 * Append the new tokens' keys, normed and rotated as by palu_norm_rope, and their values to the pages,
 * and norm and rotate their queries into q_out, in one launch. k, v (and q) as q, k above with
 * n_kv_heads heads; q and q_out (device [n_tokens][n_heads][head_dim] contiguous, dtype) may both be
 * NULL; q_out may be q itself where dtype = x_dtype and q is contiguous. The inputs do not overlap the
 * pages. Rotation positions are rows->positions, or the slots. A token whose slot is negative, lies past the
 * page table or in a page outside the pool is recorded in the error word and not stored; a length outside
 * [0, max_kv_len], a row with more than max_new new tokens and a decreasing row_start are recorded as by
 * palu_attend_kv (the tokens that have a row and a slot are stored). Two tokens that
 * fall on one slot (a page shared by two rows that both append to it) leave a mixture of the two, in 16-byte
 * pieces.
 *
 * A window that rolls (palu_decode_hybrid): one new token in a row with kv_len = slot + 1 and its own position in
 * `positions` overwrites that slot; the order of a dense segment's tokens does not matter.
 */
palu_status_t palu_append_kv(palu_kv_t h, const palu_kv_pages* pages, const palu_kv_rows* rows, const void* q,
                             int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                             const void* q_norm, const void* k_norm, void* q_out, palu_stream_t stream);

/*
 * Attention of the new tokens over the pages, causal: new token i of row b attends to the slots
 * 0 .. kv_len[b] - n_b + i (its own included; palu_append_kv comes first). Score scale
 * 1/sqrt(head_dim).
 *   q    device [n_tokens][n_heads][head_dim] in dtype, rotated, 16-byte aligned, tokens q_stride elements apart
 *        (a multiple of 8)
 *   out  device [n_tokens][n_heads][head_dim] in dtype, contiguous, 16-byte aligned; overlaps no input
 *   lse  device [n_tokens][n_heads] float32 natural log-sum-exp of the scaled scores, or NULL
 * A token that sees no slot (kv_len[b] < n_b) yields 0 and lse = -inf. Slots at or past kv_len[b] are
 * not read and may hold anything; the slots below it must be finite. fp32 scores, softmax statistics
 * and accumulation; the softmax weights are rounded to dtype for the product with the values (F16: at
 * least in steps of 2^-31 of the row's largest, as long as scores stay below 2^20 log2 units). A
 * length outside [0, max_kv_len], a row with more than max_new new tokens (both clamped), a decreasing
 * row_start (the row is skipped) and a page outside the pool (read as zeros) are recorded in the
 * error word. The result does not depend on timing: the same call gives the same bits.
 * max_new * n_heads / n_kv_heads decides the kernel: up to 16 query rows of a key/value head run on
 * the streaming kernel (one launch), more on the tensor-core kernel (one launch). Its cached
 * tokens come by TMA; page sizes without a factor of eight are gathered row by row, at about
 * half the rate. PALU_ERR_UNSUPPORTED for F32 handles, and on the tensor-core kernel where
 * n_pages * page_size * n_kv_heads >= 2^31 - 1.
 */
palu_status_t palu_attend_kv(palu_kv_t h, const palu_kv_pages* pages, const palu_kv_rows* rows, const void* q,
                             int64_t q_stride, void* out, float* lse, palu_stream_t stream);

/*
 * Paged KV cache held in 8 bits, and the steps around its attention: rows and pages planned on the device, and the
 * verification of drafted tokens. All take a handle of palu_kv_create, with its rules: no call synchronises, all can be
 * captured, what goes wrong on the device is recorded in the handle's error word. The pages give no 8-bit dense cache;
 * the layout and its rules are this library's.
 *
 *   k, v              [n_pages][page_size][n_kv_heads][head_dim] e4m3 codes (one byte each), 16-byte aligned
 *   k_scale, v_scale  [n_pages][page_size / 16][n_kv_heads] float32
 *
 * A value is its code times the scale of its head and its block of 16 slots. page_size is a multiple of 16 (with a
 * page table or without); n_pages * page_size < 2^31.
 */
#define PALU_KV8_BLOCK 16
typedef struct palu_kv8_pages {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int64_t n_pages;
  int page_size;
} palu_kv8_pages;

/*
 * palu_append_kv with pages of 8 bits. The new tokens' keys (normed, rotated) and values of a block and head share a
 * scale: the least power of two, from 2^-64 to 2^64, that brings their largest magnitude to 448 or below. Where older
 * tokens stand in the block (its first slot is none of the row's new ones) the scale is at least theirs (brought to 2^-64
 * .. 2^64; NaN to 2^-64); when it grows,
 * their codes are restated under it, which by a power of two moves the codes' exponents and loses only what falls
 * below the least subnormal. A block that begins with a new token begins anew. Codes are rounded to nearest (even), so
 * a value of at least 2^-6 scales is off by at most 2^-4 of itself. NaN is stored as NaN; values past 448 * 2^64
 * (infinities among them) as the largest code.
 * Each row appends to blocks of its own: two rows do not append to one block of 16 slots, and a dense window
 * does not roll in place, as what lies behind a row's new tokens in their last block keeps its codes while the scale
 * may change. PALU_ERR_UNSUPPORTED for F32 handles.
 */
palu_status_t palu_append_kv8(palu_kv_t h, const palu_kv8_pages* pages, const palu_kv_rows* rows, const void* q,
                              int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                              const void* q_norm, const void* k_norm, void* q_out, palu_stream_t stream);

/*
 * palu_attend_kv over pages of 8 bits. Slots at or past kv_len[b] may hold anything and change nothing (their page is
 * theirs to read, up to the end of a 128-token tile); codes and scales below it must be finite, and the scales
 * within 2^-64 .. 2^64 (any such number; one that is not positive counts as 1). fp32 scores, softmax statistics
 * and accumulation. Codes enter the products exactly, as fp16; BF16 queries are lifted by a power of two of their row's
 * own to fp16, which loses what lies 2^-38 and more below the row's largest; the softmax weights, with their values'
 * scales, are rounded to fp16 relative to the row's largest (steps of 2^-31 of it, or finer).
 * The result does not depend on timing: the same call gives the same bits. max_new * n_heads / n_kv_heads decides the
 * kernel, and for 13 to 24 query rows of a key/value head batch and max_kv_len too: few rows over much cache run on the streaming
 * kernel, others on the tensor-core kernel; that one's pairs of CTAs take heads of 128 where n_tokens, batch, max_new and
 * max_kv_len promise work enough (one launch each).
 * What is recorded in the error word, and when outputs are 0 and -inf, is as for palu_attend_kv. PALU_ERR_UNSUPPORTED for F32
 * handles.
 */
palu_status_t palu_attend_kv8(palu_kv_t h, const palu_kv8_pages* pages, const palu_kv_rows* rows, const void* q,
                              int64_t q_stride, void* out, float* lse, palu_stream_t stream);

/*
 * Pages of a batch's requests, kept on the device. Row b holds the pages page_table[b][0 .. held[b]), which cover its
 * cached tokens. Free pages stand in a ring of n_pages entries: free_state[0] is the place of the first, free_state[1]
 * their number.
 */
typedef struct palu_kv_pool {
  int32_t* page_table;        /* device [batch][table_pages] */
  int64_t table_pages;
  int32_t* held;              /* device [batch] */
  int32_t* free_pages;        /* device [n_pages] */
  int32_t* free_state;        /* device [2] */
  int64_t n_pages;
  int page_size;
} palu_kv_pool;

/*
 * The plan of a step: from each row's new tokens and cached length to the arrays of palu_kv_rows.
 *   new_tokens  device [batch]: tokens that row b brings (0: none), or a negative number: the request has ended
 *   kv_len      device [batch]: cached tokens before the step
 * Rows are admitted in order as long as the free pages and the n_tokens packed places last: the first row for which
 * one of the two does not, and every row with new tokens behind it, gets no tokens and no pages. An admitted row takes
 * the pages that its length with the new tokens needs beyond those it holds, from the front of the ring. An ended
 * row's pages go behind the ring's end and can be taken from the next call on; it holds none then, and its
 * length is 0.
 *   row_start   device [batch + 1], written: the packed tokens of the admitted rows
 *   kv_len_out  device [batch], written: the lengths with the new tokens; may be kv_len
 *   held_out, state_out   device [batch] and [2], written: what held and free_state are behind the step; NULL, or
 *               held and free_state themselves: in place. Elsewhere, the call can be repeated on the same pool
 *   positions   device [n_tokens] or NULL, written: each packed token's place in its row (0 behind the last)
 *   slots       device [n_tokens] or NULL, written: its page * page_size + offset (-1 behind the last)
 * Page table entries are written in place. A row whose length is negative or not covered by its pages, that holds
 * more pages than the table, or that brings more than max_new tokens or past max_kv_len, is recorded in the error word
 * and left as it is, without new tokens (ended rows: freed all the same, if `held` is right). A ring whose first place is
 * outside it, or whose number is not within 0 .. n_pages or would be past it with the pages given back, is recorded and
 * left as it is: no page is taken, and ended rows keep their pages and their length. A page outside the pool is
 * recorded (slot -1).
 * The outputs overlap no input but as said. batch 0: nothing is done.
 */
palu_status_t palu_plan_kv_rows(palu_kv_t h, const palu_kv_pool* pool, const int32_t* new_tokens, const int32_t* kv_len,
                                int batch, int64_t n_tokens, int max_new, int64_t max_kv_len, int32_t* row_start,
                                int32_t* kv_len_out, int32_t* held_out, int32_t* state_out, int32_t* positions,
                                int32_t* slots, palu_stream_t stream);

/*
 * Verification of drafted tokens against the target's probabilities. Row b of the batch has the target rows
 * row_start[b] .. row_start[b + 1] - 1: n_b of them, for n_b - 1 drafts (0 rows: nothing is done for it). Draft i,
 * the token x_i, is accepted while every one before it was and
 *   u_i q_i(x_i) < p_i(x_i),
 * p_i being target row i of b and q_i the draft's. Behind the last accepted one a token is drawn: from max(p - q, 0) of
 * the first rejected draft (from p where that is zero throughout), or from p of the last target row where all are
 * accepted: the lowest index whose running sum exceeds u times the whole sum.
 *   target        device [n_tokens][vocab] in p_dtype (F32, F16 or BF16), rows target_stride elements apart
 *   draft         device [batch][max_draft][vocab] in p_dtype, rows draft_stride elements apart, or NULL: each draft
 *                 was certain (q_i is 1 at x_i and 0 elsewhere)
 *   draft_tokens  device [batch][max_draft]
 *   uniforms      device [batch][max_draft + 1] in [0, 1): u_i of draft i, and last that of the drawn token
 *   tokens        device [batch][max_draft + 1], written: the accepted drafts, the drawn token, and -1 behind it
 *   accepted      device [batch], written: how many drafts were accepted
 *   kv_len, kv_len_out   device [batch], both NULL or both given (they may be one): lengths with all new tokens in, and
 *                 without the rejected ones out
 * Probabilities are finite; they need not sum to 1, and negative ones and NaN count as 0. Products and differences
 * are exact, sums are carried in twice the bits of fp32. Uniforms outside [0, 1) are brought to its
 * ends, 0 and 1 - 2^-24 (NaN to the latter), those of drafts and of the drawn token alike. A draft outside the vocabulary is rejected, and recorded in the error word; so are a row with more than
 * max_draft drafts (its first max_draft are taken, the others leave the length as rejected ones do), a decreasing row_start (nothing is done) and a distribution that is
 * zero throughout (the token is -1). vocab <= 2^20. Rows of any alignment; those whose addresses are multiples of
 * 16 bytes are read fastest.
 */
palu_status_t palu_verify_drafts(palu_kv_t h, const void* target, int64_t target_stride, const void* draft,
                                 int64_t draft_stride, palu_dtype_t p_dtype, int64_t vocab, const int32_t* row_start,
                                 int batch, int64_t n_tokens, const int32_t* draft_tokens, int max_draft,
                                 const float* uniforms, int32_t* tokens, int32_t* accepted, const int32_t* kv_len,
                                 int32_t* kv_len_out, palu_stream_t stream);

/* Free the host handle. Does not synchronise: no work on it may be in flight. NULL is fine. */
palu_status_t palu_destroy(palu_attn_t h);

/* Read and clear the device error word (synchronises `stream`). PALU_OK if nothing was recorded. */
palu_status_t palu_attn_check(palu_attn_t h, palu_stream_t stream);

/*
 * Tracing. While enabled, every palu_decode_attn call records a pair of CUDA
 * events around its main attention kernel, on the call's stream, into a ring of
 * PALU_TRACE_CAPACITY pairs (the events are created by the library and hold no
 * device memory; launches beyond the capacity are not recorded).
 * palu_attn_trace_read waits for the recorded events, returns the number of
 * recorded launches and their summed device time in milliseconds, and empties
 * the ring. Disabling destroys the events.
 */
#define PALU_TRACE_CAPACITY 4096
palu_status_t palu_attn_trace_enable(palu_attn_t h, int enable);
palu_status_t palu_attn_trace_read(palu_attn_t h, int* launches, double* total_ms);
/*
 * Like palu_attn_trace_read, but writes each recorded launch's device time in
 * milliseconds, in launch order, to ms[0 .. launches) (host memory, `capacity`
 * entries; launches beyond it are dropped) and empties the ring.
 */
palu_status_t palu_attn_trace_times(palu_attn_t h, float* ms, int capacity, int* launches);

/* Static description of a status code. */
const char* palu_status_string(palu_status_t s);

/*
 * Test hook for the int4 load path of the CUDA-core kernel (PALU_KERNEL_SIMT, which
 * runs int4 absorbed decodes and the int4 shapes the tensor-core kernel does not
 * take): writes, as float32, the dequantised latents (code * scale) of tokens
 * [0, n_tokens) of cache rows [0, batch) into out [batch][n_tokens][n_g][rank]
 * (device), with that kernel's unpack routine. which = 0 for keys, 1 for values.
 * The tensor-core kernel unpacks with other routines; palu_debug_int4_operand and
 * palu_debug_int4_dp2a export those.
 */
palu_status_t palu_debug_dequant(palu_attn_t h, const palu_cache* cache, int which, int batch,
                                 int64_t n_tokens, float* out, palu_stream_t stream);

/*
 * Test hooks for the int4 path of the tensor-core RoPE kernel (PALU_KERNEL_TC_ROPE).
 * They run that kernel's own device routines, so that a bit-exact comparison checks
 * the code that decodes. The pages fix the stored format (per-token int4 latents,
 * "补充细节" KV-quantisation paragraph; codes in [-7, 7]); the routines are this
 * library's.
 *
 * palu_debug_int4_operand -- the key side. For every 128-token tile of rows [0, batch)
 * it loads the packed key codes into shared memory with the decode kernel's TMA
 * box and 128-byte swizzle, expands each token row with the decode kernel's
 * converter into the swizzled fp16 tensor-core operand, reads the operand back and
 * writes, for tokens [0, n_tokens):
 *   codes  device [batch][n_tokens][n_g][rank_k] uint16: the fp16 bit pattern of each
 *          operand element (the signed code as an exact fp16 number), in the operand's
 *          rank order: within every run of eight consecutive ranks, position p holds
 *          rank {0, 2, 4, 6, 1, 3, 5, 7}[p] (B_k^T is stored with the same order)
 *   deq    device float, same shape and order: operand value x the token's key scale
 *          (exact in fp32), or NULL
 * Requires desc.k_dtype = PALU_INT4 and rank_k = 256 (else PALU_ERR_INVALID_ARG /
 * PALU_ERR_UNSUPPORTED) and batch * capacity >= 128 (else PALU_ERR_UNSUPPORTED). A
 * bounded wait that gives up is reported by palu_attn_check as PALU_ERR_TIMEOUT.
 *
 * palu_debug_int4_dp2a -- the value side (which = 1; which = 0 runs the same routine
 * on the key codes). For every block of 16 tokens (tokens 16 k .. 16 k + 15 of
 * [0, n_tokens), missing tokens counting as weight 0) and both heads h = 0, 1 of a
 * head pair, the decode kernel's dp2a routine forms the exact integer sums
 *   sums[b][k][g][h][c] = sum_t weights[b][t][h] * code[b][t][g][c]
 * with weights device [batch][n_tokens][2] int32, each in [0, 32767] (the 15-bit
 * weights the decode kernel feeds it; other values give undefined sums), and
 * sums device [batch][ceil(n_tokens / 16)][n_g][2][rank] int32. Requires rank 256.
 */
palu_status_t palu_debug_int4_operand(palu_attn_t h, const palu_cache* cache, int batch, int64_t n_tokens,
                                      uint16_t* codes, float* deq, palu_stream_t stream);
palu_status_t palu_debug_int4_dp2a(palu_attn_t h, const palu_cache* cache, int which, int batch, int64_t n_tokens,
                                   const int32_t* weights, int32_t* sums, palu_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* PALU_ATTN_H */
