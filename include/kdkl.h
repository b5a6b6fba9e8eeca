/*
 * kdkl.h — C ABI of libkdkl.so: an offline top-K teacher cache and a fused,
 * chunked KL(p_teacher || q_student) distillation loss for one GB300 (sm_103a).
 *
 * The method is the one described in "Efficient Knowledge Distillation for
 * LLMs: Offline Top-K Logits and a Fused Chunked KL Loss" (Multiverse Computing,
 * Hugging Face blog, 10 Aug 2026), as reported by:
 *   [ART] aiexpert.news, "Making knowledge distillation cheap enough to run in
 *         production" — the offline top-K cache, the three loss formulations
 *         (dense, forward-chunked, fused chunked) and the top-K limitation;
 *   [DAI] dailyai.com.br launch report, section "As duas inovações";
 *   [EPO] epoka.news, sections "Adónde se va la memoria" and "Los dos cambios
 *         propuestos".
 *
 * Conventions shared by every entry point
 *   - Every pointer argument is DEVICE memory owned by the caller, unless the
 *     argument says otherwise.  The library allocates no device memory: scratch
 *     space is the caller's workspace `ws` of at least the size that the matching
 *     *_workspace() query returns, 256-byte aligned.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Every call
 *     only enqueues work on it and returns without synchronising.
 *   - Matrices are row-major.  bf16 is IEEE binary32 with the low 16 bits
 *     dropped (the raw uint16 pattern).  Token rows are the flattened B*T
 *     positions.
 *   - Argument errors are detected on the host, before anything is enqueued,
 *     and returned as KD_ERR_INVALID_ARG / KD_ERR_WORKSPACE / KD_ERR_UNSUPPORTED;
 *     no CUDA call is made in that case.  A failed launch returns KD_ERR_CUDA.
 *     Conditions that only the device can see (a teacher id outside [0, V), a
 *     bounded wait inside a kernel that ran out) are recorded in an error word
 *     inside the workspace and read with kd_get_device_error().
 *   - Calls that share a workspace must be ordered (same stream, or events).
 */
#ifndef KDKL_H_
#define KDKL_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define KD_API __attribute__((visibility("default")))
#else
#define KD_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  KD_OK = 0,
  KD_ERR_INVALID_ARG = 1,   /* a size, pointer, alignment or K out of range     */
  KD_ERR_UNSUPPORTED = 2,   /* no sm_103a device, or a shape the kernels refuse */
  KD_ERR_WORKSPACE = 3,     /* ws is NULL, misaligned or smaller than required  */
  KD_ERR_CUDA = 4,          /* a CUDA runtime/driver call or launch failed      */
  KD_ERR_TIMEOUT = 5,       /* device: a bounded wait inside a kernel ran out   */
  KD_ERR_DEVICE = 6,        /* device: an input value out of range (teacher id) */
  KD_ERR_IO = 7             /* cache file: open/read/write failed, truncated or corrupt */
} kd_status;

/* Element type of a logits matrix. */
typedef enum {
  KD_BF16 = 0,
  KD_F16 = 1,
  KD_F32 = 2
} kd_dtype;

/* What kd_fused_logprobs_bwd does with grad_W [V, d]. */
typedef enum {
  KD_GRAD_ADD_F32 = 0,    /* fp32, added into what the caller passes           */
  KD_GRAD_STORE_F32 = 1,  /* fp32, overwritten                                 */
  KD_GRAD_STORE_BF16 = 2  /* bf16, overwritten, rounded once: N <= chunk alone */
} kd_grad_kind;

#define KD_MAX_K 1024
#define KD_MAX_TOP 128        /* alternatives per position of kd_token_logprobs_fwd */

/* Human-readable name of a kd_status value (static string, never NULL). */
KD_API const char* kd_status_string(int status);

/* Library version as major*10000 + minor*100 + patch. */
KD_API int kd_version(void);

/* ------------------------------------------------------------------------ *
 * Offline top-K teacher cache.
 * [ART] paragraph on the first fix (offline distillation); [DAI] "As duas
 * inovações" item 1; [EPO] "Los dos cambios propuestos", first item: the
 * teacher runs once and only its K highest logits per position, with their
 * token ids, are kept and reused.
 * ------------------------------------------------------------------------ */

/* Workspace bytes kd_topk_cache needs (>= 256; it holds the control block: the error
 * word read by kd_get_device_error, and as its third uint32 (byte offset 8) a count, which
 * the caller may read and reset, of rows selected a second time, see below). */
KD_API size_t kd_topk_cache_workspace(int64_t N, int64_t V, int K);

/*
 * For each of the N rows of a dense bf16 teacher-logits matrix, the K largest
 * logits and their column (token) ids.
 *   logits_bf16 : [N, ld] bf16, row r at logits_bf16 + r*ld; columns [0, V) are
 *                 read.  16-byte aligned; ld >= V and ld*2 a multiple of 16.
 *   K           : 1 <= K <= min(V, KD_MAX_K).
 *   ids_out     : [N, K] int32, written.   vals_out: [N, K] fp32, written.
 *   lse_out     : [N] fp32 or NULL.  If given, also the full-row logsumexp of the
 *                 logits (fp32 running max and sum of exponentials).
 *   dropped_out : [N] fp32 or NULL.  If given, the teacher probability the cache
 *                 drops per row, 1 - sum_k exp(vals_k - lse) (the softmax of the
 *                 full row outside its K kept logits, [ART] paragraph on the top-K
 *                 limitation: the cache loses the teacher's tail), computed in the
 *                 same pass (fp32, compensated sum; NaN where lse is not finite).
 * Each output row is ordered by value, highest first; equal values are ordered
 * by ascending id and the cut at K keeps the lowest ids; -0.0 equals +0.0.
 * Values are the bf16 inputs widened exactly.  NaN inputs take their place in
 * the IEEE 754 totalOrder (positive NaNs above +inf, negative NaNs below -inf,
 * a larger payload further out); apart from the zeros, that is the order.
 * Performance note: each row is streamed once by one warp.  Its selection starts
 * from a threshold taken from the row's first 4096 values, extrapolated into its
 * upper tail (invariant to the row's offset and scale); when fewer than K values
 * reach it (rows whose first 4096 values are far above the rest, for instance),
 * the row is read and selected a second time from an exact bound, the count in
 * the control block's third word goes up, and that warp stops extrapolating for
 * the rest of the call.  The result never depends on the start.
 */
KD_API int kd_topk_cache(const void* logits_bf16, int64_t N, int64_t V, int64_t ld, int K,
                  int32_t* ids_out, float* vals_out, float* lse_out, float* dropped_out,
                  void* ws, size_t ws_bytes, void* stream);

/*
 * The teacher's single pass fused with the cache extraction: for N positions of
 * teacher hidden states Ht [N, dt] bf16 and the teacher's LM-head Wt [V, dt] bf16,
 * the logits Ht Wt^T are formed on the tensor cores `chunk` positions at a time
 * (fp32 accumulation, rounded once to bf16 as a bf16 teacher would emit them) into a
 * [chunk, V] workspace buffer and reduced to their top K right away, so the dense
 * [N, V] teacher logits never exist.  Outputs as kd_topk_cache (ids, vals, optional
 * row logsumexp and dropped mass).  dt % 8 == 0; chunk a multiple of 128.  The
 * workspace holds the [chunk, V] bf16 logits and, per row and 256-column tile, the
 * tile's largest logit, which the projection's epilogue emits: with at least K
 * tiles, their K-th largest is an exact start for the row's selection.  When the
 * row logsumexp or the dropped mass is asked for (K <= 256), the epilogue also
 * emits per row and tile the sum of exp(z - tile max) over the tile's stored
 * (bf16) logits; the row logsumexp is combined from those, and the selection runs
 * without computing it.
 */
KD_API size_t kd_teacher_topk_workspace(int64_t N, int64_t dt, int64_t V, int K, int64_t chunk);
KD_API int kd_teacher_topk(const void* Ht_bf16, const void* Wt_bf16, int64_t N, int64_t dt, int64_t V, int K,
                           int64_t chunk, int32_t* ids_out, float* vals_out, float* lse_out, float* dropped_out,
                           void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------ *
 * Fused chunked KL loss.
 * [ART] paragraph on the second fix; [DAI] "As duas inovações" item 2; [EPO]
 * "Los dos cambios propuestos", second item.  Per position t (reading: forward
 * KL, teacher renormalised over its K cached logits, student normalised over
 * the full vocabulary):
 *   z_t   = H_t W^T / tau                            (never stored)
 *   p_t,k = softmax_k(t_logits_t,k / tau)
 *   KL_t  = sum_k p_t,k (log p_t,k - z_t,id_k + logsumexp_v z_t,v)
 *   loss  = sum over valid t of KL_t / N_valid       (0 when N_valid == 0)
 * The positions are processed `chunk` rows at a time; the [chunk, V] logits
 * live only in tensor memory, tile by tile.
 * ------------------------------------------------------------------------ */

/* Workspace bytes for kd_fused_kl_fwd and kd_fused_kl_bwd with these sizes
 * (one query covers both calls).  Grows with chunk*V, not with N*V. */
KD_API size_t kd_fused_kl_workspace(int64_t N, int64_t d, int64_t V, int K, int64_t chunk);

/*
 * Forward pass.
 *   H_bf16   : [N, d] bf16 student hidden states (16-byte aligned rows: d % 8 == 0).
 *   W_bf16   : [V, d] bf16 LM-head (output projection) weight.
 *   t_ids    : [N, K] int32 cached teacher token ids, distinct within a row.
 *   t_logits : [N, K] fp32 cached teacher logits (any order).
 *   mask     : [N] uint8, 1 = valid position, 0 = padding; NULL = all valid.
 *   chunk    : positions per chunk, a multiple of 128 (the last chunk may be short).
 *   tau      : temperature > 0, divides both teacher and student logits.
 *   loss_out : device fp32 scalar, written.
 *   lse_out  : [N] fp32, logsumexp_v z_t,v, written; keep it for the backward.
 *   kl_per_token_out : [N] fp32 KL_t (also for padding rows) or NULL.
 */
KD_API int kd_fused_kl_fwd(const void* H_bf16, const void* W_bf16,
                    const int32_t* t_ids, const float* t_logits, const uint8_t* mask,
                    int64_t N, int64_t d, int64_t V, int K, int64_t chunk, float tau,
                    float* loss_out, float* lse_out, float* kl_per_token_out,
                    void* ws, size_t ws_bytes, void* stream);

/*
 * Backward pass: recomputes each chunk's logits from H and W ([ART], the
 * backward recomputes every chunk instead of storing it) and forms
 *   dZ_t = grad_loss * mask_t / (N_valid * tau) * (softmax(z_t) - p_t scattered to its ids)
 *   grad_H = dZ W            (overwritten; bf16, or fp32 if grad_H_is_fp32)
 *   grad_W += dZ^T H         (fp32, ACCUMULATED into what the caller passes)
 * with fp32 tensor-core accumulation; dZ is rounded to bf16 before the two
 * gradient products.  Inputs as in kd_fused_kl_fwd, plus
 *   lse       : [N] fp32 from the forward pass with the same inputs.
 *   grad_loss : device fp32 scalar, the upstream gradient of the loss.
 *   grad_H    : [N, d] bf16 or fp32.   grad_W : [V, d] fp32.
 */
KD_API int kd_fused_kl_bwd(const void* H_bf16, const void* W_bf16,
                    const int32_t* t_ids, const float* t_logits, const uint8_t* mask,
                    int64_t N, int64_t d, int64_t V, int K, int64_t chunk, float tau,
                    const float* lse, const float* grad_loss,
                    void* grad_H, int grad_H_is_fp32, float* grad_W,
                    void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------ *
 * Forward-chunked KL: the same loss, keeping each chunk's student logits.
 * [ART] fused-loss paragraph, second formulation: the teacher stays sparse and
 * the loss is taken one chunk at a time, but the full student logits are kept
 * for the backward pass (so memory grows with sequence x vocabulary), which
 * saves the backward recompute; the page calls it the fastest of the three.
 * z_store holds the raw logits H W^T (bf16, before 1/tau) in a blocked layout:
 * element (t, v) at ((v / 64) * N + t) * 64 + v % 64, i.e.
 * kd_chunked_kl_logits_bytes(N, V) = ceil(V / 64) * N * 128 bytes, 16-byte
 * aligned, owned by the caller; the forward writes it, the backward only reads
 * it.  Everything else (arguments, workspace, outputs, errors) is as for
 * kd_fused_kl_fwd / kd_fused_kl_bwd; the backward uses the bf16-rounded
 * logits, so its gradients differ from the fused ones by that rounding.
 * ------------------------------------------------------------------------ */

KD_API size_t kd_chunked_kl_logits_bytes(int64_t N, int64_t V);

KD_API int kd_chunked_kl_fwd(const void* H_bf16, const void* W_bf16,
                    const int32_t* t_ids, const float* t_logits, const uint8_t* mask,
                    int64_t N, int64_t d, int64_t V, int K, int64_t chunk, float tau,
                    float* loss_out, float* lse_out, float* kl_per_token_out,
                    void* z_store, size_t z_bytes, void* ws, size_t ws_bytes, void* stream);

KD_API int kd_chunked_kl_bwd(const void* H_bf16, const void* W_bf16,
                    const int32_t* t_ids, const float* t_logits, const uint8_t* mask,
                    int64_t N, int64_t d, int64_t V, int K, int64_t chunk, float tau,
                    const float* lse, const float* grad_loss, const void* z_store, size_t z_bytes,
                    void* grad_H, int grad_H_is_fp32, float* grad_W,
                    void* ws, size_t ws_bytes, void* stream);

/*
 * Forward pass without a caller workspace, for callers that cannot allocate
 * device memory (no counterpart in the paper: it is an integration variant).
 * Some callers may not call cudaMalloc: plugins whose host framework owns all
 * device memory through its own pre-sized pool, and latency-critical paths that
 * cannot take the device-wide synchronisation cudaMalloc/cudaFree may cause;
 * they cannot provide the workspace kd_fused_kl_fwd needs either.  This call
 * computes exactly what kd_fused_kl_fwd computes (same arguments minus ws,
 * ws_bytes), using a scratch array of KD_STATIC_SCRATCH_BYTES compiled into
 * the library instead of a workspace:
 *   - every GPU that loads the library holds that array until the process exits;
 *   - the array's device address is looked up on the first call made with a
 *     given device current, so make that first call before any stream capture
 *     (it is looked up again after a device reset gives the device a new context);
 *   - it returns KD_ERR_WORKSPACE, before any launch, when the problem needs more
 *     than the array holds, i.e. when kd_fused_kl_workspace(N, d, V, K, chunk)
 *     exceeds KD_STATIC_SCRATCH_BYTES;
 *   - it allocates nothing; all calls share the one array, which keeps the last
 *     call's contents (its control block is cleared at the start of each call),
 *     so calls whose GPU work overlaps (other streams or host threads) race and
 *     must be serialised by the caller;
 *   - device-side conditions (a teacher id out of range) are recorded in the
 *     shared array's error word: kd_get_device_error(NULL, stream, &detail)
 *     reads and clears it.
 * Argument errors that kd_fused_kl_fwd detects are returned as there; the
 * scratch set-up and the clearing of its control block may already have been
 * enqueued when an alignment or shape check fails.
 */
#define KD_STATIC_SCRATCH_BYTES (32u * 1024u * 1024u)
KD_API int kd_fused_kl_fwd_static(const void* H_bf16, const void* W_bf16,
                    const int32_t* t_ids, const float* t_logits, const uint8_t* mask,
                    int64_t N, int64_t d, int64_t V, int K, int64_t chunk, float tau,
                    float* loss_out, float* lse_out, float* kl_per_token_out, void* stream);

/* Clears the control block (error word included) of a new workspace: one asynchronous
 * memset of its first 256 bytes.  A workspace of zeroed memory needs no call. */
KD_API int kd_workspace_clear(void* ws, size_t ws_bytes, void* stream);

/*
 * Reads (synchronising `stream`) and clears the device error word of a
 * workspace used by the calls above; ws == NULL names the scratch array of
 * kd_fused_kl_fwd_static on the current device.  Returns KD_OK, KD_ERR_TIMEOUT or
 * KD_ERR_DEVICE; *detail_out (may be NULL) receives a call-specific detail
 * (for a bad teacher id: the first offending row).  A library built with
 * KD_DEBUG (libkdkl_debug.so) also checks the indices its kernels compute and
 * reports one out of range as KD_ERR_DEVICE with the place of the check as the
 * detail (0x7xxx: top-K and the calls on dense logits), after skipping the access.
 */
KD_API int kd_get_device_error(void* ws, void* stream, int64_t* detail_out);

/* ------------------------------------------------------------------------ *
 * Scoring and distillation on dense logits.  No page has a counterpart: they are the
 * calls that a training loop or a server needs next to the cache and the fused loss
 * once a model hands out its logits.
 *
 * Conventions shared by these calls
 *   logits : [N, ld] of type `dtype`, row r at logits + r * ld elements, columns [0, V)
 *            read, V <= ld, V <= 2^30.  Any row stride and any alignment of the element
 *            type; rows that start on 16 bytes are read fastest.
 *   mask   : [N] uint8, 1 = valid, 0 = padding (its logits, tokens and cached entries
 *            are not looked at; its outputs are 0 and its gradients 0); NULL = all valid.
 *   tau    : temperature > 0; x = logits / tau.
 *   Logits of -inf take no part.  A row whose logits are all -inf has logsumexp -inf,
 *   log probabilities -inf, entropy 0 and zero gradients; a logsumexp beyond fp32's range is
 *   infinite as well, with log probabilities and gradients of the row as it is.  A NaN or +inf logit makes
 *   its row's results NaN.  Sums and statistics are fp32.
 * ------------------------------------------------------------------------ */

/* Workspace bytes of kd_token_logprobs_fwd / _bwd (control block only). */
KD_API size_t kd_token_logprobs_workspace(int64_t N, int64_t V);

/*
 * Log probabilities of M given tokens per position, with the entropy and the top
 * alternatives of the position's distribution:
 *   tokens      : [N, M] int32 in [0, V), 1 <= M <= KD_MAX_K (one outside is recorded
 *                 in the error word with its row; its output is NaN).
 *   logp_out    : [N, M] fp32, x[token] - logsumexp(x).    lse_out : [N] fp32, logsumexp(x).
 *   entropy_out : [N] fp32 or NULL, -sum_v p_v ln p_v.
 *   top         : alternatives per position, 0 <= top <= min(V, KD_MAX_TOP).
 *   top_ids_out : [N, top] int32 and top_logp_out: [N, top] fp32: the largest logits of
 *                 the row, largest first, equal ones by ascending id (-0 equals +0), as
 *                 log probabilities; both NULL when top == 0.  In a row with a NaN or
 *                 +inf logit the ids are 0, 1, ... and carry no meaning.
 */
KD_API int kd_token_logprobs_fwd(const void* logits, int dtype, int64_t N, int64_t V, int64_t ld,
                    const int32_t* tokens, int M, const uint8_t* mask, float tau, int top,
                    float* logp_out, float* lse_out, float* entropy_out, int32_t* top_ids_out, float* top_logp_out,
                    void* ws, size_t ws_bytes, void* stream);

/*
 * Gradient of the logits from the gradients of the log probabilities and entropies:
 *   dz_v = (1 / tau) (sum_m g_m [v = token_m] - p_v (sum_m g_m + h (ln p_v + H)))
 *   lse, entropy : [N] fp32 from the forward pass with the same inputs (entropy may be
 *                  NULL when grad_entropy is).
 *   grad_logp    : [N, M] fp32.   grad_entropy: [N] fp32 or NULL.  A token that occurs
 *                  more than once in a row receives the sum of its gradients.
 *   grad_logits  : [N, ld_grad] of type `dtype`, columns [0, V) written (rounded once from
 *                  fp32); may be `logits` itself with ld_grad == ld, otherwise the two
 *                  must not overlap.
 */
KD_API int kd_token_logprobs_bwd(const void* logits, int dtype, int64_t N, int64_t V, int64_t ld,
                    const int32_t* tokens, int M, const uint8_t* mask, float tau,
                    const float* lse, const float* entropy, const float* grad_logp, const float* grad_entropy,
                    void* grad_logits, int64_t ld_grad, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes of kd_logits_kl_fwd / _bwd / _step. */
KD_API size_t kd_logits_kl_workspace(int64_t N, int64_t V, int K);

/*
 * KL(teacher || student) of dense student logits against cached top-K teacher logits,
 * with q = softmax(x) over the V logits and S the row's cached ids:
 *   t_lse == NULL : p = softmax(t / tau) over S, as kd_fused_kl_fwd;
 *                   KL_t = sum_k p_k (ln p_k - ln q_k).
 *   t_lse given   : the teacher's mass outside its cache is kept as one more class:
 *                   p_k = exp(t_k / tau - t_lse), p_R = 1 - sum_k p_k, q_R = the student's
 *                   mass outside S;  KL_t gains p_R (ln p_R - ln q_R).  Where S is the whole
 *                   vocabulary there is no such class, and a p_R below 2^-21 (1 + |t_lse|),
 *                   which is the rounding of t_lse and the sum, is taken as 0.
 *                   t_lse: [N] fp32, logsumexp of the teacher's full row of logits / tau
 *                   (for tau = 1 the lse_out of kd_topk_cache and kd_teacher_topk); p_k is as
 *                   exact as fp32 holds it (|t_lse| 2^-24 of itself).
 *   loss          = sum over valid t of KL_t / N_valid   (0 when N_valid == 0).
 *   t_ids    : [N, K] int32, 1 <= K <= min(V, KD_MAX_K).  An id that repeats within a row
 *              adds up its entries' probabilities.  One outside [0, V) is recorded in the
 *              error word with its row and its entry left out.
 *   t_logits : [N, K] fp32, any order; an entry of -inf is absent (its id is not looked
 *              at).  Without t_lse, a row with no entry has KL 0 and zero gradient.
 *   loss_out : device fp32 scalar.     kl_per_token_out: [N] fp32 or NULL.
 *   stats_out: [N, 4] fp32, the row statistics that the backward pass takes: the largest
 *              logit and sum exp((logit - largest) / tau) over the row (to the rounding of
 *              largest / tau, which cancels where they are used together), then over the ids
 *              outside S (with t_lse; -inf and 0 without).
 * KD_ERR_UNSUPPORTED when the bitmap of S and the K entries of two rows do not fit into the
 * shared memory of an SM (V over about 0.7 million, 0.35 million for fp32).
 */
KD_API int kd_logits_kl_fwd(const void* logits, int dtype, int64_t N, int64_t V, int64_t ld,
                    const int32_t* t_ids, const float* t_logits, int K, const float* t_lse, const uint8_t* mask,
                    float tau, float* loss_out, float* stats_out, float* kl_per_token_out,
                    void* ws, size_t ws_bytes, void* stream);

/*
 * Its gradient, with c = grad_loss / (N_valid tau):
 *   dz_v = c (q_v - p_v) on S, c q_v outside; with t_lse, outside S
 *   c (q_v - p_R q_v / q_R).
 *   stats     : from the forward pass with the same inputs.   grad_loss: device fp32 scalar.
 *   grad_logits as for kd_token_logprobs_bwd (may be `logits` itself).
 */
KD_API int kd_logits_kl_bwd(const void* logits, int dtype, int64_t N, int64_t V, int64_t ld,
                    const int32_t* t_ids, const float* t_logits, int K, const float* t_lse, const uint8_t* mask,
                    float tau, const float* stats, const float* grad_loss, void* grad_logits, int64_t ld_grad,
                    void* ws, size_t ws_bytes, void* stream);

/* Loss and gradient in one call, for callers that know grad_loss beforehand: the logits
 * come from memory once.  Arguments as above. */
KD_API int kd_logits_kl_step(const void* logits, int dtype, int64_t N, int64_t V, int64_t ld,
                    const int32_t* t_ids, const float* t_logits, int K, const float* t_lse, const uint8_t* mask,
                    float tau, const float* grad_loss, float* loss_out, float* kl_per_token_out,
                    void* grad_logits, int64_t ld_grad, void* ws, size_t ws_bytes, void* stream);

/* The same calls with the error word in a control block of the caller's (256 bytes, 256-byte
 * aligned, cleared once by kd_workspace_clear) instead of the workspace's first bytes: for callers
 * whose workspaces do not outlive the call.  `ws` may then be memory of any content.  `control` may
 * be `ws` itself, and may serve any number of calls: it holds the first error since it was read. */
KD_API int kd_logits_kl_fwd_ctl(const void* logits, int dtype, int64_t N, int64_t V, int64_t ld,
                    const int32_t* t_ids, const float* t_logits, int K, const float* t_lse, const uint8_t* mask,
                    float tau, float* loss_out, float* stats_out, float* kl_per_token_out,
                    void* ws, size_t ws_bytes, void* control, void* stream);
KD_API int kd_logits_kl_bwd_ctl(const void* logits, int dtype, int64_t N, int64_t V, int64_t ld,
                    const int32_t* t_ids, const float* t_logits, int K, const float* t_lse, const uint8_t* mask,
                    float tau, const float* stats, const float* grad_loss, void* grad_logits, int64_t ld_grad,
                    void* ws, size_t ws_bytes, void* control, void* stream);
KD_API int kd_logits_kl_step_ctl(const void* logits, int dtype, int64_t N, int64_t V, int64_t ld,
                    const int32_t* t_ids, const float* t_logits, int K, const float* t_lse, const uint8_t* mask,
                    float tau, const float* grad_loss, float* loss_out, float* kl_per_token_out,
                    void* grad_logits, int64_t ld_grad, void* ws, size_t ws_bytes, void* control, void* stream);

/* ------------------------------------------------------------------------ *
 * The same scores straight from hidden states: log probability of one given token per
 * position and the entropy under softmax(H W^T / tau), formed `chunk` positions at a
 * time by the fused loss's projection, so that the [N, V] logits never exist (no page
 * has a counterpart: the hard-label term next to the KL, and scoring without logits).
 *   H_bf16, W_bf16, mask, chunk, tau : as for kd_fused_kl_fwd.
 *   tokens : [N] int32 in [0, V) (one outside is recorded in the error word with its
 *            row; its log probability is NaN, its one-hot gradient is left out).
 *   logp_out, lse_out : [N] fp32.   entropy_out: [N] fp32 or NULL.  Padding rows give 0;
 *            their tokens are not looked at (their hidden states are multiplied by zeros in
 *            the backward pass, and so have to be finite).
 * The backward pass recomputes each chunk's logits and takes, per valid position,
 *   dZ_v = (1 / tau) (g [v = token] - p_v (g + h (ln p_v + H)))
 * with g = grad_logp, h = grad_entropy ([N] fp32; grad_entropy and entropy may be NULL
 * together); grad_H and the rounding of dZ to bf16 as for kd_fused_kl_bwd; grad_W as
 * grad_W_kind (kd_grad_kind) says.  p is taken from lse, so it is as exact as fp32 holds lse
 * (|lse| 2^-24 of itself); for tau < 1/64 the rows' statistics are taken again instead (the
 * projection runs once more).
 * Workspace: `backward` != 0 asks for what the backward pass needs (both calls may use
 * it; it grows with chunk * V), 0 for the forward pass alone (chunk * V / 16 bytes).
 * ------------------------------------------------------------------------ */

KD_API size_t kd_fused_logprobs_workspace(int64_t N, int64_t d, int64_t V, int64_t chunk, int backward);

KD_API int kd_fused_logprobs_fwd(const void* H_bf16, const void* W_bf16, const int32_t* tokens, const uint8_t* mask,
                    int64_t N, int64_t d, int64_t V, int64_t chunk, float tau,
                    float* logp_out, float* lse_out, float* entropy_out, void* ws, size_t ws_bytes, void* stream);

KD_API int kd_fused_logprobs_bwd(const void* H_bf16, const void* W_bf16, const int32_t* tokens, const uint8_t* mask,
                    int64_t N, int64_t d, int64_t V, int64_t chunk, float tau,
                    const float* lse, const float* entropy, const float* grad_logp, const float* grad_entropy,
                    void* grad_H, int grad_H_is_fp32, void* grad_W, int grad_W_kind,
                    void* ws, size_t ws_bytes, void* stream);

/* With the error word in a control block of the caller's, as kd_logits_kl_fwd_ctl. */
KD_API int kd_fused_logprobs_fwd_ctl(const void* H_bf16, const void* W_bf16, const int32_t* tokens,
                    const uint8_t* mask, int64_t N, int64_t d, int64_t V, int64_t chunk, float tau,
                    float* logp_out, float* lse_out, float* entropy_out, void* ws, size_t ws_bytes,
                    void* control, void* stream);
KD_API int kd_fused_logprobs_bwd_ctl(const void* H_bf16, const void* W_bf16, const int32_t* tokens,
                    const uint8_t* mask, int64_t N, int64_t d, int64_t V, int64_t chunk, float tau,
                    const float* lse, const float* entropy, const float* grad_logp, const float* grad_entropy,
                    void* grad_H, int grad_H_is_fp32, void* grad_W, int grad_W_kind,
                    void* ws, size_t ws_bytes, void* control, void* stream);

/* ------------------------------------------------------------------------ *
 * Softmax cross entropy against hard labels from hidden states and the LM head: the hard-label term of
 * a distillation loss, the [N, V] logits never formed (no page has a counterpart).  With z' = h W^T, or
 * c tanh(h W^T / c) for a softcap c, and lse = logsumexp(z'),
 *   loss_n = lse - (1 - e) z'_y - (e / V) sum_v z'_v + l lse^2     e label_smoothing, l z_loss
 *   loss   = sum over valid n of loss_n / n_valid                  (0 when none is)
 *   H_bf16, W_bf16, chunk : as for kd_fused_kl_fwd; N, d and V at most 2^31 - 1024, as in every call on
 *            hidden states and a head.
 *   labels : [N] int32.  A position is valid if its label is not ignore_index and mask ([N] uint8, NULL:
 *            all) is not 0; only those are projected, the hidden states of the others are not read.
 *            A valid position's label outside [0, V) is recorded in the error word with its position;
 *            its loss is NaN, its gradient left out.
 *   0 <= label_smoothing < 1; z_loss >= 0; softcap >= 1e-6, or 0 for none.
 *   loss_out: device fp32 scalar.  lse_out, loss_per_token_out: [N] fp32 (the latter may be NULL), 0 for
 *            positions that are not valid.
 * kd_fused_cross_entropy_step returns the gradients with the loss, for a grad_loss (device fp32 scalar,
 * NULL: 1) known beforehand: one projection and two products in place of the two and two that a
 * separate backward pass needs.
 *   grad_H : [N, d] bf16 or fp32, zero rows where not valid.  grad_W, grad_W_kind as for
 *            kd_fused_logprobs_bwd.  dZ is rounded to bf16, from logits kept in 16 bits: a probability
 *            is off by 2.4e-4 of itself at most (with a softcap c below 16: 3.1e-5 c), a cap's slope by 6e-5 (3e-5
 *            from c = 16 on), and by 0.04 % of a slope of 0.01 up to c = 16; probabilities below e^-32 (with a
 *            softcap above 16: e^-28) of the largest of their 128 columns are known to be that small only.
 * kd_fused_cross_entropy_keep and _bwd are the step in two calls, for a grad_loss that is known only after the
 * loss (autograd's), all positions in one chunk: the first is the forward pass and leaves in `kept`
 * (kd_fused_cross_entropy_kept bytes, of any content before) what the second, given the same W, sizes and
 * options, makes the gradients of, once: it writes dZ where the logits lay.  A `kept` that holds nothing for these
 * sizes and options (never filled, spent) is recorded in the error word; the gradients are then zero.
 * Workspace, in bytes, for chunk positions or N where that is less, to whole tiles: 0 for `step` asks for the forward
 * pass's, chunk * (V / 8 + 2 d + 20) + 8 N; anything else for the step's, chunk * (2 V + 32 d) more, for the 16-bit
 * logits and for up to eight fp32 parts of grad_H.  `ws` may be memory of any content; the error word is in `control`
 * (see kd_logits_kl_fwd_ctl), which may be `ws` itself once kd_workspace_clear has cleared it.
 * ------------------------------------------------------------------------ */

KD_API size_t kd_fused_cross_entropy_workspace(int64_t N, int64_t d, int64_t V, int64_t chunk, int step);

KD_API int kd_fused_cross_entropy_fwd(const void* H_bf16, const void* W_bf16, const int32_t* labels,
                    const uint8_t* mask, int64_t N, int64_t d, int64_t V, int64_t chunk, float label_smoothing,
                    float z_loss, float softcap, int ignore_index, float* loss_out, float* lse_out,
                    float* loss_per_token_out, void* ws, size_t ws_bytes, void* control, void* stream);

KD_API int kd_fused_cross_entropy_step(const void* H_bf16, const void* W_bf16, const int32_t* labels,
                    const uint8_t* mask, int64_t N, int64_t d, int64_t V, int64_t chunk, float label_smoothing,
                    float z_loss, float softcap, int ignore_index, const float* grad_loss, float* loss_out,
                    float* lse_out, float* loss_per_token_out, void* grad_H, int grad_H_is_fp32, void* grad_W,
                    int grad_W_kind, void* ws, size_t ws_bytes, void* control, void* stream);

KD_API size_t kd_fused_cross_entropy_kept(int64_t N, int64_t d, int64_t V);

KD_API int kd_fused_cross_entropy_keep(const void* H_bf16, const void* W_bf16, const int32_t* labels,
                    const uint8_t* mask, int64_t N, int64_t d, int64_t V, float label_smoothing, float z_loss,
                    float softcap, int ignore_index, float* loss_out, float* lse_out, float* loss_per_token_out,
                    void* kept, size_t kept_bytes, void* control, void* stream);

KD_API size_t kd_fused_cross_entropy_bwd_workspace(int64_t N, int64_t d, int64_t V);

KD_API int kd_fused_cross_entropy_bwd(const void* W_bf16, int64_t N, int64_t d, int64_t V, float label_smoothing,
                    float softcap, const float* grad_loss, void* grad_H, int grad_H_is_fp32, void* grad_W,
                    int grad_W_kind, void* kept, size_t kept_bytes, void* ws, size_t ws_bytes, void* control,
                    void* stream);

/* x[0 .. n) *= *factor (device fp32 scalar), bf16 or fp32, n a multiple of 8; nothing is read or
 * written where the factor is 1.  What a backward pass does to a step's fp32 gradients before they are
 * rounded (bf16 ones are rounded a second time by it). */
KD_API int kd_scale_gradient(void* x, int64_t n, int is_fp32, const float* factor, void* stream);

/* ------------------------------------------------------------------------ *
 * 8-bit integers with one scale a row: a quantised teacher head (no page has a counterpart).
 *
 * kd_quantize_int8: rows of x [N, d] (bf16, fp16 or fp32, kd_dtype, any row stride ld >= d) to integers,
 *   scale_n = max |x_n| / 127 (fp32),   q_nk = the whole number nearest to x_nk / scale_n, ties to even,
 * the quotient taken exactly.  A row of zeros has scale 0; one that holds a NaN or an infinity has
 * scale NaN and integers 0.  q_out: [N, d] with row stride ld_q >= d; d at most 2^31 - 1024.
 *
 * kd_gemm_int8: C_mn = (sum_k A_mk B_nk) a_scale_m b_scale_n, A [M, K] the tokens and B [N, K] the channels,
 * 1 <= K <= KD_MAX_INT8_K, M and N at most 2^31 - 1024, any row strides lda, ldb >= K, ldc >= N; C bf16, fp16 or
 * fp32 (kd_dtype).  The
 * integer sum is exact while it stays below 2^24 (always for K <= 1024); from there on the tensor cores add in
 * fp32 and cut off, up to a step of the sum for each 16 products.  Each of the two products with a scale rounds
 * once to fp32, and the result once to C's type.  Weights whose rows start on
 * 16-byte boundaries (B and ldb multiples of 16) are read in place, others are copied to such rows
 * in the workspace by every call (kd_teacher_topk_int8: once for all its chunks).  Workspace:
 * `b_rows_aligned` as B's rows are; memory of any content, the error word in `control` (see
 * kd_logits_kl_fwd_ctl).
 *
 * kd_teacher_topk_int8: kd_teacher_topk from quantised hidden states Ht [N, dt] and head Wt [V, dt]; any
 * chunk >= 1.
 * ------------------------------------------------------------------------ */

#define KD_MAX_INT8_K 65536

KD_API int kd_quantize_int8(const void* x, int dtype, int64_t N, int64_t d, int64_t ld, int8_t* q_out, int64_t ld_q,
                    float* scale_out, void* stream);

KD_API size_t kd_gemm_int8_workspace(int64_t M, int64_t N, int64_t K, int b_rows_aligned);

KD_API int kd_gemm_int8(const int8_t* A, int64_t lda, const float* a_scale, const int8_t* B, int64_t ldb,
                    const float* b_scale, void* C, int dtype, int64_t ldc, int64_t M, int64_t N, int64_t K,
                    void* ws, size_t ws_bytes, void* control, void* stream);

KD_API size_t kd_teacher_topk_int8_workspace(int64_t N, int64_t dt, int64_t V, int K, int64_t chunk,
                    int w_rows_aligned);

KD_API int kd_teacher_topk_int8(const int8_t* Ht, int64_t ld_h, const float* h_scale, const int8_t* Wt, int64_t ld_w,
                    const float* w_scale, int64_t N, int64_t dt, int64_t V, int K, int64_t chunk,
                    int32_t* ids_out, float* vals_out, float* lse_out, float* dropped_out,
                    void* ws, size_t ws_bytes, void* control, void* stream);

/* ------------------------------------------------------------------------ *
 * On-disk teacher cache ([ART] paragraph on the first fix: run the teacher once,
 * keep its top-K logits per position on disk, reuse them across experiments).
 * HOST memory and host files only; no CUDA call.  One file per contiguous range
 * of positions (a shard): a 64-byte header (magic, version, K, V, N, row0,
 * logits type, flags, FNV-1a 64 checksum of the payload), then ids int32 [N, K],
 * logits fp32 or bf16 [N, K] and optionally the teacher's full-row logsumexp
 * fp32 [N].  bf16 logits round to nearest even (exact for caches extracted from
 * bf16 teacher logits) and are widened back to fp32 on reading.
 * ------------------------------------------------------------------------ */

/* Write a shard atomically (temporary file + rename).  lse may be NULL. */
KD_API int kd_cache_write(const char* path, const int32_t* ids, const float* logits, const float* lse,
                          int64_t N, int K, int64_t V, int64_t row0, int logits_bf16);
/* Header fields of a shard (any out pointer may be NULL); checks the file size. */
KD_API int kd_cache_info(const char* path, int64_t* N, int* K, int64_t* V, int64_t* row0,
                         int* logits_bf16, int* has_lse);
/* Recompute the payload checksum: KD_OK, or KD_ERR_IO if the file is corrupt or truncated. */
KD_API int kd_cache_verify(const char* path);
/* Read positions [first, first + count) into host buffers ids_out [count, K] and
 * logits_out [count, K] (fp32); lse_out [count] or NULL. */
KD_API int kd_cache_read(const char* path, int64_t first, int64_t count, int32_t* ids_out,
                         float* logits_out, float* lse_out);
/* Streaming reader: batches of up to rows_per_batch consecutive positions; the next
 * batch is read on a background thread while the caller uses the current one.
 * kd_cache_reader_next copies one batch into host buffers (rows_out = 0 at the end). */
KD_API int kd_cache_reader_open(const char* path, int64_t rows_per_batch, void** handle);
KD_API int kd_cache_reader_next(void* handle, int32_t* ids_out, float* logits_out, int64_t* rows_out);
KD_API int kd_cache_reader_close(void* handle);

/* ------------------------------------------------------------------------ *
 * Building blocks, exposed for testing and profiling.  No page describes these
 * separately; they are the pieces the calls above are made of.
 * ------------------------------------------------------------------------ */

/*
 * C[M, N] (op)= A · B^T-or-B with bf16 inputs and fp32 tensor-core accumulation,
 * the projection engine shared by the loss kernels.
 *   a_mn_major = 0: A is [M, K] row-major (K contiguous); 1: A is [K, M] (M contiguous).
 *   b_mn_major = 0: B is [N, K] row-major;                 1: B is [K, N].
 *   C is [M, N] fp32 row-major; accumulate != 0 adds into C.
 * All leading dimensions are the contiguous extents above; K % 8 == 0 for
 * K-major operands and M % 8 / N % 8 == 0 for MN-major ones.
 */
KD_API int kd_gemm_bf16(const void* A, const void* B, float* C, int64_t M, int64_t N, int64_t K,
                 int a_mn_major, int b_mn_major, int accumulate,
                 void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes for kd_gemm_bf16. */
KD_API size_t kd_gemm_workspace(void);

/*
 * Self-check of the bounded waits every kernel uses: launches one block that
 * waits on a shared-memory barrier nothing arrives at, with a limit of
 * `limit_ns` (1 us .. 1 s) instead of the kernels' 2 s.  The wait gives up, the
 * kernel records a timeout in the error word of `ws` and exits normally, so
 * kd_get_device_error(ws) then returns KD_ERR_TIMEOUT and the CUDA context
 * stays usable.
 */
KD_API int kd_check_wait_timeout(void* ws, size_t ws_bytes, int64_t limit_ns, void* stream);

/*
 * Per-launch timing of this library's kernels, for profiling.  While enabled,
 * each launch on `stream` is bracketed by two CUDA events (at most `capacity`
 * launches are recorded).  kd_profile_read synchronises, then fills up to `n`
 * entries of names[] (static strings), ms[] and returns how many launches were
 * recorded since kd_profile_begin.  Host-side state; not thread-safe.
 */
KD_API int kd_profile_begin(int capacity);
KD_API int kd_profile_end(void);
KD_API int kd_profile_read(const char** names, float* ms, int n);

#ifdef __cplusplus
}
#endif
#endif /* KDKL_H_ */
