/*
 * specprefill.h -- C ABI of libspecprefill.so: SpecPrefill token-importance
 * scoring and chunk selection on one NVIDIA GB300 (sm_103a).
 *
 * The method (paper review "Speculative Prefill: Turbocharging TTFT with
 * Lightweight and Training-Free Token Importance Estimation", sections "core
 * algorithm" and "core formulas"; llama.cpp guide "SpecPrefill --
 * Implementation Guide", sections "How It Works", "v3 Improvements" and
 * "v3.1 Optimizations"): a small speculator model has a post-RoPE key cache for
 * an M-token prompt and the queries of N look-ahead decode steps.  Every
 * prompt token i gets the importance
 *
 *     importance_i = (1/N) sum_j max_{l,h} softmax(Q_{M+j,l,h} K_{l,g(h)}^T / sqrt(d))_i
 *
 * where the softmax of look-ahead step j runs over the M prompt keys and the
 * look-ahead keys 0..j.  The prompt is then cut into contiguous chunks, chunk
 * scores are averaged (and pooled), chunks are selected, and the original
 * position IDs of the kept tokens are returned in ascending order.  Decoding
 * continues at positions M, M+1, ... (paper review, "position ID recovery").
 *
 * Conventions of every entry point:
 *  - All tensor pointers are DEVICE pointers owned by the caller, except
 *    arguments whose name ends in "_host".  Layouts are row-major, last index
 *    contiguous.  Data pointers must be 16-byte aligned.
 *  - The library never allocates, frees or synchronises (except
 *    sp_workspace_status).  Work is enqueued on `stream` (a cudaStream_t;
 *    NULL = the legacy default stream) and runs asynchronously; outputs are
 *    valid once the stream reaches that point.
 *  - `ws` is a caller-owned device workspace of at least the size the matching
 *    *_workspace_size function returns; its contents need not be initialised
 *    and are overwritten.  One workspace must not be used by two calls that
 *    may run at the same time.
 *  - Errors: arguments are validated before anything is enqueued; on failure
 *    the call returns a non-zero sp_status, enqueues nothing and
 *    sp_last_error() describes the problem.  CUDA launch failures return
 *    SP_ECUDA.  A kernel that detects a problem at run time (a bounded wait
 *    that gave up) records it in the workspace; sp_workspace_status() reads it.
 *    Nothing aborts the process.
 */
#ifndef SPECPREFILL_H
#define SPECPREFILL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SP_OK = 0,
    SP_EINVAL = 1,        /* bad argument (shape, pointer, parameter range)          */
    SP_ENOMEM = 2,        /* workspace smaller than *_workspace_size() asks for      */
    SP_ECUDA = 3,         /* a CUDA runtime call or kernel launch failed             */
    SP_EDEVICE = 4,       /* a kernel recorded an internal error in the workspace    */
    SP_ETIMEOUT = 5,      /* a bounded device-side wait gave up                      */
    SP_EUNSUPPORTED = 6   /* valid, but outside what this build implements          */
} sp_status;

typedef enum { SP_BF16 = 0, SP_F32 = 1 } sp_dtype;

typedef enum {
    SP_SELECT_TOPK = 0,   /* chunk mean -> 1D average pool -> exactly kc chunks      */
    SP_SELECT_MASS = 1    /* v3: chunks by mean until the cumulative mass >= tau    */
} sp_mode;

/* v3 structural boost (llama.cpp guide, "v3 Improvements: Structural Token
 * Boosting" and "v3.1: Score Normalization").  Token scores are first min-max
 * normalised to [0,1] over the prompt if `normalize` != 0 (all 1.0 when every
 * score is equal), then multiplied by first_mult at positions [0, first_n) and
 * by last_mult at positions [M - last_n, M) (both when the ranges overlap).
 * The guide's defaults are {64, 1.5, 128, 1.3, 1}. */
typedef struct {
    int32_t first_n;
    double  first_mult;
    int32_t last_n;
    double  last_mult;
    int32_t normalize;
} sp_boost;

/* The guide's v2 keep rules applied after the chunk selection (llama.cpp
 * guide, "Full Source Code": select_chunks and its main program's sparse-
 * prefill cap).  min_tok > 0 sets eff_min = min(min_tok, max(4, M / 10)): a
 * prompt of at most eff_min tokens keeps every token, otherwise tokens of the
 * chunks the selection left out are added, chunk by chunk and token by token
 * in order, until eff_min are kept.  always_keep != 0 adds tokens 0, 1, 2, 3
 * and, if M > 4, M-2 and M-1.  max_keep > 0 caps the result: with n > max_keep
 * kept, every (n / max_keep)-th token is kept, at most max_keep, the last one
 * replaced by the last kept token.  The guide runs with {128, 1, 2000}. */
typedef struct {
    int32_t min_tok;        /* 0 = off; at most 4096 */
    int32_t always_keep;
    int64_t max_keep;       /* 0 = no cap */
} sp_keep_rules;

/* ------------------------------------------------------------------------ */
/* Scoring                                                                  */
/* ------------------------------------------------------------------------ */

/* Workspace bytes sp_score needs for this shape (0 if the shape is invalid). */
size_t sp_score_workspace_size(int L, int H, int H_kv, int d, int64_t M, int N, sp_dtype dtype);

/* Token importance of one prompt.
 *
 * Defines: a[l,h,j,i] = softmax over {prompt keys 0..M-1, look-ahead keys
 * 0..j} of Q_la[j,l,h,:] . key / sqrt(d), evaluated at prompt key i;
 * importance[i] = (1/N) sum_j max_{l,h} a[l,h,j,i]   (paper review, "core
 * formulas": attention score and importance aggregation; llama.cpp guide,
 * "Token Importance": max over heads, max over layers, mean over look-ahead
 * steps).  Query head h reads KV head h / (H / H_kv).
 *
 *   Q_la      [N, L, H, d]      look-ahead queries (post-RoPE), dtype
 *   K_prompt  [L, H_kv, M, d]   prompt keys (post-RoPE), dtype
 *   K_la      [L, H_kv, N, d]   look-ahead keys (post-RoPE), dtype
 *   importance[M]               fp32 output
 *   dtype     SP_BF16 or SP_F32 (all three inputs)
 *
 * Requirements: L, H, H_kv >= 1, H % H_kv == 0, 1 <= d <= 256, d % 8 == 0,
 * M >= 0, 0 <= N, N * (H / H_kv) <= 256.  N == 0 writes importance 1.0 to
 * every token (the guide's fallback when no look-ahead step was captured).
 * M == 0 is a no-op.  Accuracy: importance within 1e-3 absolute and 1e-2
 * relative of an fp64 evaluation on the same bf16 inputs; 1e-5 for fp32. */
sp_status sp_score(const void* Q_la, const void* K_prompt, const void* K_la,
                   int L, int H, int H_kv, int d, int64_t M, int N, sp_dtype dtype,
                   float* importance, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes sp_score_prefill needs (N = decode steps; 0 if the shape is invalid). */
size_t sp_score_prefill_workspace_size(int L, int H, int H_kv, int d, int64_t M, int N, sp_dtype dtype);

/* sp_score for the capture the llama.cpp guide makes ("How It Works": the
 * prefill's last row, then the look-ahead decode steps): N + 1 query rows,
 * where row 0 is the prompt's last query at prefill -- its softmax covers only
 * the M prompt keys -- and row j >= 1 is decode step j - 1, whose softmax also
 * covers look-ahead keys 0..j-1.  importance[i] = (1/(N+1)) sum_j max_{l,h} a[l,h,j,i].
 *
 *   Q_rows    [N + 1, L, H, d]  row 0: the prompt's last query; rows 1..N: decode queries
 *   K_prompt  [L, H_kv, M, d]
 *   K_la      [L, H_kv, N, d]   the decode steps' keys (may be NULL when N == 0)
 *
 * Requirements as sp_score with N + 1 rows ((N + 1) * (H / H_kv) <= 256). */
sp_status sp_score_prefill(const void* Q_rows, const void* K_prompt, const void* K_la,
                           int L, int H, int H_kv, int d, int64_t M, int N, sp_dtype dtype,
                           float* importance, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes sp_score_lse needs for this shape (0 if the shape is invalid). */
size_t sp_score_lse_workspace_size(int L, int H, int H_kv, int d, int64_t M, int N, sp_dtype dtype);

/* Token importance of one prompt when each row's softmax normaliser is
 * already known (single pass: K is read once, no statistics pass).
 *
 * Defines: importance[i] = (1/N) sum_j max_{l,h} exp(Q_la[j,l,h,:] . K[l,g,i,:] / sqrt(d)
 * - lse[l,h,j]), g = h / (H / H_kv) -- the aggregation of sp_score (paper
 * review, "core formulas"; llama.cpp guide, "Token Importance"), with lse
 * supplied by the caller.  With lse[l,h,j] the log of the sum of exp over
 * the M prompt logits and the look-ahead logits 0..j -- the normaliser the
 * speculator's own look-ahead decode attention computes -- the result equals
 * sp_score's.  The pages have no separate call for this; it is the
 * "lse-in" variant of the same definition.
 *
 *   Q_la      [N, L, H, d]      look-ahead queries (post-RoPE), dtype
 *   K_prompt  [L, H_kv, M, d]   prompt keys (post-RoPE), dtype
 *   lse       [L, H, N]         fp32 natural-log normalisers (device memory, 4-byte aligned)
 *   importance[M]               fp32 output
 *
 * Requirements and errors as sp_score; N == 0 writes 1.0 and reads no lse.
 * Accuracy: within 1e-3 absolute and 1e-2 relative of an fp64 evaluation on
 * the same inputs (bf16), 1e-5 (fp32). */
sp_status sp_score_lse(const void* Q_la, const void* K_prompt, const float* lse,
                       int L, int H, int H_kv, int d, int64_t M, int N, sp_dtype dtype,
                       float* importance, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes for sp_score_varlen (cu_M_host: B+1 host prefix sums).  The
 * batch is planned for the current device's SM count: query the size with the
 * device that will run the call current (a smaller workspace is rejected with
 * SP_EINVAL, never overrun). */
size_t sp_score_varlen_workspace_size(int B, const int64_t* cu_M_host, int L, int H, int H_kv,
                                      int d, int N, sp_dtype dtype);

/* Token importance of B independent prompts in one call.  Prompt b has
 * M_b = cu_M_host[b+1] - cu_M_host[b] tokens (cu_M_host[0] == 0, non-
 * decreasing; empty prompts allowed).  Keys are packed along the token axis:
 *
 *   Q_la      [B, N, L, H, d]
 *   K_prompt  [L, H_kv, T, d]   T = cu_M_host[B]; prompt b occupies rows cu_M[b]..cu_M[b+1]-1
 *   K_la      [B, L, H_kv, N, d]
 *   importance[T]               fp32; entries of prompt b at offsets cu_M[b]..
 *
 * Same definition and requirements as sp_score, per prompt. */
sp_status sp_score_varlen(const void* Q_la, const void* K_prompt, const void* K_la,
                          int B, const int64_t* cu_M_host,
                          int L, int H, int H_kv, int d, int N, sp_dtype dtype,
                          float* importance, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes for sp_score_lse_varlen (planned for the current device, as
 * sp_score_varlen_workspace_size; 0 if the shape or cu_M_host is invalid). */
size_t sp_score_lse_varlen_workspace_size(int B, const int64_t* cu_M_host, int L, int H, int H_kv,
                                          int d, int N, sp_dtype dtype);

/* sp_score_lse for B independent prompts in one call: the packing of
 * sp_score_varlen, with each prompt's row normalisers given instead of its
 * look-ahead keys (single pass per prompt, K read once).
 *
 *   Q_la      [B, N, L, H, d]
 *   K_prompt  [L, H_kv, T, d]   T = cu_M_host[B]; prompt b occupies rows cu_M[b]..cu_M[b+1]-1
 *   lse       [B, L, H, N]      fp32 natural-log normalisers of prompt b's rows (device, 4-byte aligned)
 *   importance[T]               fp32; entries of prompt b at offsets cu_M[b]..
 *
 * Same definition as sp_score_lse per prompt; requirements and errors as
 * sp_score_varlen.  lse holds all B prompts' rows; those of empty prompts are
 * not used. */
sp_status sp_score_lse_varlen(const void* Q_la, const void* K_prompt, const float* lse,
                              int B, const int64_t* cu_M_host,
                              int L, int H, int H_kv, int d, int N, sp_dtype dtype,
                              float* importance, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* Selection                                                                */
/* ------------------------------------------------------------------------ */

/* Workspace bytes sp_select needs for a prompt of M tokens and this chunk size. */
size_t sp_select_workspace_size(int64_t M, int chunk);

/* Kept original position IDs of one prompt.
 *
 * Token scores x_i are the fp32 importance values as fp64, optionally
 * normalised and boosted (`boost`, NULL = neither).  Chunks are the contiguous
 * ranges [c*chunk, min((c+1)*chunk, M)), nc = ceil(M/chunk); a chunk's mean is
 * its fp64 sum (added left to right) divided by its real size (paper review,
 * chunk formula; llama.cpp guide, select_chunks).
 *
 * SP_SELECT_TOPK (rate = keep_rate, 0 < rate <= 1): chunk means are smoothed
 * by a stride-1, centred average pool of pool_k chunks (odd; an edge window
 * averages only its in-range chunks), and exactly kc = max(1,
 * ceil(f32(nc) * f32(rate))) chunks with the largest pooled score are kept,
 * ties to the lower chunk index (paper review, "chunk selection and pooling
 * denoising"; the guide's kc formula).
 *
 * SP_SELECT_MASS (rate = tau, 0 < tau <= 1; pool_k must be 1): chunks are
 * ranked by mean (descending, ties to the lower index) and the shortest ranked
 * prefix whose running sum of chunk sums (added in ranked order) reaches
 * tau * total (chunk sums added in chunk order) is kept; all chunks if it never
 * does (llama.cpp guide, "v3 Improvements: Cumulative Attention Mass
 * Selection").  Supports nc <= 16384.
 *
 *   importance [M] fp32 (finite values)
 *   kept_pos   [M] int32 output capacity; the first *n_kept entries receive the
 *              kept tokens' original positions, ascending
 *   n_kept     device int64 output
 *
 * Every fp64 operation follows the fixed order above, so the result is
 * reproducible bit for bit by any IEEE-754 implementation of the same steps. */
sp_status sp_select(const float* importance, int64_t M, int chunk, int pool_k, sp_mode mode,
                    double rate, const sp_boost* boost, int32_t* kept_pos, int64_t* n_kept,
                    void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes for sp_select_rules. */
size_t sp_select_rules_workspace_size(int64_t M, int chunk);

/* sp_select followed by the keep rules (sp_keep_rules) on the same prompt.
 * kept_pos receives the final ascending positions (capacity M) and n_kept
 * their count.  rules == NULL behaves as sp_select.  Errors: SP_EINVAL for a
 * negative min_tok or max_keep, SP_EUNSUPPORTED for min_tok > 4096. */
sp_status sp_select_rules(const float* importance, int64_t M, int chunk, int pool_k, sp_mode mode,
                          double rate, const sp_boost* boost, const sp_keep_rules* rules,
                          int32_t* kept_pos, int64_t* n_kept, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes for sp_select_varlen. */
size_t sp_select_varlen_workspace_size(int B, const int64_t* cu_M_host, int chunk);

/* Per-prompt selection of B packed prompts (importance packed as in
 * sp_score_varlen).  Prompt b's kept positions (relative to its own start,
 * i.e. its original position IDs) go to kept_pos[cu_M[b] ...] and its count
 * to n_kept[b] (device int64[B]).  Same rules as sp_select per prompt. */
sp_status sp_select_varlen(const float* importance, int B, const int64_t* cu_M_host, int chunk,
                           int pool_k, sp_mode mode, double rate, const sp_boost* boost,
                           int32_t* kept_pos, int64_t* n_kept, void* ws, size_t ws_bytes,
                           void* stream);

/* sp_select for callers that cannot allocate device memory.  The method's
 * pages have no counterpart to this entry point; it exists for deployment.
 *
 * Who needs it: code that runs inside a device-memory allocator or its
 * out-of-memory handler (allocating there would re-enter the allocator),
 * serving loops whose latency budget forbids cudaMalloc (it can synchronise
 * the whole device), and plug-ins that a host framework hands only input and
 * output buffers.  The caller passes inputs and outputs exactly as for
 * sp_select; the scratch lives in a fixed 3 MiB array of device memory inside
 * the library.  The array comes into being on a device when the library's
 * code is loaded there: with CUDA's lazy module loading (the default) that is
 * the first call of this entry point on the device, which looks up the
 * array's address with that device current and may itself allocate device
 * memory (the array and the selection kernels' code).  So make one call on
 * every device ahead of time -- before the allocator or out-of-memory path
 * that needs it, and before any stream capture.  Later calls allocate and
 * free nothing; the array stays until the process exits.
 *
 * Limits: one prompt, at most 65536 chunks (ceil(M / chunk)); larger requests
 * return SP_EUNSUPPORTED before any work is enqueued.  All calls on a device
 * share the array and leave their contents behind: calls whose work may
 * overlap on the GPU (e.g. on two unordered streams) race and must not be
 * issued.  Results are identical to sp_select's. */
sp_status sp_select_noalloc(const float* importance, int64_t M, int chunk, int pool_k, sp_mode mode,
                            double rate, const sp_boost* boost, int32_t* kept_pos, int64_t* n_kept,
                            void* stream);

/* ------------------------------------------------------------------------ */
/* Sparse-prefill input                                                     */
/* ------------------------------------------------------------------------ */

/* The target's sparse-prefill batch: for B packed prompts, each prompt's kept
 * token IDs and original position IDs, packed prompt after prompt (paper
 * review, "core algorithm: position ID recovery": the kept tokens keep their
 * positions and decoding continues at M_b, M_b + 1, ...).
 *
 *   token_ids     [T] int32, packed by cu_M_host (needed only if out_tokens is given)
 *   kept_pos      [T] int32, prompt b's ascending kept positions (relative to its
 *                 start) at kept_pos[cu_M[b] ...], as sp_select_varlen writes them
 *   n_kept        device int64[B], as sp_select_varlen writes it
 *   out_tokens    [T] int32 capacity or NULL: out_tokens[cu_kept[b] + i] = token_ids[cu_M[b] + kept_pos[cu_M[b] + i]]
 *   out_positions [T] int32 capacity or NULL: out_positions[cu_kept[b] + i] = kept_pos[cu_M[b] + i]
 *   cu_kept       device int64[B + 1]: prefix sums of n_kept
 *
 * Requirements: 1 <= B <= 256, cu_M_host as for sp_select_varlen; at least one
 * of out_tokens / out_positions.  No workspace. */
sp_status sp_gather_kept(const int32_t* token_ids, int B, const int64_t* cu_M_host, const int32_t* kept_pos,
                         const int64_t* n_kept, int32_t* out_tokens, int32_t* out_positions, int64_t* cu_kept,
                         void* stream);

/* ------------------------------------------------------------------------ */
/* Positions, the paged cache, and attention over it                        */
/* ------------------------------------------------------------------------ */

/* Rows of a tensor [rows, heads, d]: entry i of (row, head) is at
 * data[row * stride_row + head * stride_head + i] (strides in entries).  data
 * is 16-byte aligned and both strides are multiples of 16 bytes, so a slice
 * of a fused projection is taken as it lies. */
typedef struct {
    void*   data;
    int64_t stride_row, stride_head;
} sp_rows;

/* Rotary frequencies.  Filled by sp_rotary_plan_init and then read only;
 * `turns` holds each pair's turns per position as a 64-bit fraction. */
typedef struct {
    int32_t  rot;             /* entries of a head that are rotated (the first ones) */
    int32_t  interleaved;
    int32_t  axes;
    uint64_t turns[128];
    uint8_t  axis[128];
} sp_rotary_plan;

/* Fills `plan` (host memory).  rot: a multiple of 16, 16 .. 256.  Pair i
 * (i < rot / 2) is entries (i, i + rot / 2) of a head, or (2i, 2i + 1) if
 * `interleaved`; it turns by inv_freq_host[i] radians a position (at most 2^40 either way) of
 * axis axis_of_pair_host[i] (< axes <= 8; NULL: axis 0).  Several axes are the
 * positions of image and video tokens: time, height, width. */
sp_status sp_rotary_plan_init(sp_rotary_plan* plan, int rot, const double* inv_freq_host,
                              const uint8_t* axis_of_pair_host, int axes, int interleaved);

/* Rotates queries and keys at their original positions (paper review,
 * "position ID recovery": the kept tokens keep their positions): each pair
 * (x0, x1) becomes (x0 cos a - x1 sin a, x1 cos a + x0 sin a), a = position *
 * frequency, or -a if `inverse` != 0 (which undoes the rotation and is its
 * gradient).  Entries past plan->rot are copied.
 *
 *   positions   device int32 [axes, T], axis a at positions[a * pos_stride]; any int32 value, the
 *               angle is exact to fp32 rounding at all of them (sp_gather_kept's out_positions)
 *   q, q_out    [T, H, d]     in and out may be the same rows, and must not overlap otherwise
 *   k, k_out    [T, H_kv, d]  H or H_kv may be 0: that pair of tensors is left out
 *
 * Requirements: T >= 0, 8 <= d <= 256, d % 8 == 0, rot <= d, at most 65535 heads each.  No workspace.
 * Products and sums are fp32, rounded once. */
sp_status sp_rotary(const sp_rotary_plan* plan, const int32_t* positions, int64_t pos_stride, int64_t T, int d,
                    sp_dtype dtype, int inverse, const sp_rows* q, const sp_rows* q_out, int H, const sp_rows* k,
                    const sp_rows* k_out, int H_kv, void* stream);

/* How a cache holds its rows.  A row is one token's d entries of one head.
 *   SP_CACHE_SAME  as they are, in `dtype`
 *   SP_CACHE_E4M3  8-bit floats (4 exponent bits, 3 mantissa bits), largest 448
 *   SP_CACHE_INT8  8-bit integers in [-127, 127]
 * The 8-bit kinds divide each row by its own scale, a power of two: the
 * smallest 2^k, k >= -100, with max|x| / 2^k <= 448 or 127 (1 for a row of
 * zeros), and round x / 2^k to the nearest code, ties to even.  With a power
 * of two the division is exact, and code * scale is a bf16 value, so reading
 * a cache back rounds nothing (but an entry whose code rounds up to 2^128 reads back as infinity).  A row that holds a NaN or an infinity gets
 * the scale NaN and reads back as NaN.
 * A cache that another program has filled may have any fp32 scales: code * scale is then rounded once to `dtype` when
 * it is read back, and sp_attend takes it as read back in its kernel for bf16 chunks (d = 64 and 128, sequences of more
 * than 16 query rows per KV head) and unrounded elsewhere.
 * The NaN codes of e4m3 (0x7f, 0xff) are never written, and a cache must not hold them: sp_cache_read makes NaN of
 * them, and sp_attend NaN or +-480, as the kernel that the call takes has it.  (A row that is to be NaN has the scale NaN.) */
typedef enum { SP_CACHE_SAME = 0, SP_CACHE_E4M3 = 1, SP_CACHE_INT8 = 2 } sp_cache_kind;

/* One layer's keys and values in pages of `page` tokens: the row of (page p,
 * head h, slot s) starts at entry p * stride_page + h * stride_head + s *
 * stride_slot of k and of v (entries of `dtype`, or bytes of the 8-bit kinds);
 * 16-byte aligned (8-byte for the 8-bit kinds), strides likewise.  So
 * [pages, H_kv, page, d] and [pages, page, H_kv, d] are both taken. */
typedef struct {
    void*         k;
    void*         v;
    float*        k_scale;     /* 8-bit kinds: [pages, H_kv, page], contiguous (see sp_cache_kind); else NULL */
    float*        v_scale;
    int64_t       stride_page, stride_head, stride_slot;
    int64_t       pages;
    int32_t       page, H_kv, d;
    sp_dtype      dtype;       /* of the rows written, read back and attended */
    sp_cache_kind kind;
} sp_cache;

/* The new tokens of B sequences, and where they stand.  Sequence b's new
 * tokens are rows cu_new[b] .. cu_new[b+1] - 1 of the call's tensors and the
 * last ones of its kv_len[b] tokens: row cu_new[b] + t is token
 * kv_len[b] - (cu_new[b+1] - cu_new[b]) + t.  Token i of the sequence is in
 * slot i % page of page table[b * table_stride + i / page].  All arrays are on
 * the device and read when the work runs, so a captured call follows their
 * contents; sp_gather_kept's cu_kept and sp_select_varlen's n_kept are such
 * arrays.  Rows before cu_new[0] and from cu_new[B] on are not touched.
 *
 * What the device arrays say is checked when the work runs.  A sequence is
 * left out, and SP_EDEVICE recorded in the workspace, unless
 * 0 <= cu_new[b] <= cu_new[b+1] <= T, cu_new[b+1] - cu_new[b] <= max_new and
 * 0 <= kv_len[b] <= table_width * page (and <= 2^30).  Table entries of tokens that a
 * call does not touch (outside every row's window, say) are not read.  A page index outside
 * [0, pages) is never followed: SP_EDEVICE is recorded, its tokens are not
 * written, read back as zeros, and are attended as if they were zeros or left out. */
typedef struct {
    int32_t        B;          /* 1 .. 65535 */
    int32_t        max_new;    /* at least the largest number of new tokens of a sequence */
    int64_t        T;          /* rows of the call's tensors, at most 2^31 - 1 */
    const int64_t* cu_new;     /* device [B + 1] */
    const int64_t* kv_len;     /* device [B] */
    const int32_t* table;      /* device [B, table_width] */
    int32_t        table_width;
    int64_t        table_stride;
} sp_batch;

/* Workspace bytes of sp_cache_write and sp_cache_read (they keep their status there). */
size_t sp_cache_workspace_size(void);

/* Writes the new tokens' keys and values, k_new and v_new [T, H_kv, d], to
 * their places in the cache, quantising as the cache's kind says.  A new
 * token whose place would be negative (kv_len below the number of new tokens) is
 * skipped.  No other slot of the cache is touched.  No two new tokens may have the same place, nor
 * two pages, heads or slots of the cache (checked: each stride passes over what the smaller ones
 * span).  A cache that is only read may be expanded along pages or heads. */
sp_status sp_cache_write(const sp_cache* cache, const sp_batch* batch, const sp_rows* k_new, const sp_rows* v_new,
                         void* ws, size_t ws_bytes, void* stream);

/* Reads the batch's "new" tokens back into out_k and out_v [T, H_kv, d] in the
 * cache's dtype; either may be NULL.  With cu_new the prompts' offsets, kv_len
 * their lengths and the rows of layer l of a [L, H_kv, T, d] tensor
 * (stride_row d, stride_head T * d) this makes sp_score's K_prompt, or
 * sp_score_varlen's, from a paged cache.  A token whose place would be
 * negative reads as zeros. */
sp_status sp_cache_read(const sp_cache* cache, const sp_batch* batch, const sp_rows* out_k, const sp_rows* out_v,
                        void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes sp_attend needs for this cache, batch and number of query
 * heads on the current device (0 if they are invalid).  Does not depend on the
 * contents of the batch's device arrays. */
size_t sp_attend_workspace_size(const sp_cache* cache, const sp_batch* batch, int H);

/* Causal attention of the new tokens over their sequences' cached tokens (the
 * new tokens' own keys and values are already in the cache):
 *
 *   out[r, h] = sum_i softmax_i(scale * q[r, h] . k_i) v_i,  lse[r, h] = ln sum_i exp(scale * q[r, h] . k_i)
 *
 * over the tokens i <= p of the row's sequence, p its own place, and i > p -
 * window if window > 0.  Query head h reads KV head h / (H / H_kv).  A row
 * that sees no token (p < 0) gets out = 0 and lse = -inf.  One call is a
 * prefill chunk, a decode step, or a mixture of them.  The same call gives the
 * same bits; in another batch a sequence's sums may be added in another order.  The lse of the
 * look-ahead decode steps is what sp_score_lse takes.
 *
 *   q, out   [T, H, d] in the cache's dtype; out must not overlap q, and rows of neither may overlap
 *            each other
 *   lse      fp32, lse[r * lse_stride_row + h * lse_stride_head], or NULL.  Step j of N
 *            look-ahead steps of one request (T = 1, layer l of sp_score_lse's lse [L, H, N]):
 *            pointer lse + l * H * N + j, lse_stride_head = N
 *
 * Requirements: 8 <= d <= 256, d % 8 == 0, H % H_kv == 0, scale in 8.2e-39 .. 2.3e38
 * (scale * log2(e) is a normal fp32 number).  Before a call of a kind is captured into a graph, one of that kind should have run,
 * as CUDA may load a kernel at its first launch.  What unwritten slots hold (NaN too) has no effect, nor have rows
 * that are not a token of the batch.  A NaN or an infinity in a key or value of a token that
 * some rows of the sequence see may reach its other rows as well.
 * Statistics and sums are fp32; bf16 softmax weights are rounded to bf16 for
 * the product with the values.
 * The tensor cores are used for bf16 with d = 64 or 128, where no sequence has more than 16 query rows per KV head or the cache's
 * pages are a multiple of 8 tokens (any page for the 8-bit kinds, 16-byte aligned with such strides), H / H_kv is at most 128 and
 * B at most 16384.  All else is right, but runs on the
 * CUDA cores: a chunk of 256 over 4096 takes 30 us at d = 128 and 2.1 ms at d = 96. */
sp_status sp_attend(const sp_rows* q, const sp_cache* cache, const sp_batch* batch, int H, double scale,
                    int64_t window, const sp_rows* out, float* lse, int64_t lse_stride_row,
                    int64_t lse_stride_head, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* Trees of drafted tokens                                                  */
/* ------------------------------------------------------------------------ */

/* The new tokens of a batch's sequences may be drafted ones that form a tree: parent[r] says on which new token of its own
 * sequence row r hangs, counted from the sequence's first (so parent[r] < its own number), or -1 for a root, which hangs on
 * the cached tokens.  A round: sp_tree_seen, sp_rotary at its positions, sp_cache_write, sp_attend_tree in each layer, then
 * sp_tree_accept and sp_cache_keep (drafted != 0) in each layer. */

/* Workspace bytes of sp_tree_seen and sp_tree_accept (they keep their status there). */
size_t sp_tree_workspace_size(void);

/* From the parents, what sp_attend_tree and sp_rotary take.
 *
 *   parent     device int32 [T]
 *   seen       device, or NULL: bit u % 32 of word seen[r * seen_stride + u / 32] is set if row r is new token u of its
 *              sequence or hangs on it, directly or over others.  All seen_words words are written; 32 * seen_words >= max_new
 *   positions  device int32 [T], or NULL: kv_len - (new tokens) + the number of tokens that row r hangs on
 *
 * Rows that are not a token of the batch are not written.  The batch's table is not read.  A parent that is not a token before
 * its row counts as -1, and SP_EDEVICE is recorded in the workspace; a sequence of more than 4096 new tokens is left out, and
 * SP_EDEVICE recorded as well. */
sp_status sp_tree_seen(const sp_batch* batch, const int32_t* parent, uint32_t* seen, int64_t seen_stride, int seen_words,
                       int32_t* positions, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes of sp_attend_tree (0 if the arguments are invalid). */
size_t sp_attend_tree_workspace_size(const sp_cache* cache, const sp_batch* batch, int H);

/* sp_attend where a row sees the cached tokens before the new ones, and of the new ones those whose bits are set (as
 * sp_tree_seen lays them out; any bits will do, also none, or such of later tokens; bits of tokens that the sequence does not
 * have are ignored).  A row's place, which a window > 0 goes by, is kv_len - (new tokens) + max(bits set, 1) - 1; the window
 * hides tokens before the new ones only.  A row that sees nothing gets out = 0 and lse = -inf.
 * All else as sp_attend: types, layouts, kernels and their speed. */
sp_status sp_attend_tree(const sp_rows* q, const sp_cache* cache, const sp_batch* batch, int H, double scale,
                         int64_t window, const uint32_t* seen, int64_t seen_stride, int seen_words, const sp_rows* out,
                         float* lse, int64_t lse_stride_row, int64_t lse_stride_head, void* ws, size_t ws_bytes, void* stream);

/* The drafted tokens that the target agrees with, by its choice after each of them (draft and target device int32 [T]:
 * the token that row r is, and the one that the target chooses after it).  The first new token of a sequence is accepted (it
 * is the target's own choice of the round before); after an accepted token r its first child c with draft[c] == target[r] is.
 *
 *   path    device int32: path[b * path_stride + i] is the i-th accepted new token of sequence b, ascending, counted from the
 *           sequence's first; -1 behind the last one, up to max_new
 *   n_path  device int64 [B]: how many (0 for a sequence without new tokens)
 *   next    device int32 [B] or NULL: the target's choice after the last accepted token (-1 without one)
 *
 * Parents as for sp_tree_seen.  path and n_path are what sp_cache_keep takes with drafted != 0 and heads = 1. */
sp_status sp_tree_accept(const sp_batch* batch, const int32_t* parent, const int32_t* draft, const int32_t* target, int32_t* path,
                         int64_t path_stride, int64_t* n_path, int32_t* next, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* Cutting a cache                                                          */
/* ------------------------------------------------------------------------ */

/* Workspace bytes of sp_attend_weights for this cache, batch and number of query heads on the current device (0 if they
 * are invalid).  Does not depend on the contents of the batch's device arrays. */
size_t sp_attend_weights_workspace_size(const sp_cache* cache, const sp_batch* batch, int H);

/* Adds the attention weights that the new tokens' queries give their sequences' cached tokens to what these have gathered:
 *
 *   weights[i, g] = decay * weights[i, g] + sum over rows r that see i, heads h of KV head g of exp(scale * q[r, h] . k_i - lse[r, h])
 *
 * for token i of the sequence and KV head g, with the new tokens, visibility (causal, window) and lse of sp_attend.  A new
 * token's weight starts from 0; with decay = 0 every token's does, and what was there is not read.  Weights of tokens that
 * no row sees (outside every row's window, or of a sequence without new tokens) are not touched.  A row whose lse is -inf saw
 * nothing and adds nothing.
 *
 *   q        [T, H, d]   lse  fp32, lse[r * lse_stride_row + h * lse_stride_head], as sp_attend writes it
 *   weights  device fp32 [pages, H_kv, page], contiguous: of the token in slot s of page p, KV head g
 *
 * Requirements as sp_attend; 0 <= decay <= 1.  A token whose page index is out of range is left out, and SP_EDEVICE recorded.
 * No two tokens of the batch may have the same place.  Sums are fp32 in a fixed order: the same call gives the same bits. */
sp_status sp_attend_weights(const sp_rows* q, const sp_cache* cache, const sp_batch* batch, int H, double scale, int64_t window,
                            const float* lse, int64_t lse_stride_row, int64_t lse_stride_head, double decay, float* weights,
                            void* ws, size_t ws_bytes, void* stream);

/* Which of its tokens each sequence keeps: all if it has at most `budget`, else the first `first`, the last `last`, and of those
 * between the budget - first - last with the largest weights, ties to the lower token.  -0 equals 0, and NaN ranks below all
 * else.  The batch's kv_len and table say where the tokens are; its new tokens count like the others.
 *
 *   shared  0: a list for every KV head, by its own weights; otherwise one list a sequence, by the maximum over the KV heads
 *   kept    device int32: kept[b * kept_stride_seq + g * kept_stride_head + i] is the i-th kept token of sequence b and KV head
 *           g (0 if shared), ascending; -1 behind the last one, up to `budget`
 *   n_kept  device int64 [B]: min(kv_len[b], budget); not the batch's kv_len itself
 *
 * 0 <= first + last <= budget <= 2^30.  Workspace: sp_cache_workspace_size().  A sequence whose lengths are impossible keeps
 * nothing (n_kept 0); a token whose page index is out of range ranks lowest; either records SP_EDEVICE. */
sp_status sp_cache_choose(const sp_cache* cache, const sp_batch* batch, const float* weights, int shared, int64_t budget,
                          int64_t first, int64_t last, int32_t* kept, int64_t kept_stride_seq, int64_t kept_stride_head,
                          int64_t* n_kept, void* ws, size_t ws_bytes, void* stream);

/* Keeps the listed tokens of each sequence and drops the others: the i-th listed token's keys, values, scales and (unless
 * NULL) weights become those of token i, and kv_out[b] = n_kept[b].  The lists are ascending.  They are sp_cache_choose's, the
 * kept positions of a prompt that sp_select has cut, or any others.  With drafted != 0 they count from the sequence's first new
 * token, as sp_tree_accept's do, the i-th becomes new token i, and kv_out[b] = kv_len[b] - (new tokens) + n_kept[b]:
 * the tokens before the new ones stay.
 *
 *   kept    device int32, kept[b * kept_stride_seq + g * kept_stride_head + i]; heads = H_kv lists a sequence, or 1 for all heads
 *   n_kept  device int64 [B], each at most `most`
 *   to      NULL: the rows move within the sequence's own pages, whose last ones fall free.  Otherwise device int32
 *           [B, to_width], rows to_stride apart: new token i is in slot i % page of page to[b * to_stride + i / page], and
 *           what was there before stays as it was.  No page of `to` may be one that holds a listed token of the batch
 *   weights [pages, H_kv, page], as sp_attend_weights gathers them, or NULL
 *   kv_out  device int64 [B], not the batch's kv_len itself
 *
 * Keys keep the positions that they were rotated at, so attention over the kept tokens is what it was without the others; a
 * window counts kept tokens.  Nothing is quantised again.  Slots from kv_out on hold what they held.  Workspace:
 * sp_cache_workspace_size().  SP_EDEVICE is recorded, and the sequence is left as it was with kv_out[b] = kv_len[b], where
 * lengths or counts are impossible (also a `to` too narrow for them); an entry that is out of range is passed over, and one that
 * is not above the entry before it is recorded as well (the sequence's rows are then not determined).  No two sequences may
 * have a page in common that either has rows moved in. */
sp_status sp_cache_keep(const sp_cache* cache, const sp_batch* batch, const int32_t* kept, int heads, int64_t kept_stride_seq,
                        int64_t kept_stride_head, const int64_t* n_kept, int64_t most, int drafted, const int32_t* to, int to_width,
                        int64_t to_stride, float* weights, int64_t* kv_out, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* Status                                                                   */
/* ------------------------------------------------------------------------ */

/* Synchronises `stream` and returns the run-time status a kernel recorded in
 * the workspace `ws` of the last call that used it: SP_OK, SP_ETIMEOUT (a
 * bounded wait gave up) or SP_EDEVICE.  Also returns SP_ECUDA if the stream
 * reports an error. */
sp_status sp_workspace_status(const void* ws, void* stream);

/* Message of the last failing call on this host thread ("" if none). */
const char* sp_last_error(void);

/* Name of a status code. */
const char* sp_status_string(sp_status s);

/* ABI version (major * 100 + minor). */
int sp_version(void);

/* Number of CUDA kernels this process has launched through the library
 * (all entry points, all threads).  For accounting in benchmarks. */
uint64_t sp_kernel_launches(void);

/* ------------------------------------------------------------------------ */
/* Test hook (not for production use)                                       */
/* ------------------------------------------------------------------------ */

/* Sets the limit, in nanoseconds, of the tensor-core scoring kernel's waits
 * on other CTAs' exchange entries (each token range's softmax statistics and
 * each row's lse); 0 restores the default of 4 s.  Returns the previous limit.
 * Calls enqueued afterwards use the new limit (it is read when a call is
 * planned); waits inside one CTA and the drain of its in-flight copies and
 * MMAs keep 4 s.  Tests lower it to about a microsecond so that an exchange
 * wait runs out: the kernel then records SP_ETIMEOUT in the workspace, stops
 * every warp role, waits for its in-flight copies and MMAs, frees its tensor
 * memory and returns, and sp_workspace_status reports SP_ETIMEOUT.  Process-
 * wide, not synchronised with calls running on other threads. */
uint64_t sp_test_set_exchange_wait_ns(uint64_t ns);

/* Test hook (host only, no device work): the tensor-core scoring path's plan
 * for one bf16 prompt of M tokens (L layers, H query heads, H_kv KV heads, head
 * dim d, N look-ahead steps; the first pass when N needs several) on `sms` SMs.
 * Writes nine ints to out9 (caller-owned host memory): slab classes F, CTAs per
 * class Pc, CTAs P = F * Pc, tiles of 128 tokens per CTA per slab, tiles per
 * epilogue group, landing tiles per group, held slabs per group, the
 * statistics-to-normalise lag in slabs, and the shared memory per CTA in bytes.
 * Returns 1, or 0 when that path does not take the shape (or an argument is
 * out of range); nothing is launched and nothing else is written. */
int sp_test_score_plan(int L, int H, int H_kv, int d, int64_t M, int N, int sms, int* out9);

#ifdef __cplusplus
}
#endif

#endif /* SPECPREFILL_H */
