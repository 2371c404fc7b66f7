/*
 * dvl.h -- C ABI of the GB300 draft-head argmax library (libdvl.so).
 *
 * The operation: a speculative-decoding draft head projects M hidden rows
 * h[M][K] against the rows of its LM head W[N][K] and keeps, per hidden row,
 * the best token -- logits = h . W^T, reduced on the device to an id and its
 * logit, so no logit tensor is ever written to memory.  N is either the full
 * vocabulary or a frequency-ranked shortlist of it, in which case a d2t map
 * turns a shortlist row index into a full-vocabulary id.
 *   - the projection and its shape ("Shortlist MTP", section "What I was
 *     testing": hidden width 2,560 against 248,320 rows; M is 1 for a draft
 *     step and 3 for an MTP2 verify step);
 *   - the shortlist and its on-device reduction ("Shortlist MTP", sections
 *     "What was actually happening" and "Re-running the comparison fairly":
 *     the shortlist projection and local argmax reduction);
 *   - the trim at load and the d2t map ("Masked MTP drafts": a ranks .txt
 *     next to the model, the head weight trimmed at load; EAGLE-3's d2t
 *     index mapping reused for a frequency-ranked subset);
 *   - the NVFP4 head ("Masked MTP drafts": the trimmed head requantized to
 *     NVFP4) and the FP8 head ("Masked MTP drafts", section "Update
 *     (November 2026)": a drafter's own FP8 head; "[DGX Spark]
 *     Qwen3.8-Flash-Next on two DGX Sparks", section "The costs: a 69%
 *     smaller KV pool and FP8 GDN weights": weights read as FP8 E4M3);
 *   - the ranks builder ("Shortlist MTP", section "Building the 16k
 *     shortlist"; "[DGX Spark] Qwen3.8-Flash-Next on two DGX Sparks",
 *     section "Build the draft vocabulary from your own text").
 *
 * Conventions for every entry point:
 *   - Memory: the caller owns every buffer.  "device" pointers are CUDA
 *     device memory on the current device; "host" pointers are ordinary host
 *     memory.  The GPU entry points never allocate, free or synchronize; they
 *     enqueue work on `stream` (a cudaStream_t; NULL is the legacy default
 *     stream) and return.  Results are ready in stream order.
 *   - Errors: arguments are checked on the host before anything is enqueued;
 *     a bad argument returns a non-zero dvl_status and enqueues nothing.  A
 *     failed launch returns DVL_ERR_CUDA (the outputs are then undefined).
 *   - Threading: calls are thread-safe.  One workspace serves one stream at a
 *     time: two calls that may run concurrently on the GPU must not share a
 *     workspace.
 *   - Alignment: W, h, scales and the workspace start on 16-byte boundaries;
 *     d2t, ids and logits on 4-byte boundaries.
 */
#ifndef DVL_H
#define DVL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    DVL_OK = 0,
    DVL_ERR_INVALID_ARG = 1,  /* NULL pointer, bad size, misalignment        */
    DVL_ERR_OUT_OF_RANGE = 2, /* an id outside [0, V) (host-checked ids; as a
                                 device-side bit: a d2t entry outside [0, V)) */
    DVL_ERR_UNSUPPORTED = 3,  /* a shape this build has no kernel for        */
    DVL_ERR_WORKSPACE = 4,    /* workspace missing or smaller than required  */
    DVL_ERR_CUDA = 5,         /* a CUDA runtime call or a launch failed      */
    DVL_ERR_TIMEOUT = 6       /* device-side bit: a bounded wait gave up     */
} dvl_status;

typedef enum {
    DVL_BF16 = 0,  /* W: bfloat16 [N][K] row-major                          */
    DVL_NVFP4 = 1, /* W: E2M1 codes [N][K/2] (low nibble = even k), E4M3
                      scales [N][K/16] (one per 16 consecutive k of a row),
                      one fp32 tensor scale                                  */
    DVL_FP8 = 2    /* W: E4M3 codes [N][K], one fp32 tensor scale; no
                      per-block scales                                       */
} dvl_dtype;

/* Limits of this build. */
#define DVL_MAX_M 32        /* hidden rows per call                            */
#define DVL_MAX_TOPK 4      /* k of draft_topk                                 */
#define DVL_K_MULTIPLE 64   /* K must be a positive multiple of this           */
#define DVL_MAX_K 24576     /* largest hidden width                            */

/* dvl_head.flags: the caller promises that no work still pending on the
 * stream when the call is enqueued writes w, scales or d2t (true of weights
 * loaded long before; not of a head trim_head has just filled on the same
 * stream unless the caller synchronized since).  The kernel may then start
 * streaming the head before the preceding kernel on the stream has finished
 * (programmatic dependent launch); without the flag it reads nothing before
 * that kernel completes. */
#define DVL_HEAD_STATIC 1

/* A draft head as the kernels read it.  Every pointer is device memory. */
typedef struct dvl_head {
    int32_t dtype;        /* dvl_dtype                                         */
    int32_t N;            /* rows of W (>= 1)                                  */
    int32_t K;            /* hidden width (multiple of 64, <= DVL_MAX_K)       */
    int32_t flags;        /* DVL_HEAD_* bits; 0 when none applies              */
    int64_t V;            /* full vocabulary size: ids lie in [0, V)           */
    int64_t id_base;      /* with d2t == NULL, row n has full id id_base + n;
                             id_base + N <= V.  0 for a whole head; the first
                             id of a slice when a head is split by rows.       */
    const void *w;        /* bf16 [N][K], NVFP4 codes [N][K/2] or FP8 [N][K]   */
    const uint8_t *scales;/* NVFP4: E4M3 [N][K/16]; NULL for bf16 and FP8      */
    float global_scale;   /* NVFP4 / FP8 tensor scale; ignored for bf16        */
    int32_t reserved2;    /* must be 0                                         */
    const int32_t *d2t;   /* int32 [N]: full-vocabulary id of each row, each in
                             [0, V); NULL means the identity map shifted by
                             id_base.  The kernels read no memory through a
                             d2t entry; a returned id outside [0, V) is
                             returned as it is and reported as the
                             device-side status bit DVL_ERR_OUT_OF_RANGE (see
                             dvl_workspace_status)                           */
} dvl_head;

/* Human-readable name of a status code (static storage). */
const char *dvl_status_string(int status);

/* Library version, major * 10000 + minor * 100 + patch. */
int dvl_version(void);

/* The CUDA runtime's description of the error behind the calling thread's
 * most recent DVL_ERR_CUDA ("no error" if there was none).  Static storage. */
const char *dvl_last_error(void);

/* ---------------------------------------------------------------------- */
/* Workspace                                                              */
/* ---------------------------------------------------------------------- */

/* Bytes of device workspace one draft_argmax (k = 1) or draft_topk call
 * with M hidden rows needs.  Returns 0 for M or k outside their limits.
 * The workspace holds the cross-block reduction state: a ticket counter,
 * the per-row best keys and, for k > 1, one candidate list per thread block.
 * It is self-cleaning: every call leaves it as it found it. */
size_t dvl_workspace_bytes(int32_t M, int32_t k);

/* Zero a workspace before its first use (enqueued on `stream`).  Only
 * needed once; also restores a workspace whose last call did not complete.
 * ws: device, 16-byte aligned; bytes >= dvl_workspace_bytes(M, k) of every
 * call that will use it. */
dvl_status dvl_workspace_init(void *ws, size_t bytes, void *stream);

/* Device-side failures recorded in a workspace since it was last read: a
 * bitmask with bit (1 << s) set for each dvl_status s a kernel reported:
 *   DVL_ERR_TIMEOUT       a bounded wait of the tcgen05 kernel gave up; that
 *                         call's results are not valid;
 *   DVL_ERR_OUT_OF_RANGE  a draft call returned an id outside [0, V): a d2t
 *                         entry out of range won, and is returned as it is.
 * The status word is read after the work already enqueued on `stream` (this
 * synchronizes `stream`), then cleared on `stream`.
 *   ws:          a workspace from dvl_workspace_init.
 *   status_bits: HOST (out).
 * Errors: DVL_ERR_INVALID_ARG, DVL_ERR_CUDA. */
dvl_status dvl_workspace_status(void *ws, uint32_t *status_bits, void *stream);

/* ---------------------------------------------------------------------- */
/* The hot path                                                           */
/* ---------------------------------------------------------------------- */

/* Per hidden row m: the full-vocabulary id of the head row with the largest
 * logit sum_k W[n][k] * h[m][k], and that logit.  The dot products run in
 * fp32 on the device (products of bf16 values are exact; the order of the
 * additions is the kernel's).  Exactly equal logits go to the lowest full
 * id; a NaN logit ranks below every number (among NaN logits the lowest id
 * wins, reported with a NaN logit); -0 and +0 compare equal and +0 is
 * reported.  For NVFP4,
 * weight = e2m1(code) * e4m3(scale) * global_scale; for FP8,
 * weight = e4m3(code) * global_scale; the kernel applies global_scale to the
 * finished dot product.
 *   head:      the head (see dvl_head); host struct, device pointers.
 *   h:         device bf16 [M][K], row-major.
 *   M:         1 .. DVL_MAX_M.
 *   ids:       device int32 [M] (out).
 *   max_logit: device fp32 [M] (out).
 *   ws:        device workspace of at least dvl_workspace_bytes(M, 1)
 *              bytes, zeroed once by dvl_workspace_init.
 * Errors: DVL_ERR_INVALID_ARG (NULL, misaligned, N < 1, K not a multiple of
 * 64 or above DVL_MAX_K, M out of range, unknown flags, reserved2 non-zero, dtype
 * unknown, NVFP4 without scales, FP8 with scales, d2t == NULL with
 * id_base + N > V),
 * DVL_ERR_WORKSPACE, DVL_ERR_CUDA. */
dvl_status dvl_draft_argmax(const dvl_head *head, const void *h, int32_t M,
                            int32_t *ids, float *max_logit, void *ws,
                            size_t ws_bytes, void *stream);

/* Per hidden row m: the k best head rows by (logit desc, full id asc), as
 * full ids and logits, best first.  Same arithmetic, rules and errors as
 * dvl_draft_argmax; k = 1 gives exactly its result.  Rows are distinct; a
 * d2t that repeats an id can make an id appear twice.
 *   k:      1 .. DVL_MAX_TOPK, and k <= N.
 *   ids:    device int32 [M][k] (out).
 *   logits: device fp32 [M][k] (out).
 *   ws:     at least dvl_workspace_bytes(M, k) bytes. */
dvl_status dvl_draft_topk(const dvl_head *head, const void *h, int32_t M, int32_t k,
                          int32_t *ids, float *logits, void *ws, size_t ws_bytes,
                          void *stream);

/* Which kernels a dvl_draft_argmax (k = 1) or dvl_draft_topk call with this
 * head, M and k launches, for logs and tests; enqueues nothing.  *kernel is
 * a static string owned by the library:
 *   "bf16-cuda-cores"  CUDA-core kernel (one or two hidden rows, widths
 *                      other than 2,560 / 5,120, short heads);
 *   "bf16-mma"         register-path tensor cores (3 .. 8 hidden rows at
 *                      width 2,560 or 5,120, and argmax at 9 .. 16 rows at
 *                      2,560, on a 32-byte aligned head of at least 8 rows
 *                      per warp of the grid);
 *   "bf16-tcgen05"     5th-generation tensor cores (5 .. 32 hidden rows, when
 *                      the register-path kernel does not apply);
 *   "nvfp4-mma", "fp8-mma"  the low-bit heads.
 * *launches is the number of kernel launches of the call.  The choice
 * depends on the current device's SM count.
 * Errors: those of dvl_draft_topk's head and M / k checks, and
 * DVL_ERR_CUDA when the device cannot be queried. */
dvl_status dvl_draft_plan(const dvl_head *head, int32_t M, int32_t k, const char **kernel,
                          int32_t *launches);

/* dvl_draft_argmax for callers that cannot allocate device memory.  The
 * pages have no counterpart of this entry point.
 *
 * Who needs it: code running as a plugin inside an inference engine that
 * owns every device allocation (raw cudaMalloc is not available to it), and
 * latency-critical decode loops where a cudaMalloc would stall the pipeline
 * (it may synchronize the device).  Such a caller passes the head, h and the
 * outputs only; the reduction scratch lives in a fixed 512-byte array in the
 * library's own device memory (a static __device__ array: every GPU that
 * loads the library keeps it until the process exits).  This entry point
 * allocates nothing and frees nothing.
 *   Same arguments, arithmetic and results as dvl_draft_argmax, without
 *   ws / ws_bytes; the same argument errors.  M above DVL_MAX_M (32), the
 *   most the fixed scratch holds, returns DVL_ERR_INVALID_ARG before
 *   anything is enqueued.
 *   The first call in a CUDA context looks up the array's device address
 *   (cudaGetSymbolAddress, with that context's device current) and keeps it
 *   for that context; make that first call before any stream capture.
 *   Every call clears the scratch's reduction state (ticket and best keys)
 *   with memsets enqueued on `stream`, then runs the argmax on it.  The
 *   scratch's status word is not cleared: device-side failures (the bits of
 *   dvl_workspace_status) accumulate there until dvl_noalloc_status reads
 *   them.  All calls on a device share the one array: two calls that may
 *   run at the same time on the GPU (on different streams, or from
 *   different threads) race on it and may return wrong results.  Keep them
 *   in one stream order. */
dvl_status dvl_draft_argmax_noalloc(const dvl_head *head, const void *h, int32_t M,
                                    int32_t *ids, float *max_logit, void *stream);

/* The device-side failure bits that dvl_draft_argmax_noalloc calls on the
 * current device recorded since the last read (the bits and meaning of
 * dvl_workspace_status), read after the work already enqueued on `stream`
 * (this synchronizes `stream`) and then cleared on `stream`.  No
 * counterpart on the pages; allocates nothing.
 *   status_bits: HOST (out).
 * Errors: DVL_ERR_INVALID_ARG, DVL_ERR_CUDA. */
dvl_status dvl_noalloc_status(uint32_t *status_bits, void *stream);

/* Candidate scores through a head ("Masked MTP drafts", section "Update
 * (November 2026)": a drafter that carries no head of its own scores its
 * candidates through the target's LM head, bf16 or NVFP4, and the trim
 * stacks on top).  For m < M and j < c:
 *   logits[m][j] = sum_k W[ids[m][j] - id_base][k] * h[m][k]
 * with the head's dtype and arithmetic (fp32 accumulation; NVFP4 weights
 * e2m1 * e4m3, FP8 weights e4m3, with the tensor scale on the finished dot),
 * in any summation
 * order.  The head's rows are ids id_base .. id_base + N - 1: a full head
 * (id_base 0) or any contiguous slice of one.  An id outside them scores
 * NaN; the ids live on the device and are not checked on the host.
 *   head:   a head without d2t (d2t == NULL).
 *   h:      device bf16 [M][K], row-major, 16-byte aligned.
 *   M:      1 .. DVL_MAX_M.
 *   ids:    device int32 [M][c], row-major (the candidates of row m).
 *   c:      candidates per row, >= 1, with M * c < 2^31.
 *   logits: device fp32 [M][c] (out), row-major.
 * Nothing is allocated; no workspace.  The call is enqueued on `stream`.
 * Errors: DVL_ERR_INVALID_ARG (the head checks of dvl_draft_argmax, a head
 * with d2t, NULL or misaligned pointers, M or c out of range), DVL_ERR_CUDA. */
dvl_status dvl_score_ids(const dvl_head *head, const void *h, int32_t M,
                         const int32_t *ids, int32_t c, float *logits, void *stream);

/* ---------------------------------------------------------------------- */
/* The drafting step around the head                                      */
/*                                                                        */
/* What a drafter's own layer runs between two draft calls: attention of  */
/* the new tokens over its paged cache, the residual addition and norm in */
/* front of a projection or of the head, the choice of the next beams     */
/* from the head's logits, and the reordering of what belongs to a beam.  */
/* The pages describe the step (M = 1 for a draft step, 3 for an MTP2     */
/* verify step, a concurrent batch of 8), not these operators.            */
/* ---------------------------------------------------------------------- */

/* Limits of these operators. */
#define DVL_F32 3             /* fp32 activations (dvl_norm.residual_dtype, beam logits) */
#define DVL_MAX_QUERY 8       /* new tokens per sequence (T)                    */
#define DVL_MAX_QUERY_ROWS 64 /* T * query heads per cached head                */
#define DVL_MAX_HEAD_DIM 256  /* D                                              */
#define DVL_MAX_BEAMS 32      /* beams in, and beams selected, per request      */
#define DVL_MAX_STATES 8      /* state tensors of one reordering                */

/* Arguments of dvl_add_rmsnorm.  Every pointer is device memory; strides are
 * in elements of the tensor they belong to, between consecutive rows. */
typedef struct dvl_norm {
    int64_t rows;             /* >= 0; 0 enqueues nothing                          */
    int32_t K;                /* row width, 1 .. DVL_MAX_K                         */
    int32_t residual_dtype;   /* DVL_BF16 or DVL_F32: residual and residual_out    */
    int32_t group;            /* values per scale of codes: 16, 32, 64, 128, 256,
                                 or 0 for one scale per row                        */
    float eps;                /* added to the mean square, >= 0                    */
    const void *x;            /* bf16 [rows][K]                                    */
    int64_t x_stride;
    const void *weight;       /* bf16 [K]                                          */
    const void *residual;     /* [rows][K], or NULL                                */
    int64_t residual_stride;
    void *residual_out;       /* [rows][K] (out); NULL goes with residual NULL; may
                                 be residual itself, or x when residual is bf16    */
    int64_t residual_out_stride;
    void *out;                /* bf16 [rows][K] (out), or NULL                     */
    int64_t out_stride;
    uint8_t *codes;           /* E4M3 [rows][K] (out), or NULL                     */
    int64_t codes_stride;
    float *scales;            /* fp32 [rows][ceil(K / group)] contiguous (out);
                                 with codes only                                   */
} dvl_norm;

/* Residual addition and root-mean-square norm of each row, in fp32:
 *   u = x + residual (u = x without one);  residual_out = u rounded to its type;
 *   y = u * weight / sqrt(mean(u^2) + eps)      (u before that rounding);
 *   out = y rounded to bf16;
 *   per group of a row: a = max |y|, scale = a / 448,
 *   code = RNE_e4m3(y * (448 / a)), saturating at 448,
 * so y ~ code * scale.  All in fp32: the mean square, its reciprocal root and
 * 448 / a are off by a few 2^-24, so a value as near as that to the middle
 * between two codes can take either.  Squares above fp32's range make y 0; where
 * all lie below it and eps is 0, y is infinite or NaN.  A group with a < 2^-119
 * has scale a / 448 and codes 0 (1 / scale is no fp32 number there).  A NaN or
 * an infinity in a row shows: the values it reaches are NaN, in scale and codes
 * too.
 * Any K and any strides run; rows whose tensors all start on 16-byte
 * boundaries with K % 8 == 0 use 16-byte accesses.  No workspace.
 * Errors: DVL_ERR_INVALID_ARG (NULL x or weight; neither out nor codes; codes
 * without scales or the reverse; residual without residual_out or the
 * reverse; rows, K, group, eps, dtype out of range; with more than one row a
 * negative input stride or an output stride below K; a pointer not aligned to
 * its element), DVL_ERR_CUDA. */
dvl_status dvl_add_rmsnorm(const dvl_norm *args, void *stream);

/* A paged key-value cache.  Strides are in elements, not negative; the D
 * values of a head are consecutive.  Every (page, token, head) row starts on a
 * 16-byte boundary, and a page spans at most 10^9 elements (page_size token
 * strides plus heads head strides: offsets within a page are 32-bit; pages may
 * lie any distance apart). */
typedef struct dvl_kv_cache {
    int32_t dtype;            /* DVL_BF16, or DVL_FP8 (E4M3 codes, one scale each) */
    int32_t pages;            /* pages of the pool                                 */
    int32_t page_size;        /* tokens per page, >= 1                             */
    int32_t heads;            /* key-value heads                                   */
    int32_t D;                /* head width: a multiple of 16, <= DVL_MAX_HEAD_DIM */
    int32_t reserved;         /* must be 0                                         */
    void *k, *v;              /* [pages][page_size][heads][D]                      */
    int64_t k_page_stride, k_token_stride, k_head_stride;
    int64_t v_page_stride, v_token_stride, v_head_stride;
    float k_scale, v_scale;   /* value of code 1 (DVL_FP8); 1 for bf16             */
} dvl_kv_cache;

/* Bytes of device workspace a dvl_paged_attention call with this cache, T new
 * tokens and Hq query heads needs on the current device, whatever the batch
 * and its lengths.  0 for arguments outside the limits or without a device.
 * Zero it once (dvl_workspace_init); every call leaves it as it found it.
 * Attention calls of any sizes that fit may share one, calls of other entry
 * points may not.  dvl_workspace_status reads its status word. */
size_t dvl_attention_workspace_bytes(const dvl_kv_cache *cache, int32_t T, int32_t Hq);

/* Attention of the T newest tokens of each of B sequences over their cached
 * keys and values (their own included: lengths counts them).  With
 * G = Hq / heads, query head h reads cached head h / G, and token t sees
 * n = max(0, length - (T - 1 - t)) positions:
 *   s_j = scale * k_scale * (q . k_j),  m = max_j s_j,  j < n
 *   out = v_scale * sum_j exp(s_j - m) v_j / sum_j exp(s_j - m)
 *   lse = m + ln(sum_j exp(s_j - m))
 * n = 0 gives out 0 and lse -inf.  Positions at or above n are not read into
 * the result, whatever the cache holds there.  Sums and softmax statistics are
 * fp32.  Products are exact, except that with an FP8 cache query values below
 * 2^-29 of their row's largest are rounded to a grid of 2^-38 of it.  The
 * weights exp(s_j - m) are rounded before they meet V: to bf16 (2^-8
 * relative), or with an FP8 cache to f16 (2^-11 relative down to 2^-29, a grid
 * of 2^-39 below).  The result does not depend on timing: the same call on the
 * same device gives the same bits.
 *   q:        device bf16 [B][T][Hq][D]; strides in elements for the first
 *             three, the last is 1; 16-byte aligned rows.
 *   table:    device int32 [B][table_width], row stride table_stride: the
 *             page of each page_size tokens.  Entries past a sequence's
 *             length are not read.  An entry outside [0, pages) sets the
 *             status bit DVL_ERR_OUT_OF_RANGE, and page 0 is read in its
 *             place: that sequence's result says nothing, other sequences are not touched.
 *   lengths:  device int32 [B].  Below 0 counts as 0; above
 *             table_width * page_size is cut to that, with the same bit.
 *   out:      device bf16 [B][T][Hq][D] contiguous, 16-byte aligned.
 *   lse:      device fp32 [B][T][Hq] contiguous, or NULL.
 *   ws:       dvl_attention_workspace_bytes, from dvl_workspace_init.
 * B = 0 enqueues nothing.
 * Errors: DVL_ERR_INVALID_ARG (NULL or misaligned, B < 0, T or Hq < 1, T above
 * DVL_MAX_QUERY, Hq not a multiple of heads, T * G above DVL_MAX_QUERY_ROWS,
 * D not a multiple of 16 or above DVL_MAX_HEAD_DIM, page_size * table_width
 * above 2^31 - 128, scale not finite), DVL_ERR_WORKSPACE, DVL_ERR_CUDA. */
dvl_status dvl_paged_attention(const dvl_kv_cache *cache, const void *q, int64_t q_batch_stride,
                               int64_t q_token_stride, int64_t q_head_stride, int32_t B, int32_t T,
                               int32_t Hq, const int32_t *table, int64_t table_stride,
                               int32_t table_width, const int32_t *lengths, float scale, void *out,
                               float *lse, void *ws, size_t ws_bytes, void *stream);

/* Bytes of device workspace a dvl_beam_select call needs; 0 for arguments
 * outside the limits.  Zero it once (dvl_workspace_init); every call leaves
 * it as it found it.  Selections of any sizes that fit may share one, calls
 * of other entry points may not. */
size_t dvl_beam_workspace_bytes(int32_t batch, int32_t beams, int32_t N);

/* Beam search's choice of the next beams.  For request b, beam j and row n of
 * the head:
 *   x = logits[b][j],  m = max_i x[i],
 *   score(j, n) = scores[b][j] + ((x[n] - m) - ln sum_i exp(x[i] - m))   (in fp32),
 * and the k best candidates of the request, best first.  Equal scores: the
 * lower beam first; within a beam the larger logit, then the lower row.  A
 * score of -inf or NaN is no candidate (a dead beam's -inf score, a banned
 * row's -inf logit; a beam whose logits hold a NaN or +inf, or nothing but
 * -inf, has none).  Slots left over get score -inf, parent -1, token -1.
 *   logits:     device [batch][beams][N], dtype DVL_BF16 or DVL_F32, rows
 *               contiguous, batch and beam strides in elements, aligned to
 *               the element.
 *   scores:     device fp32 [batch][beams] contiguous.
 *   batch:      >= 0 (0 enqueues nothing).  beams, k: 1 .. DVL_MAX_BEAMS.
 *   N:          1 .. 2^31 - 65,536.
 *   d2t:        device int32 [N], or NULL (token = n).
 *   out_scores: device fp32 [batch][k], parents and tokens: device int32
 *               [batch][k] (out).
 *   ws:         dvl_beam_workspace_bytes(batch, beams, N) bytes, from
 *               dvl_workspace_init.
 * Errors: DVL_ERR_INVALID_ARG, DVL_ERR_WORKSPACE, DVL_ERR_CUDA. */
dvl_status dvl_beam_select(const void *logits, int32_t dtype, int64_t batch_stride,
                           int64_t beam_stride, const float *scores, int32_t batch, int32_t beams,
                           int32_t N, int32_t k, const int32_t *d2t, float *out_scores,
                           int32_t *parents, int32_t *tokens, void *ws, size_t ws_bytes,
                           void *stream);

/* One tensor of per-beam rows: src [batch][beams] rows, dst [batch][k] rows,
 * each row row_bytes consecutive bytes. */
typedef struct dvl_state {
    const void *src;
    void *dst;
    int64_t row_bytes;  /* >= 1 */
    int64_t src_stride; /* bytes from one beam's row to the next (beams * src_stride per request) */
    int64_t dst_stride;
} dvl_state;

/* The page tables of beams that share a paged cache. */
typedef struct dvl_beam_pages {
    const int32_t *table;   /* [batch][beams][width] contiguous                   */
    int32_t *table_out;     /* [batch][k][width] contiguous (out)                 */
    const int32_t *lengths; /* [batch][beams]: cached tokens of each beam         */
    int32_t *lengths_out;   /* [batch][k] (out)                                   */
    const int32_t *spare;   /* [batch][k]: a page of the pool for each new beam,
                               each different and in no table                     */
    int32_t width;
    int32_t reserved;       /* must be 0                                          */
} dvl_beam_pages;

/* Reorder what belongs to a beam after a selection: new beam i of request b
 * takes the rows of its parent,
 *   dst[b][i] = src[b][parents[b][i]]   for every state,
 * and zeros where the parent is outside [0, beams) (an unused slot).  With
 * pages, table_out and lengths_out take the parent's rows the same way, and
 * the new beam gets a page of its own for the token it will append: with
 * L = the parent's length, s = L / page_size and r = L % page_size, page
 * spare[b][i] receives the first r tokens of the parent's page s (keys and
 * values) and table_out[b][i][s] = spare[b][i] (when s < width).  Full pages
 * stay shared.  An unused slot's table of zeros names page 0: a caller that
 * keeps appending to such a slot puts a page of its own there first.  One
 * launch.
 *   states:  HOST array of n_states (0 .. DVL_MAX_STATES), device pointers.
 *   pages:   HOST struct, or NULL; cache goes with it.
 *   parents: device int32 [batch][k].
 *   batch:   >= 0 (0 enqueues nothing).  beams, k: 1 .. DVL_MAX_BEAMS.
 * A page id outside the pool (a parent's or a spare one) copies nothing.
 * Rows are copied in no order: a row of an output (of a state, table_out,
 * lengths_out) may share no byte with a row of any input (of any state, table,
 * lengths, spare, parents) or of another output; it is refused.  Rows of one
 * tensor may lie between another's.
 * Errors: DVL_ERR_INVALID_ARG, DVL_ERR_CUDA. */
dvl_status dvl_beam_reorder(const dvl_state *states, int32_t n_states, const dvl_beam_pages *pages,
                            const dvl_kv_cache *cache, const int32_t *parents, int32_t batch,
                            int32_t beams, int32_t k, void *stream);

/* ---------------------------------------------------------------------- */
/* Load time                                                              */
/* ---------------------------------------------------------------------- */

/* Trim a full head to the rows a ranks list names, in the list's order:
 * W_trim[i] = W_full[ranks[i]] (byte copy of the row, in any dtype; for NVFP4 the codes
 * and the scales), d2t[i] = ranks[i].  The ranks are checked on the host
 * before anything is enqueued; duplicates are accepted (padded lists exist)
 * and counted.
 *   full:      the full head: N == V, d2t == NULL, id_base == 0.
 *   ranks:     HOST int32 [n_ranks], each in [0, V).
 *   n_ranks:   >= 1.
 *   w_trim:    device, rows of the same format: bf16 [n][K] or codes [n][K/2].
 *   scales_trim: device E4M3 [n][K/16] for NVFP4; NULL for bf16.
 *   d2t:       device int32 [n_ranks] (out); the trimmed head's d2t.
 *   n_duplicates: HOST (out, may be NULL): entries that repeat an earlier id.
 * The ranks are copied to d2t with a host-to-device copy from pageable
 * memory, which returns once the source has been read.
 * Errors: DVL_ERR_INVALID_ARG, DVL_ERR_OUT_OF_RANGE (nothing enqueued),
 * DVL_ERR_CUDA. */
dvl_status dvl_trim_head(const dvl_head *full, const int32_t *ranks, int32_t n_ranks,
                         void *w_trim, uint8_t *scales_trim, int32_t *d2t,
                         int32_t *n_duplicates, void *stream);

/* Requantize a bf16 head to NVFP4 or FP8 at load ("Masked MTP drafts": the
 * trimmed head requantized to NVFP4 at no measured acceptance cost; the
 * pages give no recipe).  In fp32, each operation rounded once, in order:
 *   NVFP4: g = amax / (6 * 448); per 16 consecutive weights of a row
 *          s = RNE_e4m3(amax_b / (6 g)), code = RNE_e2m1(w / (s g)), all
 *          codes 0 when s is 0;
 *   FP8:   g = amax / 448; code = RNE_e4m3(w / g);
 * amax is the head's largest |w| (g = 1 for an all-zero head); RNE rounds
 * to the nearest value of the format, ties to even, saturating at its
 * largest finite value; a code's sign is its quotient's.  The weights must
 * be finite.
 *   src:    a bf16 head (only dtype, N, K and w are read).
 *   dtype:  DVL_NVFP4 or DVL_FP8.
 *   codes:  device, 16-byte aligned: NVFP4 [N][K/2] (low nibble = even k) or
 *           FP8 [N][K].
 *   scales: device, 16-byte aligned NVFP4 E4M3 [N][K/16]; NULL for FP8.
 *   global_scale: HOST float (out): g.
 *   ws:     a workspace from dvl_workspace_init (at least
 *           dvl_workspace_bytes(1, 1) bytes); left as it was found.
 * This load-time call synchronizes `stream` once, to read amax back.
 * Errors: DVL_ERR_INVALID_ARG, DVL_ERR_WORKSPACE, DVL_ERR_CUDA. */
dvl_status dvl_quantize_head(const dvl_head *src, int32_t dtype, void *codes, uint8_t *scales,
                             float *global_scale, void *ws, size_t ws_bytes, void *stream);

/* Learn escaped ids into spare rows of a trimmed head while serving ("Masked
 * MTP drafts", section "Update (November 2026)": a static trim can miss;
 * the server learns the escaped ids into spare head rows).  For i < n:
 *   W_trim[row0 + i] = W_full[ids[i]] (the row's bytes; NVFP4 codes and
 *   scales), d2t[row0 + i] = ids[i],
 * the same copy as dvl_trim_head, into rows row0 .. row0 + n - 1.  Allocate
 * the trimmed buffers with room for the rows they may learn; a head of
 * row0 + n rows over the same buffers then includes the learned ids.
 *   full:   the full head: N == V, d2t == NULL, id_base == 0.
 *   ids:    HOST int32 [n], each in [0, V), checked before anything is
 *           enqueued (DVL_ERR_OUT_OF_RANGE).
 *   n:      >= 1.   row0: >= 0, with row0 + n < 2^31.
 *   w_trim, scales_trim (NVFP4; NULL for bf16), d2t: the trimmed head's
 *           device buffers from their row 0 (not offset); the caller owns
 *           them and sizes them for rows up to row0 + n (not checkable here).
 * Ordering: rows and d2t entries are written by kernels on `stream`; later
 * calls on that stream see them.  The first reducing call after the learn
 * on that stream must not set DVL_HEAD_STATIC on the trimmed head (the flag
 * lets a kernel read the head before the preceding kernel has finished);
 * later calls may set it again.  The ids are copied from pageable memory;
 * the call returns once they have been read.
 * Errors: DVL_ERR_INVALID_ARG, DVL_ERR_OUT_OF_RANGE (nothing enqueued),
 * DVL_ERR_CUDA. */
dvl_status dvl_learn_rows(const dvl_head *full, const int32_t *ids, int32_t n, int32_t row0,
                          void *w_trim, uint8_t *scales_trim, int32_t *d2t, void *stream);

/* The whole repair step of a shortlist that learns while serving ("Masked
 * MTP drafts", section "Update (November 2026)": the ids a static trim
 * missed, learned into spare head rows): given the ids the target emitted,
 * pick those the list does not hold -- each id's first occurrence, in the
 * order given, while spare rows remain -- and copy them in as
 * dvl_learn_rows does, into rows *n_rows, *n_rows + 1, ...
 *   full:     the full head: N == V, d2t == NULL, id_base == 0.
 *   ids:      HOST int32 [n], each in [0, V), in any order, repeats allowed
 *             (n may be 0).
 *   row_of:   HOST int32 [V] (in/out): the trimmed row that holds id t, or
 *             -1 for an id the list lacks; learned ids get their rows.
 *   n_rows:   HOST (in/out): rows in use; the first spare row.
 *   capacity: rows the trimmed buffers hold (>= *n_rows).
 *   w_trim, scales_trim (NVFP4; NULL otherwise), d2t: the trimmed head's
 *             device buffers from row 0, sized for `capacity` rows.
 *   learned:  HOST int32 [n] (out): the ids learned, in row order; also the
 *             source of the d2t copy, read before the call returns.
 *   n_learned: HOST (out): how many.
 * Nothing is enqueued when nothing is learned.  Ordering as for
 * dvl_learn_rows: the first reducing call after a learn on that stream
 * must not set DVL_HEAD_STATIC on the trimmed head.  The host work is
 * O(n); nothing is allocated.
 * Errors: DVL_ERR_INVALID_ARG, DVL_ERR_OUT_OF_RANGE (an id outside [0, V):
 * nothing changed, nothing enqueued), DVL_ERR_CUDA (row_of and *n_rows
 * unchanged). */
dvl_status dvl_learn_missing(const dvl_head *full, const int32_t *ids, int32_t n,
                             int32_t *row_of, int32_t *n_rows, int32_t capacity, void *w_trim,
                             uint8_t *scales_trim, int32_t *d2t, int32_t *learned,
                             int32_t *n_learned, void *stream);

/* ---------------------------------------------------------------------- */
/* Host-only ranks builder (no GPU involved)                              */
/* ---------------------------------------------------------------------- */

/* counts[t] += 1 for every token t of tokens[0..n).  All host memory.
 * DVL_ERR_OUT_OF_RANGE (nothing counted) if a token lies outside [0, V). */
dvl_status dvl_histogram(const int32_t *tokens, int64_t n, int64_t V, int64_t *counts);

/* A shortlist of N ids from a histogram: the distinct forced ids first, in
 * rank order, then the other ids in rank order, cut at N (rank order =
 * higher count first, then lower id).  sorted != 0 sorts the result by id.
 * All host memory; ranks_out holds min(N, V) entries; *n_out receives that
 * count.  DVL_ERR_OUT_OF_RANGE if a forced id lies outside [0, V). */
dvl_status dvl_build_ranks(const int64_t *counts, int64_t V, const int32_t *forced,
                           int32_t n_forced, int32_t N, int32_t sorted,
                           int32_t *ranks_out, int32_t *n_out);

/* The sorted set union of two id lists (each taken as a set).  All host
 * memory; out holds na + nb entries; *n_out receives the union's size. */
dvl_status dvl_union_sorted(const int32_t *a, int32_t na, const int32_t *b, int32_t nb,
                            int32_t *out, int32_t *n_out);

#ifdef __cplusplus
}
#endif
#endif /* DVL_H */
