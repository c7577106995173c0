/*
 * moe_ep.h -- C ABI of the MI355X (gfx950) MoE expert-parallel exchange.
 *
 * One call covers all P *virtual* EP ranks that share one GPU's HBM: every
 * per-rank tensor of the exchange is stacked over ranks, and every rank
 * owns one region of a [P][size_per_rank] workspace (the workspace shape of
 * FlashInfer's moe_a2a_dispatch, "workspace" parameter).
 *
 * Semantics follow these documentation pages:
 *  - FlashInfer "flashinfer.moe_ep.NVLinkTwoSidedAlltoAll": dispatch()
 *    delivers every token to each rank that holds one of its chosen
 *    experts, together with the token's top-k ids, top-k weights and scale
 *    row; combine() adds up, over ranks, each token's expert outputs
 *    (each rank having weighted them and summed over its own experts); destroy() is
 *    idempotent; is_platform_supported() performs no collective work.
 *  - FlashInfer "flashinfer.moe_ep.NVLinkOneSidedConfig", lamport
 *    paragraph: token t of rank src lands in slot src * tokens_per_rank + t
 *    of a receiving rank, where tokens_per_rank equals the step's
 *    runtime_max_tokens_per_rank; BF16, MXFP8 and NVFP4 dispatch formats;
 *    at most 64 EP ranks.  First options paragraph: with
 *    use_low_precision_combine the combine moves its rows as FP8 values.
 *    cft paragraph: a payload row's size is a whole number of 16-byte
 *    units.
 *  - FlashInfer "flashinfer.comm.moe_a2a_dispatch": runtime_max_tokens_per_rank
 *    may not exceed the capacity given at initialisation; the outputs are
 *    views into the workspace, one per payload, and the workspace offset
 *    that the combine of the same step will use.
 *  - vLLM "device_communicators.all2all", FlashInferNVLinkTwoSidedManager:
 *    MoEEpCommParams(num_experts, top_k, max_tokens_per_rank, hidden_size,
 *    invalid_expert_id=num_experts); a received row without a token is
 *    marked with expert id invalid_expert_id, an id outside every rank's
 *    range.
 *  - vLLM "device_communicators.all2all", AgRsAll2AllManager: dispatch is
 *    all_gatherv of [hidden, topk_weights, topk_ids] along dim 0 with
 *    per-rank sizes; combine is reduce_scatterv of the hidden rows with
 *    the same sizes (combine_into_output: into a caller buffer).
 *
 * Readings taken where the pages are silent:
 *  - expert e lives on rank e / (E / P) (contiguous blocks; E % P == 0);
 *    ids outside [0, E) route nowhere but are still forwarded;
 *  - a token reaches a rank once however many of its experts live there;
 *  - every receive slot without a token carries invalid_expert_id in all
 *    k id entries after each dispatch (its payload, scale and weight bytes
 *    are left as they were);
 *  - combine sums in fp32 and rounds to bf16 to nearest-even;
 *  - the FP8 combine payload is OCP e4m3fn with one e8m0 scale per 32
 *    elements, the scale being the smallest power of two keeping the
 *    block's magnitudes within 448 (no saturation ever happens).
 *
 * Ownership: the caller owns every buffer (workspace, inputs, outputs).
 * The library allocates no device memory.  A handle keeps the last
 * dispatch's step size and per-rank token counts; combine uses them.
 * Handles are not thread-safe.  All launches go to the caller's stream,
 * in stream order, with no host synchronisation, and may be captured into
 * a HIP graph: the host-side arguments of a call (per-rank token counts,
 * the step size, the active rank mask, buffer pointers) are fixed into the
 * captured launches, so a graph replays exactly the calls it captured and
 * must be captured again when they change.
 *
 * Errors: every entry point validates all arguments before launching
 * anything (no partial launches) and returns one of the MOE_EP_* codes
 * below; moe_ep_last_error() gives a message for the calling thread.
 */
#ifndef MOE_EP_H
#define MOE_EP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_EP_OK 0
#define MOE_EP_ERR_INVALID_ARG (-1) /* bad argument or shape             */
#define MOE_EP_ERR_UNSUPPORTED (-2) /* no gfx950 device / format         */
#define MOE_EP_ERR_BAD_STATE (-3)   /* e.g. combine before any dispatch  */
#define MOE_EP_ERR_CAPACITY (-4)    /* workspace or step too large       */
#define MOE_EP_ERR_HIP (-5)         /* a HIP runtime call failed         */

#define MOE_EP_MAX_RANKS 64         /* one 64-bit destination mask word  */
#define MOE_EP_MAX_TOP_K 64

/* Dispatch payload formats (NVLinkOneSidedConfig, lamport paragraph). */
#define MOE_EP_FMT_BF16 0  /* row = 2H bytes, no scale row               */
#define MOE_EP_FMT_MXFP8 1 /* row = H e4m3 bytes, scale row = H/32 e8m0  */
#define MOE_EP_FMT_NVFP4 2 /* row = H/2 packed e2m1, scale row = H/16 e4m3 */
#define MOE_EP_FMT_DEEPSEEK_FP8 3 /* row = H e4m3, scale row = H/128 fp32 (1x128 blocks) */

/* Combine payload formats. */
#define MOE_EP_COMBINE_BF16 0
#define MOE_EP_COMBINE_FP8 1 /* e4m3fn + e8m0 per 32 on the wire */

/* Exchange parameters (vLLM MoEEpCommParams + NVLinkOneSidedConfig). */
typedef struct moe_ep_params {
    int32_t ep_size;             /* P, 1..64                                   */
    int32_t num_experts;         /* E, E % 4 == 0 and E % P == 0               */
    int32_t top_k;               /* k, 1..64                                   */
    int32_t max_tokens_per_rank; /* capacity C >= 1                            */
    int32_t hidden_size;         /* H: BF16 H % 8 == 0; MXFP8/NVFP4/FP8 combine H % 32 == 0 */
    int32_t dispatch_format;     /* MOE_EP_FMT_*                               */
    int32_t combine_format;      /* MOE_EP_COMBINE_*                           */
    int32_t has_weights;         /* 1: top-k weights travel with tokens        */
    int32_t invalid_expert_id;   /* id written to empty slots (usually E)      */
    int32_t extra_payload_bytes_per_token; /* >= 0: room for extra bytes per token */
    int32_t eplb_stats_num_experts; /* n in [0, num_experts] of the EPLB statistics
                                       all-gather (0: none)                        */
} moe_ep_params;

/* Where a dispatch's receive planes live.  Plane X of rank r starts at
 * workspace + r * region_bytes + X_offset; slot q of that plane at
 * X_offset + q * (row bytes of X).  q = src * tokens_per_rank + t.
 * Views stay valid until the next dispatch on the handle. */
typedef struct moe_ep_dispatch_views {
    int32_t tokens_per_rank;     /* T of this step                            */
    int32_t ep_size;             /* P                                         */
    int64_t region_bytes;        /* size_per_rank                             */
    int64_t payload_offset;      /* [P*T][payload_row_bytes] token rows       */
    int64_t payload_row_bytes;
    int64_t scales_offset;       /* [P*T][scale_row_bytes] (0 bytes if none)  */
    int64_t scale_row_bytes;
    int64_t ids_offset;          /* [P*T][k] int32 global expert ids          */
    int64_t weights_offset;      /* [P*T][k] fp32 (meaningful if has_weights) */
    int64_t slots_offset;        /* [P*T] int32: valid q ascending, first recv_total entries */
    int64_t counts_offset;       /* [P] int32 rows received from each source  */
    int64_t src_offsets_offset;  /* [P+1] int32 exclusive prefix of counts; [P] = recv_total */
    int64_t combine_payload_offset; /* FP8 combine landing codes [P*T][H], or -1 */
    int64_t combine_scales_offset;  /* FP8 combine landing scales [P*T][H/32], or -1 */
    int64_t extra_offset;        /* [P*T][extra_row_bytes] extra per-token bytes */
    int64_t extra_row_bytes;     /* extra_payload_bytes_per_token (0: none)   */
    int64_t eplb_offset;         /* [P][n] int32 gathered statistics (row s = rank s),
                                    -1 when this dispatch carried none        */
    int64_t eplb_num_experts;    /* n                                         */
} moe_ep_dispatch_views;

typedef struct moe_ep_handle moe_ep_handle;

/* 1 when the current HIP device is a gfx950 GPU, else 0.  Collective-free
 * (NVLinkTwoSidedAlltoAll.is_platform_supported). */
int moe_ep_is_supported(void);

/* size_per_rank of the [ep_size, size_per_rank] workspace
 * (moe_a2a_dispatch, workspace parameter; NVLinkOneSidedConfig, first
 * options paragraph: the dispatch workspace holds each token's activations
 * in the dispatch format plus its routing, extra_payload_bytes_per_token
 * more bytes per token and the EPLB statistics): bytes of one rank's
 * region for these parameters, every plane 256-byte aligned.  0 when the
 * parameters are invalid (see moe_ep_last_error), including a region above
 * 2^46 bytes or more than 2^31 - 1 slots (ep_size * max_tokens_per_rank),
 * which moe_ep_create rejects with MOE_EP_ERR_CAPACITY.  Host-only, no
 * device work. */
size_t moe_ep_workspace_bytes(const moe_ep_params *params);

/* Create a handle (NVLinkOneSidedConfig, first paragraph: a communication
 * is made by create_communication with the exchange's parameters and
 * backend options; vLLM FlashInferNVLinkTwoSidedManager: MoEEpCommParams)
 * over a caller-owned device workspace of P regions of size_per_rank bytes
 * each (region r at workspace + r * size_per_rank, size_per_rank >=
 * moe_ep_workspace_bytes and a multiple of 256, workspace 256-byte
 * aligned).  The workspace needs no initialisation; the handle keeps host
 * state only.  Errors: MOE_EP_ERR_INVALID_ARG (bad parameters, NULL or
 * misaligned workspace), MOE_EP_ERR_CAPACITY (region too small or too
 * large), MOE_EP_ERR_UNSUPPORTED (no gfx950 device current). */
int moe_ep_create(const moe_ep_params *params, void *workspace, size_t size_per_rank,
                  moe_ep_handle **out);

/*
 * Dispatch (NVLinkTwoSidedAlltoAll.dispatch / moe_a2a_dispatch).
 *  hidden            device [P][T][payload_row_bytes], 16-byte aligned;
 *                    row t of rank s is token t of rank s
 *  scales            device [P][T][scale_row_bytes]; required for MXFP8 /
 *                    NVFP4 / DeepSeekFp8, must be NULL for BF16
 *  extra_payload     device [P][T][extra_payload_bytes_per_token] or NULL:
 *                    more bytes per token, forwarded like the scale row
 *                    (NVLinkOneSidedConfig, extra_payload_bytes_per_token)
 *  eplb_local_stats  device [P][eplb_stats_num_experts] int32 or NULL: each
 *                    rank's per-expert counters for load balancing; every live rank receives
 *                    the [P][n] matrix (row s = rank s's statistics) in its
 *                    region (moe_a2a_dispatch, eplb_local_stats ->
 *                    eplb_gathered_stats)
 *  topk_ids          device [P][T][k] int32 global expert ids
 *  topk_weights      device [P][T][k] fp32; required iff has_weights
 *  num_tokens        host [P]: local_num_tokens n_s, 0 <= n_s <= T
 *  runtime_max_tokens_per_rank  T (the step's tokens_per_rank); <= 0
 *                    means the capacity; T <= capacity
 *  active_rank_mask  host, one word (NULL = every rank): bit r set when
 *                    rank r takes part in the step (moe_a2a_dispatch,
 *                    active_rank_mask).  A masked-off rank neither sends
 *                    nor receives: tokens routed to it are dropped, nothing
 *                    is written into its region, and the following combine
 *                    produces no rows for it.  Bits >= P must be clear.
 *  views             out (may be NULL): where the receive planes are
 * Rows t >= n_s of the inputs are never read.  Writes, for every rank r and
 * slot q = s*T + t: the token's payload row, scale row, k ids and k weights
 * when t < n_s and r owns one of its experts; otherwise k copies of
 * invalid_expert_id in the ids plane.  Also per-destination counts, source
 * offsets and the ascending list of valid slots.
 */
int moe_ep_dispatch(moe_ep_handle *h, const void *hidden, const void *scales,
                    const void *extra_payload, const int32_t *eplb_local_stats,
                    const int32_t *topk_ids, const float *topk_weights,
                    const int32_t *num_tokens, int32_t runtime_max_tokens_per_rank,
                    const uint64_t *active_rank_mask, void *stream,
                    moe_ep_dispatch_views *views);

/*
 * Combine (NVLinkTwoSidedAlltoAll.combine) of the last dispatch (and of
 * its active rank mask).
 *  expert_output  device [P][P*T][H] bf16: rank r's row for slot q at
 *                 (r*P*T + q)*H; only slots that received a token are read
 *  output         device [P][T][H] bf16: row t of rank s receives the sum
 *                 over ranks r that got token (s, t) of expert_output[r][s*T+t]
 *                 (fp32 accumulation from +0 in ascending rank order, RNE to
 *                 bf16); rows t >= n_s untouched
 * With MOE_EP_COMBINE_FP8 each sending rank first quantises its rows into
 * the source rank's landing plane (e4m3fn + e8m0 per 32), and the sum is
 * taken over the dequantised rows.
 */
int moe_ep_combine(moe_ep_handle *h, const void *expert_output, void *output, void *stream);

/*
 * moe_ep_combine for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid it): the
 * same combine of the last dispatch, with the same arguments and result,
 * but an FP8 combine stages its landing planes (e4m3 codes [P][P*T][H],
 * then e8m0 scales [P][P*T][H/32], per source rank) in the library's own
 * static device array of MOE_EP_STATIC_SCRATCH_BYTES instead of the
 * workspace; a BF16 combine stages nothing and runs as moe_ep_combine.
 * Allocates nothing (no hipMalloc, no allocating library call).
 *  - MOE_EP_ERR_CAPACITY when the step's landing planes,
 *    P * round_up_256(P*T*(H + H/32)) bytes for the last dispatch's T,
 *    exceed the array (e.g. P = 8, H = 7168 fits up to T = 128);
 *  - each GPU holds one array from library load until the process ends,
 *    shared by every call on that GPU; it keeps the last call's contents
 *    and needs no clearing (every landing row a call reads, it writes
 *    first), so calls on one GPU that overlap in time (other streams, other
 *    threads) race on it;
 *  - the workspace's landing-plane views (combine_payload_offset) are not
 *    written by this call.
 */
#define MOE_EP_STATIC_SCRATCH_BYTES (64ll << 20)
int moe_ep_combine_noalloc(moe_ep_handle *h, const void *expert_output, void *output, void *stream);

/* Release the handle.  Idempotent and NULL-safe; frees no caller memory. */
int moe_ep_destroy(moe_ep_handle *h);

/* One plane of an all-gatherv: rank q's sizes[q] input rows start at
 * in + q * in_rank_stride; rank r's gathered [sum(sizes)][row_bytes]
 * output starts at out + r * out_rank_stride. */
typedef struct moe_ep_plane {
    const void *in;
    int64_t in_rank_stride;      /* bytes */
    void *out;
    int64_t out_rank_stride;     /* bytes */
    int64_t row_bytes;           /* > 0 */
} moe_ep_plane;

/*
 * all_gatherv along dim 0 (AgRsAll2AllManager.dispatch): every rank r
 * receives, for every plane, the concatenation in rank order of each rank
 * q's first sizes[q] rows.  sizes: host [P], >= 0; 1 <= num_planes <= 8.
 */
int moe_ep_allgatherv(int32_t ep_size, const int32_t *sizes, int32_t num_planes,
                      const moe_ep_plane *planes, void *stream);

/*
 * reduce_scatterv along dim 0 (AgRsAll2AllManager.combine /
 * combine_into_output): rank q's full-length bf16 partial [sum(sizes)][H]
 * starts at in + q * in_rank_stride (bytes); rank r's result
 * [sizes[r]][H] at out + r * out_rank_stride (bytes) is the fp32 sum over
 * q (from +0, ascending q) of rows off_r .. off_r + sizes[r] - 1
 * (off_r = sum of sizes[q < r]), rounded to bf16 (RNE).
 */
int moe_ep_reduce_scatterv(int32_t ep_size, const int32_t *sizes, int32_t hidden_size,
                           const void *in, int64_t in_rank_stride, void *out,
                           int64_t out_rank_stride, void *stream);

/* ---------------------------------------------------------------------
 * The expert layer between a dispatch and its combine, and the norm that
 * makes the next layer's payload.  These calls need no handle and keep no
 * state: the caller owns every buffer, launches go to the caller's stream
 * without host synchronisation, nothing is allocated, and a call may be
 * captured into a HIP graph.  Buffers belong to the current HIP device; an
 * output overlaps no other buffer of its call unless stated otherwise.
 * Calls whose output, workspace or index buffers overlap must be ordered by
 * the caller; calls on buffers of their own may run at the same time.  A call
 * that launches clears an error that an earlier HIP call of its thread left
 * pending (hipGetLastError), and does not report it as its own.
 * Every call takes one argument block, all pointers device pointers.
 * --------------------------------------------------------------------- */

#define MOE_EP_BF16_ROWS 0 /* element types of the expert layer's rows   */
#define MOE_EP_FP32_ROWS 1

#define MOE_EP_MAX_SORT_EXPERTS 4096 /* ranks * experts_per_rank          */

/*
 * Expert sort: rows to expert order.  Slot q of rank r holds one row and
 * top_k global expert ids (the planes that a dispatch leaves in rank r's
 * region; with ranks = 1 simply a batch of tokens).  A pair (r, q, j) counts
 * when its id lies on its rank: r*e <= id < (r+1)*e, e = experts_per_rank;
 * other ids (other ranks' experts, the invalid id, anything out of range)
 * are passed over, and so are all ids of the ranks in masked_ranks: a
 * dispatch leaves a masked-off rank's region as it was, earlier steps' ids
 * among it.  Counted pairs are placed by ascending (id, q, j): the
 * order depends on the ids alone.
 *  position  [R][S][k]: a pair's place, -1 where it has none
 *  counts    [R*e]: pairs of each expert
 *  offsets   [R*e + 1]: exclusive prefix of counts, clamped to capacity;
 *            expert x's rows are offsets[x] .. offsets[x+1] - 1
 *  out_rows, out_scales: row position[r][q][j] is a copy of the row and
 *            scale row of (r, q); rows from offsets[R*e] on are left alone.
 * Pairs from place `capacity` on are dropped (position -1, not in offsets;
 * counts still holds them), so no row is written past the capacity.
 * capacity >= sum over ranks of num_tokens * k never drops one after a
 * dispatch.  An id that a row carries twice gives two pairs.
 * quantize = 1: rows are row_type elements, row_bytes of them, and out_rows
 * holds int8 codes with out_scales one fp32 scale a row: scale = amax / 127,
 * code = row / scale rounded to nearest even (scale 0 and codes 0 for a row
 * of zeros; scale NaN and codes 0 for a row with a NaN or an infinity).
 * row_bytes: a multiple of 16 up to 2^24, with quantize also of 16 elements;
 * scale_row_bytes: any size up to 2^24.  workspace: moe_ep_expert_sort_workspace_bytes(),
 * 16-byte aligned, for this call alone.
 * Limits: ranks 1..64, slots >= 0, top_k 1..64, ranks*experts_per_rank in
 * 1..4096, ranks*slots*top_k and capacity below 2^31.
 */
typedef struct moe_ep_sort_args {
    const int32_t *ids;          /* [R][S][k]                                */
    int64_t ids_rank_stride;     /* bytes from rank to rank                  */
    const void *rows;            /* [R][S][row_bytes]                        */
    int64_t rows_rank_stride;
    int64_t row_bytes;
    const void *scales;          /* [R][S][scale_row_bytes] or NULL          */
    int64_t scales_rank_stride;
    int64_t scale_row_bytes;
    void *out_rows;              /* [capacity][row_bytes], int8 [capacity][H] */
    void *out_scales;            /* [capacity][scale_row_bytes], fp32 [capacity] */
    int32_t *position;
    int32_t *offsets;
    int32_t *counts;
    void *workspace;
    int64_t workspace_bytes;
    int64_t capacity;
    int32_t ranks;
    int32_t slots;
    int32_t top_k;
    int32_t experts_per_rank;
    int32_t quantize;            /* 0: copy, 1: int8 codes and scales        */
    int32_t row_type;            /* MOE_EP_*_ROWS, read when quantize = 1    */
    uint64_t masked_ranks;       /* bit r: rank r's slots hold nothing; bits >= R clear */
} moe_ep_sort_args;

/* Bytes of workspace an expert sort of this shape needs (0: none; -1: bad
 * shape, see moe_ep_last_error).  Host-only. */
int64_t moe_ep_expert_sort_workspace_bytes(int32_t ranks, int32_t slots, int32_t top_k,
                                           int32_t experts_per_rank);

int moe_ep_expert_sort(const moe_ep_sort_args *args, void *stream);

/*
 * Expert unsort: out[r][q] = sum over j of weights[r][q][j] *
 * rows[position[r][q][j]] (weights NULL: 1), fp32 from +0 in ascending j,
 * rounded once to row_type.  Pairs with a position outside [0, num_rows)
 * add nothing; a slot without any is filled with zeros (keep_empty = 0) or
 * left alone (keep_empty = 1: a combine never reads a slot without a token,
 * but it does read one whose pairs a capacity dropped, so that a sort that
 * may drop pairs goes with 0).  With weights
 * NULL it is the gradient of the expert sort.  hidden_size elements a row, a
 * multiple of 16 bytes up to 2^24.
 */
typedef struct moe_ep_unsort_args {
    const int32_t *position;     /* [R][S][k], contiguous                    */
    const void *rows;            /* [num_rows][H]                            */
    const float *weights;        /* [R][S][k] or NULL                        */
    int64_t weights_rank_stride; /* bytes                                    */
    void *out;                   /* [R][S][H]                                */
    int64_t out_rank_stride;     /* bytes                                    */
    int64_t num_rows;
    int32_t ranks;
    int32_t slots;
    int32_t top_k;
    int32_t hidden_size;
    int32_t row_type;
    int32_t keep_empty;
} moe_ep_unsort_args;

int moe_ep_expert_unsort(const moe_ep_unsort_args *args, void *stream);

/*
 * Gradient of the expert unsort, for grad_out [R][S][H]:
 *  grad_rows[position[r][q][j]] = weights[r][q][j] * grad_out[r][q],
 *            rounded once (rows that no pair names are left alone); or NULL
 *  grad_weights[r][q][j] = sum over h of rows[position[r][q][j]][h] *
 *            grad_out[r][q][h] in fp32, in an order that the shape alone
 *            fixes, 0 for a pair without a row; or NULL
 * A place may appear in `position` once, as the sort makes it.
 */
typedef struct moe_ep_unsort_grad_args {
    const int32_t *position;     /* [R][S][k], contiguous                    */
    const void *grad_out;        /* [R][S][H]                                */
    int64_t grad_out_rank_stride;
    const void *rows;            /* [num_rows][H], needed for grad_weights   */
    const float *weights;        /* [R][S][k] or NULL                        */
    int64_t weights_rank_stride;
    void *grad_rows;             /* [num_rows][H] or NULL                    */
    float *grad_weights;         /* [R][S][k], contiguous, or NULL           */
    int64_t num_rows;
    int32_t ranks;
    int32_t slots;
    int32_t top_k;
    int32_t hidden_size;
    int32_t row_type;
    int32_t reserved;            /* 0                                        */
} moe_ep_unsort_grad_args;

int moe_ep_expert_unsort_backward(const moe_ep_unsort_grad_args *args, void *stream);

/*
 * Product of int8 rows with each expert's int8 weights:
 *  out[m][n] = x_scales[m] * w_scales[e][n] * sum over k of x[m][k] * w[e][n][k]
 * for the rows offsets[e] <= m < offsets[e+1] of every expert e, the sum
 * exact in int32, the scaling in fp32 ((sum * w_scale) * x_scale, so that rows
 * of any magnitude keep their result), one rounding to out_type.  offsets
 * [E + 1] ascends and is read on the device, each entry taken as at most
 * num_rows; rows outside every expert's range are left alone.  offsets NULL:
 * a dense product, num_experts = 1 and every row.  k a multiple of 16 and at
 * most 131056 (|sum| < 2^31 also at -128 * -128); n >= 1; x and w 16-byte
 * aligned and contiguous.
 */
typedef struct moe_ep_matmul_args {
    const int8_t *x;             /* [num_rows][k]                            */
    const float *x_scales;       /* [num_rows]                               */
    const int8_t *w;             /* [E][n][k]                                */
    const float *w_scales;       /* [E][n]                                   */
    const int32_t *offsets;      /* [E + 1] or NULL                          */
    void *out;                   /* [num_rows][n]                            */
    int64_t num_rows;
    int32_t num_experts;
    int32_t n;
    int32_t k;
    int32_t out_type;            /* MOE_EP_*_ROWS                            */
} moe_ep_matmul_args;

int moe_ep_expert_matmul(const moe_ep_matmul_args *args, void *stream);

/*
 * Gated activation between the two expert products: for the first
 * min(*num_valid, num_rows) rows (num_valid NULL: all; offsets + E of the
 * sort), a = silu(x[:, :I]) * x[:, I:] in fp32, as int8 codes and one scale
 * a row (as the quantising sort's); other rows are left alone.  silu(g) is
 * g / (1 + exp(-g)), relative error up to (2 |g| + 10) * 2^-24; where exp(-g)
 * passes fp32 (g below -88.7) it is -0, and NaN for g = -infinity.  I a
 * multiple of 16, at most 32768.
 */
typedef struct moe_ep_silu_args {
    const void *x;               /* [num_rows][2 * I] row_type               */
    const int32_t *num_valid;    /* one device int32, or NULL                */
    int8_t *out;                 /* [num_rows][I]                            */
    float *out_scales;           /* [num_rows]                               */
    int64_t num_rows;
    int32_t inter_size;          /* I                                        */
    int32_t row_type;
} moe_ep_silu_args;

int moe_ep_silu_mul_quantize(const moe_ep_silu_args *args, void *stream);

#define MOE_EP_NORM_INT8 0        /* int8 codes, one fp32 scale a row         */
#define MOE_EP_NORM_MXFP8 1       /* the MXFP8 payload: e4m3, e8m0 a 32-block */
#define MOE_EP_NORM_DEEPSEEK_FP8 2 /* the DeepSeekFp8 payload: e4m3, fp32 a 128-block */

/*
 * Root-mean-square norm with the residual's addition and an 8-bit output:
 *  s = x + residual (residual NULL: x), residual_out = s rounded to row_type,
 *  y = s / sqrt(mean(s^2) + eps) * weight, from the unrounded s, all in fp32,
 *  out / scales = y in `format`:
 *   INT8: scale = amax(y) / 127, as the quantising sort's rows
 *   MXFP8: scale 2^(b - 127), the smallest power of two that keeps the
 *    block's magnitudes within 448 (b = 0 for a block of zeros; the FP8
 *    combine's rule: nothing saturates), code = y / scale to nearest even; a
 *    block with a NaN or an infinity in y has b = 255 and codes 0x7F
 *   DEEPSEEK_FP8: scale = amax / 448, code = y * (448 / amax), product and
 *    quotient each rounded to fp32, to nearest even (scale 0 and codes 0 for
 *    a block of zeros; NaN and codes 0x7F for one with a NaN or an infinity)
 * A row in which s holds a NaN or an infinity, or whose sum of squares passes
 * fp32, has y = NaN throughout; a row of zeros with eps = 0 too.  Squares lose
 * bits below 2^-126 and vanish below 2^-150, which only an eps near 0 shows.
 * H a multiple of 16 (INT8), 32, 128, at most 32768.  residual_out may be
 * residual or x itself; NULL: not written.
 */
typedef struct moe_ep_norm_args {
    const void *x;               /* [num_rows][H] row_type                   */
    const void *residual;        /* [num_rows][H] row_type or NULL           */
    const void *weight;          /* [H] row_type                             */
    void *residual_out;          /* [num_rows][H] row_type or NULL           */
    void *out;                   /* [num_rows][H] bytes                      */
    void *scales;                /* fp32 [num_rows], [num_rows][H/32] bytes,
                                    fp32 [num_rows][H/128]                   */
    int64_t num_rows;
    int32_t hidden_size;
    int32_t row_type;
    int32_t format;              /* MOE_EP_NORM_*                            */
    float eps;                   /* >= 0                                     */
} moe_ep_norm_args;

int moe_ep_add_rms_norm(const moe_ep_norm_args *args, void *stream);

/* Message of the calling thread's last failed call ("" if none). */
const char *moe_ep_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EP_H */
