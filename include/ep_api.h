/*
 * ep_api.h -- C ABI of the GB300 (sm_103a) MoE expert-parallel token
 * layout / dispatch / combine library (libep_gb300.so).
 *
 * What it computes follows the ROCm MORI documentation, "Communication APIs"
 * page, section "MORI-EP (Expert Parallelism)", table "EpDispatchCombineOp
 * methods":
 *   dispatch(input, weights, scales, indices)
 *       -> (output, weights, scales, indices, recv_count)   sends each token
 *          to the ranks that hold its experts
 *   combine(input, weights, indices) -> (output, weights)    brings the
 *          experts' results back to the source tokens
 *   dispatch_send()/dispatch_recv(), combine_send()/combine_recv()  split
 *          phases for overlapping independent work
 *   reset(), get_dispatch_src_token_pos(),
 *   get_registered_combine_input_buffer(dtype)
 * and the "AsyncLL v2 SDMA overlap" section of the same page (send posts the
 * payload, then a ready notification; receive waits, then data and counts
 * are ready on the stream; zero-token peers notify too; the receive step
 * writes the count, zero included; options are frozen at construction).
 *
 * Model.  All W logical EP ranks live in ONE GPU's HBM.  The caller passes
 * one device workspace; the library carves it into a layout-state region and
 * W identical per-rank segments (the symmetric-heap analogue).  A "send" to
 * rank r is a store into segment r.  There is no collective.
 *
 * Notation: W ranks (1..32), E experts (multiple of W), Er = E/W, k = top-k
 * (1..32), T = max tokens per source rank, n_s = tokens present on source
 * rank s in this call (0..T), H = hidden size, cap = receive rows per rank.
 * D(s,t) = { idx[s][t][j] / Er : j < k } is the set of distinct destination
 * ranks of token t on rank s; duplicate experts collapse.
 *
 * Results:
 *  - layout: C[s][r] = #{t < n_s : r in D(s,t)}; recv_count[r] = sum_s
 *    C[s][r]; rows on rank r are ordered by (source rank, source token);
 *    pos[s][t][r] = sum_{s'<s} C[s'][r] + #{t' < t : r in D(s,t')} when
 *    r in D(s,t), else -1.  Deterministic; no atomics decide any position.
 *  - dispatch: row p = pos[s][t][r] of rank r receives x[s][t] (bf16 bits,
 *    or FP8 E4M3 codes plus one fp32 scale per 128 elements with
 *    scale = fl32(amax/448) and q = RNE-satfinite(fl32(x/scale)); an
 *    all-zero block gives scale 0 and codes 0x00; the quantised input is
 *    taken to be finite: a block holding an infinity or a NaN gets an
 *    unspecified scale and codes), all k weights and all k expert ids
 *    unchanged, and src_pos = s*T + t.
 *  - combine: out[s][t] = bf16_rne( fp32 sum over r in D(s,t), r ascending,
 *    starting from +0.0f, of y_r[pos[s][t][r]] ); out_w the same ordered
 *    fp32 sum of the expert-side weight rows.  No weighting is applied.
 *
 * Conventions.
 *  - Pointers named d_* are device pointers, h_* host pointers.  Streams are
 *    cudaStream_t passed as void* (NULL = the legacy default stream).
 *  - Every call after ep_create is asynchronous on the given stream and
 *    allocates nothing (ep_create takes one pinned host word for
 *    ep_get_error).  ep_get_error synchronises the stream it is given.
 *  - Device-side problems (an expert id outside [0,E), a rank receiving more
 *    than cap rows, a wait that timed out, combine indices that differ from
 *    the dispatch's) set bits of a sticky device error word; the kernels skip
 *    the offending entry or row, never write out of bounds and never trap.
 *  - Host-detectable problems return a status at once and launch nothing.
 *
 * Status codes: the first eight mirror the StatusCode enum of the same
 * page's MORI-IO section (SUCCESS, INIT, IN_PROGRESS, ERR_INVALID_ARGS,
 * ERR_NOT_FOUND, ERR_RDMA_OP, ERR_BAD_STATE, ERR_GPU_OP), the only error
 * convention the pages give; EP_ERR_RDMA_OP is never returned here.
 */
#ifndef EP_API_H
#define EP_API_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    EP_SUCCESS = 0,
    EP_INIT = 1,
    EP_IN_PROGRESS = 2,
    EP_ERR_INVALID_ARGS = 3,
    EP_ERR_NOT_FOUND = 4,
    EP_ERR_RDMA_OP = 5,       /* reserved: no RDMA on one GPU */
    EP_ERR_BAD_STATE = 6,     /* call out of order (recv w/o send, ...) */
    EP_ERR_GPU_OP = 7,        /* a CUDA runtime call failed */
    EP_ERR_TIMEOUT = 8,       /* a bounded device wait gave up */
    EP_ERR_CAPACITY = 9,      /* a rank would receive more than cap rows */
    EP_ERR_BAD_INDEX = 10     /* an expert id outside [0, E) */
} ep_status_t;

/* Bits of the device error word (ep_get_error). */
#define EP_DEVERR_BAD_INDEX        0x1u
#define EP_DEVERR_CAPACITY         0x2u
#define EP_DEVERR_TIMEOUT          0x4u
#define EP_DEVERR_COMBINE_MISMATCH 0x8u

typedef enum {
    EP_DT_BF16 = 0,
    EP_DT_FP8_E4M3 = 1,       /* OCP E4M3 ("fn"), max 448 */
    EP_DT_FP32 = 2,
    EP_DT_FP16 = 3            /* routing and expert products only */
} ep_dtype_t;

#define EP_MAX_WORLD 32
#define EP_MAX_TOPK 32
#define EP_QUANT_BLOCK 128

/* Op configuration (the EpDispatchCombineConfig analogue).  Frozen into the
 * handle by ep_create; ops with different options coexist. */
typedef struct {
    int32_t world_size;               /* W, 1..32 */
    int32_t num_experts;              /* E, multiple of W */
    int32_t topk;                     /* k, 1..32 */
    int32_t hidden;                   /* H, multiple of 8 (of 128 for FP8),
                                         8..2^24 (16384 at most for the fused
                                         FP8 dispatch) */
    int32_t max_tokens_per_rank;      /* T >= 1 */
    int32_t max_recv_tokens_per_rank; /* cap; 0 selects W*T (exact worst case) */
    int32_t dispatch_dtype;           /* EP_DT_BF16, or EP_DT_FP8_E4M3 for the
                                         fused per-128-element quantisation */
    int32_t early_notify;             /* 1: the send phase posts per-(source,
                                         destination) ready flags after its
                                         payload, zero-token pairs included;
                                         the receive phase checks them */
    int32_t fused_recv;               /* 1 (needs early_notify): combine's
                                         gather kernel does the receive wait
                                         itself, one warp per CTA, then a CTA
                                         barrier releases the gather warps */
    int32_t combine_dtype;            /* element type of the expert rows that
                                         combine reads: EP_DT_BF16 (0),
                                         EP_DT_FP32, or EP_DT_FP8_E4M3 (codes
                                         + one fp32 scale per 128 elements,
                                         registered buffer only; H % 128 == 0);
                                         the output is bf16 */
    int64_t wait_timeout_ns;          /* bound of every device wait; 0 = 1 s */
    int32_t max_grouped_rows_per_rank;/* rows of the standard-MoE grouped
                                         buffers per rank (0: no grouping);
                                         cap * k is the exact worst case */
    int32_t combine_mode;             /* EP_COMBINE_GATHER (0): combine_recv
                                         gathers the expert rows from the
                                         destination segments.
                                         EP_COMBINE_SCATTER: combine_send pushes
                                         every received row's expert output to a
                                         per-token staging area on the source
                                         side (slot = the rank's order among the
                                         token's destinations) and combine_recv
                                         reduces the staged rows; bf16 rows from
                                         the registered buffer only */
} ep_config_t;

#define EP_COMBINE_GATHER 0
#define EP_COMBINE_SCATTER 1

/* A handle is not thread-safe: drive it from one host thread at a time. */
typedef struct ep_handle ep_handle_t;

/* Device views of the dispatch results (valid until the next dispatch,
 * reset or destroy).  Every per-rank buffer of rank r starts at
 * base + r * rank_stride_bytes; rows hold H payload elements (bf16 or u8),
 * H/128 scales, k weights, k expert ids, one src_pos. */
typedef struct {
    void     *out;            /* [W] x [cap][H]  bf16 or e4m3 codes */
    float    *out_scales;     /* [W] x [cap][H/128]; NULL unless FP8 */
    float    *out_w;          /* [W] x [cap][k] */
    int32_t  *out_idx;        /* [W] x [cap][k] global expert ids */
    int32_t  *src_pos;        /* [W] x [cap]   s*T + t */
    int64_t   rank_stride_bytes;
    int32_t  *recv_count;     /* [W], written by the receive step */
    int32_t  *send_counts;    /* [W][W], C[s][r] */
    int32_t  *pos;            /* [W][T][W], -1 where r is not in D(s,t) */
    uint32_t *dispatch_flags; /* [W dst][W src] ready epochs (early_notify) */
    uint32_t *combine_flags;  /* [W src][W dst] ready epochs (early_notify) */
    uint32_t  dispatch_epoch; /* value the flags carry for the last send */
    uint32_t  combine_epoch;
    int32_t   cap;
    int32_t   max_dest;       /* min(W, k) */
    void     *combine_stage;  /* scatter combine: [W][T][max_dest][H] bf16, or NULL */
} ep_dispatch_out_t;

const char *ep_status_str(ep_status_t s);

/* Bytes of device workspace ep_create needs for this config.
 * INVALID_ARGS if the config is outside the limits above. */
ep_status_t ep_workspace_size(const ep_config_t *cfg, size_t *bytes);

/* Validate cfg, carve d_workspace (>= ep_workspace_size bytes, 256-byte
 * aligned, owned by the caller and kept alive until ep_destroy), zero the
 * flags, counters and error word (synchronously), take one pinned host word
 * (cudaHostAlloc) for ep_get_error, and return a host handle.
 * Reads EP_EARLY_NOTIFY / EP_FUSED_RECV / EP_LOG_LEVEL from the environment
 * once, here.  Must be called with the workspace's device current. */
ep_status_t ep_create(const ep_config_t *cfg, void *d_workspace, size_t bytes,
                      ep_handle_t **out);

/* Free the host handle and its CUDA events (not the workspace). */
ep_status_t ep_destroy(ep_handle_t *h);

/* Layout only (step "routing layout"): from d_idx int32 [W][T][k] and the
 * per-call token counts h_num_tokens int32 [W] (host), compute per-token
 * destination masks, the W x W send counts, recv_count and the chunk bases
 * that fix every position.  Sets BAD_INDEX / CAPACITY device bits. */
ep_status_t ep_layout(ep_handle_t *h, const int32_t *d_idx,
                      const int32_t *h_num_tokens, void *stream);

/* Send phase of dispatch: layout, then the copy of every token row to each
 * of its destination ranks (with its k weights, k ids and src_pos), then
 * (early_notify) the ready flags.  d_w: [W][T][k] fp32; d_idx: [W][T][k]
 * int32.  d_x and d_scales, 16-byte aligned:
 *  - d_scales == NULL: d_x is [W][T][H] bf16; with an FP8 dispatch_dtype
 *    every row is quantised on the way (fused per-128-element E4M3);
 *  - d_scales != NULL (FP8 dispatch_dtype only; the pages' dispatch takes
 *    `scales` beside `input`, and a backend may pass FP8 input that is
 *    quantised already): d_x is [W][T][H] E4M3 codes and d_scales [W][T][H/128]
 *    fp32 block scales, both copied unchanged.
 * Inputs must stay unchanged until the receive phase has been enqueued.
 * The copy kernel is launched as a programmatic dependent of the layout
 * kernel just before it (both enqueued by this call), so stream capture
 * records a programmatic edge between them.  When the routing spans at most
 * 8 chunks of 32 tokens (W * ceil(T/32) <= 8), no layout kernel runs: the
 * copy computes the layout itself and is launched as a programmatic
 * dependent of whatever kernel precedes it.  Either way anything enqueued
 * earlier on the stream is complete before the first read of the inputs. */
ep_status_t ep_dispatch_send(ep_handle_t *h, const void *d_x, const float *d_w,
                             const float *d_scales, const int32_t *d_idx,
                             const int32_t *h_num_tokens, void *stream);

/* Receive phase of dispatch on `stream` (may differ from the send stream):
 * wait for the send (stream-ordered via an event the send recorded); with
 * early_notify, check the ready flags (bounded wait, TIMEOUT bit on expiry)
 * and then write recv_count (zero included).  Without early_notify the
 * send's layout kernel has produced recv_count and this phase launches no
 * kernel.  Either way the received rows and recv_count are ready on
 * `stream` once this call's work there is done.  BAD_STATE without a
 * pending send. */
ep_status_t ep_dispatch_recv(ep_handle_t *h, void *stream);

/* Send + receive on one stream. */
ep_status_t ep_dispatch(ep_handle_t *h, const void *d_x, const float *d_w,
                        const float *d_scales, const int32_t *d_idx,
                        const int32_t *h_num_tokens, void *stream);

/* Routing replay: the copy (and notify) of ep_dispatch_send, reusing the
 * layout of the last ep_layout / ep_dispatch_send call for the same indices
 * and token counts, without recomputing it.  d_x / d_scales as in
 * ep_dispatch_send; h_num_tokens must equal the layout's.  BAD_STATE
 * without a layout. */
ep_status_t ep_dispatch_send_replay(ep_handle_t *h, const void *d_x,
                                    const float *d_w, const float *d_scales,
                                    const int32_t *d_idx,
                                    const int32_t *h_num_tokens, void *stream);

ep_status_t ep_dispatch_outputs(const ep_handle_t *h, ep_dispatch_out_t *out);

/* The pre-registered combine input buffer of rank 0 (the expert writes
 * y_r rows here; rank r's rows start at *d_ptr + r * *rank_stride_bytes).
 * dtype must be the config's combine_dtype (else EP_ERR_NOT_FOUND). */
ep_status_t ep_get_combine_input_buffer(const ep_handle_t *h, int32_t dtype,
                                        void **d_ptr,
                                        int64_t *rank_stride_bytes);

/* FP8 combine payload (combine_dtype == EP_DT_FP8_E4M3): the block scales
 * of the registered combine buffer, rank r's [cap][H/128] fp32 rows at
 * *d_ptr + r * *rank_stride_bytes.  Combine dequantises each element as
 * fl32(e4m3_value(q) * scale) before its ordered fp32 sum.  NOT_FOUND for
 * other combine dtypes. */
ep_status_t ep_get_combine_input_scales(const ep_handle_t *h, float **d_ptr,
                                        int64_t *rank_stride_bytes);

/* Send phase of combine (expert side): records the completion of the
 * expert's work on `stream` and (early_notify) posts combine ready flags.
 * BAD_STATE without a dispatch, while a dispatch send waits for its receive
 * phase (the receive orders the expert side after the send's copy), or while
 * an earlier combine send waits for its receive. */
ep_status_t ep_combine_send(ep_handle_t *h, void *stream);

/* Receive phase of combine (source side): wait for the combine send, then
 * gather-reduce.  d_y: NULL for the registered buffer, else rank r's rows at
 * d_y + r*y_rank_stride_bytes ([cap][H] of combine_dtype, 16-byte aligned).
 * d_w_in: NULL, or rank r's expert-side weight rows [cap][k] fp32 at
 * d_w_in + r*w_rank_stride_bytes.  d_idx: NULL, or the [W][T][k] ids of the
 * dispatch (checked: a token whose destination set differs sets the
 * COMBINE_MISMATCH bit; the dispatch's layout is used).  d_out: [W][T][H]
 * bf16; d_out_w: [W][T][k] fp32 (written iff d_w_in).  Rows t >= n_s are
 * not written.  BAD_STATE without a dispatch or without a combine send.
 * The gather kernel is launched as a programmatic dependent of the kernel
 * before it on the stream and waits for that kernel's completion before
 * its first read, so it may be enqueued right after the expert's kernel. */
ep_status_t ep_combine_recv(ep_handle_t *h, const void *d_y,
                            int64_t y_rank_stride_bytes, const float *d_w_in,
                            int64_t w_rank_stride_bytes, const int32_t *d_idx,
                            void *d_out, float *d_out_w, void *stream);

/* Send + receive on one stream.  BAD_STATE without a dispatch, while a
 * dispatch send waits for its receive phase, or while a combine send waits
 * for its receive. */
ep_status_t ep_combine(ep_handle_t *h, const void *d_y,
                       int64_t y_rank_stride_bytes, const float *d_w_in,
                       int64_t w_rank_stride_bytes, const int32_t *d_idx,
                       void *d_out, float *d_out_w, void *stream);

/* Standard-MoE conversion ("Choosing an EP API and backend", EPv2 row:
 * "standard-MoE conversion"), needs max_grouped_rows_per_rank > 0.
 * After the receive phase of a dispatch, on every rank r the entries
 * (received row p < min(recv_count[r], cap), top-k slot j) whose expert
 * lives on r are grouped per local expert e = idx - r*Er: groups in e order,
 * entries in (p, j) order inside a group.  count[r][e], offset[r][e] (its
 * exclusive prefix) and entry_slot[r][p][j] (-1 if non-local) describe it;
 * slot q of rank r gets the payload row (and FP8 scale row), g_src = p*k + j
 * and g_w = the row's weight j.  Entries whose slot is >= the grouped
 * capacity are dropped and set the CAPACITY bit. */
typedef struct {
    void     *xg;             /* [W] x [gcap][H] payload (bf16 or e4m3) */
    float    *xg_scales;      /* [W] x [gcap][H/128] (FP8) or NULL */
    int32_t  *g_src;          /* [W] x [gcap] p*k + j */
    float    *g_w;            /* [W] x [gcap] routing weight of the entry */
    void     *yg;             /* [W] x [gcap][H] bf16: registered expert-output rows */
    int32_t  *entry_slot;     /* [W] x [cap][k] */
    int64_t   rank_stride_bytes;
    int32_t  *count;          /* [W][Er] */
    int32_t  *offset;         /* [W][Er] */
    int32_t   gcap;
    int32_t   experts_per_rank;
} ep_moe_out_t;

ep_status_t ep_moe_group(ep_handle_t *h, void *stream);
ep_status_t ep_moe_outputs(const ep_handle_t *h, ep_moe_out_t *out);

/* The inverse before combine: for every received row p of rank r,
 * y_r[p][h] = bf16_rne(+0.0f + sum over its entries j ascending of
 * fl32(g_w * fp32(yg[slot][h]))) written to the registered combine input
 * buffer (combine_dtype must be bf16).  d_yg: NULL for the registered
 * expert-output buffer, else rank r's [gcap][H] bf16 rows at
 * d_yg + r*yg_rank_stride_bytes.  BAD_STATE without a grouping. */
ep_status_t ep_moe_ungroup(ep_handle_t *h, const void *d_yg,
                           int64_t yg_rank_stride_bytes, void *stream);

/* Reset between iterations: zero the ready flags, epochs and error word on
 * `stream` and forget the layout (combine then needs a new dispatch). */
ep_status_t ep_reset(ep_handle_t *h, void *stream);

/* Read and clear the device error word in `stream` order (one atomic
 * exchange on the device, so no bit set concurrently is lost), then wait for
 * that stream alone (cudaStreamSynchronize; work on other streams keeps
 * running, and what it sets later shows in a later call).  *mask gets the
 * EP_DEVERR_* bits; the return is EP_SUCCESS for 0, else the status of the
 * lowest set bit (BAD_INDEX, CAPACITY, TIMEOUT, BAD_STATE for a combine
 * mismatch). */
ep_status_t ep_get_error(ep_handle_t *h, uint32_t *mask, void *stream);

/* Test harness, not part of the hot path: the identity expert of the
 * benchmark's correctness check ("Validation before tuning").  For each
 * received row p < min(recv_count[r], cap) of every rank r:
 * alpha = ordered fp32 sum of the row's weights whose expert lives on r,
 * y_r[p][h] = bf16_rne(fl32(v_h * alpha)) (fp32 rows: fl32(v_h * alpha);
 * FP8 payload: those fp32 products quantised per 128-element block with the
 * dispatch formula),
 * v = the bf16 payload, or fl32(e4m3_value(q) * scale) for FP8.  d_y as in
 * ep_combine_recv. */
ep_status_t ep_test_identity_expert(ep_handle_t *h, void *d_y,
                                    int64_t y_rank_stride_bytes, void *stream);

/* Test harness, not part of the hot path: checks the arithmetic behind the
 * fused FP8 quantisation of dispatch (per 128-element block a = max|x|,
 * scale = fl32(a/448), q = RNE-satfinite(fl32(x/scale)); OCP E4M3, "Choosing
 * an EP API and backend", "EPv2 configuration and lifecycle") over every
 * positive finite bf16 block maximum a and every finite bf16 x with
 * |x| <= a, both signs (1 065 402 238 pairs), using the dispatch kernel's
 * own device functions.  d_counts: 4 device uint64 (8-byte aligned), zeroed
 * here, then [0] = pairs checked, [1] = pairs whose E4M3 code differs from
 * the code of the IEEE quotient x / (a / 448), [2] = block maxima whose scale
 * differs from the IEEE quotient a / 448, [3] = pairs that took the
 * reciprocal-and-correction quotient.  Asynchronous on `stream`. */
ep_status_t ep_test_fp8_quotient_check(uint64_t *d_counts, void *stream);

/* Routing layout without any allocation, for callers that cannot allocate
 * device memory or pass a workspace: code living inside another
 * framework's memory pool that only sees raw tensor pointers, and serving
 * paths that forbid cudaMalloc (it can synchronise the device and can fail
 * under memory pressure).  The pages have no counterpart of this call; it
 * computes the same layout as ep_layout + ep_dispatch (pos, send counts,
 * recv_count) with no handle.
 *   d_idx [W][T][k] int32, h_num_tokens [W] host; outputs (caller-owned,
 *   device): d_pos [W][T][W] (-1 where r is not a destination),
 *   d_send_counts [W][W], d_recv_count [W]; d_error: NULL or a device u32
 *   that gets EP_DEVERR_BAD_INDEX OR-ed in (out-of-range ids contribute no
 *   destination).
 * Scratch is a fixed device array inside the library (about 0.66 MB, held
 * by every GPU that loads the library until the process exits); it limits
 * the layout to W <= 32 and W * ceil(T/32) <= 4128 32-token chunks: any
 * W * T <= 131072 is accepted whatever T is, and up to 132096 tokens when T
 * is a multiple of 32.  Larger sizes return EP_ERR_INVALID_ARGS.  Every call
 * looks the array's device address up with the caller's device current (a
 * host-side lookup once the library's device code is loaded, so a context
 * reset in between is harmless); the first call on a device may load that
 * code, so make it before any stream capture.  All calls share the array:
 * calls whose work overlaps on the GPU race; order them on one stream. */
ep_status_t ep_layout_noalloc(int32_t world_size, int32_t num_experts,
                              int32_t topk, int32_t max_tokens_per_rank,
                              const int32_t *d_idx, const int32_t *h_num_tokens,
                              int32_t *d_pos, int32_t *d_send_counts,
                              int32_t *d_recv_count, uint32_t *d_error,
                              void *stream);

/* ---------------------------------------------------------------------
 * Routing, balance loss and expert products: what stands before and between
 * dispatch and combine in a MoE layer.  These calls need no handle; sizes
 * and options come in a descriptor, scratch (where a call needs any) from
 * the caller, and everything is asynchronous on `stream`.  d_error: NULL, or
 * a device u32 (zeroed once by the caller) that gets EP_DEVERR_* bits OR-ed
 * in.  Call them with the tensors' device current. */

typedef enum { EP_SCORE_SOFTMAX = 0, EP_SCORE_SIGMOID = 1 } ep_score_t;

#define EP_MAX_ROUTE_EXPERTS 1024

/* Router logits [W][T][E]: element (s,t,e) at d_logits[s * rank_stride +
 * t * row_stride + e].  x below is the logit in fp32 with NaN read as -inf
 * and +inf as the largest finite number; an expert with x = -inf is closed:
 * it has probability and weight 0 and is chosen only where fewer than k
 * experts are open.  Token t of rank s is present when t < h_num_tokens[s]. */
typedef struct {
    int32_t world_size;   /* W, 1..32 */
    int32_t tokens;       /* T >= 1, W * T <= 2^30 */
    int32_t num_experts;  /* E, 1..EP_MAX_ROUTE_EXPERTS */
    int32_t topk;         /* k, 1..min(E, 32) */
    int32_t dtype;        /* EP_DT_BF16, EP_DT_FP16 or EP_DT_FP32 logits */
    int32_t score;        /* ep_score_t */
    int32_t renormalize;  /* 1: the k weights are divided by their sum (softmax:
                             the softmax is taken over the chosen experts) */
    float   scale;        /* factor on the weights */
    float   balance_coef; /* of the balance loss (loss calls only) */
    float   z_coef;       /* of the mean squared log-sum-exp (loss calls only) */
    int64_t row_stride;   /* elements, >= E */
    int64_t rank_stride;  /* elements; unused when W == 1 */
} ep_route_desc_t;

/* Top-k routing.  The k experts with the largest x_e + bias_e (an fp32 add;
 * d_bias NULL: no bias) are chosen, in descending order, ties to the lowest
 * expert id.  The bias takes no part in the weights.  It is one of the logits:
 * balancing without a loss, as published, adds its bias to the score, which is
 * another choice wherever scores differ by less than their biases; pass the
 * scores as d_logits for that one, -inf for experts that are to stay closed.
 *   softmax:  w_j = scale * exp(x_j) / sum exp(x), the sum over the chosen
 *             experts (renormalize) or over all
 *   sigmoid:  w_j = scale * v_j, v_j = 1 / (1 + exp(-x_j)), divided by the sum
 *             of the chosen v (renormalize; weights 0 where every chosen x is
 *             below -745)
 * d_w [W][T][k] fp32 and d_idx [W][T][k] int32, dense, are dispatch's weights
 * and indices.  Tokens that are not present get ids -1 and weights 0. */
ep_status_t ep_route(const ep_route_desc_t *d, const void *d_logits,
                     const float *d_bias, const int32_t *h_num_tokens,
                     float *d_w, int32_t *d_idx, void *stream);

/* The balance and z losses of a routing, with n = number of tokens present:
 *   counts_e = choices of e among present tokens (ids outside [0, E) are
 *              skipped and set BAD_INDEX)
 *   probs_e  = (1/n) sum over present tokens of softmax(x)_e
 *   d_loss[1] = sum_e (counts_e * E / (k n)) * probs_e
 *   d_loss[2] = (1/n) sum of (log sum exp x)^2   (0 for a token that sees no
 *               open expert)
 *   d_loss[0] = balance_coef * d_loss[1] + z_coef * d_loss[2], with z_coef 0
 *               without the second term, whatever d_loss[2] is
 * All 0 when n = 0.  Sums are fp32, in an order that the sizes alone fix.
 * d_idx [W][T][k]; d_loss [3], d_counts [E] int32, d_probs [E] fp32.
 * d_workspace: ep_balance_loss_workspace bytes, 16-byte aligned, any
 * contents. */
ep_status_t ep_balance_loss_workspace(const ep_route_desc_t *d, size_t *bytes);
ep_status_t ep_balance_loss(const ep_route_desc_t *d, const void *d_logits,
                            const int32_t *d_idx, const int32_t *h_num_tokens,
                            float *d_loss, int32_t *d_counts, float *d_probs,
                            void *d_workspace, size_t workspace_bytes,
                            uint32_t *d_error, void *stream);

/* Gradient by the logits, in their type, dense [W][T][E]; 0 for tokens that
 * are not present.  The sum of two parts, either of which may be left out:
 *  - of the weights (d_grad_w [W][T][k] fp32 with the forward's d_idx; both
 *    NULL: left out);
 *  - of d_loss[0] (d_grad_loss, one fp32, with the forward's d_counts; both
 *    NULL: left out).  counts are constants of the gradient.
 * Ids outside [0, E) are skipped and set BAD_INDEX. */
ep_status_t ep_route_backward(const ep_route_desc_t *d, const void *d_logits,
                              const float *d_grad_w, const int32_t *d_idx,
                              const float *d_grad_loss, const int32_t *d_counts,
                              const int32_t *h_num_tokens, void *d_grad_logits,
                              uint32_t *d_error, void *stream);

typedef enum {
    EP_ACT_NONE = 0,
    EP_ACT_RELU = 1,
    EP_ACT_GELU = 2,      /* v * Phi(v), the error-function form */
    EP_ACT_SILU = 3,
    EP_ACT_SWIGLU = 4     /* silu(first N features) * (last N of 2N features) */
} ep_activation_t;

/* Rows grouped by expert, as ep_moe_group leaves them: R segments ("ranks")
 * of `rows` rows, and in each segment `groups` groups; group e of segment r
 * is rows offset[r][e] .. offset[r][e] + count[r][e] - 1 (device int32 [R][groups]).
 * Rows of a group past the segment's end are left out; d_count == NULL means one
 * group per segment that holds all its rows.  Groups of a segment must not
 * overlap.  Strides are in elements; every row is contiguous, every pointer is
 * 16-byte aligned and every stride is a multiple of 8 elements. */
typedef struct {
    void   *ptr;
    int64_t rank_stride;  /* unused when R == 1 */
    int64_t row_stride;
} ep_rows_t;

typedef struct {
    int32_t ranks;        /* R >= 1 */
    int32_t groups;       /* groups per segment >= 1; R * groups <= 65535 */
    int32_t rows;         /* rows per segment, 0..2^30 */
    int32_t in_features;  /* K, multiple of 8 */
    int32_t out_features; /* N, multiple of 8 */
    int32_t dtype;        /* EP_DT_BF16 or EP_DT_FP16, of every tensor */
    int32_t activation;   /* ep_activation_t */
    int32_t reserved;     /* 0 */
    const int32_t *d_count, *d_offset;  /* both NULL, or both [R][groups] */
    /* weight[g][f][c], g = r * groups + e, f < wide = N (2N for SWIGLU), c < K:
     * at weight.ptr + g * rank_stride + f * row_stride + c */
    ep_rows_t weight;
    ep_rows_t x;          /* [R][rows][K] */
} ep_product_desc_t;

/* For every row i of group g:
 *   pre = x_i W_g^T + bias_g,   y_i = act(pre) + residual_i
 * with fp32 products' sums and epilogue, one rounding per output.  d_bias:
 * [R*groups][wide] dense or NULL; residual, pre: ptr NULL to leave out;
 * pre gets the wide pre-activations (what the gradient needs).  Rows outside
 * every group are not written.  y may be the residual itself; otherwise y and
 * pre overlap nothing that the call reads.  The kernel is launched as a
 * programmatic dependent of the kernel before it on the stream and waits for
 * it before its first read or write; so are the gradient's, the balance
 * loss's, and ep_route's and ep_route_backward's from 2^18 logits on. */
ep_status_t ep_expert_product(const ep_product_desc_t *d, const void *d_bias,
                              const ep_rows_t *residual, const ep_rows_t *y,
                              const ep_rows_t *pre, uint32_t *d_error,
                              void *stream);

/* The gradient, from grad = dL/dy [R][rows][N] and the forward's pre
 * (EP_ACT_NONE: not read):
 *   d = grad * act'(pre), rounded once to the tensors' type for the products
 *   grad_x_i = d_i W_g;  grad_w_g = sum over g's rows of d_i^T x_i
 *   grad_bias_g = sum over g's rows of d_i (of d before that rounding)
 * grad_x: like x (rows outside every group are not written); d_grad_w: dense
 * [R*groups][wide][K]; d_grad_bias: dense [R*groups][wide] or NULL.  A group
 * without rows gets zeros.  grad_x->ptr or d_grad_w may be NULL to leave that
 * part out.  The gradient of the residual is grad itself.  d_workspace:
 * ep_expert_product_workspace bytes, 256-byte aligned, any contents. */
ep_status_t ep_expert_product_workspace(const ep_product_desc_t *d, size_t *bytes);
ep_status_t ep_expert_product_backward(const ep_product_desc_t *d,
                                       const ep_rows_t *grad, const ep_rows_t *pre,
                                       const ep_rows_t *grad_x, void *d_grad_w,
                                       void *d_grad_bias, void *d_workspace,
                                       size_t workspace_bytes, uint32_t *d_error,
                                       void *stream);

/* ---------------------------------------------------------------------
 * Norm, checkpoints in 8 bits, and the experts of a few tokens: no handle,
 * asynchronous on `stream`, as the calls above; every kernel is launched as a
 * programmatic dependent of the one before it on the stream and waits for it
 * before it reads or writes what that one may (ep_moe_few's second kernel reads the
 * call's inputs, which its first has waited for, ahead of that).
 *
 * 8 bits are E4M3 codes with one fp32 scale for every block of 128 values of a
 * row (the last block of a row may be a part), as dispatch quantises:
 * a = max|v|, scale = fl32(a / 448), code = the E4M3 value nearest to
 * fl32(v / scale), ties to even; the quotient is the IEEE one for bf16 values and
 * within a unit of fp32's last place for others.  A block of zeros has scale 0
 * and codes 0; a block that holds an infinity or a NaN has scale NaN and every
 * code NaN (0x7F), so that all of it comes back as NaN. */

#define EP_MAX_NORM_WIDTH 32768
#define EP_MAX_FEW_TOKENS 64

/* Rows here are contiguous, aligned to their element alone, with any strides >=
 * width (rank_stride > 0), in elements; 16-byte aligned ones are read faster. */
typedef struct {
    int32_t ranks;        /* R, 1..65535 */
    int32_t rows;         /* rows per rank, 0..2^30, R * rows <= 2^30 */
    int32_t width;        /* H, 1..EP_MAX_NORM_WIDTH */
    int32_t dtype;        /* EP_DT_BF16, EP_DT_FP16 or EP_DT_FP32, of every row */
    int32_t weight_dtype; /* dtype or EP_DT_FP32 */
    float   eps;          /* >= 0; with 0 a row's root mean square has to be 2^-127 or more, or its r passes fp32 */
    ep_rows_t x;          /* [R][rows][H] */
    const void *weight;   /* [H] */
} ep_norm_desc_t;

/* Root-mean-square norm of every row, after the residual's addition:
 *   total = x + residual, rounded once to dtype (residual->ptr NULL: x itself)
 *   r = 1 / sqrt(mean(total^2) + eps),  y = total * r * weight
 * The norm is that of the rounded total, which is what the next block adds to
 * and what the gradient sees.  Sums in fp32, y rounded once.  total->ptr NULL:
 * not written.  total may be x or the residual itself; y overlaps nothing that is
 * read.  scales->ptr NULL: y has dtype; else y gets codes (one byte each) and scales the
 * [R][rows][H/128] fp32 block scales, with H a multiple of 128: what a
 * pre-quantised dispatch takes. */
ep_status_t ep_rms_norm(const ep_norm_desc_t *d, const ep_rows_t *residual,
                        const ep_rows_t *total, const ep_rows_t *y,
                        const ep_rows_t *scales, void *stream);

/* The gradient, d->x being the forward's total, grad = dL/dy:
 *   u = grad * weight
 *   grad_x = r * (u - total * r^2 * mean(u * total)) + grad_total
 *   grad_weight = sum over rows of grad * total * r
 * grad_total (ptr NULL: none) is what comes to total from elsewhere, the residual
 * stream.  grad_x is the gradient of x and of the residual alike, and may be
 * grad_total itself.  d_grad_weight [H] in weight_dtype; rows are summed in an
 * order that sizes, strides, alignment and whether there is a grad_total fix.  d_workspace: ep_rms_norm_workspace bytes, 16-byte
 * aligned, any contents. */
ep_status_t ep_rms_norm_workspace(const ep_norm_desc_t *d, size_t *bytes);
ep_status_t ep_rms_norm_backward(const ep_norm_desc_t *d, const ep_rows_t *grad,
                                 const ep_rows_t *grad_total,
                                 const ep_rows_t *grad_x, void *d_grad_weight,
                                 void *d_workspace, size_t workspace_bytes,
                                 uint32_t *d_error, void *stream);

/* Activations kept in 8 bits between forward and backward, over rows grouped as in
 * ep_product_desc_t.  Rows outside every group are neither read nor written. */
typedef struct {
    int32_t ranks, groups, rows;    /* as in ep_product_desc_t */
    int32_t features;     /* values of a kept row, multiple of 8, <= 2^24 */
    int32_t dtype;        /* EP_DT_BF16 or EP_DT_FP16, of x and y */
    int32_t activation;   /* of restore */
    const int32_t *d_count, *d_offset;
} ep_checkpoint_desc_t;

/* x [R][rows][features] -> codes (one byte each, strides in bytes, multiples of 8)
 * and scales [R][rows][ceil(features / 128)] fp32. */
ep_status_t ep_checkpoint_save(const ep_checkpoint_desc_t *d, const ep_rows_t *x,
                               const ep_rows_t *codes, const ep_rows_t *scales,
                               void *stream);
/* y = act(code * scale), the product in fp32, rounded once; with EP_ACT_SWIGLU
 * features is a multiple of 16 and y has half of them.  Also turns the grouped 8-bit rows of
 * an FP8 dispatch into rows that ep_expert_product takes. */
ep_status_t ep_checkpoint_restore(const ep_checkpoint_desc_t *d, const ep_rows_t *codes,
                                  const ep_rows_t *scales, const ep_rows_t *y,
                                  void *stream);
/* ep_expert_product_backward with pre = code * scale (in fp32, not rounded to
 * the tensors' type), codes [R][rows][wide] and scales [R][rows][ceil(wide /
 * 128)] as ep_checkpoint_save leaves them. */
ep_status_t ep_expert_product_backward_checkpoint(
    const ep_product_desc_t *d, const ep_rows_t *grad, const ep_rows_t *codes,
    const ep_rows_t *scales, const ep_rows_t *grad_x, void *d_grad_w,
    void *d_grad_bias, void *d_workspace, size_t workspace_bytes,
    uint32_t *d_error, void *stream);

/* A whole MoE layer's experts for a few tokens, without dispatch:
 *   out[t] = residual[t] + sum over j of w[t][j] * y(t, e), e = idx[t][j],
 *   y(t, e) = act(x[t] up_e^T + up_bias_e) down_e^T + down_bias_e
 * Every sum is fp32; the activations between the products are kept in fp32 (little
 * work: up to 48 MB of weights over all choices) or in two 16-bit halves (a value and what
 * its rounding left), and out is rounded once.  Halves are within 2^-16 of the value; those of
 * fp16 only from 2^-16 on, within 2^-32 below, and infinite from 2^20 on.  Sums are in an order that sizes and indices alone fix; an expert that is
 * named twice counts twice.  idx < 0: no expert (ep_route's -1); idx >=
 * experts: skipped, and sets BAD_INDEX.  A token without experts gets its
 * residual, or 0. */
typedef struct {
    int32_t tokens;       /* T, 0..EP_MAX_FEW_TOKENS */
    int32_t experts;      /* E, 1..EP_MAX_ROUTE_EXPERTS */
    int32_t topk;         /* k, 1..32 */
    int32_t hidden;       /* H, multiple of 8, <= 2^20 */
    int32_t inner;        /* F, multiple of 8, <= 2^20 */
    int32_t dtype;        /* EP_DT_BF16 or EP_DT_FP16, of every tensor but w */
    int32_t activation;   /* ep_activation_t; SWIGLU: up has 2F features, the gate's first */
    int32_t reserved;     /* 0 */
    ep_rows_t up;         /* [E][wide][H]; rows as in ep_product_desc_t */
    ep_rows_t down;       /* [E][H][F] */
    const void *up_bias, *down_bias;    /* [E][wide], [E][H] dense, or NULL */
} ep_few_desc_t;

/* x, residual (ptr NULL: none), out: [T][H] (rank_stride unused).  out may be the
 * residual itself and overlaps nothing else.  d_workspace: ep_moe_few_workspace bytes,
 * 256-byte aligned, any contents. */
ep_status_t ep_moe_few_workspace(const ep_few_desc_t *d, size_t *bytes);
ep_status_t ep_moe_few(const ep_few_desc_t *d, const ep_rows_t *x, const float *d_w,
                       const int32_t *d_idx, const ep_rows_t *residual,
                       const ep_rows_t *out, void *d_workspace,
                       size_t workspace_bytes, uint32_t *d_error, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* EP_API_H */
