/*
 * ep.h -- C ABI of the GB300 MoE dispatch / combine layout library
 * (libep_gb300.so, CUDA sm_103a).
 *
 * The library implements the data-parallel hot path of expert-parallel MoE
 * communication as a layout transformation on ONE GPU: expert-parallel ranks
 * are logical destination partitions of a single HBM buffer.
 *
 *   ep_get_layout : topk_idx            -> counts, aligned offsets, slots
 *   ep_dispatch   : token-major x       -> expert-major rows (bf16 or FP8)
 *   ep_combine    : expert-major rows   -> token-major y (gate-weighted)
 *
 * with what stands before and between them in a layer:
 *
 *   ep_route      : router logits       -> topk_idx, gate weights (losses,
 *                                          gradient: ep_route_balance,
 *                                          ep_route_backward)
 *   ep_expert_w4  : expert-major rows   -> rows times 4-bit expert weights
 *
 * Sources (page title, section):
 *  "GPU Microarchitecture: DeepEP from First Principles" -- 1.1 and 1.2
 *  (dispatch token-major -> destination-major -> expert-major; combine back,
 *  Output(T0) = 0.73 x Expert2(T0) + 0.27 x Expert7(T0)), 6.1 / 6.2 (layout
 *  and identity metadata), 7.1 (count -> prefix sum -> scatter).
 *  "Deep Dive - DeepEP" -- "V2's single interface: ElasticBuffer" (problem
 *  statement: max tokens, hidden, top-k, FP8 dispatch), "Dispatch: layout,
 *  move, and epilogue" (topk_idx / topk_weights contract, -1 = unused,
 *  expanded mode, expert alignment, psum semantics, zero padding, CPU sync),
 *  "Combine: reverse routing plus reduction" (fp32 accumulation, one bf16
 *  cast), "Precision: FP8 on the wire, BF16 for the reduction" (one fp32
 *  scale per 128 values), "EPHandle: route metadata with a lifetime" (the
 *  handle carries route metadata, not gate values; deterministic order).
 *
 * Conventions for every entry point
 *  - Pointers named d_* or documented "device" are CUDA device pointers; all
 *    buffers are allocated and owned by the CALLER.  The library never
 *    allocates or frees memory and keeps no pointer after a call returns.
 *    (The host-buffer entry points, when they copy in chunks, create two
 *    copy streams -- one a direction -- and a few events per device on
 *    first use, kept until exit.)
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream).  Work is enqueued asynchronously on it; a call returns before
 *    the GPU has finished unless documented otherwise.
 *  - Calls that do not synchronise can be recorded into a CUDA graph by
 *    stream capture: the device entry points, and the host-buffer entry
 *    points in both modes (in chunked mode the library's copy streams join
 *    the capture through events; make one chunked call outside any capture
 *    first, which creates them).  ep_get_layout with h_expert_count,
 *    ep_check_error and the self-tests synchronise and cannot be captured.
 *  - Argument errors are detected on the host before anything is launched
 *    and returned synchronously (EP_ERR_INVALID_ARG).  Errors in the routing
 *    data (an expert id outside [-1, E), an expert repeated within a token)
 *    can only be seen on the GPU: they are recorded in the layout's device
 *    error word and reported by ep_check_error (or by ep_get_layout when it
 *    is asked to synchronise).  Kernels never trap.
 *  - Every device pointer must be 16-byte aligned.
 *  - Row-major layouts throughout.  T = num_tokens of the ep_get_layout call
 *    (<= cfg.max_tokens), H = hidden, K = num_topk, E = num_experts,
 *    R = num_ranks, A = expert_alignment, cap = ep_recv_capacity(cfg).
 */
#ifndef EP_GB300_H
#define EP_GB300_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define EP_API __attribute__((visibility("default")))
#else
#define EP_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes returned by every entry point (int32_t). */
enum {
  EP_OK = 0,
  EP_ERR_INVALID_ARG = 1,   /* bad config, pointer, alignment or size      */
  EP_ERR_EXPERT_RANGE = 2,  /* a topk_idx entry outside [-1, E)            */
  EP_ERR_DUP_EXPERT = 3,    /* an expert selected twice by one token       */
  EP_ERR_CAPACITY = 4,      /* a buffer or built-in scratch is too small   */
  EP_ERR_CUDA = 5,          /* a CUDA runtime call failed                  */
  EP_ERR_TIMEOUT = 6,       /* a bounded on-chip wait gave up (no hang)    */
  EP_ERR_TIMEOUT_PENDING = 7 /* as EP_ERR_TIMEOUT, and a bulk copy the
                                waiting CTA had issued was still not done
                                when it returned: it may still write that
                                SM's shared memory, so treat the CUDA
                                context as unreliable                     */
};

/* Problem statement, as in the pages' buffer constructor: max tokens,
 * hidden size, top-k, expert count, FP8 dispatch; plus the logical rank
 * count, the expert alignment and the zero-padding switch of dispatch. */
typedef struct {
  int32_t max_tokens;        /* tokens a layout may hold (capacity planning)   */
  int32_t hidden;            /* H: bf16 channels per row, H <= 2^20; H % 8
                                == 0 for bf16 rows, H % 128 == 0 when
                                use_fp8_dispatch                              */
  int32_t num_topk;          /* K in [1, 32], K <= E                           */
  int32_t num_experts;       /* E in [1, 2048]                                  */
  int32_t num_ranks;         /* R logical ranks, E % R == 0; rank r owns the
                                experts [r*E/R, (r+1)*E/R)                     */
  int32_t expert_alignment;  /* A in [1, 1024]: every expert segment starts
                                at a multiple of A rows                        */
  int32_t use_fp8_dispatch;  /* 0: bf16 rows; 1: E4M3 rows + 1x128 fp32 scales */
  int32_t zero_padding;      /* 1: dispatch clears the alignment gap rows      */
} ep_config;

/* The layout handle: route metadata only (no gate values).  Every pointer is
 * a caller-allocated DEVICE buffer of the size given; ep_get_layout fills
 * them and sets num_tokens.  The handle stays valid, and may be reused by
 * any number of dispatch / combine calls, while the route is unchanged. */
typedef struct {
  int32_t *expert_count;     /* [E]   rows routed to each expert (unaligned)   */
  int32_t *expert_start;     /* [E+1] aligned start row of each expert segment;
                                expert_start[E] = rows in use                  */
  int32_t *expert_end;       /* [E]   expert_start[e] + expert_count[e]: the
                                end of expert e's valid rows (psum semantics)  */
  int32_t *rank_start;       /* [R+1] first row of each logical rank's range
                                (= expert_start[r*E/R])                        */
  int32_t *tokens_per_rank;  /* [R]   tokens sent to each rank, counted once
                                per (token, rank)                              */
  uint8_t *is_token_in_rank; /* [max_tokens*R] 1 if token t has an expert
                                on rank r                                      */
  int32_t *slot_of;          /* [max_tokens*K] row of (t,k) in the expert-major
                                buffer, -1 for an unused (-1) selection        */
  int32_t *src_info;         /* [cap*2] (token, k) of each row in use;
                                (-1,-1) for alignment padding rows             */
  int32_t *err;              /* [1]   device error word                        */
  void *workspace;           /* ep_layout_workspace_bytes(cfg) bytes           */
  /* Optional destination-major rows (all three set, or all NULL): rank r
   * owns rows [rank_row_start[r], rank_row_start[r+1]), one per token sent
   * to it (a token is sent once to every rank owning one of its experts),
   * in token order. */
  int32_t *rank_row_start;   /* [R+1]                                          */
  int32_t *rank_slot_of;     /* [max_tokens*R] rank row of (t, r), or -1       */
  int32_t *rank_src;         /* [max_tokens*min(K,R)] token of each rank row   */
  int32_t num_tokens;        /* set by ep_get_layout                           */
  int32_t reserved;
} ep_layout;

/* Rows the expert-major buffer needs in the worst case:
 * max_tokens*K + E*(A-1).  Returns -1 if the config is invalid. */
EP_API int64_t ep_recv_capacity(const ep_config *cfg);

/* Bytes of device scratch memory ep_get_layout needs in layout->workspace
 * (per-tile expert and rank counts, per-tile error bits); layouts of at
 * most 4096 (t, k) pairs do not touch it.  Returns -1 if the config is
 * invalid. */
EP_API int64_t ep_layout_workspace_bytes(const ep_config *cfg);

/* Layout ("GPU Microarchitecture: DeepEP from First Principles", 6.1 and 7.1;
 * "Deep Dive - DeepEP", "Dispatch: layout, move, and epilogue").
 *
 * d_topk_idx: device int64 [num_tokens, K]; -1 marks an unused selection.
 * Counts rows per expert and per destination rank (a token counts once per
 * rank), lays the experts out contiguously with every segment rounded up to
 * A rows, and assigns each (t, k) its row: within an expert, rows follow
 * source-global order (source rank, token, k) -- the pages' deterministic
 * mode, produced directly.  Logical source ranks own contiguous token
 * blocks, so that order is (t, k) order.  Runs one kernel on `stream` when
 * num_tokens * K <= 4096, else two.  The layout's error word is cleared by
 * the call itself before anything is recorded in it.
 *
 * h_expert_count: NULL for a fully asynchronous call.  If non-NULL (host
 * memory, E int32), the call synchronises `stream`, copies the per-expert
 * counts there and returns the device error status (the pages' CPU-sync
 * path).  Without it, consumers must use only rows [expert_start[e],
 * expert_end[e]) and call ep_check_error to see routing errors.
 * num_tokens may be 0.  Returns EP_OK or an error. */
EP_API int32_t ep_get_layout(const ep_config *cfg, int32_t num_tokens,
                      const int64_t *d_topk_idx, ep_layout *layout,
                      int32_t *h_expert_count, void *stream);

/* Dispatch, expanded mode ("GPU Microarchitecture: DeepEP from First
 * Principles", 1.1; "Deep Dive - DeepEP", "Dispatch: layout, move, and
 * epilogue" and "Precision: FP8 on the wire, BF16 for the reduction").
 *
 * d_x: device bf16 [T, H] (raw 16-bit patterns).
 * d_topk_weights: device fp32 [T, K] or NULL.
 * d_recv_x: device [cap, H]: bf16 rows, or E4M3 bytes when use_fp8_dispatch.
 *   Row slot_of[t,k] receives token t.  bf16 rows are bit copies.  FP8 rows:
 *   per 128-channel block, amax = max|x| (exact), scale = amax / 448 (fp32,
 *   round to nearest), q = E4M3(x / scale) rounded to nearest even with
 *   saturation to +-448; an all-zero block has scale 0 and q = 0.
 * d_recv_scale: device fp32 [cap, H/128] (FP8 only, else ignored; may be
 *   NULL for bf16): the dequantisation multipliers, x ~ q * scale.
 * d_recv_w: device fp32 [cap] or NULL: recv_w[slot_of[t,k]] = w[t,k], one
 *   gate weight per expert row (requires d_topk_weights).
 * With cfg->zero_padding, rows [expert_end[e], expert_start[e+1]) get
 * zero payload, zero scales and zero weight.  Rows at or past
 * expert_start[E] are never written.  Returns EP_OK or an error. */
EP_API int32_t ep_dispatch(const ep_config *cfg, const ep_layout *layout,
                    const void *d_x, const float *d_topk_weights,
                    void *d_recv_x, float *d_recv_scale, float *d_recv_w,
                    void *stream);

/* Combine ("GPU Microarchitecture: DeepEP from First Principles", 1.2;
 * "Deep Dive - DeepEP", "Combine: reverse routing plus reduction").
 *
 * d_expert_out: device bf16 [cap, H] in the layout's row order (the expert
 *   outputs of the dispatched rows).
 * d_topk_weights: device fp32 [T, K], or NULL.  For each token and channel,
 *   acc = +0.0f; for k = 0..K-1 with slot_of[t,k] >= 0:
 *   acc = fmaf(w[t,k], expert_out[slot_of[t,k], i], acc); y = bf16(acc),
 *   round to nearest even.  Each gate weight is applied exactly once; with
 *   NULL every weight is 1, i.e. the plain sum of rows the caller already
 *   weighted (the pages' V2 contract).  Unused selections contribute
 *   nothing and the remaining weights are not renormalised; padding rows
 *   are never read.
 * d_y: device bf16 [T, H].  Returns EP_OK or an error. */
EP_API int32_t ep_combine(const ep_config *cfg, const ep_layout *layout,
                   const void *d_expert_out, const float *d_topk_weights,
                   void *d_y, void *stream);

/* Layout and dispatch in one call ("Deep Dive - DeepEP", "Dispatch: layout,
 * move, and epilogue": a dispatch counts and lays out rows by rank and
 * expert, then moves them -- conceptual stages that kernels can overlap).
 *
 * Same arguments and results as ep_get_layout (with h_expert_count NULL)
 * followed by ep_dispatch of the same num_tokens tokens, and the same errors
 * for the same arguments.  For inputs of at most 4096 (t, k) pairs whose
 * one-launch layout gives each of its CTAs at most 64 pairs, one kernel does
 * both: each CTA of the layout copies the x rows of its own tokens into
 * shared memory while it computes the layout (when they fit beside its
 * other arrays), then dispatches them as soon as their rows are known, so
 * the dispatch costs no second launch.  Larger inputs run the two paths in
 * turn.  (Column-major scales and pre-quantised input are ep_dispatch_fp8's
 * and are not offered here.)  Returns EP_OK or an error. */
EP_API int32_t ep_layout_and_dispatch(const ep_config *cfg, int32_t num_tokens,
                                      const int64_t *d_topk_idx, ep_layout *layout,
                                      const void *d_x, const float *d_topk_weights,
                                      void *d_recv_x, float *d_recv_scale,
                                      float *d_recv_w, void *stream);

/* Allocation-free layout.  The pages have no counterpart: this entry point
 * exists for callers that cannot allocate device memory -- code inside a
 * framework that owns all device memory and has no spare buffer to give, a
 * serving loop that must not allocate after warm-up (cudaMalloc can
 * synchronise the device and fragment a sized pool), or a plugin that only
 * receives the tensors it computes on.
 *
 * Same arguments and results as ep_get_layout, except that
 * layout->workspace is ignored (it may be NULL): the per-tile scratch lives
 * in a 1 MiB array in the library's own device memory, which every GPU that
 * loads the library holds until the process exits.  Only layouts of more
 * than 4096 (t, k) pairs (num_tokens * K > 4096, which take two launches)
 * use scratch; of those, configurations whose ep_layout_workspace_bytes
 * exceeds 1 MiB (152 * 4 * (E rounded up to 4 + R rounded up to 4) + 608
 * bytes) are rejected with EP_ERR_CAPACITY before anything is launched.
 * Smaller layouts are accepted whatever E and R.  Nothing is allocated or
 * freed, by this call or by any routine it calls.
 *
 * The first call on each device looks up the array's device address (with
 * that device current) and caches it; make that first call before any
 * stream capture.  All calls share the one array and it keeps the last
 * call's contents; every call writes the scratch it reads before reading
 * it, so nothing has to start at zero.  Calls whose work overlaps on the GPU
 * (e.g. on two streams at once) race on the array: order them. */
EP_API int32_t ep_get_layout_noalloc(const ep_config *cfg, int32_t num_tokens,
                                     const int64_t *d_topk_idx,
                                     ep_layout *layout,
                                     int32_t *h_expert_count, void *stream);

/* Leading dimension (in fp32 entries) of column-major FP8 scales:
 * ep_recv_capacity(cfg) rounded up to a multiple of 4, so that every
 * block's column starts on a 16-byte boundary.  -1 if the config is
 * invalid. */
EP_API int64_t ep_scale_ld(const ep_config *cfg);

/* FP8 dispatch with options ("Deep Dive - DeepEP", "Precision: FP8 on the
 * wire, BF16 for the reduction": the input may arrive as FP8 values plus
 * scale factors; a column-major scale layout serves TMA-fed consumers).
 *
 * Input, exactly one of:
 *   d_x       device bf16 [T, H], quantised as in ep_dispatch (1x128 blocks,
 *             scale = amax / 448, E4M3 round to nearest even, saturating);
 *   d_x_q + d_x_scale  device E4M3 bytes [T, H] and fp32 scales [T, H/128]
 *             of pre-quantised rows, copied bit for bit.
 * d_recv_q: device [cap, H] E4M3 rows (row slot_of[t,k] gets token t).
 * d_recv_scale: device fp32; scale_col_major = 0: [cap, H/128] row-major;
 *   1: [H/128, ep_scale_ld(cfg)] column-major (entry (row, block) at
 *   block * ld + row).
 * d_topk_weights / d_recv_w: as in ep_dispatch.  cfg->zero_padding clears
 * the alignment gap rows (payload, scales in the chosen layout, weights).
 * H % 128 == 0 is required; cfg->use_fp8_dispatch is not consulted.
 * Returns EP_OK or an error. */
EP_API int32_t ep_dispatch_fp8(const ep_config *cfg, const ep_layout *layout,
                               const void *d_x, const uint8_t *d_x_q,
                               const float *d_x_scale,
                               const float *d_topk_weights, uint8_t *d_recv_q,
                               float *d_recv_scale, int32_t scale_col_major,
                               float *d_recv_w, void *stream);

/* Combine with its epilogue ("Deep Dive - DeepEP", "Combine: reverse routing
 * plus reduction": zero, one or two bf16 bias tensors in the combine
 * epilogue; optional return of the top-k weights).
 *
 * As ep_combine, then in fp32 and in this order: acc += bias0[t,i] (if
 * d_bias0), acc += bias1[t,i] (if d_bias1), then one bf16 rounding.  Biases
 * are device bf16 [T, H]; a NULL bias is no term.
 * d_combined_w (device fp32 [T, K], optional; needs d_recv_w, the per-row
 * weights dispatch wrote): combined_w[t,k] = recv_w[slot_of[t,k]], 0 for an
 * unused selection.  With both biases and d_combined_w NULL this is exactly
 * ep_combine.  Returns EP_OK or an error. */
EP_API int32_t ep_combine_epilogue(const ep_config *cfg, const ep_layout *layout,
                                   const void *d_expert_out,
                                   const float *d_topk_weights,
                                   const void *d_bias0, const void *d_bias1,
                                   const float *d_recv_w, void *d_y,
                                   float *d_combined_w, void *stream);

/* Backward of dispatch ("Deep Dive - DeepEP", combine section, backward
 * duality: dispatch and combine are transposes -- copying rows forward
 * becomes summing their gradients backward).
 * d_grad_recv: device bf16 [cap, H], the gradient of the dispatched rows.
 * d_grad_x: device bf16 [T, H]; grad_x[t,i] = bf16( sum over k ascending,
 *   slot_of[t,k] >= 0, of grad_recv[slot_of[t,k], i] ), fp32 from +0.
 * d_grad_recv_w / d_grad_w (both or neither; device fp32 [cap] / [T, K]):
 *   the weights rode along as copies, so grad_w[t,k] =
 *   grad_recv_w[slot_of[t,k]], 0 for an unused selection.
 * Returns EP_OK or an error. */
EP_API int32_t ep_dispatch_backward(const ep_config *cfg, const ep_layout *layout,
                                    const void *d_grad_recv,
                                    const float *d_grad_recv_w, void *d_grad_x,
                                    float *d_grad_w, void *stream);

/* Backward of combine (same source: the transpose of the weighted row sum,
 * and the gate gradient the surrounding autograd needs).
 * d_dy: device bf16 [T, H], the gradient of y.
 * d_grad_expert_out: device bf16 [cap, H]; grad[slot_of[t,k], i] =
 *   bf16( w[t,k] * dy[t,i] ) (fp32 product, one rounding); with
 *   d_topk_weights NULL the weight is 1 and the rows are bit copies of dy
 *   (a dispatch of dy).  Rows of unused selections are not written;
 *   alignment gap rows are zeroed when cfg->zero_padding.
 * d_grad_w (optional, device fp32 [T, K]; needs d_expert_out, the forward
 *   expert rows): grad_w[t,k] = sum_i dy[t,i] * Y[slot_of[t,k], i] in fp32 in
 *   a fixed order (deterministic run to run), 0 for an unused selection.
 * Gradients of the combine biases are dy itself.  Returns EP_OK or an
 * error. */
EP_API int32_t ep_combine_backward(const ep_config *cfg, const ep_layout *layout,
                                   const void *d_dy, const float *d_topk_weights,
                                   const void *d_expert_out,
                                   void *d_grad_expert_out, float *d_grad_w,
                                   void *stream);

/* ---- Non-expanded (destination-major) stage ------------------------------
 * ("Deep Dive - DeepEP", "Why expert parallelism needs a communication
 * layer": a token travels once to each selected destination rank and an
 * optional expansion then makes one slot per expert; "Dispatch: layout,
 * move, and epilogue": in non-expanded mode a received row is a source token
 * with its top-k metadata; "GPU Microarchitecture: DeepEP from First
 * Principles" 2.1 and 1.2: receive buffer -> expert buffer, and on the way
 * back expert-major -> destination-major -> token-major.)
 * All four need a layout computed with the rank-row pointers set
 * (layout->rank_row_start / rank_slot_of / rank_src); rows = rank_row_start[R]
 * <= ep_rank_rows_capacity(cfg).  bf16 rows; d_topk_idx is the int64 [T, K]
 * routing the layout was computed from. */

/* Rows the destination-major buffer may need: max_tokens * min(K, R). */
EP_API int64_t ep_rank_rows_capacity(const ep_config *cfg);

/* rank_x[row(t,r)] = x[t] for every rank r that owns one of token t's
 * experts.  Per rank row, K entries of metadata: d_rank_topk_idx (int32) =
 * local expert id e - r*E/R where the token's k-th expert is on rank r, -1
 * elsewhere; d_rank_topk_w (fp32, optional) = that selection's weight, 0
 * elsewhere.  Returns EP_OK or an error. */
EP_API int32_t ep_dispatch_ranks(const ep_config *cfg, const ep_layout *layout,
                                 const void *d_x, const int64_t *d_topk_idx,
                                 const float *d_topk_weights, void *d_rank_x,
                                 int32_t *d_rank_topk_idx, float *d_rank_topk_w,
                                 void *stream);

/* Expansion: recv_x[slot_of[t,k]] = rank_x[row(t, rank of expert k)] for
 * every (t,k) that is not an unused (-1) selection; d_recv_w[slot] = d_rank_topk_w[row, k] (both or
 * neither).  expand(dispatch_ranks(x)) equals ep_dispatch(x) row for row.
 * cfg->zero_padding clears the alignment gap rows.  Returns EP_OK or an
 * error. */
EP_API int32_t ep_expand(const ep_config *cfg, const ep_layout *layout,
                         const int64_t *d_topk_idx, const void *d_rank_x,
                         const float *d_rank_topk_w, void *d_recv_x,
                         float *d_recv_w, void *stream);

/* Per-rank reduction, the destination rank's partial sum before the rows go
 * back: rank_y[row(t,r), i] = bf16( fold over k ascending whose expert is on
 * rank r of acc = fmaf(w[t,k], expert_out[slot_of[t,k], i], acc) ), acc from
 * +0, weight 1 when d_topk_weights is NULL.  The bf16 partial is the extra
 * rounding of a two-stage reduction ("Combine: reverse routing plus
 * reduction": 256 + 1 rounds to 256, then 256 - 256 = 0).  Returns EP_OK or
 * an error. */
EP_API int32_t ep_reduce_ranks(const ep_config *cfg, const ep_layout *layout,
                               const int64_t *d_topk_idx, const void *d_expert_out,
                               const float *d_topk_weights, void *d_rank_y,
                               void *stream);

/* Token-major sum over destination ranks: y[t,i] = bf16( fold over r
 * ascending with a row for (t, r) of acc += rank_y[row, i] ), fp32 from +0.
 * Needs R <= 64.  Returns EP_OK or an error. */
EP_API int32_t ep_combine_ranks(const ep_config *cfg, const ep_layout *layout,
                                const void *d_rank_y, void *d_y, void *stream);

/* ---- Host buffers ---------------------------------------------------------
 * For callers whose token rows live in host memory (CPU-resident activations,
 * a serving loop that stages batches on the host).  Results equal
 * ep_dispatch / ep_combine bit for bit.  num_chunks selects how the rows
 * cross the host link:
 *  - 0 (direct): no copy and no staging buffer.  The kernel reads
 *    (dispatch) or writes (combine) the host rows in place, each byte once
 *    over the link, on `stream` alone.  The host buffer must be page-locked
 *    memory the device can address (cudaHostAlloc, or cudaHostRegister with
 *    mapping) whose device address is 16-byte aligned, else
 *    EP_ERR_INVALID_ARG; the staging pointer is not used and may be NULL.
 *    Where kernels reach the link's rate, this saves the staging traffic
 *    and the chunk hand-offs.
 *  - 1..64 (chunked): the rows move in token chunks on a copy stream the
 *    library owns, and each chunk's dispatch or combine waits only for its
 *    own chunk's copy ("Deep Dive - DeepEP", "EventOverlap: a stream
 *    contract": streams let data movement and compute overlap; readiness is
 *    a stream dependency on an event, not a host wait).  num_chunks is an
 *    upper bound: a chunk carries at least 4 MiB of rows (T rows of 2H
 *    bytes split into n = min(num_chunks, max(1, floor(2HT / 4 MiB)))
 *    chunks of ceil(T / n) tokens, the last ragged); a single chunk is
 *    copied on `stream` itself, with no copy stream involved.  The first
 *    chunked call on a device creates that device's two copy streams, one
 *    for rows coming in (ep_dispatch_from_host) and one for rows going out
 *    (ep_combine_to_host), and their events (kept until exit).  Calls of
 *    one direction on one device share its stream, so their copies run in
 *    call order; the two directions run at once, so a combine's rows going
 *    out can overlap the next batch's rows coming in when the two calls
 *    are on different streams.  Calls are made from one host thread at a
 *    time.  Host buffers should be pinned (page-locked): pageable memory
 *    works but its copies do not overlap. */

/* As ep_dispatch with x in host memory (h_x: host bf16 [T, H]).  Direct
 * (num_chunks = 0): the dispatch kernel reads h_x in place; d_x is unused.
 * Chunked: h_x is copied into d_x (device bf16 [T, H], a staging buffer the
 * caller owns and that holds x afterwards) chunk by chunk, overlapped with
 * the dispatch of the chunks already copied; the copies start once the work
 * enqueued on `stream` before this call is done (so d_x may still be read
 * by it).  cfg->use_fp8_dispatch and cfg->zero_padding act as in
 * ep_dispatch.  Returns EP_OK or an error. */
EP_API int32_t ep_dispatch_from_host(const ep_config *cfg, const ep_layout *layout,
                                     const void *h_x, void *d_x,
                                     const float *d_topk_weights, void *d_recv_x,
                                     float *d_recv_scale, float *d_recv_w,
                                     int32_t num_chunks, void *stream);

/* As ep_combine with y returned to host memory (h_y: host bf16 [T, H]).
 * Direct (num_chunks = 0): the combine kernel writes h_y in place; d_y is
 * unused.  Chunked: each chunk of tokens is combined into d_y (device bf16
 * [T, H], staging owned by the caller) and then copied to h_y while later
 * chunks combine.  Either way, work enqueued on `stream` after this call
 * starts after the last row reached h_y, so a synchronisation of `stream`
 * makes h_y readable.  Returns EP_OK or an error. */
EP_API int32_t ep_combine_to_host(const ep_config *cfg, const ep_layout *layout,
                                  const void *d_expert_out, const float *d_topk_weights,
                                  void *d_y, void *h_y, int32_t num_chunks, void *stream);

/* Synchronises `stream` and returns the status recorded in the layout's
 * device error word by the last layout call (EP_OK if none): routing errors,
 * else EP_ERR_TIMEOUT_PENDING or EP_ERR_TIMEOUT if one of its bounded
 * on-chip waits gave up.  Each layout call clears the word before its
 * kernels record anything, so a status never carries over from an earlier
 * call.  After a timeout, part of the layout was not written: do not use it
 * for dispatch or combine. */
EP_API int32_t ep_check_error(const ep_layout *layout, void *stream);

/* Self-test of the FP8 dispatch arithmetic ("Deep Dive - DeepEP",
 * "Precision: FP8 on the wire, BF16 for the reduction": one fp32 scale per
 * 128 values; the scale here is amax / 448 and each value is quantised from
 * x / scale rounded to nearest).  The dispatch forms x / scale as a product
 * with the block's reciprocal plus one fused multiply-add correction, which
 * may differ from the IEEE quotient in its last bit (blocks whose scale is
 * below 2^-100 or infinite divide); this runs the dispatch's quotient for
 * every positive bf16 block maximum, finite or +inf, and every bf16 value x
 * with |x| <= amax (about 2^31 pairs: the whole non-NaN input domain)
 * beside the IEEE division and compares the E4M3 codes.
 * d_counts: device uint64 [3], 16-byte aligned: [0] = pairs whose E4M3
 * codes differ (0: the dispatch's codes equal those of the IEEE division),
 * [1] = pairs whose fp32 quotients differ, [2] = those of them whose IEEE
 * quotient is a normal fp32 number (information only).  d_first: device
 * int32, -1 or (amax bits << 16 | x bits) of one code mismatch.
 * Asynchronous on `stream`.  Returns EP_OK or an error. */
EP_API int32_t ep_selftest_fp8_quotient(uint64_t *d_counts, int32_t *d_first,
                                        void *stream);

/* Self-test of the bounded on-chip wait (the layout kernel's wait for its
 * bulk copies):
 * launches one CTA that waits on a shared-memory barrier nothing will ever
 * complete, with a limit of timeout_ns nanoseconds.  The wait gives up, the
 * kernel records EP_ERR_TIMEOUT in d_err (device int32, OR-ed in) and
 * returns; the GPU context stays usable.  Synchronises `stream` and returns
 * the recorded status (EP_ERR_TIMEOUT when the mechanism works).
 * timeout_ns must be in [1000, 10^9]. */
EP_API int32_t ep_selftest_wait_timeout(int64_t timeout_ns, int32_t *d_err,
                                        void *stream);

/* Self-test of the layout's own bounded wait ("Deep Dive - DeepEP",
 * "Benchmark and failure-mode checklist": a timeout is a failure boundary,
 * reported, never a hang).  Runs the two-launch layout of ep_get_layout
 * (same arguments; num_tokens * K above 4096 or E above 2048, so that the
 * layout takes two launches) except that CTA `stall_tile` of its second
 * kernel issues no copy of the per-tile counts and waits for it with a
 * limit of timeout_ns nanoseconds (in [1000, 10^9]).  That wait gives up,
 * the CTA records EP_ERR_TIMEOUT in the layout's error word and returns
 * without writing its rows; the other CTAs finish.  stall_tile must be in
 * [0, CTAs of that kernel): 0 .. max(tiles, min(E, 152)) - 1, where tiles
 * is the number of token tiles (at most 152).  Synchronises `stream` and
 * returns the recorded status (EP_ERR_TIMEOUT when the mechanism works);
 * the layout it leaves is incomplete and must not be used. */
EP_API int32_t ep_selftest_layout_timeout(const ep_config *cfg, int32_t num_tokens,
                                          const int64_t *d_topk_idx, ep_layout *layout,
                                          int32_t stall_tile, int64_t timeout_ns,
                                          void *stream);

/* ---- Router gate ----------------------------------------------------------
 * What produces topk_idx and topk_weights: scores, choice, gate weights, the
 * balance and z losses over them, and the gradient by the logits.
 *
 * Score s_te of token t for expert e: softmax over e of the logits l_te, or
 * sigmoid(l_te).  Choice score: l_te itself (softmax; the same order), or
 * s_te + bias_e (sigmoid; the bias orders, it never enters a weight; a bias
 * of -inf or NaN takes its expert out of the choice, not out of the scores).  A
 * logit of -inf takes its expert out of service for that token (score 0,
 * never chosen); a NaN logit is never chosen either and its row's softmax
 * scores are NaN.  With num_groups > 1, groups of E / num_groups consecutive
 * experts are ranked by their highest choice score (softmax) or the sum of
 * their two highest (sigmoid), and only experts of the topk_groups best
 * groups can be chosen.  The K highest choice scores are chosen in
 * descending order; equal scores, of experts or of groups, go to the lower
 * index.  w_tk = route_scale * s of choice k, divided by the sum of the
 * chosen s when renormalize is set (0 where that sum is 0).  Where fewer than
 * K experts can be chosen, and for masked tokens, idx = -1 and w = 0 (an
 * unused selection of ep_get_layout).  A score under 2^-126 is taken as 0;
 * its expert can be chosen all the same. */
enum { EP_SCORE_SOFTMAX = 0, EP_SCORE_SIGMOID = 1 };

typedef struct {
  int32_t num_experts;   /* E in [1, 2048]                                  */
  int32_t num_topk;      /* K in [1, 32], K <= topk_groups * E / num_groups */
  int32_t score;         /* EP_SCORE_SOFTMAX or EP_SCORE_SIGMOID            */
  int32_t num_groups;    /* in [1, 32], divides E; 1: no groups             */
  int32_t topk_groups;   /* in [1, num_groups]                              */
  int32_t renormalize;   /* 1: the chosen scores are divided by their sum   */
  int32_t logits_bf16;   /* logits and their gradient: 0 fp32, 1 bf16       */
  float route_scale;     /* factor of every gate weight                     */
} ep_router_config;

/* Choice and gate weights of num_tokens (T, at most 2^30) tokens.
 * d_logits: device [T, ld_logits] fp32 or bf16, ld_logits >= E (entries past
 *   E are not read).
 * d_bias: device fp32 [E] or NULL; sigmoid scores only.
 * d_token_mask: device uint8 [T] or NULL; 0 marks a padding token.
 * d_topk_idx: device int64 [T, K]; d_topk_weights: device fp32 [T, K].
 * Returns EP_OK or an error. */
EP_API int32_t ep_route(const ep_router_config *cfg, int32_t num_tokens,
                        const void *d_logits, int64_t ld_logits, const float *d_bias,
                        const uint8_t *d_token_mask, int64_t *d_topk_idx,
                        float *d_topk_weights, void *stream);

/* Bytes of device scratch memory ep_route_balance needs on the current
 * device, for any number of tokens.  -1 if the arguments are invalid. */
EP_API int64_t ep_route_workspace_bytes(const ep_router_config *cfg, int32_t num_seqs);

/* ep_route together with the balance statistics and losses of its tokens.
 *
 * The tokens form B = num_seqs (1 to 2^20) sequences: d_seq_start (device
 * int32 [B + 1], NULL when B = 1) ascends from 0 to T, sequence b owns tokens
 * [seq_start[b], seq_start[b+1]) and may be empty.  Masked tokens count
 * nowhere.  With n_b the tokens of sequence b, c_be their selections of
 * expert e, and p_te = s_te / (sum of s_t over the experts):
 *   d_expert_count: int32 [B, E]  c_be
 *   d_expert_prob:  fp32 [B, E]   P_be = mean of p_te over the n_b tokens
 *   d_seq_tokens:   int32 [B+2]   n_b; then sum n_b; then how many n_b > 0
 *   d_loss[0] = mean over sequences with n_b > 0 of
 *               sum_e (c_be E / (K n_b)) P_be       (1 when balanced)
 *   d_loss[1] = mean over tokens of logsumexp(l_t)^2 (softmax; else 0)
 * A row with no expert in service adds nothing to P or the z loss.  Both
 * losses are 0 without tokens.  Sums are fp32 in a fixed order: the same
 * inputs give the same bits.  d_workspace: ep_route_workspace_bytes bytes,
 * used until the call's work is done.  num_tokens may be 0.
 * Returns EP_OK or an error. */
EP_API int32_t ep_route_balance(const ep_router_config *cfg, int32_t num_tokens,
                                const void *d_logits, int64_t ld_logits,
                                const float *d_bias, const uint8_t *d_token_mask,
                                int32_t num_seqs, const int32_t *d_seq_start,
                                int64_t *d_topk_idx, float *d_topk_weights,
                                int32_t *d_expert_count, float *d_expert_prob,
                                int32_t *d_seq_tokens, float *d_loss, void *d_workspace,
                                void *stream);

/* Gradient by the logits of  sum_tk grad_w_tk w_tk + grad_loss . loss, the
 * choice and the counts c_be held constant.
 * d_grad_w: device fp32 [T, K] or NULL (no gate term; ep_combine_backward
 *   writes it); d_topk_idx: the forward's choice, needed with d_grad_w.
 * d_expert_count, d_seq_tokens (ep_route_balance's) and d_grad_loss (device
 *   fp32 [2]): all three, or all NULL (no loss terms).  grad_loss[1] is not
 *   used with sigmoid scores.
 * d_grad_logits: device [T, ld_grad], the type of the logits; columns past E
 *   are not written.  Masked tokens get 0, and so do experts out of service
 *   where their token's gradients and coefficients are finite.
 * Everything else is recomputed from the logits.  Returns EP_OK or an
 * error. */
EP_API int32_t ep_route_backward(const ep_router_config *cfg, int32_t num_tokens,
                                 const void *d_logits, int64_t ld_logits,
                                 const uint8_t *d_token_mask, const int64_t *d_topk_idx,
                                 const float *d_grad_w, int32_t num_seqs,
                                 const int32_t *d_seq_start,
                                 const int32_t *d_expert_count,
                                 const int32_t *d_seq_tokens, const float *d_grad_loss,
                                 void *d_grad_logits, int64_t ld_grad, void *stream);

/* ---- Experts' products with 4-bit weights ----------------------------------
 * y_r = W_e x_r for the rows r of every expert e, between ep_dispatch and
 * ep_combine, with W_e [N, H] held as 4-bit codes: W = (code - zero) * scale,
 * one bf16 scale (and optionally one zero point; 8 otherwise) per row and
 * group of group_size inputs.  With `gated`, W_e stacks a gate and an up
 * matrix ([N/2, H] each) and y = silu(gate x) * (up x), N/2 wide.
 *
 * Made for few rows an expert (decode: one to some dozens), where reading
 * the weights once is the cost; any number of rows is computed correctly.
 *
 * Packed weights: tiles of 64 packed rows by blocks of 128 inputs.  Packed
 * row n of a tile is row 64 * tile + n of W; when gated, a tile covers 32
 * outputs and packed row 8 g + p is gate row 32 * tile + 4 g + p for p < 4,
 * up row 32 * tile + 4 g + p - 4 for p >= 4.
 *   codes:  uint32 [E, tiles, blocks, 8, 32, 4]; word (p, l, i) holds inputs
 *           32 i + 8 (l % 4) + 2 j and + 2 j + 1 of the block, for packed row
 *           8 (l / 4) + p, in its 4-bit fields j and j + 4 (j = 0..3)
 *   scales: bf16 [E, tiles, blocks * 128 / group_size, 64] (group, packed row)
 *   zeros:  uint8, as the scales
 * Rows past N and inputs past H are padding: code 8, scale 0, zero 8. */
typedef struct {
  int32_t num_experts;   /* E in [1, 2048]                                   */
  int32_t in_features;   /* H: a multiple of group_size, <= 2^20; of 128 when
                            x_fp8                                            */
  int32_t out_features;  /* N in [1, 2^20]; even when gated                  */
  int32_t group_size;    /* 32, 64 or 128 inputs a scale                     */
  int32_t x_fp8;         /* 0: bf16 rows; 1: E4M3 rows with 1x128 fp32 scales */
  int32_t gated;         /* 1: silu(gate) * up                               */
  int32_t has_zeros;     /* 1: zero points, in [0, 15]                       */
} ep_w4_config;

/* Bytes of the packed codes, scales and zeros (0 without zero points);
 * -1 if the config is invalid. */
EP_API int64_t ep_w4_codes_bytes(const ep_w4_config *cfg);
EP_API int64_t ep_w4_scales_bytes(const ep_w4_config *cfg);
EP_API int64_t ep_w4_zeros_bytes(const ep_w4_config *cfg);

/* Packs weights once, before serving.  d_codes: device uint8 [E, N, H / 2],
 * input 2 i in the low four bits of byte i; d_scales: device bf16
 * [E, N, H / group_size]; d_zeros: device uint8, as the scales (has_zeros).
 * Returns EP_OK or an error. */
EP_API int32_t ep_w4_pack(const ep_w4_config *cfg, const uint8_t *d_codes,
                          const void *d_scales, const uint8_t *d_zeros,
                          void *d_packed_codes, void *d_packed_scales,
                          uint8_t *d_packed_zeros, void *stream);

/* The product.  cap: rows that d_x and d_out hold.  num_rows: how many rows
 * the experts have together, at most (T * K of the layout's call; it sizes
 * the launch, and more rows are still computed; 0 launches nothing).
 * d_x: device [cap, H] bf16, or E4M3 bytes with d_x_scale (device fp32
 *   [cap, H / 128]), as ep_dispatch writes them.
 * d_expert_start, d_expert_end: device int32 [E] at least, a layout's: expert
 *   e owns rows [start[e], end[e]), clipped to [0, cap); none when empty.
 * d_out: device bf16 [cap, N] ([cap, N/2] when gated); rows of no expert
 *   are not written.
 * Products and sums are fp32 (codes and inputs enter them exactly), rounded
 * once at the end; the same call gives the same bits.  A value of x that is
 * not finite shows in its own row alone.  Returns EP_OK or an error. */
EP_API int32_t ep_expert_w4(const ep_w4_config *cfg, int32_t cap, int32_t num_rows,
                            const void *d_x, const float *d_x_scale, const void *d_codes,
                            const void *d_scales, const uint8_t *d_zeros,
                            const int32_t *d_expert_start, const int32_t *d_expert_end,
                            void *d_out, void *stream);

/* The cudaError_t of the last CUDA runtime call of this library that failed
 * in the calling thread (0 if none since the previous query); reading it
 * clears it.  Explains an EP_ERR_CUDA status. */
EP_API int32_t ep_last_cuda_error(void);

/* Static, human-readable name of a status code. */
EP_API const char *ep_status_str(int32_t status);

#ifdef __cplusplus
}
#endif
#endif /* EP_GB300_H */
