/*
 * ep.h -- C ABI of a single-GPU MoE token dispatch / combine library for
 * NVIDIA GB300 (sm_103a).
 *
 * The operations follow the DeepEP pages this library is built from:
 *  - "Redundant atomics in internode_ll" (DeepEP issue #282), the quoted
 *    low-latency dispatch excerpt: a token count per expert, and expert e
 *    living on partition e / (experts per partition) as local expert
 *    e % (experts per partition).
 *  - "Reasons for not calling NVSHMEM public APIs?" (DeepEP issue #18), the
 *    answer on low-latency mode: data for one expert keeps its order.
 *  - "Pipeline direct NVLink dispatch with triple-buffered prefetch" (DeepEP
 *    PR #693), Summary: each token carries hidden data, scale factors,
 *    metadata and routing; the next token is prefetched while earlier stores
 *    drain.  Validation table: dispatch and combine are the measured pair.
 * Here all experts live in one GPU's HBM; partitions are logical only.
 *
 * Conventions for every entry point
 *  - Device pointers are raw CUDA device addresses.  The caller allocates and
 *    frees every buffer (including the layout workspace); the library never
 *    allocates, frees or synchronises.
 *  - All work is enqueued on `stream` (NULL = the legacy default stream).  A
 *    return of EP_OK means the work was enqueued; results are ready once the
 *    stream reaches that point.  Calls are stateless and thread-safe.
 *  - Most kernels launch with programmatic stream serialization and let the
 *    next kernel of the stream start early: each waits for the previous
 *    kernel to complete before it writes memory or reads what that kernel may
 *    write (before the wait it only prefetches into L2).  A caller's kernel
 *    that follows and is itself launched programmatically must likewise
 *    execute griddepcontrol.wait (cudaGridDependencySynchronize) before it
 *    reads this library's outputs; kernels launched normally need nothing.
 *  - Arguments are checked on the host before anything is launched; a bad
 *    argument returns EP_ERR_INVALID_ARG (unsupported sizes EP_ERR_UNSUPPORTED)
 *    with nothing enqueued.  A failed launch returns EP_ERR_CUDA.  The text of
 *    the last failure on the calling thread is available from ep_last_error().
 *  - Conditions found on the device never trap: they are OR-ed into the
 *    caller's 32-bit `err_flags` word (EP_ERRF_*), which the caller clears and
 *    reads back.  `err_flags` may be NULL, in which case they are dropped.
 *  - A buffer of zero elements may be passed as NULL.
 *  - Element types: bf16 is stored as 16-bit IEEE bfloat16; fp8 as one byte of
 *    OCP e4m3 ("e4m3fn": bias 7, max 448, no infinities); f32 / i32 native.
 *  - All arrays are dense and row-major.
 */
#ifndef EP_GB300_H_
#define EP_GB300_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define EP_API __attribute__((visibility("default")))
#else
#define EP_API
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st *ep_stream_t;

typedef enum {
    EP_OK = 0,
    EP_ERR_INVALID_ARG = 1,   /* null or misaligned pointer, bad shape       */
    EP_ERR_UNSUPPORTED = 2,   /* valid but beyond this library's limits, or no
                                 sm_103 device current                        */
    EP_ERR_CUDA = 3           /* a CUDA runtime call or launch failed         */
} ep_status_t;

typedef enum {
    EP_LAYOUT_PACKED = 0,     /* R = T*k rows, expert e owns rows
                                 [offsets[e], offsets[e+1])                   */
    EP_LAYOUT_CAPACITY = 1    /* R = E*capacity rows, expert e owns rows
                                 [e*capacity, (e+1)*capacity)                 */
} ep_layout_mode_t;

/* Payload format of ep_dispatch. */
typedef enum {
    EP_PAYLOAD_BF16 = 0,      /* recv is bf16 [R, H], a bit copy of x         */
    EP_PAYLOAD_FP8_E4M3 = 1,  /* recv is e4m3 [R, H] plus f32 scales [R, H/128] */
    EP_PAYLOAD_FP8_E4M3_UE8M0 = 2 /* e4m3 [R, H] plus power-of-two scales stored
                                 as u8 biased exponents [R, H/128] (UE8M0:
                                 scale = 2^(e - 127))                          */
} ep_payload_t;

/* Bits of the device error word. */
enum {
    EP_ERRF_BAD_EXPERT = 1u,  /* a topk_idx entry outside [-1, E); treated as -1 */
    EP_ERRF_CAPACITY = 2u,    /* capacity mode dropped at least one copy      */
    EP_ERRF_TIMEOUT = 4u,     /* an internal bounded wait ran out; outputs of
                                 that call are incomplete                     */
    EP_ERRF_BAD_SLOT = 8u,    /* a slot_of entry >= R (or < -1); that copy was
                                 skipped                                      */
    EP_ERRF_BAD_SEQ = 16u     /* ep_route: seq_offsets does not rise from 0 to T */
};

/* Limits of this library. */
#define EP_MAX_EXPERTS 1024
#define EP_MAX_TOPK 32

typedef struct {
    int32_t T;                /* tokens, >= 0                                  */
    int32_t H;                /* hidden channels, > 0, multiple of 8 (of 128
                                 for fp8 payloads)                             */
    int32_t E;                /* experts, 1..EP_MAX_EXPERTS                    */
    int32_t k;                /* experts per token, 1..min(E, EP_MAX_TOPK)     */
    int32_t num_partitions;   /* P >= 1, divides E; partition p holds experts
                                 [p*E/P, (p+1)*E/P)                            */
    int32_t mode;             /* ep_layout_mode_t                              */
    int32_t capacity;         /* rows per expert, >= 1 in capacity mode        */
} ep_shape_t;

/* Rows R of the receive buffer for this shape; -1 if the shape is invalid. */
EP_API int64_t ep_recv_rows(const ep_shape_t *shape);

/* Bytes of device workspace ep_get_layout needs for this shape (may be 0);
 * (size_t)-1 if the shape is invalid. */
EP_API size_t ep_layout_workspace_bytes(const ep_shape_t *shape);

/*
 * ep_get_layout -- turn top-k routing into the per-expert layout.
 *
 * Passages: the per-expert token count and the division of experts into
 * partitions (expert e on partition e / (E/P)) follow the low-latency
 * dispatch excerpt quoted in "Redundant atomics in internode_ll" (DeepEP
 * issue #282, question); the order inside an expert follows "Reasons for not
 * calling NVSHMEM public APIs?" (DeepEP issue #18, answer on low-latency
 * mode: the data of one expert keeps its order).  The pages do not give the
 * layout as a separate call; on one GPU the count exchange they describe
 * becomes this call.
 *
 * In:  topk_idx   i32 [T, k]  expert of copy (t, j); -1 = masked slot.
 * Out: counts       i32 [E]    copies routed to each expert (true demand,
 *                              also in capacity mode).
 *      offsets      i32 [E+1]  exclusive prefix sum of counts.
 *      part_counts  i32 [P]    counts summed over each partition.
 *      part_offsets i32 [P+1]  exclusive prefix sum of part_counts.
 *      slot_of      i32 [T, k] receive row of copy (t, j); -1 if masked or
 *                              dropped for capacity.
 *      src_token    i32 [R]    token of each receive row; -1 if the row holds
 *                              no copy.
 *      src_k        i32 [R]    top-k position j of each receive row; -1 if
 *                              the row holds no copy.
 * Order: rows of one expert hold its copies in increasing (t, j), so the
 * result is deterministic and equals a stable sort of the flattened ids.
 *   packed:   slot = offsets[e] + rank(t, j),
 *   capacity: slot = e*capacity + rank if rank < capacity, else dropped
 *             (EP_ERRF_CAPACITY),
 * rank(t, j) = number of copies (t', j') < (t, j) routed to the same expert.
 * workspace: device buffer of ep_layout_workspace_bytes(shape) bytes, owned
 * by the caller, contents on entry ignored; NULL allowed when that is 0.
 * err_flags: EP_ERRF_BAD_EXPERT, EP_ERRF_CAPACITY.
 */
EP_API ep_status_t ep_get_layout(const ep_shape_t *shape, const int32_t *topk_idx,
                          int32_t *counts, int32_t *offsets,
                          int32_t *part_counts, int32_t *part_offsets,
                          int32_t *slot_of, int32_t *src_token, int32_t *src_k,
                          void *workspace, size_t workspace_bytes,
                          uint32_t *err_flags, ep_stream_t stream);

/*
 * ep_get_layout_static -- ep_get_layout without a caller-supplied workspace.
 * The pages have no counterpart of this entry point: it exists for callers
 * that cannot allocate device memory where they compute the layout (code
 * confined to a fixed memory budget owned by a host framework, or a latency-
 * critical path on which a device allocation could stall the device).
 *
 * Same arguments, outputs, ordering and err_flags as ep_get_layout, minus
 * workspace / workspace_bytes.  Scratch comes from a 1 MiB array built into
 * the library (every GPU that loads the library holds it until the process
 * exits): shapes needing more than 1 MiB of layout workspace, i.e.
 * ceil(T*k / 1024) * E * 4 bytes > 1 MiB (about 2^20 routing entries at
 * E = 256), return EP_ERR_UNSUPPORTED; smaller shapes that need no workspace
 * use none.  The array's device address is looked up on the first call that
 * needs it in each device context, with that context current, and reused
 * while the same context lives (a context created later, e.g. after
 * cudaDeviceReset, gets its own lookup); make that first call before any
 * stream capture.  All calls share the array and it keeps the
 * last call's contents (each call writes every entry it reads, so nothing
 * needs clearing); calls whose work overlaps on the GPU race on it and must
 * be ordered by the caller.  Allocates nothing.
 */
EP_API ep_status_t ep_get_layout_static(const ep_shape_t *shape, const int32_t *topk_idx,
                          int32_t *counts, int32_t *offsets,
                          int32_t *part_counts, int32_t *part_offsets,
                          int32_t *slot_of, int32_t *src_token, int32_t *src_k,
                          uint32_t *err_flags, ep_stream_t stream);

/*
 * ep_dispatch -- copy every token's hidden row to each receive row it is
 * routed to (slot_of from ep_get_layout; R = ep_recv_rows(shape)).
 *
 * In:  x        bf16 [T, H], 16-byte aligned.
 *      topk_w   f32 [T, k] routing weights, or NULL.
 *      slot_of  i32 [T, k] receive row of each copy, -1 = none; each
 *               non-negative value should appear at most once (rows written
 *               twice end up with either copy); values outside [-1, R) are
 *               skipped and flagged EP_ERRF_BAD_SLOT.
 * Out: recv     EP_PAYLOAD_BF16:     bf16 [R, H]: recv[slot_of[t,j]] = x[t].
 *               EP_PAYLOAD_FP8_E4M3: e4m3 [R, H]; per token t and channel
 *               block b of 128: s = max(amax, 1e-4) / 448 (fp32, round to
 *               nearest), q = e4m3(x / s) (fp32 division rounded to nearest,
 *               then nearest e4m3, ties to even, saturating at +-448).
 *               16-byte aligned.
 *               EP_PAYLOAD_FP8_E4M3_UE8M0: as E4M3 but s is the smallest
 *               power of two >= max(amax, 1e-4) / 448 (that quotient rounded
 *               to nearest in fp32), so x / s is exact ("Support UE8M0 data
 *               format", referenced from "Redundant atomics in
 *               internode_ll").
 *      recv_scales (fp8 only, else ignored): E4M3: f32 [R, H/128], s of each
 *               block, 16-byte aligned; E4M3_UE8M0: u8 [R, H/128], the biased
 *               exponent e of each block's s = 2^(e - 127).
 *      recv_w   f32 [R] or NULL: recv_w[slot_of[t,j]] = topk_w[t,j]
 *               (needs topk_w).
 * Rows of recv / recv_scales / recv_w that receive no copy are not written.
 * err_flags: EP_ERRF_TIMEOUT, EP_ERRF_BAD_SLOT.
 */
EP_API ep_status_t ep_dispatch(const ep_shape_t *shape, const void *x,
                        const float *topk_w, const int32_t *slot_of,
                        int32_t payload, void *recv, void *recv_scales,
                        float *recv_w, uint32_t *err_flags, ep_stream_t stream);

/*
 * ep_layout_dispatch -- ep_get_layout followed by ep_dispatch, in one launch
 * when the batch is small (T*k <= 2048 and T <= 2048), otherwise as those two
 * calls.  Small decode batches are where a launch matters ("Why does DeepEP
 * LL kernel use double send/recv/signal buffers?", last answer: the design
 * targets high tokens per second), and the v1 low-latency path avoided a
 * separate count exchange ("Why did DeepEP v2 drop the double-buffer
 * design...", question).
 *
 * Arguments, outputs, ordering, checks and err_flags are exactly those of
 * ep_get_layout (topk_idx .. src_k, workspace, workspace_bytes) and
 * ep_dispatch (x, topk_w, payload, recv, recv_scales, recv_w) on the same
 * shape; every output is bit-identical to the two separate calls.  The
 * workspace is only used on the two-call path (size from
 * ep_layout_workspace_bytes).
 */
EP_API ep_status_t ep_layout_dispatch(const ep_shape_t *shape, const int32_t *topk_idx,
                          const void *x, const float *topk_w, int32_t payload,
                          int32_t *counts, int32_t *offsets,
                          int32_t *part_counts, int32_t *part_offsets,
                          int32_t *slot_of, int32_t *src_token, int32_t *src_k,
                          void *recv, void *recv_scales, float *recv_w,
                          void *workspace, size_t workspace_bytes,
                          uint32_t *err_flags, ep_stream_t stream);

/*
 * ep_combine -- weighted top-k reduce of expert outputs back to token order.
 *
 * Passage: combine is the reverse of dispatch and is measured beside it in
 * "Pipeline direct NVLink dispatch with triple-buffered prefetch" (DeepEP PR
 * #693), Validation table (combine GB/s unchanged by the dispatch pipeline,
 * balanced and unbalanced); the pages do not spell out its arithmetic, which
 * is read here as the weighted sum of the token's k expert outputs.
 *
 * In:  y        bf16 [R, H] expert outputs in the receive layout, 16-byte
 *               aligned.
 *      topk_w   f32 [T, k], or NULL for an unweighted sum (weights applied on
 *               the expert side, e.g. from ep_dispatch's recv_w).
 *      slot_of  i32 [T, k] from ep_get_layout (-1 = skipped; values outside
 *               [-1, R) are skipped and flagged EP_ERRF_BAD_SLOT).
 * Out: out      bf16 [T, H], 16-byte aligned:
 *               out[t] = bf16( sum_{j: slot_of[t,j] >= 0} topk_w[t,j] * y[slot_of[t,j]] ),
 *               accumulated in fp32 in increasing j from 0 (each product and
 *               sum rounded to nearest), rounded once to bf16 (nearest even).
 *               A token with no valid slot gets 0.
 * err_flags: EP_ERRF_BAD_SLOT.
 */
EP_API ep_status_t ep_combine(const ep_shape_t *shape, const void *y,
                       const float *topk_w, const int32_t *slot_of, void *out,
                       uint32_t *err_flags, ep_stream_t stream);

/*
 * ep_combine_fp8 -- ep_combine over fp8 expert outputs (the e4m3 variant of
 * the combine the pages measure beside dispatch, "Pipeline direct NVLink
 * dispatch with triple-buffered prefetch", Validation table).
 *
 * In:  y        e4m3 [R, H] expert outputs in the receive layout, 16-byte
 *               aligned; H % 128 == 0.
 *      y_scales payload EP_PAYLOAD_FP8_E4M3: f32 [R, H/128] (4-byte aligned);
 *               EP_PAYLOAD_FP8_E4M3_UE8M0: u8 [R, H/128] biased exponents,
 *               scale = 2^(e - 127).
 *      topk_w, slot_of, out, err_flags as ep_combine.
 * Each element is dequantised as v = value(code) * scale (fp32 product,
 * rounded to nearest), then out[t] = bf16( sum_j topk_w[t,j] * v ) in fp32 in
 * increasing j, as ep_combine.
 */
EP_API ep_status_t ep_combine_fp8(const ep_shape_t *shape, const void *y,
                       const void *y_scales, int32_t payload,
                       const float *topk_w, const int32_t *slot_of, void *out,
                       uint32_t *err_flags, ep_stream_t stream);

/*
 * ep_combine_src -- the combine addressed from the expert side.  The caller
 * holds, for every row of the expert-major buffer, the token and top-k
 * position the row was dispatched from (ep_get_layout's src_token / src_k)
 * and, optionally, the row's own weight (ep_dispatch's recv_w: the routing
 * information that travels with each token, "Pipeline direct NVLink dispatch
 * with triple-buffered prefetch", Summary), instead of the token-side slot_of.
 * Copy j of token t is the row r with (src_token[r], src_k[r]) = (t, j); the
 * rows are read in place (no copy of y is made).
 *
 * In:  y, y_scales, payload  as ep_combine (payload EP_PAYLOAD_BF16, y_scales
 *               NULL) or ep_combine_fp8 (the two fp8 payloads).
 *      row_w    f32 [R] weight of each row, or NULL for an unweighted sum.
 *      src_token, src_k  i32 [R]: the pair each row holds, src_token = -1 in a
 *               row that holds no copy.  Each pair appears in at most one row
 *               (as ep_get_layout writes them; if several rows claim a pair,
 *               which one is used is unspecified).  A row whose pair lies
 *               outside [0,T) x [0,k) (other than src_token = -1) is skipped
 *               and flags EP_ERRF_BAD_SLOT.
 *      workspace  device memory of ep_combine_src_workspace_bytes(shape)
 *               bytes, 4-byte aligned, caller-owned; its contents on entry do
 *               not matter.  It receives the token-side map rebuilt from the
 *               source maps, [T, k] rows then [T, k] weights.
 * Out: out      bf16 [T, H]: exactly what ep_combine / ep_combine_fp8 give
 *               with slot_of[t,j] = r and topk_w[t,j] = row_w[r] (bit for
 *               bit): fp32 sum in increasing j, one rounding to bf16; a pair
 *               that no row holds (a dropped or masked copy) adds nothing.
 * err_flags: EP_ERRF_BAD_SLOT.
 */
EP_API size_t ep_combine_src_workspace_bytes(const ep_shape_t *shape);
EP_API ep_status_t ep_combine_src(const ep_shape_t *shape, const void *y,
                       const void *y_scales, int32_t payload, const float *row_w,
                       const int32_t *src_token, const int32_t *src_k, void *out,
                       void *workspace, size_t workspace_bytes,
                       uint32_t *err_flags, ep_stream_t stream);

/* ------------------------------------------------------------------------
 * The ends of a mixture-of-experts block.  No page of the design describes
 * these; they are the calls a block needs around dispatch and combine.
 * Conventions as above (caller-owned buffers, host checks before any launch,
 * nothing allocated, nothing synchronised).  Exception: inputs marked `ld`
 * have rows ld elements apart.
 * ------------------------------------------------------------------------ */

/* Element type of a stream that may be held in either precision. */
typedef enum {
    EP_TYPE_BF16 = 0,
    EP_TYPE_F32 = 1
} ep_type_t;

/* What the block's gate is held for. */
typedef enum {
    EP_GATE_NONE = 0,         /* gate = 1                                     */
    EP_GATE_CHANNEL = 1,      /* f32 [H]                                      */
    EP_GATE_TOKEN = 2         /* f32 [T]                                      */
} ep_gate_kind_t;

#define EP_MAX_NORM_WIDTH 16384

typedef struct {
    int32_t T;                /* rows, >= 0                                    */
    int32_t H;                /* channels, > 0, multiple of 8, at most
                                 EP_MAX_NORM_WIDTH                             */
    int32_t stream_type;      /* ep_type_t of h, h_out, d_h_out and d_h        */
    int32_t gate_kind;        /* ep_gate_kind_t                                */
    float eps;                /* 1e-30..1e30, added to the mean square of both
                                 norms                                         */
} ep_norm_t;

/*
 * ep_block_norm -- the end of one block and the start of the next, one pass
 * over the rows:
 *   u     = y * r1 * w_post,   r1 = 1 / sqrt(mean(y^2) + eps)
 *           (u = y without w_post)
 *   h_out = res_scale * h + gate * u
 *   n     = h_out * r2 * w_pre,  r2 = 1 / sqrt(mean(h_out^2) + eps)
 * Everything is computed in fp32; h_out enters the second norm before it is
 * rounded to the stream's type, and h_out and n are each rounded once.
 *
 * In:  h         stream type [T, H], rows ld_h elements apart.
 *      y         bf16 [T, H], rows ld_y apart (the block's output, e.g. from
 *                ep_combine); NULL: h_out = res_scale * h (the first norm of
 *                a network), w_post and gate must then be absent.
 *      w_post    f32 [H] or NULL;  gate  f32 by gate_kind, NULL for
 *                EP_GATE_NONE;  res_scale  f32 [1] on the device or NULL (1).
 *      w_pre     f32 [H], or NULL when n is not wanted.
 * Out: h_out     stream type [T, H], or NULL when not wanted.
 *      n         bf16 [T, H] (needs w_pre), NULL exactly when w_pre is.
 *      rstd      f32 [2, T]: r1 then r2 of every row, for the backward pass
 *                (entries of a norm that is absent are not written), or NULL.
 * There are no err_flags: should a copy inside the kernel not end within its
 * time limit, the rows of that thread block come out as NaN (rstd too).
 * h and h_out may be the same buffer when ld_h = H.  16-byte alignment of h,
 * y, w_post, w_pre, h_out, n and a channel gate; ld_h and ld_y multiples of 8
 * and at least H.
 */
EP_API ep_status_t ep_block_norm(const ep_norm_t *norm, const void *h, int64_t ld_h,
                          const void *y, int64_t ld_y, const float *w_post,
                          const float *gate, const float *res_scale,
                          const float *w_pre, void *h_out, void *n, float *rstd,
                          ep_stream_t stream);

/* Bytes of device workspace ep_block_norm_backward needs (column sums in
 * progress); (size_t)-1 if the description is invalid. */
EP_API size_t ep_block_norm_workspace_bytes(const ep_norm_t *norm);

/*
 * ep_block_norm_backward -- gradients of ep_block_norm.  With
 * t = d_n * w_pre, hn = h_out * r2, yn = y * r1:
 *   dH     = d_h_out + r2 * (t - hn * mean(t * hn))
 *   d_h    = res_scale * dH              d_res_scale = sum(dH * h)
 *   d_w_pre = sum over rows of d_n * hn
 *   du     = gate * dH                   d_gate = dH * u summed over what the
 *                                        gate is shared by
 *   d_w_post = sum over rows of du * yn
 *   d_y    = r1 * (du * w_post - yn * mean(du * w_post * yn))
 *            (du without w_post)
 * in fp32, h_out recomputed from h and y.  Sums over rows are taken in an
 * order that depends on the sizes alone: a repeated call gives the same bits.
 *
 * In:  the inputs of ep_block_norm and the rstd it wrote; d_h_out stream type
 *      [T, H] or NULL (zero); d_n bf16 [T, H], NULL exactly when w_pre is; at
 *      least one of the two.
 * Out: d_h       stream type [T, H].
 *      d_y       bf16 [T, H], NULL exactly when y is.
 *      d_w_post, d_w_pre  f32 [H], NULL exactly when w_post / w_pre is.
 *      d_gate    f32 [H] or [T], NULL exactly when gate is.
 *      d_res_scale  f32 [1], NULL exactly when res_scale is.
 * workspace: ep_block_norm_workspace_bytes(norm) bytes, 16-byte aligned,
 * contents on entry ignored.  T = 0 sets the sums to zero.
 * err_flags: EP_ERRF_TIMEOUT.
 */
EP_API ep_status_t ep_block_norm_backward(const ep_norm_t *norm, const void *h, int64_t ld_h,
                          const void *y, int64_t ld_y, const float *w_post,
                          const float *gate, const float *res_scale,
                          const float *w_pre, const float *rstd,
                          const void *d_h_out, const void *d_n, void *d_h, void *d_y,
                          float *d_w_post, float *d_gate, float *d_res_scale,
                          float *d_w_pre, void *workspace, size_t workspace_bytes,
                          uint32_t *err_flags, ep_stream_t stream);

#define EP_MAX_ROUTE_GROUPS 32

typedef struct {
    int32_t T;                /* tokens, >= 0                                  */
    int32_t E;                /* experts, 1..EP_MAX_EXPERTS                    */
    int32_t k;                /* experts per token, 1..min(E, EP_MAX_TOPK)     */
    int32_t groups;           /* expert groups, divides E, at most
                                 EP_MAX_ROUTE_GROUPS; 1 = no groups            */
    int32_t topk_groups;      /* groups a token may choose from, 1..groups     */
    int32_t full_softmax;     /* 0: topk_w is the softmax over the chosen
                                 logits; 1: the chosen experts' probabilities
                                 in the softmax over all experts               */
    int32_t logits_type;      /* ep_type_t of logits and d_logits              */
    int32_t num_seqs;         /* sequences the batch consists of, >= 1         */
    float balance_coef;       /* factors of the two losses                     */
    float z_coef;
} ep_route_t;

/* Bytes of device workspace ep_route needs when it computes the losses;
 * (size_t)-1 if the description is invalid. */
EP_API size_t ep_route_workspace_bytes(const ep_route_t *route);

/*
 * ep_route -- choose each token's experts from the router's logits and, for
 * training, count the copies of every expert and compute the balance loss.
 *
 * Choice: an expert's rank is decided by logit + select_bias (one fp32
 * addition).  With groups > 1 only the topk_groups groups with the largest
 * such value stay; then the k largest, in decreasing order.  Ties go to the
 * lower index, for groups and experts.  Logits of -inf and NaN are never
 * chosen.  A token without k experts to choose has topk_idx = -1 and topk_w =
 * 0 in the remaining places (the masked slot of ep_get_layout).
 * Live tokens: token_mask (u8 [T], NULL: all ones) is not 0 and some logit is
 * above -inf.  The logits of other tokens are not used in any way; their
 * places are -1 and 0.
 * With p = softmax(logits) over all experts and lse its log normaliser, n_s
 * the live tokens of sequence s, n their sum, S the sequences that have any:
 *   losses[0] = balance_coef / S * sum_s E / (k * n_s^2)
 *                                        * sum_e counts[s,e] * prob_sums[s,e]
 *   losses[1] = z_coef / n * sum over live tokens of lse^2
 * (a loss over no tokens is 0).  All sums in fp32 in an order that depends on
 * the sizes alone; counts are exact.
 *
 * In:  logits       [T, E], rows ld elements apart (ld >= E).
 *      select_bias  f32 [E] or NULL: shifts the choice, not the weights (for
 *                   balancing without a loss).
 *      seq_offsets  i32 [num_seqs + 1]: sequence s is the tokens
 *                   [seq_offsets[s], seq_offsets[s+1]); must rise from 0 to T
 *                   (else EP_ERRF_BAD_SEQ, and the outputs of that call mean
 *                   nothing).  NULL for one sequence, or without losses.
 * Out: topk_idx     i32 [T, k];  topk_w  f32 [T, k].
 *      lse          f32 [T] (-inf for tokens that are not live), or NULL.
 *      counts i32 [num_seqs, E], prob_sums f32 [num_seqs, E], seq_tokens i32
 *      [num_seqs + 2] (live tokens of each sequence, then of all, then the
 *      number of sequences that have any), losses f32 [2]: all four, with lse,
 *      or all NULL (the choice alone, as for serving).
 * workspace: ep_route_workspace_bytes(route) bytes, 16-byte aligned, when the
 * losses are wanted; contents on entry ignored.
 * err_flags: EP_ERRF_BAD_SEQ.
 */
EP_API ep_status_t ep_route(const ep_route_t *route, const void *logits, int64_t ld,
                     const float *select_bias, const uint8_t *token_mask,
                     const int32_t *seq_offsets, int32_t *topk_idx, float *topk_w,
                     float *lse, int32_t *counts, float *prob_sums,
                     int32_t *seq_tokens, float *losses, void *workspace,
                     size_t workspace_bytes, uint32_t *err_flags, ep_stream_t stream);

/*
 * ep_route_backward -- gradient of topk_w and the losses with respect to the
 * logits.  The choice and the counts are constants in it:
 *   g[e]  = d_losses[0] * balance_coef * E / (S * k * n_s^2) * counts[s,e]
 *           (+ d_topk_w of e if chosen, with full_softmax)
 *   d_logits[e] = p[e] * (g[e] - sum_e' p[e'] g[e'])
 *               + d_losses[1] * 2 * z_coef / n * lse * p[e]
 *               + (softmax over the chosen) w_j * (d_topk_w_j - sum w d_topk_w)
 *                 for the chosen expert of place j
 * in fp32, rounded once to the logits' type.  Rows of tokens that are not
 * live are 0.
 *
 * In:  logits, ld, seq_offsets and the outputs of ep_route; d_topk_w f32
 *      [T, k] and d_losses f32 [2] on the device, each NULL for zero.
 * Out: d_logits  [T, E], dense, of the logits' type.
 */
EP_API ep_status_t ep_route_backward(const ep_route_t *route, const void *logits, int64_t ld,
                     const int32_t *seq_offsets, const int32_t *topk_idx,
                     const float *topk_w, const float *lse, const int32_t *counts,
                     const int32_t *seq_tokens, const float *d_topk_w,
                     const float *d_losses, void *d_logits, ep_stream_t stream);

typedef struct {
    int32_t E;                /* matrices (experts), 1..EP_MAX_EXPERTS         */
    int32_t N;                /* output channels, > 0, multiple of 8           */
    int32_t K;                /* input channels, > 0, multiple of 8 (of 128 for
                                 fp8 rows)                                     */
    int32_t group;            /* input channels that share a scale: 32, 64 or
                                 128 (the last group of a row may be shorter)  */
    int32_t paired;           /* 1: each expert has 2N rows, N gate rows and
                                 then N up rows, and y = silu(gate) * up       */
} ep_w4_t;

/* Bytes of the packed weights (codes and scales of all experts);
 * (size_t)-1 if the description is invalid. */
EP_API size_t ep_w4_bytes(const ep_w4_t *w);

/*
 * ep_w4_pack -- lay 4-bit weights out for ep_expert_w4, once per model load.
 *
 * In:  codes   u8 [E, rows, K/2] (rows = N, or 2N when paired): input channel
 *              2i in the low half of byte i, 2i + 1 in the high half; a code c
 *              of 0..15 stands for (c - 8) * scale.  4-byte aligned.
 *      scales  bf16 [E, rows, ceil(K / group)].
 * Out: packed  ep_w4_bytes(w) bytes, 16-byte aligned.
 */
EP_API ep_status_t ep_w4_pack(const ep_w4_t *w, const uint8_t *codes, const void *scales,
                       void *packed, ep_stream_t stream);

/*
 * ep_expert_w4 -- every expert's product over its rows of the receive buffer:
 *   y[r, n] = sum_k x[r, k] * (code[e, n, k] - 8) * scale[e, n, k / group]
 * for the rows r of expert e (paired: silu of the gate product times the up
 * product), accumulated in fp32 and rounded once to bf16.  Codes and fp8
 * values enter the tensor cores exactly; scales are applied in fp32.  Made for
 * the few rows an expert has in a decode batch, where the weights' bytes decide
 * the time; correct for any number of rows.
 *
 * In:  mode, capacity  as in ep_shape_t: packed rows [offsets[e],
 *              offsets[e+1]), or in capacity mode the first min(counts[e],
 *              capacity) rows of [e*capacity, (e+1)*capacity).
 *      counts  i32 [E] (capacity mode), offsets i32 [E+1] (packed), from
 *              ep_get_layout; the other may be NULL.  With E = 1, packed and
 *              offsets NULL all R rows belong to the one matrix.
 *      R       rows of x and y (at least E*capacity in capacity mode).
 *      max_rows  no more than this many rows hold a copy in all experts
 *              together (T*k): sizes the launch.  If they hold more, the rest
 *              is not computed and EP_ERRF_CAPACITY is flagged.
 *      x, x_scales, payload  the receive buffer as ep_dispatch writes it:
 *              bf16 [R, K], or e4m3 [R, K] with f32 (4-byte aligned) or u8
 *              UE8M0 scales [R, K/128].  x 16-byte aligned.
 * Out: y       bf16 [R, N], 16-byte aligned.  Rows that hold no copy are not
 *              written.
 * err_flags: EP_ERRF_BAD_SLOT (rows outside [0, R), skipped),
 * EP_ERRF_CAPACITY, EP_ERRF_TIMEOUT.
 */
EP_API ep_status_t ep_expert_w4(const ep_w4_t *w, const void *packed, int32_t mode,
                         int32_t capacity, int64_t R, int64_t max_rows,
                         const int32_t *counts, const int32_t *offsets, const void *x,
                         const void *x_scales, int32_t payload, void *y,
                         uint32_t *err_flags, ep_stream_t stream);

#define EP_MAX_QUANT_WIDTH 16384

/*
 * Random numbers of dropout: the generator Philox4x32 with ten rounds (Salmon
 * and others, SC11).  `rng` is two i64 on the device, a seed (the generator's
 * key, low half first) and a step; `site` tells the dropouts of one step apart.
 * Eight neighbours of a row share a counter: words 0 and 1 are the number of
 * the eight, row * ceil(H / 8) + column / 8 (low half first), words 2 and 3 are
 * step + site modulo 2^64.  Element j of the eight has the 16 bits of the low
 * (j even) or high half of result word j / 2 and is dropped when they are below
 * limit = round(65536 p), halves to even; what stays is multiplied by
 * 65536 / (65536 - limit), rounded to fp32, so that the mean stays what it was.
 * A dropped value counts as 0, whatever it is.  With p = 1 all are dropped.
 * rng = NULL: nothing is dropped.
 *
 * Only the sum of step and site enters: site 3 of one step has the random
 * numbers of site 2 of the next if the step goes up by 1.  For masks that are
 * never used twice under a seed, either the step goes up by more than the
 * largest site each time (sites 0..n-1: by n), or the sites lie further apart
 * than the steps reach (sites i * 2^32, steps below 2^32, counted by 1).
 */

/*
 * ep_dropout -- y = residual + dropout(x), computed in fp32, each product and
 * sum rounded, the result rounded once to the type.  The gradient with respect
 * to x is the same call on the gradient of y, without the residual.
 *
 * In:  x         type (ep_type_t) [T, H], rows ld_x elements apart; T >= 0,
 *                H >= 1.
 *      residual  type [T, H], rows ld_res apart, or NULL.
 *      p         probability of being dropped, 0..1.
 * Out: y         type [T, H], rows ld_y apart; may be x or residual where the
 *                rows lie the same.
 * Rows are at least H apart.  Pointers are aligned to their elements; rows at
 * 16-byte boundaries with H a multiple of 8 go by wide accesses.
 */
EP_API ep_status_t ep_dropout(int64_t T, int64_t H, int32_t type, const void *x, int64_t ld_x,
                       const void *residual, int64_t ld_res, double p,
                       const int64_t *rng, uint64_t site, void *y, int64_t ld_y,
                       ep_stream_t stream);

typedef struct {
    int32_t T;                /* rows, >= 0                                    */
    int32_t H;                /* channels, > 0, multiple of 8, at most
                                 EP_MAX_NORM_WIDTH                             */
    int32_t stream_type;      /* ep_type_t of h, h_out, d_h_out and d_h        */
    float eps;                /* 1e-30..1e30, added to the variance            */
    double p;                 /* dropout of y, 0..1                            */
    uint64_t site;            /* which dropout of the network it is            */
} ep_layer_norm_t;

/*
 * ep_layer_norm -- the end of one block and the start of the next in a network
 * of layer norms, one pass over the rows:
 *   h_out = h + dropout(y)                         (h_out = h without y)
 *   n     = (h_out - mean) * r * w + b,   r = 1 / sqrt(variance + eps)
 * mean and variance over a row's H channels.  In fp32; h_out is rounded once
 * to the stream's type and the norm is taken of what is stored; n is rounded
 * once.
 *
 * In:  h      stream type [T, H], rows ld_h elements apart.
 *      y      bf16 [T, H], rows ld_y apart (the block's output, e.g. from
 *             ep_combine), or NULL (the first norm of a network).
 *      w, b   f32 [H], each NULL for 1 or 0.
 *      rng    as above; NULL: nothing is dropped (as for serving).
 * Out: h_out  stream type [T, H], NULL exactly when y is; may be h when
 *             ld_h = H.
 *      n      bf16 [T, H].
 *      stats  f32 [2, T]: mean, then r of every row, or NULL.
 * 16-byte alignment of h, y, w, b, h_out and n; ld_h and ld_y multiples of 8
 * and at least H.
 * err_flags: EP_ERRF_TIMEOUT.
 */
EP_API ep_status_t ep_layer_norm(const ep_layer_norm_t *norm, const void *h, int64_t ld_h,
                          const void *y, int64_t ld_y, const float *w, const float *b,
                          const int64_t *rng, void *h_out, void *n, float *stats,
                          uint32_t *err_flags, ep_stream_t stream);

/* Bytes of device workspace ep_layer_norm_backward needs (column sums in
 * progress); (size_t)-1 if the description is invalid. */
EP_API size_t ep_layer_norm_workspace_bytes(const ep_layer_norm_t *norm);

/*
 * ep_layer_norm_backward -- gradients of ep_layer_norm.  With
 * xn = (h_out - mean) * r and t = d_n * w:
 *   d   = d_h_out + r * (t - mean(t) - xn * mean(t * xn))
 *   d_h = d          d_y = d where y stayed, times its factor, else 0
 *   d_w = sum over rows of d_n * xn        d_b = sum over rows of d_n
 * in fp32.  Sums over rows are taken in an order that depends on the sizes
 * alone: a repeated call gives the same bits.
 *
 * In:  h_out (h where there was no y), rows ld_h apart; w, rng and the stats
 *      of ep_layer_norm; d_h_out stream type [T, H] or NULL (zero); d_n bf16
 *      [T, H].
 * Out: d_h  stream type [T, H]; may be d_h_out.
 *      d_y  bf16 [T, H], or NULL when not wanted (without dropout and with a
 *           bf16 stream it equals d_h).
 *      d_w, d_b  f32 [H], each NULL when not wanted.
 * workspace: ep_layer_norm_workspace_bytes(norm) bytes, 16-byte aligned,
 * contents on entry ignored.  T = 0 sets the sums to zero.
 * err_flags: EP_ERRF_TIMEOUT.
 */
EP_API ep_status_t ep_layer_norm_backward(const ep_layer_norm_t *norm, const void *h_out, int64_t ld_h,
                          const float *w, const int64_t *rng, const float *stats,
                          const void *d_h_out, const void *d_n, void *d_h, void *d_y,
                          float *d_w, float *d_b, void *workspace, size_t workspace_bytes,
                          uint32_t *err_flags, ep_stream_t stream);

/*
 * ep_quant_i8 -- rows of the receive buffer (or of what a product made of it)
 * to 8-bit integers with a scale each:
 *   scale[r] = amax(|x[r]|) / 127      q[r, k] = round(127 * x[r, k] / amax)
 * rounded to nearest, halves to even, -127..127; the codes are exactly those of
 * the real numbers.  A row of zeros has scale 0 and codes 0, a row that holds an
 * infinity or a NaN scale NaN and codes 0.
 *
 * In:  mode, capacity, counts, offsets  as in ep_expert_i8: which rows hold a
 *      copy.  Packed with offsets NULL: all R rows.
 *      x       bf16 [R, K], rows ld_x elements apart, 16-byte aligned; K a
 *              multiple of 16, at most EP_MAX_QUANT_WIDTH; ld_x a multiple of 8.
 * Out: q       i8 [R, K], 16-byte aligned;  scales  f32 [R].  Rows that hold no
 *              copy are not written.
 * err_flags: EP_ERRF_BAD_SLOT (offsets beyond R, cut off).
 */
EP_API ep_status_t ep_quant_i8(int32_t E, int32_t K, int32_t mode, int32_t capacity, int64_t R,
                        const int32_t *counts, const int32_t *offsets, const void *x,
                        int64_t ld_x, int8_t *q, float *scales, uint32_t *err_flags,
                        ep_stream_t stream);

typedef struct {
    int32_t E;                /* matrices (experts), 1..EP_MAX_EXPERTS         */
    int32_t N;                /* output channels, > 0, multiple of 8           */
    int32_t K;                /* input channels, > 0, multiple of 16           */
    int32_t paired;           /* 1: each expert has 2N rows, N gate rows and
                                 then N up rows, and y = silu(gate) * up       */
} ep_i8_t;

/* Bytes of the packed weights (codes and scales of all experts, padded to whole
 * blocks of 128 rows, or 64 gate and 64 up rows, and 128 input channels: K = 16
 * takes eight times its codes); (size_t)-1 if the description is invalid. */
EP_API size_t ep_i8_bytes(const ep_i8_t *w);

/*
 * ep_i8_pack -- lay 8-bit weights out for ep_expert_i8, once per model load.
 *
 * In:  codes   i8 [E, rows, K] (rows = N, or 2N when paired), 16-byte aligned.
 *      scales  f32 [E, rows].
 * Out: packed  ep_i8_bytes(w) bytes, 16-byte aligned.
 */
EP_API ep_status_t ep_i8_pack(const ep_i8_t *w, const int8_t *codes, const float *scales,
                       void *packed, ep_stream_t stream);

/*
 * ep_expert_i8 -- every expert's product over its rows of the receive buffer:
 *   y[r, n] = x_scale[r] * scale[e, n] * sum_k x[r, k] * code[e, n, k]
 * for the rows r of expert e (paired: silu of the gate product times the up
 * product).  Products of codes are exact and summed in fp32 (a batch of little
 * work: in 32-bit integers), which is exact as long as no partial sum passes
 * 2^24; scales are applied in fp32 and the result is rounded once to bf16.
 *
 * In:  mode, capacity, counts, offsets, R, max_rows  as in ep_expert_w4 (if
 *                more than max_rows rows hold a copy, the rest is computed, or
 *                left out and EP_ERRF_CAPACITY flagged).
 *      x         i8 [R, K], 16-byte aligned;  x_scales  f32 [R].
 * Out: y         bf16 [R, N], 16-byte aligned.  Rows that hold no copy are not
 *                written.
 * err_flags: EP_ERRF_BAD_SLOT (rows outside [0, R), skipped),
 * EP_ERRF_CAPACITY, EP_ERRF_TIMEOUT.
 */
EP_API ep_status_t ep_expert_i8(const ep_i8_t *w, const void *packed, int32_t mode,
                         int32_t capacity, int64_t R, int64_t max_rows,
                         const int32_t *counts, const int32_t *offsets, const int8_t *x,
                         const float *x_scales, void *y, uint32_t *err_flags,
                         ep_stream_t stream);

/* Static description of a status code. */
EP_API const char *ep_status_string(ep_status_t status);

/* The same function under the shorter name of the original interface plan. */
EP_API const char *ep_status_str(ep_status_t status);

/* Detail of the last non-EP_OK status returned on the calling thread
 * ("" if none).  The pointer stays valid until the next call on this thread. */
EP_API const char *ep_last_error(void);

/* ABI version of this library (major * 100 + minor). */
EP_API int32_t ep_abi_version(void);

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif  /* EP_GB300_H_ */
