/*
 * gdr2.h -- C ABI of the Gated DeltaNet-2 library for AMD MI355X
 * (gfx950).  Plain C: no C++ or HIP types.  Streams are passed as void*
 * holding a hipStream_t (NULL = the default stream).
 *
 * The operation (page "Gated DeltaNet-2: 선형 어텐션에서 삭제와 쓰기 게이트
 * 분리", section "Gated Delta Rule-2 업데이트 수식", the update equation and
 * its symbol table), for every batch row b and head h independently:
 *
 *     S_t = (I - k_t (b_t * k_t)^T) D_t S_{t-1} + k_t (w_t * v_t)^T
 *     o_t = S_t^T q_t
 *
 *   S_t    d_k x d_v memory state (fp32 here), row index = key channel
 *   k_t    key (the pages take it L2-normalised; the caller normalises, the
 *          library computes the formula for any k)
 *   b_t    erase gate, per key channel (width d_k) or one scalar (width 1)
 *   w_t    write gate, per value channel (width d_v) or one scalar (width 1)
 *   D_t    diag(exp(g_t)): per-key-channel decay, passed as its logarithm g_t
 *          (fp32, width d_k or 1; g <= 0 is expected but not required)
 *   o_t    readout after the update at t, without scaling (the pages give no
 *          readout; this is the usual linear-attention convention)
 *   '*'    elementwise product
 *
 * Width-1 gates broadcast over their channels: b = w = one scalar beta is
 * KDA, and a scalar decay on top is Gated DeltaNet (same section).
 *
 * Optional initial state S0: a learned prefilled memory (page "[논문리뷰]
 * Sparse Delta Memory: Scaling the State of Linear RNNs through Sparsity",
 * section 3, the learned initial state M_0).  S_out of one call may be passed
 * as S0 of the next to continue a sequence segment by segment (page "Memory
 * Caching(MC): ...", section "체크포인트를 캐싱할까, 독립 압축기를 쓸까?");
 * the result equals one call over the whole sequence up to rounding.
 *
 * Chunked prefill: fixed-size chunks (page "Gated DeltaNet-2 ...", section
 * "효율적 구현": a chunkwise algorithm with a WY form that absorbs the
 * cumulative per-channel decay into the rank-1 erase factors).  The decode
 * step is the pure recurrent mode of the same page (section "개요"): one
 * token per sequence, state updated in place.
 *
 * Common rules for every entry point
 *   Ownership : the caller allocates and frees every device buffer (inputs,
 *               outputs, workspace).  The library allocates no device memory,
 *               does not synchronise, and keeps no pointer after returning.
 *               Work is enqueued on `stream` and runs asynchronously.
 *   Errors    : arguments are validated on the host before any launch; on
 *               error the call returns a non-zero gdr2_status, records a
 *               message for gdr2_last_error() in the calling thread, launches
 *               nothing and leaves every output untouched.  A failed HIP
 *               launch returns GDR2_ERR_HIP with the HIP error text.  NaN or
 *               Inf inputs are not checked; they propagate.
 *   Layout    : every tensor is dense, row-major, contiguous, in device memory,
 *               16-byte aligned.
 *   Threads   : calls are reentrant; calls on different streams run
 *               concurrently as long as their buffers do not overlap.
 */
#ifndef GDR2_H
#define GDR2_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GDR2_ABI_VERSION 8

typedef enum gdr2_status {
    GDR2_OK = 0,
    GDR2_ERR_INVALID_ARG = 1,  /* null / misaligned / overlapping pointer, bad size */
    GDR2_ERR_UNSUPPORTED = 2,  /* valid but outside the supported set below */
    GDR2_ERR_WORKSPACE = 3,    /* workspace missing or smaller than required */
    GDR2_ERR_HIP = 4,          /* the HIP runtime reported an error */
    GDR2_STATUS_RANGE_ = 0x7fffffff  /* not a status: makes every 32-bit value a
                                        valid gdr2_status, so an unknown code
                                        passed to gdr2_status_string is defined */
} gdr2_status;

/* Element type of q, k, v, b, w and o.  g, S0, S_out and state are fp32. */
typedef enum gdr2_dtype {
    GDR2_F32 = 0,
    GDR2_BF16 = 1  /* bfloat16; o is rounded to nearest-even once, at store */
} gdr2_dtype;

/*
 * Optional input prologue, fused into the kernels (bit flags; 0 = inputs are
 * used as given).  The page "Gated DeltaNet-2 ..." (section "Gated Delta
 * Rule-2 업데이트 수식", symbol table) takes the key L2-normalised, the
 * erase and write gates in [0, 1] and the decay in (0, 1); these bits let a
 * caller pass raw projections instead of normalising and activating them in
 * a separate pass over HBM.  The pages name no activation function: the
 * logistic sigmoid and the log-sigmoid decay below are this library's choice.
 *   NORM_QK  q and k are scaled per token and head to unit L2 norm over the
 *            d_k channels: x <- x (sum x_i^2 + 1e-6)^(-1/2)
 *   GATES    b <- sigmoid(b), w <- sigmoid(w) (applied to the scalar of a
 *            width-1 gate), and g carries a pre-activation x whose log-decay
 *            is -softplus(x) = log sigmoid(-x)
 * The backward's gradients are then with respect to the raw inputs.
 */
typedef enum gdr2_prologue {
    GDR2_PROLOGUE_NORM_QK = 1,
    GDR2_PROLOGUE_GATES = 2
} gdr2_prologue;

/* Algorithm of the chunked forward. */
typedef enum gdr2_algo {
    GDR2_ALGO_AUTO = 0,    /* the library picks */
    GDR2_ALGO_STAGED = 1,  /* intra-chunk kernel writes per-chunk factors to the
                              workspace; a propagation kernel carries the state
                              through the chunks and writes o */
    GDR2_ALGO_SEGMENTED = 2, /* STAGED with the chunks of each sequence cut into
                              segments that run in parallel: a span kernel
                              forms each segment's chunk product and local
                              state, a fold kernel chains the segments' start
                              states, and the propagation kernel runs every
                              segment from its start (a two-level scan of the
                              chunk recurrence, for few sequences x heads and
                              many chunks).  AUTO takes it when one pass would
                              leave most of the GPU idle.  Same results as
                              STAGED up to rounding order. */
    GDR2_ALGO_FUSED = 3    /* one kernel per (sequence, head, 64 value
                              columns): each workgroup forms every chunk's
                              factors in LDS and carries the state through
                              the chunks, so nothing per chunk goes through
                              device memory and no workspace is needed.
                              bf16 only (GDR2_ERR_UNSUPPORTED otherwise), and
                              only with GDR2_STAGE_ALL.  AUTO takes it for
                              bf16 at Dk = 64 when B*H is at least the GPU's
                              compute-unit count (there it is faster than
                              STAGED; at Dk = 128 each head's two column
                              workgroups would repeat the chunk's factors).
                              Same results as STAGED up to rounding order. */
} gdr2_algo;

/* Which kernels of GDR2_ALGO_STAGED one call runs.  Two calls on the same
 * stream, PREP then STATE, with identical arguments (workspace included),
 * give exactly the result of one GDR2_STAGE_ALL call; the split exists so the
 * two kernels can be timed or scheduled separately.  A STATE call reads the
 * per-chunk factors the PREP call left in the workspace. */
typedef enum gdr2_stage {
    GDR2_STAGE_ALL = 0,
    GDR2_STAGE_PREP = 1,   /* intra-chunk kernel only (writes the workspace) */
    GDR2_STAGE_STATE = 2   /* propagation/output kernel only (reads it) */
} gdr2_stage;

/*
 * Arguments of the chunked forward.
 *   q, k   [B, T, H, Dk]        dtype
 *   v      [B, T, H, Dv]        dtype
 *   b      [B, T, H, b_width]   dtype, b_width in {1, Dk}
 *   w      [B, T, H, w_width]   dtype, w_width in {1, Dv}
 *   g      [B, T, H, g_width]   fp32 log-decay, g_width in {1, Dk}
 *   S0     [B, H, Dk, Dv]       fp32, may be NULL (zero initial state)
 *   o      [B, T, H, Dv]        dtype, written
 *   S_out  [B, H, Dk, Dv]       fp32, written, may be NULL; may be the same
 *                               pointer as S0 (in-place continuation), must
 *                               not otherwise overlap anything
 *   S_chunks [B, H, NC, Dk, Dv] fp32, NC = ceil(T / chunk), may be NULL:
 *                               written with the state at the start of every
 *                               chunk (S_chunks[b, h, n] = the state before
 *                               token n*chunk; n = 0 gives S0 or zeros), the
 *                               segment-boundary memory checkpoints of the
 *                               page "Memory Caching(MC): 길이에 따라
 *                               메모리가 커지는 RNN에 대한 연구", section
 *                               "체크포인트를 캐싱할까, 독립 압축기를
 *                               쓸까?".  Written by the STATE stage; must
 *                               not overlap anything else.
 *   o must not overlap any input.
 * Supported set: Dk == Dv in {64, 128}; chunk in {32, 64}; dtype F32 or BF16;
 * B, T, H >= 0 (T need not be a multiple of chunk; T == 0 writes S0, or
 * zeros, to S_out).  Anything else returns GDR2_ERR_UNSUPPORTED.  The chunked
 * form is exact for every chunk size, so the chunk changes results only by
 * rounding; F32 with Dk = 128 and chunk 64 is evaluated in chunks of 32 (a
 * 64 x 128 fp32 chunk does not fit the intra-chunk kernel's LDS), with
 * S_chunks still sampled every 64 tokens.
 */
typedef struct gdr2_fwd_args {
    int64_t B, T, H, Dk, Dv;
    int32_t chunk;
    int32_t dtype;        /* gdr2_dtype */
    int32_t algo;         /* gdr2_algo */
    int32_t stage;        /* gdr2_stage */
    int32_t b_width, w_width, g_width;
    int32_t prologue;     /* gdr2_prologue bits */
    const void *q, *k, *v, *b, *w;
    const float *g;
    const float *S0;
    void *o;
    float *S_out;
    void *workspace;      /* device memory, >= gdr2_forward_workspace_size() bytes */
    size_t workspace_bytes;
    float *S_chunks;      /* optional chunk-start states (see above) */
} gdr2_fwd_args;

/*
 * Arguments of one batched decode step: N sequences x H heads, one token each.
 *   q, k   [N, H, Dk]   dtype        v  [N, H, Dv]   dtype
 *   b      [N, H, b_width]           w  [N, H, w_width]       (dtype)
 *   g      [N, H, g_width] fp32
 *   state  [N, H, Dk, Dv] fp32, read and overwritten in place with S_t
 *   o      [N, H, Dv] dtype, written; must not overlap any other buffer
 * Supported set: Dk == Dv in {64, 128}; dtype F32 or BF16; N, H >= 0.
 */
typedef struct gdr2_decode_args {
    int64_t N, H, Dk, Dv;
    int32_t dtype;        /* gdr2_dtype */
    int32_t b_width, w_width, g_width;
    const void *q, *k, *v, *b, *w;
    const float *g;
    float *state;
    void *o;
    int32_t prologue;     /* gdr2_prologue bits */
    int32_t reserved;     /* must be 0 */
} gdr2_decode_args;

/*
 * Arguments of the chunked backward: the gradients of a loss L with respect
 * to every input of the chunked forward, given dL/do and dL/dS_final.  The
 * derivatives are those of the update and readout above (page "Gated
 * DeltaNet-2 ...", section "Gated Delta Rule-2 업데이트 수식"), taken
 * through the chunked WY form of section "효율적 구현"; the state at every
 * chunk start comes from the forward (S_chunks), so no state is recomputed.
 *   q, k, v, b, w, g   the forward's inputs, same shapes, dtype and widths
 *   S_chunks [B, H, NC, Dk, Dv] fp32, NC = ceil(T / 64): the chunk-start
 *                      states the forward wrote with chunk = 64 (any exact
 *                      source of the states before tokens 0, 64, 128, ...
 *                      serves); S_chunks[:, :, 0] is the forward's S0
 *   dO       [B, T, H, Dv]  dtype  dL/do
 *   dS_final [B, H, Dk, Dv] fp32   dL/dS_final, may be NULL (zero)
 * Outputs, all fp32, written in full (no accumulation into them):
 *   dq, dk   [B, T, H, Dk]     dv [B, T, H, Dv]
 *   db       [B, T, H, b_width]   dw [B, T, H, w_width]   dg [B, T, H, g_width]
 *            (a width-1 gate gets the sum over the channels it broadcasts to)
 *   dS0      [B, H, Dk, Dv], may be NULL: dL/dS0
 * No output may overlap any input, another output or the workspace.
 * Supported set: Dk == Dv in {64, 128}; chunk == 64; dtype F32 or BF16;
 * B, T, H >= 0 (T == 0 writes dS_final, or zeros, to dS0).  Anything else
 * returns GDR2_ERR_UNSUPPORTED.  Accumulation is fp32; with bf16 inputs the
 * matrix-core operands are bf16, as in the forward.  The result does not
 * depend on scheduling: every sum runs in a fixed order (no atomics), so a
 * call repeated on the same arguments gives the same bits.
 */
typedef struct gdr2_bwd_args {
    int64_t B, T, H, Dk, Dv;
    int32_t chunk;        /* must be 64 */
    int32_t dtype;        /* gdr2_dtype of q, k, v, b, w, dO */
    int32_t b_width, w_width, g_width;
    int32_t prologue;     /* gdr2_prologue bits, as given to the forward */
    const void *q, *k, *v, *b, *w;
    const float *g;
    const float *S_chunks;
    const void *dO;
    const float *dS_final;
    float *dq, *dk, *dv, *db, *dw, *dg;
    float *dS0;
    void *workspace;      /* device memory, >= gdr2_backward_workspace_size() bytes */
    size_t workspace_bytes;
    int32_t algo;         /* gdr2_algo of the reverse scan over the chunks:
                             STAGED one pass per (b, h), SEGMENTED the
                             two-level scan over chunk segments (a span
                             kernel, the segment fold and the scan per
                             segment, as in the forward), AUTO the library
                             picks (the two-level scan when one pass would
                             leave most of the GPU idle) */
    int32_t reserved;     /* must be 0 */
} gdr2_bwd_args;

/* Bytes of device workspace gdr2_forward_chunked needs for these arguments
 * (pointers are not read).  0 when none is needed or the arguments are
 * invalid or unsupported. */
size_t gdr2_forward_workspace_size(const gdr2_fwd_args *args);

/* Chunked forward: o for every token and the final state S_out. */
gdr2_status gdr2_forward_chunked(const gdr2_fwd_args *args, void *stream);

/* Bytes of device workspace gdr2_backward_chunked needs for these
 * arguments (pointers are not read).  0 when none is needed or the arguments
 * are invalid or unsupported. */
size_t gdr2_backward_workspace_size(const gdr2_bwd_args *args);

/* Chunked backward: every input gradient and dS0. */
gdr2_status gdr2_backward_chunked(const gdr2_bwd_args *args, void *stream);

/* One recurrent decode step for every (sequence, head) state. */
gdr2_status gdr2_decode_step(const gdr2_decode_args *args, void *stream);

/* Bytes of the library's static device scratch used by
 * gdr2_forward_chunked_noalloc (one copy per device, held until the process
 * ends). */
#define GDR2_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

/* The chunked forward for callers that cannot allocate device memory: code
 * under HIP stream/graph capture, tight serving loops, hosts that forbid
 * hipMalloc.  Same arguments, results and checks as gdr2_forward_chunked,
 * except that args->workspace and args->workspace_bytes are ignored: the
 * workspace is the library's static device scratch of
 * GDR2_NOALLOC_SCRATCH_BYTES bytes.  The call allocates nothing (no
 * hipMalloc, no hipFree).  Arguments whose workspace
 * (gdr2_forward_workspace_size) exceeds the scratch return
 * GDR2_ERR_WORKSPACE and launch nothing.  Every call on one device shares
 * that device's scratch: calls that may overlap in time on one device (other
 * streams, other threads) race and must be serialised by the caller.  The
 * scratch's address is looked up on the first call on each device (a HIP
 * error then returns GDR2_ERR_HIP). */
gdr2_status gdr2_forward_chunked_noalloc(const gdr2_fwd_args *args, void *stream);

/* ------------------------------------------------------------------------
 * The operators around the recurrence in a sequence-mixing layer: the short
 * causal convolution in front of it, the selective state space scan beside
 * it, and the normalisation before and after it.
 *
 * Rules these entry points add to the common rules above
 *   Rows      : a token row is `C` contiguous elements.  Inputs named with a
 *               *_stride field may be column slices of a wider matrix: row r
 *               starts at r * stride elements (stride >= the row's width) and
 *               the pointer is aligned to its element only.  Every other
 *               buffer is dense and 16-byte aligned.
 *   Batches   : offsets == NULL: B sequences of T rows each, row b*T + t.
 *               offsets != NULL (device, int64 [B+1], ascending, within
 *               0..T): T rows in all, sequence s owns the rows
 *               offsets[s] .. offsets[s+1]-1 and may be empty.  Rows of no
 *               sequence are neither read nor written.  The offsets are read
 *               on the device only: values out of 0..T are clamped to it and
 *               a descending pair is an empty sequence; offsets that are
 *               not ascending give unspecified results, within the buffers.
 *   Parameters: weights, biases, A, skip are fp32 whatever the dtype of the
 *               rows, and so are their gradients and the scan's states.
 *   Gradients : of rows, in the rows' dtype, accumulated in fp32 and rounded
 *               once at the store.  Every sum runs in a fixed order (no
 *               atomics): a repeated call gives the same bits.
 *   Sizes     : all int64; rows of more than 2^24 elements, rows further apart
 *               than 2^40 (in gdr2_scan_forward and gdr2_scan_backward 2^24),
 *               2^40 or more rows, and a call one of whose launches would need
 *               2^24 or more workgroups (of 256 threads, larger ones counted as
 *               several) return GDR2_ERR_UNSUPPORTED.
 * ------------------------------------------------------------------------ */

/* Activation fused behind the convolution. */
typedef enum gdr2_act {
    GDR2_ACT_NONE = 0,
    GDR2_ACT_SILU = 1  /* y = p / (1 + exp(-p)) */
} gdr2_act;

/*
 * Short causal depthwise convolution over each sequence:
 *     p[t, c] = bias[c] + sum_{k < width} weight[c, k] x[t - (width-1) + k, c]
 *     y = act(p)
 * Rows before the sequence come from state0 (the width-1 rows before it,
 * oldest first), or are zero without one.
 *   x         [.., C]            dtype, rows of x_stride elements
 *   weight    [C, width] fp32    bias [C] fp32, may be NULL
 *   state0    [B, width-1, C]    dtype, may be NULL
 *   offsets   see "Batches"
 *   y         [.., C]            dtype, dense, written
 *   state_out [B, width-1, C]    dtype, may be NULL: the last width-1 rows of
 *             (state0, sequence), the state0 of the sequence's continuation.
 *             May be the same pointer as state0; no other overlap.
 * Supported set: width in {2, 3, 4}; C >= 1; dtype F32 or BF16; B, T >= 0.
 */
typedef struct gdr2_conv_args {
    int64_t B, T, C;
    int64_t x_stride;
    int32_t width;
    int32_t dtype;        /* gdr2_dtype */
    int32_t act;          /* gdr2_act */
    int32_t reserved;     /* must be 0 */
    const void *x;
    const float *weight, *bias;
    const void *state0;
    const int64_t *offsets;
    void *y;
    void *state_out;
} gdr2_conv_args;

/*
 * The convolution for one token of each of N sequences:
 *   state [N, width-1, C] dtype, the previous inputs oldest first; read, then
 *         overwritten with its last width-2 rows and x
 *   x     [N, C] dtype, rows of x_stride elements      y [N, C] dtype, written
 */
typedef struct gdr2_conv_step_args {
    int64_t N, C;
    int64_t x_stride;
    int32_t width;
    int32_t dtype;
    int32_t act;
    int32_t reserved;     /* must be 0 */
    void *state;
    const void *x;
    const float *weight, *bias;
    void *y;
} gdr2_conv_step_args;

/*
 * Gradients of the convolution, given dy (dL/dy, dense) and optionally dstate
 * (dL/dstate_out):
 *   dx [.., C] dtype, dense     dweight [C, width] fp32    dbias [C] fp32, may
 *   be NULL                     dstate0 [B, width-1, C] dtype, may be NULL
 * x, weight, bias, state0, offsets and act as given to the forward.
 */
typedef struct gdr2_conv_bwd_args {
    int64_t B, T, C;
    int64_t x_stride;
    int32_t width;
    int32_t dtype;
    int32_t act;
    int32_t reserved;     /* must be 0 */
    const void *x;
    const float *weight, *bias;
    const void *state0;
    const int64_t *offsets;
    const void *dy;
    const void *dstate;
    void *dx;
    float *dweight, *dbias;
    void *dstate0;
    void *workspace;      /* device, >= gdr2_conv_backward_workspace_size() bytes */
    size_t workspace_bytes;
} gdr2_conv_bwd_args;

/* Flags of the scan. */
typedef enum gdr2_scan_flags {
    GDR2_SCAN_SOFTPLUS = 1  /* the step is softplus(dt + dt_bias), not dt + dt_bias */
} gdr2_scan_flags;

/* Tokens between two recorded states of the scan (h_chunks). */
#define GDR2_SCAN_CHUNK 32

/*
 * Selective state space scan.  For every sequence and channel c, with the
 * step d_t = softplus(dt_t + dt_bias) and the group j = c / (C / G):
 *     h_t[c, n] = exp(d_t A[c, n]) h_{t-1}[c, n] + d_t x_t[c] Bt_t[j, n]
 *     v_t[c]    = sum_n Ct_t[j, n] h_t[c, n] + skip[c] x_t[c]
 *     y_t       = v_t, or v_t z_t / (1 + exp(-z_t)) with a gate z
 * (the erase-free relative of the update above, with a decay of its own for
 * every state element instead of one per key channel).  A token whose dt is
 * -inf or the dtype's lowest value, as a mask sets it, has d = 0 under softplus:
 * it leaves the state as it is, and its ddt is 0.
 *   x, dt, z  [.., C]   dtype, rows of x_stride, dt_stride, z_stride elements;
 *                       z may be NULL
 *   Bt, Ct    [.., G, N] dtype, rows (of G*N elements) b_stride, c_stride apart
 *   A         [C, N] fp32 (A <= 0 is expected but not required)
 *   skip, dt_bias [C] fp32, may be NULL
 *   h0        [B, C, N] fp32, may be NULL (zero)
 *   y         [.., C]   dtype, dense, written
 *   h_out     [B, C, N] fp32, may be NULL: the state after each sequence; may
 *             be the same pointer as h0
 *   h_chunks  [gdr2_scan_chunk_count(), C, N] fp32, may be NULL: the state
 *             before the tokens 0, 32, 64, ... of each sequence, which the
 *             backward reads.  Token 32*i of sequence s is recorded in slot
 *             s*ceil(T/32) + i, or with offsets offsets[s]/32 + s + i; other
 *             slots are left as they were.
 * Supported set: 1 <= N <= 32; G divides C; dtype F32 or BF16; B, T >= 0.
 * algo: AUTO, STAGED (one pass over each sequence) or SEGMENTED (sequences
 * cut into segments that run in parallel: a span pass forms each segment's
 * total decay and local end state, a fold chains them, and the main pass runs
 * every segment from its start state).  AUTO takes segments when one pass
 * would leave much of the GPU idle.
 */
typedef struct gdr2_scan_args {
    int64_t B, T, C, N, G;
    int64_t x_stride, dt_stride, b_stride, c_stride, z_stride;
    int32_t dtype;
    int32_t flags;        /* gdr2_scan_flags bits */
    int32_t algo;         /* gdr2_algo: AUTO, STAGED or SEGMENTED */
    int32_t reserved;     /* must be 0 */
    const void *x, *dt, *Bt, *Ct, *z;
    const float *A, *skip, *dt_bias, *h0;
    const int64_t *offsets;
    void *y;
    float *h_out, *h_chunks;
    void *workspace;      /* device, >= gdr2_scan_workspace_size() bytes */
    size_t workspace_bytes;
} gdr2_scan_args;

/*
 * The scan for one token of each of B sequences: state [B, C, N] fp32 is read
 * and overwritten in place; the rows are [B, C] and [B, G, N].  Uses the
 * fields of gdr2_scan_args except T (must be 1), offsets, h0, h_out, h_chunks
 * (must be NULL), algo and workspace (ignored).
 */
typedef struct gdr2_scan_step_args {
    gdr2_scan_args s;
    float *state;
} gdr2_scan_step_args;

/*
 * Gradients of the scan, given dy (dL/dy, dense) and optionally dh_out
 * (dL/dh_out).  `f` holds the forward's arguments, h_chunks as it wrote them
 * (the states before every 32nd token; h_chunks is required, h0, h_out, y and
 * f's workspace are not read).
 *   dx, ddt, dz [.., C] dtype     dBt, dCt [.., G, N] dtype     all dense
 *   dA [C, N], dskip, ddt_bias [C] fp32     dh0 [B, C, N] fp32
 * dskip, ddt_bias and dh0 may be NULL; dz is required with z and refused
 * without it.  dh0 may be the same pointer as dh_out.
 */
typedef struct gdr2_scan_bwd_args {
    gdr2_scan_args f;
    const void *dy;
    const float *dh_out;
    void *dx, *ddt, *dBt, *dCt, *dz;
    float *dA, *dskip, *ddt_bias, *dh0;
    void *workspace;      /* device, >= gdr2_scan_backward_workspace_size() bytes */
    size_t workspace_bytes;
} gdr2_scan_bwd_args;

/* Which norm. */
typedef enum gdr2_norm_kind {
    GDR2_NORM_LAYER = 0,  /* the row's mean is taken off */
    GDR2_NORM_RMS = 1
} gdr2_norm_kind;

/*
 * Normalisation of R rows of C elements:
 *     n = (x - m) (mean((x - m)^2) + eps)^(-1/2) weight + bias
 *     y = n, or n z / (1 + exp(-z)) with a gate z
 * with m the row's mean (LAYER) or 0 (RMS).
 *   x, z  [R, C] dtype, rows of x_stride, z_stride elements; z may be NULL
 *   weight, bias [C] fp32, may be NULL (1 and 0)
 *   y     [R, C] dtype, dense, written
 * Supported set: C >= 1, R >= 0; eps >= 0 and finite; dtype F32 or BF16.
 */
typedef struct gdr2_norm_args {
    int64_t R, C;
    int64_t x_stride, z_stride;
    int32_t dtype;
    int32_t kind;         /* gdr2_norm_kind */
    float eps;
    int32_t reserved;     /* must be 0 */
    const void *x, *z;
    const float *weight, *bias;
    void *y;
} gdr2_norm_args;

/*
 * Gradients of the norm, given dy (dL/dy, dense).  `f` holds the forward's
 * arguments (y is not read).  The row's statistics are formed again from x,
 * which the gradient reads in any case.
 *   dx [R, C] dtype, dense      dz [R, C] dtype, dense; required with z and
 *                               refused without it
 *   dweight, dbias [C] fp32, may be NULL
 */
typedef struct gdr2_norm_bwd_args {
    gdr2_norm_args f;
    const void *dy;
    void *dx, *dz;
    float *dweight, *dbias;
    void *workspace;      /* device, >= gdr2_norm_backward_workspace_size() bytes */
    size_t workspace_bytes;
} gdr2_norm_bwd_args;

/* The convolution, its single-token step, its gradients. */
gdr2_status gdr2_conv_forward(const gdr2_conv_args *args, void *stream);
gdr2_status gdr2_conv_step(const gdr2_conv_step_args *args, void *stream);
size_t gdr2_conv_backward_workspace_size(const gdr2_conv_bwd_args *args);
gdr2_status gdr2_conv_backward(const gdr2_conv_bwd_args *args, void *stream);

/* The scan, its single-token step, its gradients.  The workspace queries
 * (here and above) look at sizes, at whether an optional pointer is NULL, and
 * at the current device's compute units; 0 when none is needed or the
 * arguments are invalid or unsupported. */
int64_t gdr2_scan_chunk_count(int64_t B, int64_t T, int packed);
size_t gdr2_scan_workspace_size(const gdr2_scan_args *args);
gdr2_status gdr2_scan_forward(const gdr2_scan_args *args, void *stream);
gdr2_status gdr2_scan_step(const gdr2_scan_step_args *args, void *stream);
size_t gdr2_scan_backward_workspace_size(const gdr2_scan_bwd_args *args);
gdr2_status gdr2_scan_backward(const gdr2_scan_bwd_args *args, void *stream);

/* The norm and its gradients. */
gdr2_status gdr2_norm_forward(const gdr2_norm_args *args, void *stream);
size_t gdr2_norm_backward_workspace_size(const gdr2_norm_bwd_args *args);
gdr2_status gdr2_norm_backward(const gdr2_norm_bwd_args *args, void *stream);

/* ------------------------------------------------------------------------
 * The operators of a block around its mixing layers: the norm with the
 * residual's addition, the gated linear recurrence (a mixing layer whose
 * state is one number per channel), and rows in 8 bits, which these two write
 * as activation checkpoints and read in their gradients.  The rules of the
 * layer operators above hold for them too (rows, batches, parameters,
 * gradients, sizes), with these additions:
 *   Rows8     : rows of C columns in 8 bits are codes [R, C], one e4m3 number
 *               (4 exponent bits, 3 mantissa bits, largest finite 448) per
 *               element, and scales [R, ceil(C/32)], one byte b per 32 columns of a
 *               row (the last block may be shorter) that stands for 2^(b-127)
 *               (255, which no rounding gives, for NaN).
 *               An element's value is its code times its block's scale: the
 *               layout of block-scaled matrix operands.  Both dense.
 *   Rounding  : a block's scale is the smallest 2^e, e >= -127, with
 *               448 2^e >= the largest finite magnitude in it, so that no finite value is
 *               clipped; a code is the value over the scale, to nearest even.
 *               NaN becomes a NaN code.  e4m3 has no infinity: one becomes a
 *               NaN beside finite values, but a block without any finite
 *               value takes e = 120 and the codes +-448, which read as
 *               infinities again (a row masked with -inf, or with the
 *               dtype's lowest value, stays one).
 * ------------------------------------------------------------------------ */

/* Columns that share a scale. */
#define GDR2_ROWS8_BLOCK 32

typedef struct gdr2_rows8 {
    void *codes;          /* [R, C] bytes */
    void *scales;         /* [R, ceil(C / 32)] bytes */
} gdr2_rows8;

/*
 * Rows into 8 bits.
 *   x [R, C] dtype, rows of x_stride elements     out: written
 * Supported set: C >= 1, R >= 0; dtype F32 or BF16.
 */
typedef struct gdr2_pack_args {
    int64_t R, C;
    int64_t x_stride;
    int32_t dtype;        /* gdr2_dtype */
    int32_t reserved;     /* must be 0 */
    const void *x;
    gdr2_rows8 out;
} gdr2_pack_args;

/* Rows from 8 bits: y [R, C] dtype, dense, written (in fp32 the exact values;
 * those past the type's range read as infinite). */
typedef struct gdr2_unpack_args {
    int64_t R, C;
    int32_t dtype;        /* gdr2_dtype of y */
    int32_t reserved;     /* must be 0 */
    gdr2_rows8 rows;
    void *y;
} gdr2_unpack_args;

/*
 * Norm with the residual's addition, over R rows of C elements:
 *     h = x + residual, rounded to the residual's type
 *     n = (h - m) (mean((h - m)^2) + eps)^(-1/2) weight + bias
 *     y = n,  y8 = n in 8 bits,  h8 = h in 8 bits
 * with m the row's mean (LAYER) or 0 (RMS).  The norm is taken of h as it is
 * stored, so that the gradients see the same rows.
 *   x, residual [R, C]   dtype and res_dtype, rows of x_stride, res_stride
 *                        elements; residual may be NULL (h = x; then res_dtype
 *                        must be dtype)
 *   weight, bias [C] fp32, may be NULL (1 and 0)
 *   h    [R, C] res_dtype, dense, may be NULL; may be the same pointer as a
 *        dense residual (res_stride == C): the stream is then updated in place
 *   y    [R, C] dtype, dense, may be NULL
 *   y8, h8  may be NULL (both pointers of one); at least one of h, y, y8, h8 is given
 * The statistics and n are formed in 64 bits, so that codes do not depend on
 * how a row is spread over lanes.
 * Supported set: 1 <= C <= 16384, R >= 0; eps >= 0 and finite; dtype F32 or
 * BF16; res_dtype the same or F32.
 */
typedef struct gdr2_add_norm_args {
    int64_t R, C;
    int64_t x_stride, res_stride;
    int32_t dtype;        /* gdr2_dtype of x and y */
    int32_t res_dtype;    /* gdr2_dtype of residual and h */
    int32_t kind;         /* gdr2_norm_kind */
    float eps;
    const void *x, *residual;
    const float *weight, *bias;
    void *h, *y;
    gdr2_rows8 y8, h8;
} gdr2_add_norm_args;

/*
 * Gradients of the norm with the residual's addition, given dy (dL/dy) and
 * optionally dh (dL/dh by the stream's other uses):
 *     dresidual = dh + the norm's gradient with respect to h;  dx the same
 *   h [R, C] res_dtype, dense, as the forward wrote it; or NULL, and h8: the
 *     gradient is then that at the values the codes stand for
 *   dy [R, C] dtype   dh [R, C] res_dtype, may be NULL      all dense
 *   dresidual [R, C] res_dtype, may be the same pointer as dh
 *   dx [R, C] dtype, may be NULL      at least one of dresidual and dx is given
 *   dweight, dbias [C] fp32, may be NULL
 * A gradient through y8 or h8 is taken as one through n or h.
 * The root enters the gradients in fp32: without eps, rows whose root mean
 * square is below 2^-127 (subnormal streams) have no finite ones.
 * Supported set: as the forward's.
 */
typedef struct gdr2_add_norm_bwd_args {
    int64_t R, C;
    int32_t dtype;        /* gdr2_dtype of dy and dx */
    int32_t res_dtype;    /* gdr2_dtype of h, dh and dresidual */
    int32_t kind;         /* gdr2_norm_kind */
    float eps;
    const float *weight;
    const void *h;
    gdr2_rows8 h8;
    const void *dy, *dh;
    void *dresidual, *dx;
    float *dweight, *dbias;
    void *workspace;      /* device, >= gdr2_add_norm_backward_workspace_size() bytes */
    size_t workspace_bytes;
} gdr2_add_norm_bwd_args;

/* Tokens between two recorded states of the gated linear recurrence. */
#define GDR2_GLR_CHUNK 16

/*
 * Gated linear recurrence.  For every sequence and channel c, s the logistic
 * sigmoid:
 *     a_t = exp(A[c] s(r_t[c]))
 *     h_t = a_t h_{t-1} + sqrt(1 - a_t^2) s(i_t[c]) x_t[c],   y_t = h_t
 * A token with a_t = 1 (r = -inf or the dtype's lowest value, as a mask sets
 * it, or A = 0) leaves the state as it is; its x and i are not used, whatever they
 * hold.  A <= 0 is expected (a positive A gives NaN, the root's value there).
 *   x, r, i  [.., C]  dtype, rows of x_stride, r_stride, i_stride elements
 *   A        [C] fp32
 *   h0       [B, C] fp32, may be NULL (zero)
 *   y        [.., C]  dtype, dense, written
 *   h_out    [B, C] fp32, may be NULL: the state after each sequence; may be
 *            the same pointer as h0
 *   h_chunks [gdr2_glr_chunk_count(), C] fp32, may be NULL: the state before
 *            the tokens 0, 16, 32, ... of each sequence, which the backward
 *            reads.  Token 16*j of sequence s is recorded in row
 *            s*ceil(T/16) + j, or with offsets offsets[s]/16 + s + j; other
 *            rows are left as they were.
 *   x8, r8, i8  the rows of x, r and i in 8 bits, as gdr2_pack_rows forms
 *            them; all six pointers or none.  Rows of no sequence are left as they were.
 * algo: AUTO, STAGED (one pass over each sequence) or SEGMENTED (sequences
 * cut into tiles that run in parallel, each handing its total decay and its end
 * state on to the next through the workspace, which one call uses at a time).
 * AUTO takes tiles when one pass would leave much of the GPU idle, for packed
 * batches, and for some large arrays; results differ by roundings.
 * Supported set: C >= 1; rows at most 2^22 elements apart; dtype F32 or BF16; B, T >= 0.
 */
typedef struct gdr2_glr_args {
    int64_t B, T, C;
    int64_t x_stride, r_stride, i_stride;
    int32_t dtype;        /* gdr2_dtype */
    int32_t algo;         /* gdr2_algo: AUTO, STAGED or SEGMENTED */
    const void *x, *r, *i;
    const float *A, *h0;
    const int64_t *offsets;
    void *y;
    float *h_out, *h_chunks;
    gdr2_rows8 x8, r8, i8;
    void *workspace;      /* device, >= gdr2_glr_workspace_size() bytes */
    size_t workspace_bytes;
} gdr2_glr_args;

/*
 * The recurrence for one token of each of N sequences:
 *   state [N, C] fp32, read and overwritten in place
 *   x, r, i [N, C] dtype, rows of x_stride, r_stride, i_stride elements (at
 *   most 2^40)      y [N, C] dtype, written
 */
typedef struct gdr2_glr_step_args {
    int64_t N, C;
    int64_t x_stride, r_stride, i_stride;
    int32_t dtype;        /* gdr2_dtype */
    int32_t reserved;     /* must be 0 */
    float *state;
    const void *x, *r, *i;
    const float *A;
    void *y;
} gdr2_glr_step_args;

/*
 * Gradients of the recurrence, given dy (dL/dy, dense) and optionally dh_out
 * (dL/dh_out).  `f` holds the forward's arguments: sizes, dtype (of dy and the
 * gradients too), A, offsets, algo, h_chunks as the forward wrote them (required),
 * and either x, r, i, or, with these NULL, x8, r8, i8: the gradients are then
 * those at the values the codes stand for, with the states formed again from
 * the recorded one before every 16th token.  f's other fields are not read.
 *   dx, dr, di [.., C] dtype, dense     dA [C] fp32     dh0 [B, C] fp32
 * dh0 may be NULL, and may be the same pointer as dh_out.  Where a_t = 1 the
 * root's own derivative, which has no value there, counts as 0.
 */
typedef struct gdr2_glr_bwd_args {
    gdr2_glr_args f;
    const void *dy;
    const float *dh_out;
    void *dx, *dr, *di;
    float *dA, *dh0;
    void *workspace;      /* device, >= gdr2_glr_backward_workspace_size() bytes */
    size_t workspace_bytes;
} gdr2_glr_bwd_args;

/* Rows into 8 bits and back. */
gdr2_status gdr2_pack_rows(const gdr2_pack_args *args, void *stream);
gdr2_status gdr2_unpack_rows(const gdr2_unpack_args *args, void *stream);

/* The norm with the residual's addition, and its gradients. */
gdr2_status gdr2_add_norm_forward(const gdr2_add_norm_args *args, void *stream);
size_t gdr2_add_norm_backward_workspace_size(const gdr2_add_norm_bwd_args *args);
gdr2_status gdr2_add_norm_backward(const gdr2_add_norm_bwd_args *args, void *stream);

/* The gated linear recurrence, its single-token step, its gradients.  The
 * workspace queries (here and above) look at sizes, at whether an optional
 * pointer is NULL, and at the current device's compute units; 0 when none is
 * needed or the arguments are invalid or unsupported. */
int64_t gdr2_glr_chunk_count(int64_t B, int64_t T, int packed);
size_t gdr2_glr_workspace_size(const gdr2_glr_args *args);
gdr2_status gdr2_glr_forward(const gdr2_glr_args *args, void *stream);
gdr2_status gdr2_glr_step(const gdr2_glr_step_args *args, void *stream);
size_t gdr2_glr_backward_workspace_size(const gdr2_glr_bwd_args *args);
gdr2_status gdr2_glr_backward(const gdr2_glr_bwd_args *args, void *stream);

/* Static text for a status code (never NULL). */
const char *gdr2_status_string(gdr2_status status);

/* Message of the last failed call in this thread ("" if none). */
const char *gdr2_last_error(void);

/* GDR2_ABI_VERSION of the built library. */
int gdr2_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDR2_H */
