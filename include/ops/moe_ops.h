/*
 * moe_ops.h -- C ABI of the operators around the MXFP4 MoE expert layer
 * (include/moe_mxfp4.h), MI355X (gfx950).
 *
 * The pages keep the MoE experts, and only those, in 4 bits and the rest of
 * the model at FP8 (bjdmk.com.cn news page, co-design section; yifor-blog
 * digest, selective FP4 quantisation).  These are the operators that stand
 * directly before, beside and around the expert layer in such a block, in
 * the library's own 8-bit format (MXFP8: E4M3 elements, one E8M0 scale per
 * 32 consecutive elements, the OCP MX block rule of moe_mxfp8_quantize):
 *
 *   moe_rmsnorm            residual addition, RMS norm, MXFP8 and bf16 output
 *   moe_mxfp8_linear       act(x W^T + bias) + residual, x and W in MXFP8
 *   moe_dispatch           tokens sorted by expert (order and rows)
 *   moe_dispatch_backward  the gradient of the rows, back per token
 *   moe_combine            the experts' rows back per token, weighted
 *   moe_combine_backward   its gradients to the rows and to the weights
 *   moe_mxfp4_forward_mx8  the expert layer on activations already in MXFP8
 *
 * Conventions are the layer's: the caller owns every tensor (device memory
 * of the current device) and keeps it alive until the work enqueued on
 * `stream` has completed; arguments are checked synchronously before
 * anything is enqueued, and a failed check returns a negative MOE_E_* status
 * and enqueues nothing; no call synchronises, allocates or copies to the
 * host; nothing aborts and no C++ exception crosses this ABI.  A call may be
 * captured into a HIP graph.  num_tokens == 0 is a valid no-op (for
 * moe_dispatch it writes zero counts and offsets).
 *
 * The operators (unlike the layer) keep no state in the library, and
 * moe_mxfp4_init is not needed: scratch memory, where a call needs it, is a
 * workspace the caller passes.  Its contents need not be initialised and
 * mean nothing after the call; two calls whose work may overlap in time (on
 * two streams, in two graphs) need a workspace each.
 *
 * Rows may be strided: *_stride is the distance between rows in elements
 * (at least the row length; 0 means the row length), elements inside a row
 * are contiguous.  Sums are added in an order that the sizes alone decide
 * (no floating-point atomics), so the same inputs give the same bits.
 * Inputs must not overlap outputs, except where an argument says so.
 *
 * Element types are MOE_DT_BF16 and MOE_DT_F32 (moe_mxfp4.h); bf16 results
 * are rounded once, to nearest even, from at least float32.
 */
#ifndef MOE_OPS_H
#define MOE_OPS_H

#include <stdint.h>

#include "../moe_mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ norm
 * Per token t, with s = x + residual (x alone if residual is NULL):
 *
 *   n[t, i] = s[t, i] * weight[i] / sqrt(mean_i(s[t, i]^2) + eps)
 *
 *   residual_out[t, :] = s            in the residual's type
 *   y[t, :]            = bf16(n)
 *   codes, scales      = MXFP8(n)     the block rule of moe_mxfp8_quantize
 *
 * The sum s, its statistic, n and the 8-bit rounding are formed in 64 bits
 * from the inputs, so codes and scales are those of the formula (a block
 * with a non-finite n gets scale 0xFF and codes 0).  s is not rounded before
 * it is normalised. */
typedef struct moe_rmsnorm_args {
    const void* x;            /* [num_tokens, hidden], x_dtype */
    int64_t x_stride;
    int32_t x_dtype;          /* MOE_DT_BF16 or MOE_DT_F32 */
    int32_t residual_dtype;   /* of residual and residual_out */
    const void* residual;     /* [num_tokens, hidden] or NULL */
    int64_t residual_stride;
    void* residual_out;       /* [num_tokens, hidden]; NULL: not written.  May be `residual`
                                 itself, or `x` if its type and stride are the same.  Needs
                                 `residual` (MOE_E_NULL without) */
    int64_t residual_out_stride;
    const void* weight;       /* [hidden], weight_dtype */
    int32_t weight_dtype;     /* MOE_DT_BF16 or MOE_DT_F32 */
    int32_t reserved;         /* 0 */
    double eps;               /* finite, >= 0 */
    void* y;                  /* [num_tokens, hidden] bf16 or NULL; may be `x` itself if that is
                                 bf16 and of the same stride, not residual_out */
    int64_t y_stride;
    uint8_t* codes;           /* [num_tokens, hidden] E4M3, contiguous rows; NULL together with scales */
    uint8_t* scales;          /* [num_tokens, hidden / 32] E8M0, contiguous */
    int64_t num_tokens;       /* 0 .. 2^20 */
    int64_t hidden;           /* a multiple of 32, 32 .. 16384 */
} moe_rmsnorm_args;

/* At least one of y and codes is required.  All pointers 16-byte aligned
 * (scales: 4), and so is every row of x, residual, residual_out and y.
 * MOE_E_NULL, MOE_E_SHAPE (sizes, strides below hidden), MOE_E_DTYPE,
 * MOE_E_ALIGN, MOE_E_OPTION (eps, reserved, y over residual_out),
 * MOE_E_HIP. */
int moe_rmsnorm(const moe_rmsnorm_args* args, void* stream);

/* ---------------------------------------------------------------- linear
 *   v   = x . W^T + bias                     (float32 accumulation)
 *   out = act(v) + residual
 *
 * Products and sums are float32's at every size (about 1e-7 of the sum's
 * rms); how the sum is ordered goes by the sizes alone.  Values of x and W
 * outside float32's normal range may count as zero or infinity, and GELU's
 * results below it are zero.  SiLU's relative error is up to (8 + |v|) 2^-23,
 * GELU's up to (16 + 2 v^2) 2^-23.
 *
 * x [num_tokens, inner] and W [rows, inner] in MXFP8; W in the MXFP8 tile
 * layout of moe_mxfp8_prepack, with gate_up_pairs = 1 for MOE_EPI_SILU_MUL
 * (rows 0 .. rows/2-1 are gate, the others up) and 0 otherwise.  The output
 * has out_cols = rows columns, or rows / 2 for MOE_EPI_SILU_MUL, and goes
 * to `out` as bf16 or to `out_codes` / `out_scales` as MXFP8 (encoded from
 * float32; the form another moe_mxfp8_linear, or the expert layer, reads). */
#define MOE_EPI_NONE 0
#define MOE_EPI_SILU 1      /* v / (1 + exp(-v)) */
#define MOE_EPI_GELU 2      /* v / 2 * (1 + erf(v / sqrt 2)) */
#define MOE_EPI_SILU_MUL 3  /* SiLU(v_gate) * v_up */

typedef struct moe_mxfp8_linear_args {
    const uint8_t* x_codes;   /* [num_tokens, inner] E4M3, contiguous */
    const uint8_t* x_scales;  /* [num_tokens, inner / 32] E8M0, contiguous */
    const uint8_t* w_tiles;   /* rows * inner bytes, tile layout */
    const uint8_t* w_scales;  /* rows * inner / 32 bytes, tile layout */
    const float* bias;        /* [rows] float32 or NULL (gate rows, then up rows) */
    const void* residual;     /* [num_tokens, out_cols] bf16 or NULL; may be `out` itself */
    int64_t residual_stride;
    void* out;                /* [num_tokens, out_cols] bf16; or NULL ... */
    int64_t out_stride;
    uint8_t* out_codes;       /* ... and [num_tokens, out_cols] E4M3, contiguous, */
    uint8_t* out_scales;      /* [num_tokens, out_cols / 32] E8M0 */
    void* workspace;          /* at least moe_mxfp8_linear_workspace() bytes (NULL if that is 0) */
    int64_t workspace_bytes;
    int64_t num_tokens;       /* 0 .. 2^20 */
    int64_t rows;             /* a multiple of 64, 64 .. 2^20 */
    int64_t inner;            /* a multiple of 128, 128 .. 65536 */
    int32_t activation;       /* MOE_EPI_* */
    int32_t reserved;         /* 0 */
} moe_mxfp8_linear_args;

/* Bytes of workspace a call of these sizes needs (0: none), the same for
 * both kinds of output (MXFP8's need, asked of a bf16 call as well), or a
 * negative status for sizes moe_mxfp8_linear refuses. */
int64_t moe_mxfp8_linear_workspace(int64_t num_tokens, int64_t rows, int64_t inner, int32_t activation);

/* Exactly one of out and out_codes (with out_scales) must be given.  All
 * pointers 16-byte aligned (x_scales, out_scales: 4), rows of out and
 * residual 16-byte aligned.  MOE_E_NULL, MOE_E_SHAPE, MOE_E_ALIGN,
 * MOE_E_OPTION (activation, reserved, both or neither output), MOE_E_LIMIT
 * (workspace too small), MOE_E_HIP. */
int moe_mxfp8_linear(const moe_mxfp8_linear_args* args, void* stream);

/* -------------------------------------------------------------- dispatch
 * The slots t * top_k + j of ids [num_tokens, top_k], sorted by expert,
 * ascending inside an expert (the order of moe_mxfp4_options.sorted), and
 * the token rows in that order:
 *
 *   counts[e]    slots with ids == e          (optional)
 *   offsets[e]   exclusive prefix sum of the counts; offsets[num_experts] = n
 *   sorted[p]    the slot at position p, p < n            (optional)
 *   pos[t, j]    the position of slot t * top_k + j
 *   rows[p, :]   x[sorted[p] / top_k, :]                  (optional)
 *
 * A slot whose id is outside 0 .. num_experts-1 (an expert another rank
 * holds, a dropped slot) has no position: its pos is -1 and no row is
 * written for it.  sorted and rows are written up to position n and left as
 * they were behind it; they must hold num_tokens * top_k entries.  A token
 * may name an expert twice.  rows are copied bit for bit: bf16, float32, or
 * MXFP8 (dtype MOE_DT_U8) with the scale rows beside them. */
typedef struct moe_dispatch_args {
    const int32_t* ids;       /* [num_tokens, top_k], contiguous */
    const void* x;            /* [num_tokens, hidden] or NULL (order only) */
    int64_t x_stride;
    const uint8_t* x_scales;  /* MOE_DT_U8: [num_tokens, hidden / 32], contiguous; else NULL */
    int32_t* counts;          /* [num_experts] or NULL */
    int32_t* offsets;         /* [num_experts + 1] */
    int32_t* sorted;          /* [num_tokens * top_k] or NULL */
    int32_t* pos;             /* [num_tokens, top_k] */
    void* rows;               /* [num_tokens * top_k, hidden], contiguous; NULL with x */
    uint8_t* row_scales;      /* [num_tokens * top_k, hidden / 32]; NULL with x_scales */
    void* workspace;          /* at least moe_dispatch_workspace() bytes, 4-byte aligned */
    int64_t workspace_bytes;
    int64_t num_tokens;       /* num_tokens * top_k <= 2^25 */
    int64_t num_experts;      /* 1 .. 1024 */
    int64_t hidden;           /* 1 .. 65536 elements (MOE_DT_U8: a multiple of 32) */
    int32_t top_k;            /* 1 .. 32 */
    int32_t dtype;            /* of x and rows: MOE_DT_BF16, MOE_DT_F32, MOE_DT_U8 (MXFP8) */
} moe_dispatch_args;

/* Bytes of workspace (0: none), or a negative status for refused sizes. */
int64_t moe_dispatch_workspace(int64_t num_tokens, int64_t num_experts, int32_t top_k);

/* Pointers and row starts need only the alignment of their elements
 * (16-byte aligned rows are copied fastest).  MOE_E_NULL, MOE_E_SHAPE,
 * MOE_E_TOPK, MOE_E_DTYPE, MOE_E_ALIGN, MOE_E_LIMIT (workspace too small),
 * MOE_E_HIP. */
int moe_dispatch(const moe_dispatch_args* args, void* stream);

/* --------------------------------------------------------------- combine
 *   out[t, :] = sum_j weights[t, j] * rows[pos[t, j], :]
 *
 * in float32, j ascending, over the slots with a position (pos >= 0; the
 * weight of a slot without one is not read into the sum, nor is anything
 * else); a token without any gets zeros.  weights == NULL: weight 1, which
 * is moe_dispatch_backward.
 *
 * moe_combine_backward, given dout:
 *   drows[pos[t, j], :] = weights[t, j] * dout[t, :]
 *   dweights[t, j]      = <dout[t, :], rows[pos[t, j], :]>, 0 without a position
 * drows rows that no slot points to are left as they were; either output
 * may be NULL (not both, unless num_rows is 0). */
typedef struct moe_combine_args {
    const void* rows;         /* [num_rows, hidden], rows_dtype (backward: NULL if dweights is) */
    int64_t rows_stride;
    const float* weights;     /* [num_tokens, top_k] or NULL */
    const int32_t* pos;       /* [num_tokens, top_k], each < num_rows (a larger one: as -1) */
    void* out;                /* [num_tokens, hidden], out_dtype; unused by the backward */
    int64_t out_stride;
    const void* dout;         /* backward: [num_tokens, hidden], out_dtype */
    int64_t dout_stride;
    void* drows;              /* backward: [num_rows, hidden], rows_dtype, or NULL.  May be `rows`
                                 itself.  Two slots may not share a position. */
    int64_t drows_stride;
    float* dweights;          /* backward: [num_tokens, top_k] or NULL */
    int64_t num_tokens;       /* num_tokens * top_k <= 2^25 */
    int64_t num_rows;         /* 0 .. 2^25 */
    int64_t hidden;           /* 1 .. 65536 */
    int32_t top_k;            /* 1 .. 32 */
    int32_t rows_dtype;       /* MOE_DT_BF16 or MOE_DT_F32 */
    int32_t out_dtype;        /* MOE_DT_BF16 or MOE_DT_F32 */
    int32_t reserved;         /* 0 */
} moe_combine_args;

/* MOE_E_NULL, MOE_E_SHAPE, MOE_E_TOPK, MOE_E_DTYPE, MOE_E_ALIGN (element
 * alignment), MOE_E_OPTION (reserved), MOE_E_HIP. */
int moe_combine(const moe_combine_args* args, void* stream);
int moe_combine_backward(const moe_combine_args* args, void* stream);

/* dx[t, :] = sum_j drows[pos[t, j], :] -- the gradient of moe_dispatch's rows
 * (moe_combine with weights = NULL; `rows` is drows, `out` is dx). */
int moe_dispatch_backward(const moe_combine_args* args, void* stream);

/* ----------------------------------------- the expert layer on MXFP8 rows
 * moe_mxfp4_forward_ex with activations that are in MXFP8 already (as
 * moe_rmsnorm and moe_mxfp8_linear leave them): x_codes [num_tokens, hidden]
 * and x_scales [num_tokens, hidden / 32], both 16-byte aligned, in place of
 * x.  The same output bits as moe_mxfp4_forward_ex with MOE_ACT_MXFP8 on an
 * x whose encoding they are, without the encoding pass.  opt == NULL: the
 * plain call on weights in the tile layout; else opt->act_format must be
 * MOE_ACT_MXFP8 and opt->router_weight NULL (MOE_E_OPTION: the router product
 * reads bf16 rows).  Needs moe_mxfp4_init, and shares the layer's workspace
 * and its rules.  Status codes as moe_mxfp4_forward_ex. */
int moe_mxfp4_forward_mx8(const uint8_t* x_codes, const uint8_t* x_scales, const float* router_logits,
                          int64_t num_tokens, int32_t top_k, const uint8_t* W_gate_up,
                          const uint8_t* W_down, const moe_mxfp4_scales* scales, void* out, void* stream,
                          const moe_mxfp4_options* opt);

#ifdef __cplusplus
}
#endif

#endif /* MOE_OPS_H */
