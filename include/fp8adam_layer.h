/*
 * fp8adam_layer.h -- linear layers on 8-bit operands with 8-bit activation checkpoints, for AMD
 * MI355X: what lies between the FP8 weights that fp8adam_quantize makes and the gradients that
 * fp8adam_clip_grads and the AdamW steps take.
 *
 *   fp8adam_pack8 / unpack8       a matrix of activations to 8 bits with scales, and back
 *   fp8adam_linear8               act(x w^T + bias) + residual, x and w in 8 bits; the sum before the
 *                                 activation is kept in 8 bits where asked
 *   fp8adam_gated8                act(x wg^T) * (x wu^T): both projections, the activation and the
 *                                 product in one kernel; both projections are kept in 8 bits where asked
 *   fp8adam_linear8_backward      the gradient of the activation from the 8-bit checkpoint, and the bias's
 *   fp8adam_gated8_backward       the gradients of both projections from their 8-bit checkpoints
 *   fp8adam_weight_grad8          dy^T x from the 8-bit checkpoint of x, added to a gradient or written
 *   fp8adam_input_grad8           dy w from the 8-bit weights, summed over up to two layers of one input
 *
 * Matrices in 8 bits: FP8 codes, row after row, and one power-of-two scale for every 128 columns of
 * a row (the row's last block may be shorter).  The scale of a block is the smallest power of two s with
 * amax / s <= FMAX (448 or 57344), between 2^-126 and 2^126, and 1 for a block of zeros or one with a
 * NaN or Inf; its codes are encode(x / s), to nearest even, saturating (an Inf saturates, a NaN becomes
 * a NaN code): the block rule of fp8adam_quantize.  Where cols is a multiple of 128, codes and scales of
 * fp8adam_quantize with FP8ADAM_SCALE_BLOCK128 and FP8ADAM_SCALE_POW2 are such a matrix.
 *
 * There is no plan: activations move from step to step.  A call enqueues its kernels on the given
 * stream (0 = the null stream), which must belong to the current device, allocates nothing, does not
 * synchronize and may be captured into a graph and replayed (a replay uses the same addresses).  Calls
 * may overlap unless they share memory that one of them writes, their workspaces among it.  Results are
 * the same bits in every run.  Errors as in fp8adam.h: 0 or a negative code with fp8adam_last_error().
 * What a call writes may not overlap anything else of it (EINVAL), except where said.
 */
#ifndef FP8ADAM_LAYER_H
#define FP8ADAM_LAYER_H

#include "fp8adam_list.h"

#ifdef __cplusplus
extern "C" {
#endif

/* gelu(z) = z (1 + erf(z / sqrt 2)) / 2,  silu(z) = z / (1 + e^-z) */
typedef enum {
    FP8ADAM_ACT_NONE = 0, FP8ADAM_ACT_RELU = 1, FP8ADAM_ACT_SILU = 2, FP8ADAM_ACT_GELU = 3
} fp8adam_activation;
typedef enum { FP8ADAM_SCALES_E8M0 = 0, FP8ADAM_SCALES_F32 = 1 } fp8adam_scale_type;

#define FP8ADAM_LAYER_MAX_COLS (1 << 20) /* rows and cols of weights, columns of activations */
#define FP8ADAM_LAYER_MAX_LD (1 << 21)   /* every ld */

/* A matrix in 16 or 32 bits, row-major: rows `ld` elements apart (not used where there is
 * one row), aligned to its element.  data = NULL where it is optional: absent. */
typedef struct {
    void *data;
    int64_t ld;
    int32_t dtype;        /* fp8adam_dtype */
    int32_t reserved;     /* 0 */
} fp8adam_matrix;

/* A matrix in 8 bits.  codes: rows `ld` bytes apart, 16-byte aligned, ld a multiple of 16 that holds cols
 * rounded up to 128; the codes behind cols, up to that multiple, are zero (written as zero by the calls
 * that write such a matrix).  scales: rows `ld_scale` entries apart, 4-byte aligned.  E8M0: bytes b that
 * stand for 2^(b - 127), ld_scale a multiple of 4.  F32: powers of two in fp32 (of matrices that a call
 * reads only).  Scales lie between 2^-126 and 2^127 (b between 1 and 254); others are not checked for.  codes = NULL where it is optional: absent. */
typedef struct {
    void *codes;
    void *scales;
    int64_t ld, ld_scale;
    int32_t format;       /* fp8adam_format */
    int32_t scale_type;   /* fp8adam_scale_type */
} fp8adam_matrix8;

/* x [rows, cols] -> out (E8M0 scales), and back: decode(code) * scale, rounded once to x's type (to
 * nearest even).  rows >= 0, cols >= 1. */
int fp8adam_pack8(const fp8adam_matrix *x, const fp8adam_matrix8 *out, int64_t rows, int64_t cols, hipStream_t stream);
int fp8adam_unpack8(const fp8adam_matrix8 *in, const fp8adam_matrix *x, int64_t rows, int64_t cols, hipStream_t stream);

/* A layer's forward product over tokens, with rows outputs and cols inputs:
 *   p[t,n] = sum over k of x[t,k] w[n,k]    (of the values the codes stand for, in fp32)
 *   linear8:  z = p + bias;  y = act(z) + residual
 *   gated8:   g = x w^T, u = x w_up^T;  y = act(g) * u
 * in fp32 up to here; y is then rounded to its type (to nearest even), and y8 is y before that rounding in
 * 8 bits.  keep (z or g) and keep_up (u) are those sums in 8 bits.  Where y is fp32, with up to 64
 * tokens, and where `exact` asks for it, every product is exact and added in fp32 (with up to 64 tokens in another order
 * where something is kept).  Otherwise the FP8 matrix
 * instruction adds eight products of consecutive columns at a time, each cut at 2^-13 of the power of two of the
 * largest's exponents, and these sums in fp32: p is then off by up to 7 * 2^-13 of the sum of the largest
 * products of all eights.  Of p's rms the error is typically 1.5e-5 (normal numbers) to 2.6e-5 (a hundredth of the columns
 * eight times as large), below the roundings to 16 and 8 bits; of kept codes one in 600 to 1000 falls on the other
 * side of a border (exact: fewer than one in 100000).  Where large products cancel, what is left may be off by more of
 * itself than any rounding.  "Exact" is a product of what the codes stand for but for what lies below 2^-133 of a code
 * times its scale (scales below 2^-124 of E4M3 and 2^-117 of E5M2).  x_in: if given, x is written first
 * as x_in in 8 bits.  At least one of y and y8 is given; residual may be y itself (the same data, ld and type). */
typedef struct {
    int64_t tokens;       /* >= 0 */
    int64_t rows, cols;   /* >= 1 */
    fp8adam_matrix x_in;  /* optional: [tokens, cols] */
    fp8adam_matrix8 x;    /* [tokens, cols] */
    fp8adam_matrix8 w;    /* [rows, cols] */
    fp8adam_matrix8 w_up; /* gated8: [rows, cols], of w's format and type of scales */
    fp8adam_matrix bias;  /* linear8, optional: rows elements (ld is not used) */
    fp8adam_matrix residual; /* linear8, optional: [tokens, rows] */
    fp8adam_matrix y;     /* optional: [tokens, rows] */
    fp8adam_matrix8 y8;   /* optional: [tokens, rows] */
    fp8adam_matrix8 keep, keep_up; /* optional: [tokens, rows]; keep_up for gated8, both or neither, of one format */
    int32_t activation;   /* fp8adam_activation */
    int32_t exact;        /* 1: every product is exact and added in fp32, whatever is written (0: see above) */
} fp8adam_product8;

int fp8adam_linear8(const fp8adam_product8 *args, hipStream_t stream);
int fp8adam_gated8(const fp8adam_product8 *args, hipStream_t stream);

/* Back through an activation, elementwise in fp32, rounded to the outputs' type (dy's; to nearest even):
 *   linear8:  dz = dy act'(z);  bias_grad[n] (+)= sum over t of dy act'(z) (in fp32, before dz is rounded)
 *   gated8:   dz = dy u act'(g);  dup = dy act(g)
 * with the values that keep and keep_up stand for; act'(0) of relu is 0.  dz and dup may be dy itself.
 * linear8 with FP8ADAM_ACT_NONE: keep and dz absent, bias_grad alone. */
typedef struct {
    int64_t tokens, rows; /* tokens >= 0, rows >= 1 */
    fp8adam_matrix dy;    /* [tokens, rows] */
    fp8adam_matrix8 keep, keep_up;
    fp8adam_matrix dz, dup;
    fp8adam_matrix bias_grad; /* linear8, optional: rows elements (ld is not used) */
    void *workspace;      /* with bias_grad: 16-byte aligned, of at least the size that the function below gives */
    int64_t workspace_bytes;
    int32_t accumulate;   /* bias_grad is added to what stands there (0: written) */
    int32_t activation;
} fp8adam_act_backward8;

int64_t fp8adam_linear8_backward_workspace(const fp8adam_act_backward8 *args); /* or a negative error code */
int fp8adam_linear8_backward(const fp8adam_act_backward8 *args, hipStream_t stream);
int fp8adam_gated8_backward(const fp8adam_act_backward8 *args, hipStream_t stream);

/* Gradients of a layer's weights and of its input, from dy [tokens, rows]:
 *   weight_grad8:  out[n,k] (+)= sum over t of dy[t,n] x[t,k]            out [rows, cols], b[0] = x [tokens, cols]
 *   input_grad8:   out[t,k] (+)= sum over i < n, n of dy_i[t,n] w_i[n,k]  out [tokens, cols], b[i] = w_i [rows, cols]
 * The products are of dy as it is (bf16), or split into bf16 parts: two (fp16, whose 11 bits they hold), or of fp32
 * three with `exact`, which hold its 24 bits, and two without, which hold 16 (each product is off by at most 2^-16 of its
 * size); what lies below 2^-133 is lost, in dy and in a code times its scale.  They are taken with the values that the codes stand for and summed in fp32; out is rounded once (to nearest even). */
typedef struct {
    int64_t tokens, rows, cols;
    int32_t n;            /* input_grad8: layers, 1 or 2 (of one dtype of dy, format and type of scales); weight_grad8: 1 */
    int32_t accumulate;   /* added to what stands in out (0: written) */
    fp8adam_matrix dy[2];
    fp8adam_matrix8 b[2];
    fp8adam_matrix out;
    void *workspace;      /* 16-byte aligned, of at least the size that the functions below give; NULL if that is 0 */
    int64_t workspace_bytes;
    int32_t exact;        /* 1: fp32 dy in all of its bits (0: in 16, two thirds of the products) */
    int32_t reserved;     /* 0 */
} fp8adam_grad8;

int64_t fp8adam_weight_grad8_workspace(const fp8adam_grad8 *args); /* or a negative error code */
int64_t fp8adam_input_grad8_workspace(const fp8adam_grad8 *args);
int fp8adam_weight_grad8(const fp8adam_grad8 *args, hipStream_t stream);
int fp8adam_input_grad8(const fp8adam_grad8 *args, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8ADAM_LAYER_H */
