/*
 * fp8adam_list.h -- list operators beside the FP8-moment Adam step (fp8adam.h), for AMD MI355X:
 * what a training step with mixed tensor lists needs around it.
 *
 *   fp8adam_adamw_*     AdamW over a list whose tensors differ: fp32 / bf16 / fp16 weights and
 *                       gradients, moments in fp32 or in 8 bits tensor by tensor, parameter groups
 *                       with hyperparameters of their own, a 16-bit copy of fp32 weights written by
 *                       the same pass.
 *   fp8adam_clip_*      the global norm of a list of gradients, and the gradients clipped to it, in
 *                       place or into another list and type (accumulated fp32 gradients into the
 *                       bf16 ones fp8adam_step reads).
 *   fp8adam_quant_*     a list to FP8 codes with scales, per tensor or per 128 elements, and back
 *                       (moments between 32 and 8 bits, weights for an FP8 forward pass).
 *
 * Each works through a plan: built once over a list, it holds the list's descriptors and the
 * workspace on the device.  Building allocates and synchronizes the stream, which must not be
 * under capture (EINVAL).  A call enqueues its kernels on the given stream (0 = the null
 * stream), allocates nothing, does not synchronize, and may be captured into a graph and
 * replayed.  Calls of one plan must not overlap (they share its workspace; neither may replays of
 * graphs that captured it); calls of different plans may, unless their tensors overlap.
 *
 * A replay takes what lies in device memory as it is then, and every argument from the host as it
 * was at the capture: hyperparameters, max_norm, the scaler's factors, and fp8adam_adamw_step's
 * `step`.  A replayed fp8adam_adamw_step therefore corrects its moments with the same t every
 * time; training by replays takes fp8adam_adamw_step_amp, which counts t in device memory.  A
 * new learning rate needs a new capture.
 *
 * Conventions are fp8adam.h's: 0 or a negative FP8ADAM_E* code with fp8adam_last_error(); no
 * exception crosses the ABI; the plan belongs to the device that was current when it was built
 * and a stream of another device is refused.  Tensors are dense runs of `numel` elements at any
 * address that is a multiple of their element's size (EALIGN otherwise), owned by the caller, and
 * must stay valid and in place while the plan exists.  Nothing that a call writes may overlap
 * anything else in the list (EINVAL).  A tensor with numel 0 needs no pointers.
 */
#ifndef FP8ADAM_LIST_H
#define FP8ADAM_LIST_H

#include "fp8adam.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { FP8ADAM_F32 = 0, FP8ADAM_BF16 = 1, FP8ADAM_F16 = 2 } fp8adam_dtype;
/* A tensor's moments: two fp32 numbers per element, or two FP8 codes with one power-of-two scale
 * per 128 elements each (the block-128 POW2 state of fp8adam_step). */
typedef enum { FP8ADAM_MOMENTS_32 = 0, FP8ADAM_MOMENTS_8 = 1 } fp8adam_moments;

typedef struct fp8adam_plan fp8adam_plan;

/* Frees a plan of any kind (NULL is ignored).  The caller makes sure that no call of it is still
 * running, and that no graph that captured one is replayed again. */
void fp8adam_plan_destroy(fp8adam_plan *plan);

/* ---- AdamW over a mixed list ----
 * Per element, in fp32, with G the gradient (times the gradient factor with loss scaling):
 *   m' = fma(b1, m, (1-b1)*G)          v' = fma(b2, v, (1-b2)*(G*G))
 *   p' = p - (lr*wd*p + lr/(1-beta1^t) * m' / (sqrt(v'/(1-beta2^t)) + eps))
 * p' is then rounded to the weight's type, and for the copy to the copy's (to nearest even).  b1,
 * 1-b1, b2, 1-b2 and the other constants are fp32 numbers nearest to their values in double.
 * 8-bit moments are decoded from code * scale; every block of 128 elements then takes the POW2
 * scale of its largest |m'| (v'), and the codes are encode(m' / scale), to nearest even: codes and
 * scales are bit-exact functions of the inputs, and with bf16 gradients those of fp8adam_step with
 * FP8ADAM_SCALE_BLOCK128 (given beta1 and beta2 that are fp32 numbers).
 * Not finite: a NaN or Inf gradient makes the moments and the weight what the formulas give (8-bit
 * moments: the block takes scale 1, an Inf saturates, a NaN becomes a NaN code); eps = 0 with
 * v' = 0 gives NaN.  With eps < 2^-38, a v'/(1-beta2^t) of 2^104 or more counts as Inf (2^80
 * with an eps between 0 and 2^-114). */
typedef struct {
    void *param;          /* weights, read and written */
    const void *grad;     /* gradients, read */
    void *copy;           /* 16-bit copy of fp32 weights, written; or NULL */
    void *m, *v;          /* moments, read and written: fp32, or codes */
    float *m_scale, *v_scale; /* 8-bit moments: ceil(numel/128) scales each (4-byte aligned) */
    int64_t numel;
    int32_t param_dtype, grad_dtype, copy_dtype; /* fp8adam_dtype; copy: BF16 or F16, with F32 weights only */
    int32_t moments;      /* fp8adam_moments */
    int32_t group;        /* parameter group, 0 .. n_groups-1 */
    int32_t reserved;     /* 0 */
} fp8adam_adamw_tensor;

#define FP8ADAM_MAX_GROUPS 32
typedef struct {
    int32_t n_groups;           /* 1 .. FP8ADAM_MAX_GROUPS */
    int32_t m_format, v_format; /* fp8adam_format of 8-bit moments */
    int32_t reserved;           /* 0 */
} fp8adam_adamw_config;

/* One group's hyperparameters: lr and weight_decay finite, betas in [0, 1), eps finite and >= 0. */
typedef struct {
    double lr, beta1, beta2, eps, weight_decay;
} fp8adam_adamw_hparams;

int fp8adam_adamw_plan(fp8adam_plan **out, const fp8adam_adamw_tensor *tensors, int32_t n,
                       const fp8adam_adamw_config *cfg, hipStream_t stream);
/* One step; groups holds n_groups hyperparameters (the plan's number of groups) on the host; step
 * is the 1-based t.  One kernel launch for each combination of types and moments in the list. */
int fp8adam_adamw_step(fp8adam_plan *plan, const fp8adam_adamw_hparams *groups, int32_t n_groups,
                       int64_t step, hipStream_t stream);
/* One step with loss scaling, skipping and clipping on the device, as fp8adam_step_amp: the norm
 * over every gradient of the list, the scaler's decision in *state (device memory, 8-byte aligned),
 * then the step with every gradient multiplied by state's grad_factor and t = state's step, or
 * nothing if a gradient was not finite.  With a scale of 1 and a growth_interval out of reach
 * (INT32_MAX) it is a step with clipping alone, for as long as no step is skipped: a skipped one
 * lowers the scale, which the program then sets back. */
int fp8adam_adamw_step_amp(fp8adam_plan *plan, const fp8adam_adamw_hparams *groups, int32_t n_groups,
                           const fp8adam_amp_config *amp, fp8adam_amp_state *state, hipStream_t stream);

/* ---- global norm and clipping of a list of gradients ----
 *   N = sqrt(sum of src^2 over the list)       (in fp64, in a fixed order: the same bits every time)
 *   c = min(1, max_norm / (N + 1e-6)) in fp32  (1 if max_norm <= 0, or if N is not finite)
 *   dst = src * c, in fp32, rounded to dst's type (to nearest even)
 * dst may be src itself (the same address and type), another tensor, or NULL: then the tensor
 * counts in the norm and nothing is written.  result[0] = N, result[1] = c, in fp32 (device).  A
 * list with a NaN or Inf keeps it: N is then NaN or Inf, and c is 1. */
typedef struct {
    const void *src;
    void *dst;
    int64_t numel;
    int32_t src_dtype, dst_dtype; /* fp8adam_dtype */
} fp8adam_clip_tensor;

int fp8adam_clip_plan(fp8adam_plan **out, const fp8adam_clip_tensor *tensors, int32_t n, hipStream_t stream);
/* max_norm finite (EINVAL otherwise); result: 2 floats on the device, 4-byte aligned. */
int fp8adam_clip_grads(fp8adam_plan *plan, float max_norm, float *result, hipStream_t stream);

/* ---- a list in 8 bits with scales ----
 * quantize:   s = the scale of the largest |value| of the tensor, or of each run of 128 elements
 *             (fp8adam_scale_mode's rules); codes = encode(value * inv_s), to nearest even, saturating
 * dequantize: values = decode(code) * s in fp32 (exact for POW2), rounded to the values' type (to nearest even)
 * A tensor or block with a NaN or Inf takes scale 1 (its Inf saturates, its NaN
 * becomes a NaN code).  Both directions use the same
 * plan; quantize only reads the values and dequantize only writes them. */
typedef struct {
    void *values;
    uint8_t *codes;
    float *scale;         /* 1 float, or ceil(numel/128) with block granularity (4-byte aligned) */
    int64_t numel;
    int32_t dtype;        /* fp8adam_dtype of the values */
    int32_t format;       /* fp8adam_format of the codes */
} fp8adam_quant_tensor;

typedef struct {
    int32_t granularity;  /* fp8adam_granularity */
    int32_t scale_mode;   /* fp8adam_scale_mode */
} fp8adam_quant_config;

int fp8adam_quant_plan(fp8adam_plan **out, const fp8adam_quant_tensor *tensors, int32_t n,
                       const fp8adam_quant_config *cfg, hipStream_t stream);
int fp8adam_quantize(fp8adam_plan *plan, hipStream_t stream);
int fp8adam_dequantize(fp8adam_plan *plan, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8ADAM_LIST_H */
