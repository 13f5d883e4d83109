/* A plain C11 caller of the list operators: no torch, no Python.  Clips fp32
 * gradients into bf16 ones, takes an AdamW step with 32-bit moments and a bf16 copy
 * of the weights, and converts the weights to E4M3 blocks and back; every result is
 * checked against double arithmetic here.  Calls that do not fit their plan are
 * refused.  Exit status 0 and "c list demo ok" on success. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "fp8adam_list.h"

#define N 5003
#define CHECK_HIP(e) do { hipError_t r_ = (e); if (r_ != hipSuccess) { \
    fprintf(stderr, "%s: %s\n", #e, hipGetErrorString(r_)); return 1; } } while (0)
#define CHECK_LIB(e) do { int r_ = (e); if (r_ != 0) { \
    fprintf(stderr, "%s: %d %s\n", #e, r_, fp8adam_last_error()); return 1; } } while (0)
#define REFUSED(e, code) do { int r_ = (e); if (r_ != (code)) { \
    fprintf(stderr, "%s: %d, not %d\n", #e, r_, (code)); return 1; } } while (0)

static float from_bf16(uint16_t b) {
    uint32_t u = (uint32_t)b << 16;
    float x;
    memcpy(&x, &u, 4);
    return x;
}

static double uniform(uint64_t *s) {
    *s = *s * 6364136223846793005ULL + 1442695040888963407ULL;
    return ((double)(*s >> 33) + 0.5) / 2147483648.0 - 0.5;
}

int main(void) {
    static float p0[N], g0[N], p[N], m[N], v[N], back[N];
    static uint16_t g[N], copy[N];
    uint64_t seed = 7;
    double norm = 0.0;
    for (int i = 0; i < N; i++) {
        p0[i] = (float)(uniform(&seed) * 0.04);
        g0[i] = (float)uniform(&seed);
        norm += (double)g0[i] * g0[i];
    }
    norm = sqrt(norm);
    float *d_p, *d_g0, *d_m, *d_v, *d_scale, *d_back, *d_result;
    uint16_t *d_g, *d_copy;
    uint8_t *d_codes;
    CHECK_HIP(hipMalloc((void **)&d_p, sizeof p0));
    CHECK_HIP(hipMalloc((void **)&d_g0, sizeof g0));
    CHECK_HIP(hipMalloc((void **)&d_m, sizeof m));
    CHECK_HIP(hipMalloc((void **)&d_v, sizeof v));
    CHECK_HIP(hipMalloc((void **)&d_g, sizeof g + 2));
    CHECK_HIP(hipMalloc((void **)&d_copy, sizeof copy));
    CHECK_HIP(hipMalloc((void **)&d_codes, N));
    CHECK_HIP(hipMalloc((void **)&d_scale, sizeof(float) * ((N + 127) / 128)));
    CHECK_HIP(hipMalloc((void **)&d_back, sizeof back));
    CHECK_HIP(hipMalloc((void **)&d_result, 2 * sizeof(float)));
    CHECK_HIP(hipMemcpy(d_p, p0, sizeof p0, hipMemcpyHostToDevice));
    CHECK_HIP(hipMemcpy(d_g0, g0, sizeof g0, hipMemcpyHostToDevice));
    CHECK_HIP(hipMemset(d_m, 0, sizeof m));
    CHECK_HIP(hipMemset(d_v, 0, sizeof v));
    uint16_t *const grad = d_g + 1; /* not on a dword */

    fp8adam_clip_tensor ct = {d_g0, grad, N, FP8ADAM_F32, FP8ADAM_BF16};
    fp8adam_adamw_tensor at;
    memset(&at, 0, sizeof at);
    at.param = d_p; at.grad = grad; at.copy = d_copy; at.m = d_m; at.v = d_v; at.numel = N;
    at.param_dtype = FP8ADAM_F32; at.grad_dtype = FP8ADAM_BF16; at.copy_dtype = FP8ADAM_BF16;
    fp8adam_adamw_config ac = {1, FP8ADAM_E4M3, FP8ADAM_E5M2, 0};
    fp8adam_quant_tensor qt = {d_p, d_codes, d_scale, N, FP8ADAM_F32, FP8ADAM_E4M3};
    fp8adam_quant_tensor bt = {d_back, d_codes, d_scale, N, FP8ADAM_F32, FP8ADAM_E4M3};
    fp8adam_quant_config qc = {FP8ADAM_SCALE_BLOCK128, FP8ADAM_SCALE_POW2};
    fp8adam_adamw_hparams hp = {1e-3, 0.9, 0.95, 1e-8, 0.1};
    fp8adam_plan *clip, *adamw, *quant, *unquant;
    CHECK_LIB(fp8adam_clip_plan(&clip, &ct, 1, NULL));
    CHECK_LIB(fp8adam_adamw_plan(&adamw, &at, 1, &ac, NULL));
    CHECK_LIB(fp8adam_quant_plan(&quant, &qt, 1, &qc, NULL));
    CHECK_LIB(fp8adam_quant_plan(&unquant, &bt, 1, &qc, NULL));

    REFUSED(fp8adam_quantize(clip, NULL), FP8ADAM_EINVAL);
    REFUSED(fp8adam_clip_grads(adamw, 1.0f, d_result, NULL), FP8ADAM_EINVAL);
    REFUSED(fp8adam_adamw_step(quant, &hp, 1, 1, NULL), FP8ADAM_EINVAL);
    REFUSED(fp8adam_adamw_step(adamw, &hp, 2, 1, NULL), FP8ADAM_EINVAL);
    REFUSED(fp8adam_adamw_step(adamw, NULL, 1, 1, NULL), FP8ADAM_EINVAL);
    REFUSED(fp8adam_clip_grads(clip, INFINITY, d_result, NULL), FP8ADAM_EINVAL);
    REFUSED(fp8adam_clip_grads(clip, 1.0f, NULL, NULL), FP8ADAM_EINVAL);
    REFUSED(fp8adam_clip_grads(clip, 1.0f, (float *)((char *)d_result + 2), NULL), FP8ADAM_EALIGN);

    CHECK_LIB(fp8adam_clip_grads(clip, 1.0f, d_result, NULL));
    CHECK_LIB(fp8adam_adamw_step(adamw, &hp, 1, 1, NULL));
    CHECK_LIB(fp8adam_quantize(quant, NULL));
    CHECK_LIB(fp8adam_dequantize(unquant, NULL));
    float result[2];
    CHECK_HIP(hipMemcpy(result, d_result, sizeof result, hipMemcpyDeviceToHost));
    CHECK_HIP(hipMemcpy(g, grad, sizeof g, hipMemcpyDeviceToHost));
    CHECK_HIP(hipMemcpy(p, d_p, sizeof p, hipMemcpyDeviceToHost));
    CHECK_HIP(hipMemcpy(copy, d_copy, sizeof copy, hipMemcpyDeviceToHost));
    CHECK_HIP(hipMemcpy(back, d_back, sizeof back, hipMemcpyDeviceToHost));

    /* half steps: fp32 2^-24, bf16 2^-8, e4m3 2^-4 (relative), 2^-10 of the scale near zero */
    const double u = ldexp(1.0, -24), c = 1.0 / (norm + 1e-6);
    int bad = fabs(result[0] - norm) > 2 * u * norm || fabs(result[1] - c) > 2 * u * c;
    for (int i = 0; i < N; i++) {
        const double want_g = g0[i] * c;
        bad |= fabs(from_bf16(g[i]) - want_g) > (ldexp(1.0, -8) + 4 * u) * fabs(want_g);
        const double G = from_bf16(g[i]);
        const double upd = 1e-3 * G / (fabs(G) + 1e-8), want = p0[i] - (1e-4 * p0[i] + upd);
        bad |= fabs(p[i] - want) > u * (17 * fabs(upd) + 2e-4 * fabs(p0[i]) + fabs(want)) + 1e-38;
        bad |= fabs(from_bf16(copy[i]) - p[i]) > ldexp(1.0, -8) * fabs(p[i]);
        double amax = 0.0; /* of its block */
        for (int k = i / 128 * 128; k < N && k < i / 128 * 128 + 128; k++) amax = fmax(amax, fabs(p[k]));
        bad |= fabs(back[i] - p[i]) > ldexp(1.0, -4) * fabs(p[i]) + ldexp(amax / 224.0, -10);
        if (bad) {
            fprintf(stderr, "element %d is off\n", i);
            return 1;
        }
    }
    fp8adam_plan_destroy(clip);
    fp8adam_plan_destroy(adamw);
    fp8adam_plan_destroy(quant);
    fp8adam_plan_destroy(unquant);
    printf("c list demo ok\n");
    return 0;
}
