/* The list operators (fp8adam_list.h) against the HIP runtime's last error, on a stand-in
 * runtime (stub_hip.h): an error that the thread holds from before is not a launch's, and
 * a call that fails leaves none behind.  Exit status 0 is the pass condition. */
#include "stub_hip.h"

#include "fp8adam_list.h"

#define OLD hipErrorInvalidDevice
#define EXPECT(call, want, launches, last) \
    do { \
        const int got = call; \
        expect(#call, got, want, launches, last, fp8adam_last_error()); \
    } while (0)

static fp8adam_plan *adamw(int64_t numel) {
    /* three kinds of tensor: three launches a step */
    fp8adam_adamw_tensor t[3];
    fp8adam_adamw_config cfg = {1, FP8ADAM_E4M3, FP8ADAM_E5M2, 0};
    fp8adam_plan *p = NULL;
    memset(t, 0, sizeof t);
    for (int i = 0; i < 3; i++) {
        uintptr_t at = (uintptr_t)(i + 1) << 40;
        t[i].param = (void *)at;
        t[i].grad = (void *)(at + (1ll << 36));
        t[i].m = (void *)(at + (2ll << 36));
        t[i].v = (void *)(at + (3ll << 36));
        t[i].m_scale = (float *)(at + (4ll << 36));
        t[i].v_scale = (float *)(at + (5ll << 36));
        t[i].numel = numel;
        t[i].param_dtype = i == 2 ? FP8ADAM_BF16 : FP8ADAM_F32;
        t[i].grad_dtype = FP8ADAM_BF16;
        t[i].moments = i == 0 ? FP8ADAM_MOMENTS_32 : FP8ADAM_MOMENTS_8;
    }
    EXPECT(fp8adam_adamw_plan(&p, t, 3, &cfg, NULL), FP8ADAM_OK, 0, stub_last);
    return p;
}

int main(void) {
    const fp8adam_adamw_hparams hp = {1e-3, 0.9, 0.95, 1e-8, 0.1};
    const fp8adam_amp_config amp = {1.0f, 2.0f, 0.5f, 2000};
    static fp8adam_amp_state state;
    static float result[2];
    fp8adam_plan *p = NULL;

    /* an old error: every call launches all of its kernels, reports none, and leaves it to whom it belongs */
    stub_last = OLD;
    p = adamw(1000);
    EXPECT(fp8adam_adamw_step(p, &hp, 1, 1, NULL), FP8ADAM_OK, 3, OLD);
    EXPECT(fp8adam_adamw_step_amp(p, &hp, 1, &amp, &state, NULL), FP8ADAM_OK, 1 + 3, OLD);
    /* a launch that fails: the call ends there, reports it and leaves no error behind */
    for (int k = 0; k < 3; k++) {
        stub_fail_launch = k;
        EXPECT(fp8adam_adamw_step(p, &hp, 1, 1, NULL), FP8ADAM_EHIP, k, hipSuccess);
        EXPECT(fp8adam_adamw_step_amp(p, &hp, 1, &amp, &state, NULL), FP8ADAM_EHIP, k, hipSuccess);
    }
    stub_fail_launch = -1;
    EXPECT(fp8adam_adamw_step(p, &hp, 1, 1, NULL), FP8ADAM_OK, 3, hipSuccess);
    fp8adam_plan_destroy(p);

    stub_last = OLD;
    p = adamw(300000);  /* the decision is a launch of its own */
    EXPECT(fp8adam_adamw_step_amp(p, &hp, 1, &amp, &state, NULL), FP8ADAM_OK, 2 + 3, OLD);
    for (int k = 0; k < 5; k++) {
        stub_fail_launch = k;
        EXPECT(fp8adam_adamw_step_amp(p, &hp, 1, &amp, &state, NULL), FP8ADAM_EHIP, k, hipSuccess);
    }
    stub_fail_launch = -1;
    fp8adam_plan_destroy(p);

    fp8adam_clip_tensor c = {(void *)(1ll << 40), (void *)(2ll << 40), 5000, FP8ADAM_F32, FP8ADAM_BF16};
    stub_last = OLD;
    EXPECT(fp8adam_clip_plan(&p, &c, 1, NULL), FP8ADAM_OK, 0, OLD);
    EXPECT(fp8adam_clip_grads(p, 1.0f, result, NULL), FP8ADAM_OK, 2, OLD);
    for (int k = 0; k < 2; k++) {
        stub_fail_launch = k;
        EXPECT(fp8adam_clip_grads(p, 1.0f, result, NULL), FP8ADAM_EHIP, k, hipSuccess);
    }
    stub_fail_launch = -1;
    fp8adam_plan_destroy(p);

    for (int g = 0; g < 2; g++) {
        /* two kinds; scales by tensors take a pass of their own for the maxima */
        fp8adam_quant_tensor q[2] = {
            {(void *)(1ll << 40), (uint8_t *)(2ll << 40), (float *)(3ll << 40), 5000, FP8ADAM_F32, FP8ADAM_E4M3},
            {(void *)(4ll << 40), (uint8_t *)(5ll << 40), (float *)(6ll << 40), 70, FP8ADAM_BF16, FP8ADAM_E5M2}};
        fp8adam_quant_config cfg = {g ? FP8ADAM_SCALE_BLOCK128 : FP8ADAM_SCALE_TENSOR, FP8ADAM_SCALE_POW2};
        const int there = g ? 2 : 4;
        stub_last = OLD;
        EXPECT(fp8adam_quant_plan(&p, q, 2, &cfg, NULL), FP8ADAM_OK, 0, OLD);
        EXPECT(fp8adam_quantize(p, NULL), FP8ADAM_OK, there, OLD);
        EXPECT(fp8adam_dequantize(p, NULL), FP8ADAM_OK, 2, OLD);
        for (int k = 0; k < there; k++) {
            stub_fail_launch = k;
            EXPECT(fp8adam_quantize(p, NULL), FP8ADAM_EHIP, k, hipSuccess);
            if (k < 2) EXPECT(fp8adam_dequantize(p, NULL), FP8ADAM_EHIP, k, hipSuccess);
        }
        stub_fail_launch = -1;
        fp8adam_plan_destroy(p);

        /* a plan that cannot be built */
        stub_fail_malloc = 1;
        EXPECT(fp8adam_quant_plan(&p, q, 2, &cfg, NULL), FP8ADAM_ENOMEM, 0, hipSuccess);
        stub_fail_memcpy = 1;
        EXPECT(fp8adam_quant_plan(&p, q, 2, &cfg, NULL), FP8ADAM_EHIP, 0, hipSuccess);
    }
    stub_fail_malloc = 1;
    EXPECT(fp8adam_clip_plan(&p, &c, 1, NULL), FP8ADAM_ENOMEM, 0, hipSuccess);

    /* a plan is not built on a stream that is being captured, and the capture sees nothing of it;
     * the calls of a plan are captured */
    fp8adam_plan *q = NULL;
    EXPECT(fp8adam_clip_plan(&q, &c, 1, NULL), FP8ADAM_OK, 0, hipSuccess);
    stub_capturing = 1;
    stub_device_calls = 0;
    fp8adam_adamw_tensor t;
    memset(&t, 0, sizeof t);
    t.param = (void *)(1ll << 40), t.grad = (void *)(2ll << 40), t.m = (void *)(3ll << 40), t.v = (void *)(4ll << 40);
    t.numel = 10;
    fp8adam_adamw_config acfg = {1, FP8ADAM_E4M3, FP8ADAM_E5M2, 0};
    fp8adam_quant_tensor x = {(void *)(1ll << 40), (uint8_t *)(2ll << 40), (float *)(3ll << 40), 10, 0, 0};
    fp8adam_quant_config qcfg = {FP8ADAM_SCALE_TENSOR, FP8ADAM_SCALE_POW2};
    EXPECT(fp8adam_clip_plan(&p, &c, 1, NULL), FP8ADAM_EINVAL, 0, hipSuccess);
    EXPECT(fp8adam_adamw_plan(&p, &t, 1, &acfg, NULL), FP8ADAM_EINVAL, 0, hipSuccess);
    EXPECT(fp8adam_quant_plan(&p, &x, 1, &qcfg, NULL), FP8ADAM_EINVAL, 0, hipSuccess);
    EXPECT(fp8adam_clip_grads(q, 1.0f, result, NULL), FP8ADAM_OK, 2, hipSuccess);
    if (stub_device_calls) {
        fprintf(stderr, "%d device calls during a capture\n", stub_device_calls);
        failures++;
    }
    stub_capturing = 0;
    fp8adam_plan_destroy(q);
    if (failures) return 1;
    printf("launch errors ok\n");
    return 0;
}
