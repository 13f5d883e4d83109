/* The FP8-moment step and the codec (fp8adam.h) against the HIP runtime's last error, on a
 * stand-in runtime (stub_hip.h): an error that the thread holds from before is not a
 * launch's, a launch that fails ends its call, and no call leaves an error behind.  Exit
 * status 0 is the pass condition. */
#include "stub_hip.h"

#include "fp8adam.h"

#define OLD hipErrorInvalidDevice

static fp8adam_ctx *ctx;
static fp8adam_tensor tensors[2];
static fp8adam_config cfg;
static fp8adam_hparams hp = {1e-3f, 0.9f, 0.95f, 1e-8f, 0.1f, 1};
static const fp8adam_amp_config amp = {1.0f, 2.0f, 0.5f, 2000};
static fp8adam_amp_state state;
static char memory[16][1024] __attribute__((aligned(256)));

static int step(void) { return fp8adam_step(ctx, &hp, NULL); }
static int step_amp(void) { return fp8adam_step_amp(ctx, &hp, &amp, &state, NULL); }
static int step_noalloc(void) { return fp8adam_step_noalloc(tensors, 2, &cfg, &hp, NULL); }
static int init(void) {
    const int r = fp8adam_init(&ctx, tensors, 2, &cfg, NULL);
    if (r == FP8ADAM_OK) fp8adam_destroy(ctx);
    ctx = NULL;
    return r;
}
static int encode(void) { return fp8adam_encode(0, (float *)memory[0], (uint8_t *)memory[1], 5, NULL); }
static int encode5(void) { return fp8adam_encode(1, (float *)memory[0], (uint8_t *)memory[1], 5, NULL); }
static int decode(void) { return fp8adam_decode(0, (uint8_t *)memory[1], (float *)memory[0], 5, NULL); }
static int decode5(void) { return fp8adam_decode(1, (uint8_t *)memory[1], (float *)memory[0], 5, NULL); }
static int bits(void) { return fp8adam_encode_bits_range(0, 0, 5, (uint8_t *)memory[0], NULL); }
static int bits5(void) { return fp8adam_encode_bits_range(1, 0, 5, (uint8_t *)memory[0], NULL); }
static int sr_bits(void) { return fp8adam_encode_sr_bits_range(0, 0, 5, 1, (uint8_t *)memory[0], NULL); }
static int sr_bits5(void) { return fp8adam_encode_sr_bits_range(1, 0, 5, 1, (uint8_t *)memory[0], NULL); }
static int sr(void) {
    return fp8adam_encode_sr(0, (float *)memory[0], (uint16_t *)memory[1], (uint8_t *)memory[2], 5, NULL);
}
static int sr5(void) {
    return fp8adam_encode_sr(1, (float *)memory[0], (uint16_t *)memory[1], (uint8_t *)memory[2], 5, NULL);
}
static int copy(void) { return fp8adam_stream_copy(memory[0], memory[1], 64, NULL); }
static int rw(void) { return fp8adam_stream_rw(memory[0], 64, memory[1], 64, NULL); }
static int mix(void) {
    return fp8adam_stream_mix(0, memory[0], memory[1], memory[2], memory[3], memory[4], memory[5], 4096, NULL);
}
static int mix16(void) {
    return fp8adam_stream_mix(1, memory[0], memory[1], memory[2], memory[3], memory[4], memory[5], 4096, NULL);
}

/* One call: as it should be; with an old error pending; with each of its launches failing. */
static void check(const char *what, int (*call)(void)) {
    stub_last = hipSuccess;
    stub_launches = 0;
    int r = call();
    const int n = stub_launches;
    if (n < 1) {
        fprintf(stderr, "%s: no launch (%d, %s)\n", what, r, fp8adam_last_error());
        failures++;
    }
    expect(what, r, FP8ADAM_OK, n, hipSuccess, fp8adam_last_error());
    stub_last = OLD;
    r = call();
    expect(what, r, FP8ADAM_OK, n, OLD, fp8adam_last_error());
    for (int k = 0; k < n; k++) {
        stub_fail_launch = k;
        r = call();
        expect(what, r, FP8ADAM_EHIP, k, hipSuccess, fp8adam_last_error());
    }
    stub_fail_launch = -1;
}

static void steps(const char *what, int64_t t) {
    fp8adam_ctx *c = NULL;
    const int r = fp8adam_init(&c, tensors, 2, &cfg, NULL);
    expect(what, r, FP8ADAM_OK, stub_launches, stub_last, fp8adam_last_error());
    if (!c) return;
    ctx = c;
    hp.step = t;
    check(what, step);
    check(what, step_amp);
    /* timed: a launch that fails is not among the timed ones */
    int last = -1;
    for (int k = 0; last != FP8ADAM_OK; k++) {
        double ms[32];
        int32_t count[32], sum = 0;
        if (fp8adam_set_timing(c, 1) != FP8ADAM_OK) failures++;
        stub_launches = 0;
        stub_last = hipSuccess;
        stub_fail_launch = k;
        last = step_amp();
        if (last != FP8ADAM_OK) expect(what, last, FP8ADAM_EHIP, k, hipSuccess, fp8adam_last_error());
        const int launched = last == FP8ADAM_OK ? stub_launches : k;
        if (fp8adam_kernel_times(c, ms, count, 32) != FP8ADAM_OK) failures++;
        for (int i = 0; i < 32; i++) sum += count[i];
        if (sum != launched) {
            fprintf(stderr, "%s: %d kernels timed of %d\n", what, sum, launched);
            failures++;
        }
    }
    stub_fail_launch = -1;
    stub_launches = 0;
    fp8adam_destroy(c);
    ctx = NULL;
}

int main(void) {
    for (int i = 0; i < 2; i++) {
        fp8adam_tensor *t = &tensors[i];
        char(*m)[1024] = memory + 8 * i;
        t->param = m[0];
        t->grad = m[1];
        t->m = (uint8_t *)m[2];
        t->v = (uint8_t *)m[3];
        t->m_scale = (float *)m[4];
        t->v_scale = (float *)m[5];
        t->m_alt = (uint8_t *)m[6];
        t->v_alt = (uint8_t *)m[7];
        t->numel = 200;
    }
    static float history[2][64];
    for (int mf = 0; mf < 2; mf++)
        for (int vf = 0; vf < 2; vf++)
            for (int stats = 0; stats < 2; stats++) {
                memset(&cfg, 0, sizeof cfg);
                cfg.m_format = mf;
                cfg.v_format = vf;
                cfg.collect_stats = stats;
                steps("two passes", 1);
                cfg.granularity = FP8ADAM_SCALE_BLOCK128;
                steps("by blocks", 1);
                cfg.granularity = FP8ADAM_SCALE_TENSOR;
                cfg.schedule = FP8ADAM_SCHEDULE_SPECULATIVE;
                cfg.predictor = FP8ADAM_PREDICT_PROBE;
                steps("before the first speculative step", 3);
                steps("speculative", 4);
                cfg.schedule = FP8ADAM_SCHEDULE_TWO_PASS;
                cfg.scaling = FP8ADAM_SCALING_DELAYED;
                tensors[0].amax_history = history[0];
                tensors[1].amax_history = history[1];
                steps("delayed", 2);
                tensors[0].amax_history = tensors[1].amax_history = NULL;
                cfg.scaling = FP8ADAM_SCALING_JUST_IN_TIME;
                if (!stats) check("without allocation", step_noalloc);
            }
    memset(&cfg, 0, sizeof cfg);
    cfg.zero_state = 1;
    check("fp8adam_init", init);
    stub_fail_malloc = 1;
    int r = init();
    expect("fp8adam_init out of memory", r, FP8ADAM_ENOMEM, 0, hipSuccess, fp8adam_last_error());
    stub_fail_memcpy = 1;
    r = init();
    expect("fp8adam_init with a failed copy", r, FP8ADAM_EHIP, 0, hipSuccess, fp8adam_last_error());
    check("encode", encode);
    check("encode to E5M2", encode5);
    check("decode", decode);
    check("decode from E5M2", decode5);
    check("encode bits", bits);
    check("encode bits to E5M2", bits5);
    check("encode bits, stochastic", sr_bits);
    check("encode bits to E5M2, stochastic", sr_bits5);
    check("encode, stochastic", sr);
    check("encode to E5M2, stochastic", sr5);
    check("copy", copy);
    check("stream", rw);
    check("byte mix", mix);
    check("byte mix, bf16 weights", mix16);
    if (failures) return 1;
    printf("launch errors ok\n");
    return 0;
}
