/* The layer operators (fp8adam_layer.h) against the HIP runtime's last error, on a
 * stand-in runtime (stub_hip.h): an error that the thread holds from before is not a
 * launch's, a call that fails ends there and leaves none behind, and no call allocates,
 * copies or waits.  Exit status 0 is the pass condition. */
#include "stub_hip.h"

#include "fp8adam_layer.h"

#define OLD hipErrorInvalidDevice
#define EXPECT(call, want, launches, last) \
    do { \
        const int got = call; \
        expect(#call, got, want, launches, last, fp8adam_last_error()); \
    } while (0)

static void *at(int i) { return (void *)((uintptr_t)(i + 1) << 40); } /* far apart; nothing is read */

static fp8adam_matrix mat(int i, int64_t ld, int dtype) {
    fp8adam_matrix m = {at(i), ld, dtype, 0};
    return m;
}

static fp8adam_matrix8 mat8(int i, int64_t cols) {
    const int64_t nb = (cols + 127) / 128;
    fp8adam_matrix8 m = {at(i), (char *)at(i) + (1ll << 39), nb * 128, (nb + 3) / 4 * 4, FP8ADAM_E4M3, FP8ADAM_SCALES_E8M0};
    return m;
}

/* Every launch of a call in turn fails; then none does.  Each with and without an error from before. */
#define EACH(call, n) \
    do { \
        for (int k = 0; k < (n); k++) { \
            stub_last = k % 2 ? OLD : hipSuccess; \
            stub_fail_launch = k; \
            EXPECT(call, FP8ADAM_EHIP, k, hipSuccess); \
        } \
        stub_fail_launch = -1; \
        stub_last = OLD; \
        EXPECT(call, FP8ADAM_OK, n, OLD); \
        stub_last = hipSuccess; \
        EXPECT(call, FP8ADAM_OK, n, hipSuccess); \
    } while (0)

int main(void) {
    const int64_t N = 300, K = 200;
    const int64_t tokens[] = {1, 2, 20, 200, 3000};
    for (int i = 0; i < 5; i++) {
        const int64_t T = tokens[i];
        fp8adam_matrix x = mat(0, K, FP8ADAM_BF16), dy = mat(1, N, FP8ADAM_F32);
        fp8adam_matrix8 x8 = mat8(2, K);
        EACH(fp8adam_pack8(&x, &x8, T, K, NULL), 1);
        EACH(fp8adam_unpack8(&x8, &x, T, K, NULL), 1);

        fp8adam_product8 p;
        memset(&p, 0, sizeof p);
        p.tokens = T, p.rows = N, p.cols = K;
        p.x = x8, p.w = mat8(3, K), p.y = mat(5, N, FP8ADAM_BF16), p.activation = FP8ADAM_ACT_SILU;
        EACH(fp8adam_linear8(&p, NULL), 1);
        p.x_in = x;
        EACH(fp8adam_linear8(&p, NULL), T <= 4 ? 1 : 2); /* few tokens are packed by the product itself */
        p.keep = mat8(6, N);
        EACH(fp8adam_linear8(&p, NULL), 2);
        p.w_up = mat8(4, K), p.keep_up = mat8(7, N);
        EACH(fp8adam_gated8(&p, NULL), 2);
        p.tokens = 0;
        EACH(fp8adam_gated8(&p, NULL), 0);

        fp8adam_act_backward8 a;
        memset(&a, 0, sizeof a);
        a.tokens = T, a.rows = N, a.dy = dy, a.keep = p.keep, a.dz = mat(8, N, FP8ADAM_F32), a.activation = FP8ADAM_ACT_GELU;
        EACH(fp8adam_linear8_backward(&a, NULL), 1);
        a.bias_grad = mat(9, N, FP8ADAM_F32), a.workspace = at(10);
        a.workspace_bytes = fp8adam_linear8_backward_workspace(&a);
        EACH(fp8adam_linear8_backward(&a, NULL), 2);
        memset(&a.bias_grad, 0, sizeof a.bias_grad);
        a.keep_up = p.keep_up, a.dup = mat(9, N, FP8ADAM_F32);
        EACH(fp8adam_gated8_backward(&a, NULL), 1);

        fp8adam_grad8 g;
        memset(&g, 0, sizeof g);
        g.tokens = T, g.rows = N, g.cols = K, g.n = 1, g.dy[0] = dy, g.b[0] = x8, g.out = mat(11, K, FP8ADAM_F32), g.workspace = at(10);
        for (int weights = 0; weights < 2; weights++) {
            /* fp32: split; the parts of a long sum are joined where it has more than one */
            g.workspace_bytes = weights ? fp8adam_weight_grad8_workspace(&g) : fp8adam_input_grad8_workspace(&g);
            const int64_t split = 2 * ((T * ((N + 7) / 8 * 8) * 2 + 255) / 256 * 256);
            const int n = 2 + (g.workspace_bytes > split);
            if (g.workspace_bytes < split) failures++;
            if (weights) EACH(fp8adam_weight_grad8(&g, NULL), n);
            else EACH(fp8adam_input_grad8(&g, NULL), n);
        }
    }
    if (stub_device_calls) {
        fprintf(stderr, "%d allocations, copies or waits\n", stub_device_calls);
        failures++;
    }
    if (!failures) printf("launch errors ok\n");
    return failures != 0;
}
