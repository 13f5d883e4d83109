/* Which kernels the layer operators' calls launch, on a stand-in runtime (stub_hip.h), without a
 * GPU: each line of the standard input is a call's sizes and types, and the names of the kernels that
 * it launches are printed, as the library registers them. */
#include <hip/hip_runtime_api.h>
#define hipLaunchKernel stub_unnamed_launch
#include "stub_hip.h"
#undef hipLaunchKernel

#include "fp8adam_layer.h"

static struct {
    const void *f;
    const char *name;
} kernels[1 << 14];
static int nkernels = 0;

void __hipRegisterFunction(void **modules, const void *f, char *device, const char *name, unsigned limit, void *tid, void *bid,
                           dim3 *block, dim3 *grid, int *wave) {
    (void)modules, (void)device, (void)limit, (void)tid, (void)bid, (void)block, (void)grid, (void)wave;
    if (nkernels < 1 << 14) kernels[nkernels].f = f, kernels[nkernels++].name = name;
}

hipError_t hipLaunchKernel(const void *f, dim3 g, dim3 b, void **a, size_t lds, hipStream_t s) {
    const char *name = "unknown";
    (void)g, (void)b, (void)a, (void)lds, (void)s;
    for (int i = 0; i < nkernels; i++)
        if (kernels[i].f == f) name = kernels[i].name;
    printf("%s ", name);
    return stub_launch();
}

static void *at(int i) { return (void *)((uintptr_t)(i + 1) << 40); } /* far apart; nothing is read */

static fp8adam_matrix mat(int i, int64_t ld, int dtype) {
    fp8adam_matrix m = {at(i), ld, dtype, 0};
    return m;
}

static fp8adam_matrix8 mat8(int i, int64_t cols, int format) {
    const int64_t nb = (cols + 127) / 128;
    fp8adam_matrix8 m = {at(i), (char *)at(i) + (1ll << 39), nb * 128, (nb + 3) / 4 * 4, format, FP8ADAM_SCALES_E8M0};
    return m;
}

int main(void) {
    char op[16];
    long T, N, K;
    while (scanf("%15s %ld %ld %ld", op, &T, &N, &K) == 4) {
        int rc;
        if (!strcmp(op, "linear8") || !strcmp(op, "gated8")) {
            int xf, wf, x_dt, y_dt, keep, pack, exact; /* x_dt, y_dt, pack: -1 is absent */
            if (scanf("%d %d %d %d %d %d %d", &xf, &wf, &x_dt, &y_dt, &keep, &pack, &exact) != 7) return 2;
            const int gated = op[0] == 'g';
            fp8adam_product8 p;
            memset(&p, 0, sizeof p);
            p.tokens = T, p.rows = N, p.cols = K, p.activation = FP8ADAM_ACT_SILU, p.exact = exact;
            p.x = mat8(1, K, xf), p.w = mat8(2, K, wf);
            if (x_dt >= 0) p.x_in = mat(0, K, x_dt);
            if (gated) p.w_up = mat8(3, K, wf);
            if (y_dt >= 0) p.y = mat(4, N, y_dt);
            if (pack >= 0) p.y8 = mat8(5, N, pack);
            if (keep) p.keep = mat8(6, N, FP8ADAM_E4M3);
            if (keep && gated) p.keep_up = mat8(7, N, FP8ADAM_E4M3);
            rc = gated ? fp8adam_gated8(&p, NULL) : fp8adam_linear8(&p, NULL);
        } else {
            int n, format, dy_dt, exact;
            if (scanf("%d %d %d %d", &n, &format, &dy_dt, &exact) != 4) return 2;
            const int weights = !strcmp(op, "weight_grad8");
            fp8adam_grad8 g;
            memset(&g, 0, sizeof g);
            g.tokens = T, g.rows = N, g.cols = K, g.n = n, g.out = mat(4, K, FP8ADAM_F32), g.workspace = at(5), g.exact = exact;
            for (int i = 0; i < n; i++) g.dy[i] = mat(i, N, dy_dt), g.b[i] = mat8(2 + i, K, format);
            g.workspace_bytes = weights ? fp8adam_weight_grad8_workspace(&g) : fp8adam_input_grad8_workspace(&g);
            rc = weights ? fp8adam_weight_grad8(&g, NULL) : fp8adam_input_grad8(&g, NULL);
        }
        if (rc) printf("error %d %s", rc, fp8adam_last_error());
        printf("\n");
        (void)expect;
    }
    return failures != 0;
}
