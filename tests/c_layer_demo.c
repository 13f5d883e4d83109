/* A plain C11 caller of the layer operators: no torch, no Python.  A training step of one layer with
 * GELU: weights through fp8adam_quantize, the product with bias and kept sums, back through the
 * activation, both gradients; every result is checked against double arithmetic here.  Also calls of one
 * token whose lds say nothing.  Exit status 0 and "c layer demo ok" on success. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "fp8adam_layer.h"

#define T 70
#define N 130
#define K 256
#define NB 2 /* blocks of K, and of N */
#define CHECK_HIP(e) do { hipError_t r_ = (e); if (r_ != hipSuccess) { \
    fprintf(stderr, "%s: %s\n", #e, hipGetErrorString(r_)); return 1; } } while (0)
#define CHECK_LIB(e) do { int r_ = (e); if (r_ != 0) { \
    fprintf(stderr, "%s: %d %s\n", #e, r_, fp8adam_last_error()); return 1; } } while (0)

static double uniform(uint64_t *s) {
    *s = *s * 6364136223846793005ULL + 1442695040888963407ULL;
    return ((double)(*s >> 33) + 0.5) / 2147483648.0 - 0.5;
}

static double e4m3(uint8_t c) {
    const int e = c >> 3 & 15, m = c & 7;
    const double v = e ? ldexp(8 + m, e - 10) : ldexp(m, -9);
    return c & 0x80 ? -v : v;
}

static int bad = 0;
static void near(const char *what, int i, double got, double want, double tol) {
    if (!(fabs(got - want) <= tol) && bad++ < 10) fprintf(stderr, "%s[%d]: %g, not %g (within %g)\n", what, i, got, want, tol);
}

static float x[T * K], w[N * K], b[N], y[T * N], dy[T * N], dz[T * N], db[N], dw[N * K], dx[T * K], sw[N * NB];
static uint8_t cx[T * K], cw[N * K], sx[T * 4], cz[T * 256], sz[T * 4];
static double vx[T * K], vw[N * K], vz[T * N];

int main(void) {
    uint64_t seed = 11;
    for (int i = 0; i < T * K; i++) x[i] = (float)uniform(&seed);
    for (int i = 0; i < N * K; i++) w[i] = (float)(uniform(&seed) / 4);
    for (int i = 0; i < N; i++) b[i] = (float)uniform(&seed);
    for (int i = 0; i < T * N; i++) dy[i] = (float)uniform(&seed);
    float *d_x, *d_w, *d_b, *d_y, *d_dy, *d_dz, *d_db, *d_dw, *d_dx, *d_sw;
    uint8_t *d_cx, *d_cw, *d_sx, *d_cz, *d_sz;
    CHECK_HIP(hipMalloc((void **)&d_x, sizeof x));
    CHECK_HIP(hipMalloc((void **)&d_w, sizeof w));
    CHECK_HIP(hipMalloc((void **)&d_b, sizeof b));
    CHECK_HIP(hipMalloc((void **)&d_y, sizeof y));
    CHECK_HIP(hipMalloc((void **)&d_dy, sizeof dy));
    CHECK_HIP(hipMalloc((void **)&d_dz, sizeof dz));
    CHECK_HIP(hipMalloc((void **)&d_db, sizeof db));
    CHECK_HIP(hipMalloc((void **)&d_dw, sizeof dw));
    CHECK_HIP(hipMalloc((void **)&d_dx, sizeof dx));
    CHECK_HIP(hipMalloc((void **)&d_sw, sizeof sw));
    CHECK_HIP(hipMalloc((void **)&d_cx, sizeof cx));
    CHECK_HIP(hipMalloc((void **)&d_cw, sizeof cw));
    CHECK_HIP(hipMalloc((void **)&d_sx, sizeof sx));
    CHECK_HIP(hipMalloc((void **)&d_cz, sizeof cz));
    CHECK_HIP(hipMalloc((void **)&d_sz, sizeof sz));
    CHECK_HIP(hipMemcpy(d_x, x, sizeof x, hipMemcpyHostToDevice));
    CHECK_HIP(hipMemcpy(d_w, w, sizeof w, hipMemcpyHostToDevice));
    CHECK_HIP(hipMemcpy(d_b, b, sizeof b, hipMemcpyHostToDevice));
    CHECK_HIP(hipMemcpy(d_dy, dy, sizeof dy, hipMemcpyHostToDevice));

    hipStream_t s;
    CHECK_HIP(hipStreamCreate(&s));
    fp8adam_plan *plan;
    const fp8adam_quant_tensor q = {d_w, d_cw, d_sw, N * K, FP8ADAM_F32, FP8ADAM_E4M3};
    const fp8adam_quant_config cfg = {FP8ADAM_SCALE_BLOCK128, FP8ADAM_SCALE_POW2};
    CHECK_LIB(fp8adam_quant_plan(&plan, &q, 1, &cfg, s));
    CHECK_LIB(fp8adam_quantize(plan, s));

    fp8adam_product8 p;
    memset(&p, 0, sizeof p);
    p.tokens = T, p.rows = N, p.cols = K;
    p.x_in = (fp8adam_matrix){d_x, K, FP8ADAM_F32, 0};
    p.x = (fp8adam_matrix8){d_cx, d_sx, K, 4, FP8ADAM_E4M3, FP8ADAM_SCALES_E8M0};
    p.w = (fp8adam_matrix8){d_cw, d_sw, K, NB, FP8ADAM_E4M3, FP8ADAM_SCALES_F32};
    p.bias = (fp8adam_matrix){d_b, 0, FP8ADAM_F32, 0};
    p.y = (fp8adam_matrix){d_y, N, FP8ADAM_F32, 0};
    p.keep = (fp8adam_matrix8){d_cz, d_sz, 256, 4, FP8ADAM_E4M3, FP8ADAM_SCALES_E8M0};
    p.activation = FP8ADAM_ACT_GELU;
    CHECK_LIB(fp8adam_linear8(&p, s));

    fp8adam_act_backward8 a;
    memset(&a, 0, sizeof a);
    a.tokens = T, a.rows = N;
    a.dy = (fp8adam_matrix){d_dy, N, FP8ADAM_F32, 0};
    a.keep = p.keep;
    a.dz = (fp8adam_matrix){d_dz, N, FP8ADAM_F32, 0};
    a.bias_grad = (fp8adam_matrix){d_db, 0, FP8ADAM_F32, 0};
    a.activation = FP8ADAM_ACT_GELU;
    a.workspace_bytes = fp8adam_linear8_backward_workspace(&a);
    CHECK_HIP(hipMalloc(&a.workspace, (size_t)a.workspace_bytes));
    CHECK_LIB(fp8adam_linear8_backward(&a, s));

    fp8adam_grad8 g[2];
    for (int i = 0; i < 2; i++) {
        memset(&g[i], 0, sizeof g[i]);
        g[i].tokens = T, g[i].rows = N, g[i].cols = K, g[i].n = 1;
        g[i].dy[0] = a.dz;
        g[i].b[0] = i ? p.w : p.x;
        g[i].out = (fp8adam_matrix){i ? d_dx : d_dw, K, FP8ADAM_F32, 0};
        g[i].workspace_bytes = i ? fp8adam_input_grad8_workspace(&g[i]) : fp8adam_weight_grad8_workspace(&g[i]);
        CHECK_HIP(hipMalloc(&g[i].workspace, (size_t)g[i].workspace_bytes));
        CHECK_LIB(i ? fp8adam_input_grad8(&g[i], s) : fp8adam_weight_grad8(&g[i], s));
    }
    CHECK_HIP(hipStreamSynchronize(s));
    CHECK_HIP(hipMemcpy(cx, d_cx, sizeof cx, hipMemcpyDeviceToHost));
    CHECK_HIP(hipMemcpy(sx, d_sx, sizeof sx, hipMemcpyDeviceToHost));
    CHECK_HIP(hipMemcpy(cw, d_cw, sizeof cw, hipMemcpyDeviceToHost));
    CHECK_HIP(hipMemcpy(sw, d_sw, sizeof sw, hipMemcpyDeviceToHost));
    CHECK_HIP(hipMemcpy(cz, d_cz, sizeof cz, hipMemcpyDeviceToHost));
    CHECK_HIP(hipMemcpy(sz, d_sz, sizeof sz, hipMemcpyDeviceToHost));
    CHECK_HIP(hipMemcpy(y, d_y, sizeof y, hipMemcpyDeviceToHost));
    CHECK_HIP(hipMemcpy(dz, d_dz, sizeof dz, hipMemcpyDeviceToHost));
    CHECK_HIP(hipMemcpy(db, d_db, sizeof db, hipMemcpyDeviceToHost));
    CHECK_HIP(hipMemcpy(dw, d_dw, sizeof dw, hipMemcpyDeviceToHost));
    CHECK_HIP(hipMemcpy(dx, d_dx, sizeof dx, hipMemcpyDeviceToHost));

    for (int i = 0; i < T * K; i++) {
        vx[i] = ldexp(e4m3(cx[i]), sx[i / K * 4 + i % K / 128] - 127);
        near("x", i, vx[i], x[i], fabs(x[i]) / 16 + 1e-5); /* half a step: 2^-4 of the value, or 2^-10 of the scale (at most 2^-9) */
    }
    for (int i = 0; i < N * K; i++) vw[i] = e4m3(cw[i]) * sw[i / 128];
    for (int t = 0; t < T; t++)
        for (int n = 0; n < N; n++) {
            double z = b[n], size = fabs(b[n]);
            for (int k = 0; k < K; k++) z += vx[t * K + k] * vw[n * K + k], size += fabs(vx[t * K + k] * vw[n * K + k]);
            const int i = t * N + n;
            const double sum = 1.01 * (K + 2) * 0x1p-23 * size;
            near("y", i, y[i], 0.5 * z * erfc(-z / sqrt(2.0)), 1.13 * sum + 8 * 0x1p-23 * fabs(z) + 3e-7 * (1 + fabs(z)));
            vz[i] = ldexp(e4m3(cz[t * 256 + n]), sz[t * 4 + n / 128] - 127);
            near("z", i, vz[i], z, sum + (fabs(z) + sum) / 16 + ldexp(1, sz[t * 4 + n / 128] - 127 - 10));
            const double d = 0.5 * erfc(-vz[i] / sqrt(2.0)) + vz[i] * exp(-vz[i] * vz[i] / 2) / sqrt(2 * acos(-1.0));
            near("dz", i, dz[i], dy[i] * d, fabs(dy[i]) * (1e-6 + 8 * 0x1p-23 * (1 + fabs(vz[i]))));
        }
    for (int n = 0; n < N; n++) {
        double sum = 0, size = 0;
        for (int t = 0; t < T; t++) sum += dz[t * N + n], size += fabs(dz[t * N + n]);
        near("db", n, db[n], sum, 1.01 * (T + 2) * 0x1p-23 * size);
        for (int k = 0; k < K; k++) {
            sum = size = 0;
            for (int t = 0; t < T; t++) sum += dz[t * N + n] * vx[t * K + k], size += fabs(dz[t * N + n] * vx[t * K + k]);
            near("dw", n * K + k, dw[n * K + k], sum, (1.01 * (2 * T + 2) * 0x1p-23 + 0x1p-16) * size);
        }
    }
    for (int t = 0; t < T; t++)
        for (int k = 0; k < K; k++) {
            double sum = 0, size = 0;
            for (int n = 0; n < N; n++) sum += dz[t * N + n] * vw[n * K + k], size += fabs(dz[t * N + n] * vw[n * K + k]);
            near("dx", t * K + k, dx[t * K + k], sum, (1.01 * (2 * N + 2) * 0x1p-23 + 0x1p-16) * size);
        }

    /* one token, an Inf in a bf16 gradient of 128, and lds of 0 */
    static uint16_t h[128], out16[K];
    for (int n = 0; n < 128; n++) h[n] = n == 3 ? 0x7F80 : 0x3F80; /* Inf, and 1 */
    uint16_t *d_h;
    CHECK_HIP(hipMalloc((void **)&d_h, sizeof h));
    CHECK_HIP(hipMemcpy(d_h, h, sizeof h, hipMemcpyHostToDevice));
    for (int i = 0; i < 2; i++) {
        g[i].tokens = 1, g[i].rows = 128;
        g[i].dy[0] = (fp8adam_matrix){d_h, 0, FP8ADAM_BF16, 0};
        if (i) g[i].out = (fp8adam_matrix){d_dx, 0, FP8ADAM_BF16, 0};
        CHECK_LIB(i ? fp8adam_input_grad8(&g[i], s) : fp8adam_weight_grad8(&g[i], s));
    }
    CHECK_HIP(hipStreamSynchronize(s));
    CHECK_HIP(hipMemcpy(dw, d_dw, sizeof dw, hipMemcpyDeviceToHost));
    CHECK_HIP(hipMemcpy(out16, d_dx, sizeof out16, hipMemcpyDeviceToHost));
    for (int i = 0; i < 128 * K; i++) {
        const double v = vx[i % K];
        if (i / K != 3) near("dw of one token", i, dw[i], v, 0);
        else if (v != 0 ? !(isinf(dw[i]) && (dw[i] > 0) == (v > 0)) : !isnan(dw[i])) bad++;
    }
    for (int k = 0; k < K; k++) {
        const uint16_t want = vw[3 * K + k] > 0 ? 0x7F80 : 0xFF80;
        if (vw[3 * K + k] != 0 && out16[k] != want && bad++ < 10) fprintf(stderr, "dx of one token[%d]: %x\n", k, out16[k]);
    }
    fp8adam_plan_destroy(plan);
    if (bad) return 1;
    printf("c layer demo ok\n");
    return 0;
}
