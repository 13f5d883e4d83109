/* Calls the plan builders of the list operators (fp8adam_list.h) with lists that
 * they refuse and with lists that they accept up to the first device call, for a
 * build of the library whose host code carries AddressSanitizer.  Nothing is
 * enqueued.  Without a GPU an accepted list ends with FP8ADAM_EHIP; with one it gives
 * a plan, which is destroyed.  Exit status 0 and no sanitizer report is the pass
 * condition. */
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "fp8adam_list.h"

static int failures = 0;

static void expect(int got, int want, const char *what) {
    if (got != want) {
        fprintf(stderr, "%s: returned %d, expected %d (%s)\n", what, got, want, fp8adam_last_error());
        failures++;
    }
    (void)strlen(fp8adam_last_error());
}

static void accepted(int got, fp8adam_plan *p, const char *what) {
    if (got != FP8ADAM_OK && got != FP8ADAM_EHIP) {
        fprintf(stderr, "%s: returned %d (%s)\n", what, got, fp8adam_last_error());
        failures++;
    }
    fp8adam_plan_destroy(p);
}

#define AT(i, j) (void *)(((uintptr_t)(i) + 1) * 0x100000 + (uintptr_t)(j) * 0x10000)

int main(void) {
    const int n = 20000;
    fp8adam_plan *p = NULL;
    fp8adam_adamw_config cfg = {2, FP8ADAM_E4M3, FP8ADAM_E5M2, 0};
    fp8adam_adamw_tensor *a = calloc(n, sizeof *a);
    fp8adam_clip_tensor *c = calloc(n, sizeof *c);
    fp8adam_quant_tensor *q = calloc(n, sizeof *q);
    if (!a || !c || !q) return 2;
    for (int i = 0; i < n; i++) {
        const int odd = i % 4;  /* bytes off: 0, or a 16-bit stream that starts at an odd element */
        a[i].param = AT(i, 0);
        a[i].grad = (char *)AT(i, 1) + (odd & 2);
        a[i].copy = i % 3 == 1 ? (char *)AT(i, 2) + (odd & 2) : NULL;
        a[i].copy_dtype = FP8ADAM_F16;
        a[i].m = AT(i, 3);
        a[i].v = AT(i, 4);
        a[i].m_scale = AT(i, 5);
        a[i].v_scale = AT(i, 6);
        a[i].numel = i % 7 ? 1 + i % 9000 : 0;
        a[i].param_dtype = FP8ADAM_F32;
        a[i].grad_dtype = FP8ADAM_BF16;
        a[i].moments = i % 2;
        a[i].group = i % 2;
        c[i].src = AT(i, 0);
        c[i].dst = i % 3 == 0 ? NULL : i % 3 == 1 ? AT(i, 0) : AT(i, 1);
        c[i].src_dtype = FP8ADAM_F32;
        c[i].dst_dtype = i % 3 == 1 ? FP8ADAM_F32 : FP8ADAM_BF16;
        c[i].numel = a[i].numel;
        q[i].values = AT(i, 0);
        q[i].codes = (uint8_t *)AT(i, 1) + odd;
        q[i].scale = AT(i, 2);
        q[i].dtype = i % 3;
        q[i].format = i % 2;
        q[i].numel = a[i].numel;
    }
    accepted(fp8adam_adamw_plan(&p, a, n, &cfg, NULL), p, "a long mixed list");
    p = NULL;
    accepted(fp8adam_clip_plan(&p, c, n, NULL), p, "a long list of gradients");
    for (int g = 0; g < 2; g++)
        for (int m = 0; m < 2; m++) {
            fp8adam_quant_config qc = {g, m};
            p = NULL;
            accepted(fp8adam_quant_plan(&p, q, n, &qc, NULL), p, "a long list to convert");
        }
    /* refused late in the list */
    a[n - 2].v = a[n - 9].param;
    expect(fp8adam_adamw_plan(&p, a, n, &cfg, NULL), FP8ADAM_EINVAL, "overlap far apart");
    a[n - 2].v = AT(n - 2, 4);
    a[n - 1].group = 2;
    expect(fp8adam_adamw_plan(&p, a, n, &cfg, NULL), FP8ADAM_EINVAL, "a bad group");
    c[n - 2].dst = c[n - 5].dst;
    c[n - 2].numel = c[n - 5].numel = 100;
    c[n - 5].dst = c[n - 2].dst = AT(n, 3);
    c[n - 5].dst_dtype = c[n - 2].dst_dtype = FP8ADAM_BF16;
    expect(fp8adam_clip_plan(&p, c, n, NULL), FP8ADAM_EINVAL, "one output twice");
    q[n - 2].format = 9;
    fp8adam_quant_config qc = {0, 0};
    expect(fp8adam_quant_plan(&p, q, n, &qc, NULL), FP8ADAM_EINVAL, "a bad format");
    expect(fp8adam_adamw_plan(NULL, a, n, &cfg, NULL), FP8ADAM_EINVAL, "no place for the plan");
    expect(fp8adam_quantize(NULL, NULL), FP8ADAM_EINVAL, "no plan");
    if (p) failures++;  /* a refusal gives no plan */
    fp8adam_plan_destroy(NULL);
    free(a);
    free(c);
    free(q);
    printf("list abi driver done, %d failures\n", failures);
    return failures ? 1 : 0;
}
