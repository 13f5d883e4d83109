/* A stand-in for the calls of the HIP runtime that the library makes, for driver programs
 * that test its error handling without a GPU.  The program is linked with
 * --export-dynamic, so the library's calls come here.  As in HIP 7, a thread's last error
 * is that of the last call that failed: calls that succeed leave it, hipGetLastError()
 * takes it.  "Device" memory is host memory and launches only count. */
#ifndef STUB_HIP_H
#define STUB_HIP_H

#include <hip/hip_runtime_api.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

static hipError_t stub_last = hipSuccess;
static int stub_launches = 0;       /* launches so far */
static int stub_fail_launch = -1;   /* the launch that fails (counted from 0), or -1 */
static int stub_fail_malloc = 0;    /* the next hipMalloc runs out of memory */
static int stub_fail_memcpy = 0;    /* the next copy fails */
static int stub_capturing = 0;      /* every stream is being captured */
static int stub_device_calls = 0;   /* allocations, copies and waits so far: none belongs into a capture */

static hipError_t stub_result(hipError_t e) {
    if (e != hipSuccess) stub_last = e;
    return e;
}

hipError_t hipGetLastError(void) {
    const hipError_t e = stub_last;
    stub_last = hipSuccess;
    return e;
}

hipError_t hipGetDevice(int *dev) { *dev = 0; return hipSuccess; }
hipError_t hipStreamGetDevice(hipStream_t s, hipDevice_t *dev) { (void)s; *dev = 0; return hipSuccess; }
hipError_t hipStreamSynchronize(hipStream_t s) {
    (void)s;
    stub_device_calls++;
    return hipSuccess;
}
hipError_t hipStreamIsCapturing(hipStream_t s, hipStreamCaptureStatus *c) {
    (void)s;
    *c = stub_capturing ? hipStreamCaptureStatusActive : hipStreamCaptureStatusNone;
    return hipSuccess;
}

hipError_t hipMalloc(void **p, size_t n) {
    stub_device_calls++;
    if (stub_fail_malloc) {
        stub_fail_malloc = 0;
        return stub_result(hipErrorOutOfMemory);
    }
    *p = calloc(1, n);
    return stub_result(*p ? hipSuccess : hipErrorOutOfMemory);
}
hipError_t hipFree(void *p) { free(p); return hipSuccess; }

hipError_t hipMemcpyAsync(void *d, const void *s, size_t n, hipMemcpyKind k, hipStream_t st) {
    (void)k;
    (void)st;
    stub_device_calls++;
    if (stub_fail_memcpy) {
        stub_fail_memcpy = 0;
        return stub_result(hipErrorInvalidValue);
    }
    memcpy(d, s, n);
    return hipSuccess;
}
hipError_t hipMemsetAsync(void *d, int v, size_t n, hipStream_t s) {
    (void)s;
    memset(d, v, n);
    return hipSuccess;
}

hipError_t hipGetSymbolAddress(void **p, const void *sym) {
    static unsigned char room[4 << 20];
    (void)sym;
    *p = room;
    return hipSuccess;
}

hipError_t hipEventCreate(hipEvent_t *e) { *e = (hipEvent_t)malloc(1); return hipSuccess; }
hipError_t hipEventDestroy(hipEvent_t e) { free(e); return hipSuccess; }
hipError_t hipEventSynchronize(hipEvent_t e) { (void)e; return hipSuccess; }
hipError_t hipEventElapsedTime(float *ms, hipEvent_t a, hipEvent_t b) {
    (void)a, (void)b;
    *ms = 1.0f;
    return hipSuccess;
}

static hipError_t stub_launch(void) {
    if (stub_launches == stub_fail_launch) return stub_result(hipErrorLaunchFailure);
    stub_launches++;
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void *f, dim3 g, dim3 b, void **a, size_t lds, hipStream_t s) {
    (void)f, (void)g, (void)b, (void)a, (void)lds, (void)s;
    return stub_launch();
}
hipError_t hipExtLaunchKernel(const void *f, dim3 g, dim3 b, void **a, size_t lds, hipStream_t s, hipEvent_t e0,
                              hipEvent_t e1, int flags) {
    (void)f, (void)g, (void)b, (void)a, (void)lds, (void)s, (void)e0, (void)e1, (void)flags;
    return stub_launch();
}

static int failures = 0;

/* A call returned `want` and launched `launches` kernels, and the thread's last error is `last` now. */
static void expect(const char *what, int got, int want, int launches, hipError_t last, const char *msg) {
    if (got != want || stub_launches != launches || stub_last != last) {
        fprintf(stderr, "%s: returned %d (%s), expected %d; %d launches, expected %d; last error %d, expected %d\n", what,
                got, got ? msg : "", want, stub_launches, launches, (int)stub_last, (int)last);
        failures++;
    }
    stub_launches = 0;
}

#endif
