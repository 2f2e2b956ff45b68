/*
 * Sanitizer driver for the host side of the layer norm's and kq_mxfp4_linear's entry points
 * (test infrastructure): built by tests/test_layer_sanitizers.py against a library whose host
 * code carries -fsanitize=address,undefined, and run on the CPU with no GPU. Every call
 * fails its argument checks, or has nothing to do, before any HIP call.
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "kq.h"

#define P(x) ((void *)(uintptr_t)(x))
static const void *GOOD = P(0x10000); /* never dereferenced */
static float *F = P(0x10000);
static uint8_t *B = P(0x10000);
static int failures = 0;

static void expect(const char *what, kq_status got, kq_status want) {
    if (got != want) {
        fprintf(stderr, "%s: status %d, expected %d\n", what, (int)got, (int)want);
        ++failures;
    }
}

int main(void) {
    const int64_t sizes[] = {INT64_MIN, -1, (int64_t)1 << 31, (int64_t)1 << 40, INT64_MAX / 2, INT64_MAX};
    int64_t n = 0;
    for (int i = 0; i < 6; ++i) {
        const int64_t s = sizes[i];
        const kq_status want = s < 0 ? KQ_ERR_SHAPE : KQ_ERR_UNSUPPORTED;
        expect("norm m", kq_layernorm(GOOD, KQ_BF16, s, 64, 64, F, F, 1e-5f, F, 64, F, F, NULL), want);
        expect("norm d", kq_layernorm(GOOD, KQ_F32, 4, s, s, F, F, 1e-5f, F, s, F, F, NULL), want);
        expect("norm ldx", kq_layernorm(GOOD, KQ_F32, 4, 64, s, F, F, 1e-5f, F, 64, F, F, NULL), want);
        expect("norm ldy", kq_layernorm(GOOD, KQ_F32, 4, 64, 64, F, F, 1e-5f, F, s, F, F, NULL), want);
        expect("norm grad m", kq_layernorm_backward(GOOD, 64, GOOD, 64, KQ_F32, s, 64, F, F, F, F, 64, F, F, F, s, NULL), want);
        expect("norm grad d", kq_layernorm_backward(GOOD, s, GOOD, s, KQ_F32, 4, s, F, F, F, F, s, F, F, F, s, NULL), want);
        expect("norm grad ws", kq_layernorm_backward_workspace_bytes(s, 64, &n), want);
        expect("norm grad ws", kq_layernorm_backward_workspace_bytes(64, s, &n), want);
        expect("norm quant m", kq_layernorm_quantize_mxfp4(GOOD, KQ_F32, s, 256, 256, F, F, 1e-5f, F, B, B, 1, F, F, F, NULL), want);
        expect("linear m", kq_mxfp4_linear(B, B, B, B, 1, s, 64, 256, F, 0, KQ_F32, GOOD, 64, F, 64, F, 64, NULL), want);
        expect("linear n", kq_mxfp4_linear(B, B, B, B, 1, 4, s, 256, F, 0, KQ_F32, GOOD, s, F, s, F, s, NULL), want);
        expect("linear ldo", kq_mxfp4_linear(B, B, B, B, 0, 4, 64, 256, F, 0, KQ_F32, GOOD, 64, F, s, F, 64, NULL), want);
        expect("linear ldr", kq_mxfp4_linear(B, B, B, B, 0, 4, 64, 256, F, 0, KQ_F32, GOOD, s, F, 64, F, 64, NULL), want);
        expect("linear grad m", kq_mxfp4_linear_backward(GOOD, 64, GOOD, 64, KQ_F32, s, 64, 1, F, 64, F, F, s, NULL), want);
        expect("linear grad n", kq_mxfp4_linear_backward(GOOD, s, GOOD, s, KQ_F32, 4, s, 1, F, s, F, F, s, NULL), want);
        expect("linear grad ws", kq_mxfp4_linear_backward_workspace_bytes(s, 64, &n), want);
    }
    /* sizes that fit one by one and not together */
    const int64_t big = ((int64_t)1 << 31) - 32;
    expect("norm quant d", kq_layernorm_quantize_mxfp4(GOOD, KQ_F32, 4, big, big, F, F, 1e-5f, F, B, B, 0, F, F, F, NULL), KQ_ERR_UNSUPPORTED);
    expect("norm quant packed", kq_layernorm_quantize_mxfp4(GOOD, KQ_F32, big, 256, 256, F, F, 1e-5f, F, B, B, 1, F, F, F, NULL), KQ_ERR_UNSUPPORTED);
    expect("linear k", kq_mxfp4_linear(B, B, B, B, 0, 4, 64, big, F, 0, KQ_F32, NULL, 0, F, 64, NULL, 0, NULL), KQ_ERR_UNSUPPORTED);
    expect("linear scales", kq_mxfp4_linear(B, B, B, B, 0, big, 64, 8192, F, 0, KQ_F32, NULL, 0, F, 64, NULL, 0, NULL), KQ_ERR_UNSUPPORTED);
    expect("linear rows", kq_mxfp4_linear(B, B, B, B, 0, big, 64, 32, F, 0, KQ_F32, NULL, 0, F, big, NULL, 0, NULL), KQ_ERR_UNSUPPORTED);
    expect("linear grad short", kq_mxfp4_linear_backward(GOOD, big, GOOD, big, KQ_F32, big, big, 1, F, big, F, F, 64, NULL), KQ_ERR_SHAPE);
    expect("norm grad short", kq_layernorm_backward(GOOD, big, GOOD, big, KQ_F32, big, big, F, F, F, F, big, F, F, F, 64, NULL), KQ_ERR_SHAPE);
    /* workspaces of the largest sizes */
    expect("norm ws", kq_layernorm_backward_workspace_bytes(big, big, &n), KQ_OK);
    if (n != 256 * 2 * big * 4) ++failures;
    expect("linear ws", kq_mxfp4_linear_backward_workspace_bytes(big, big, &n), KQ_OK);
    if (n <= 0 || n % (4 * big) != 0) ++failures;
    expect("ws null", kq_layernorm_backward_workspace_bytes(1, 1, NULL), KQ_ERR_NULL);
    expect("ws null", kq_mxfp4_linear_backward_workspace_bytes(1, 1, NULL), KQ_ERR_NULL);
    /* the rest: eps, types, activations, pointers, alignment, nothing to do */
    expect("eps", kq_layernorm(GOOD, KQ_F32, 4, 64, 64, F, F, NAN, F, 64, F, F, NULL), KQ_ERR_SHAPE);
    expect("eps", kq_layernorm(GOOD, KQ_F32, 4, 64, 64, F, F, INFINITY, F, 64, F, F, NULL), KQ_ERR_SHAPE);
    expect("type", kq_layernorm(GOOD, 2, 4, 64, 64, F, F, 0.f, F, 64, F, F, NULL), KQ_ERR_UNSUPPORTED);
    expect("act", kq_mxfp4_linear(B, B, B, B, 0, 4, 64, 256, F, -1, KQ_F32, NULL, 0, F, 64, NULL, 0, NULL), KQ_ERR_UNSUPPORTED);
    expect("null", kq_layernorm(NULL, KQ_F32, 4, 64, 64, F, F, 0.f, F, 64, F, F, NULL), KQ_ERR_NULL);
    expect("null", kq_mxfp4_linear(B, B, NULL, B, 0, 4, 64, 256, F, 0, KQ_F32, NULL, 0, F, 64, NULL, 0, NULL), KQ_ERR_NULL);
    expect("null z", kq_mxfp4_linear_backward(GOOD, 64, NULL, 64, KQ_F32, 4, 64, 1, F, 64, F, F, 1 << 20, NULL), KQ_ERR_NULL);
    expect("align", kq_layernorm(P(0x10001), KQ_BF16, 4, 64, 64, F, F, 0.f, F, 64, F, F, NULL), KQ_ERR_ALIGN);
    expect("align ws", kq_layernorm_backward(GOOD, 64, GOOD, 64, KQ_F32, 64, 64, F, F, F, F, 64, F, F, P(0x10004), 1 << 20, NULL), KQ_ERR_ALIGN);
    expect("align scales", kq_mxfp4_linear(B, P(0x10004), B, B, 1, 4, 64, 256, F, 0, KQ_F32, NULL, 0, F, 64, NULL, 0, NULL), KQ_ERR_ALIGN);
    expect("no rows", kq_layernorm(NULL, KQ_F32, 0, 64, 64, NULL, NULL, 0.f, NULL, 64, NULL, NULL, NULL), KQ_OK);
    expect("no rows", kq_layernorm_backward(NULL, 64, NULL, 64, KQ_F32, 0, 64, NULL, NULL, NULL, NULL, 64, NULL, NULL, NULL, 0, NULL), KQ_OK);
    expect("no rows", kq_mxfp4_linear(NULL, NULL, NULL, NULL, 1, 0, 64, 256, NULL, 0, KQ_F32, NULL, 0, NULL, 64, NULL, 0, NULL), KQ_OK);
    expect("no columns", kq_mxfp4_linear_backward(NULL, 0, NULL, 0, KQ_F32, 4, 0, 1, NULL, 0, NULL, NULL, 0, NULL), KQ_OK);
    if (failures) {
        fprintf(stderr, "%d host-check failures\n", failures);
        return 1;
    }
    printf("layer host-check sanitizer driver: ok\n");
    return 0;
}
