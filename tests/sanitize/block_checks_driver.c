/*
 * Sanitizer driver for the host side of the heads', the cache's and kq_mxfp4_gated_linear's entry points
 * (test infrastructure): built by tests/test_block_sanitizers.py against a library whose host
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
static const int64_t *S = P(0x10000);
static int failures = 0;

static void expect(const char *what, kq_status got, kq_status want) {
    if (got != want) {
        fprintf(stderr, "%s: status %d, expected %d\n", what, (int)got, (int)want);
        ++failures;
    }
}

static kq_status head(int64_t m, int64_t heads, int64_t d, int64_t ld, int64_t hs, const kq_rope *r) {
    return kq_headnorm_rope(GOOD, KQ_BF16, m, heads, d, ld, hs, 1, F, F, 0, 1e-6f, r, F, ld, hs, NULL);
}
static kq_status back(int64_t m, int64_t heads, int64_t d, int64_t ld, int64_t hs, const kq_rope *r, int64_t ws) {
    return kq_headnorm_rope_backward(GOOD, ld, hs, GOOD, ld, hs, KQ_F32, m, heads, d, 1, F, F, 0, 1e-6f, r, F, ld, hs, F, F, F, ws, NULL);
}
static kq_status put(int64_t m, int64_t kh, int64_t vh, int64_t d, int64_t ld, int64_t hs, const kq_rope *r, int64_t n) {
    return kq_cache_write_mxfp4(GOOD, ld, hs, kh, GOOD, ld, hs, vh, KQ_BF16, m, d, 1, F, 1e-6f, r, S, n, B, B, B, B, NULL);
}
static kq_status get(int64_t m, int64_t heads, int64_t d, int64_t ld, int64_t hs, int64_t n) {
    return kq_cache_read_mxfp4(S, m, B, B, n, heads, d, KQ_BF16, F, ld, hs, NULL);
}
static kq_status gated(int64_t m, int64_t n, int64_t k, int64_t ldo, int64_t ldg, int packed) {
    return kq_mxfp4_gated_linear(B, B, B, B, B, B, packed, m, n, k, F, F, KQ_ACT_SILU, KQ_F32, F, ldo, F, ldg, F, ldg, NULL);
}
static kq_status gated_back(int64_t m, int64_t n, int64_t ld, int64_t ws) {
    return kq_mxfp4_gated_linear_backward(GOOD, ld, GOOD, ld, GOOD, ld, KQ_F32, m, n, KQ_ACT_SILU, F, ld, F, ld, F, F, F, ws, NULL);
}

int main(void) {
    const int64_t sizes[] = {INT64_MIN, INT64_MIN + 1, -1, (int64_t)1 << 31, (int64_t)1 << 40, INT64_MAX / 2, INT64_MAX};
    const int64_t big = ((int64_t)1 << 31) - 32;
    int64_t n = 0;
    kq_rope rope = {S, (const double *)GOOD, 64, 0, 1.0f, 1, {32, 0, 0, 0}};
    for (int i = 0; i < 7; ++i) {
        const int64_t s = sizes[i];
        const kq_status want = s < 0 ? KQ_ERR_SHAPE : KQ_ERR_UNSUPPORTED;
        expect("head m", head(s, 4, 64, 256, 64, NULL), want);
        expect("head heads", head(4, s, 64, 256, 64, NULL), want);
        expect("head d", head(4, 4, s, 256, 64, NULL), want);
        expect("head ld", head(4, 4, 64, s, 64, NULL), want);
        expect("head hs", head(4, 4, 64, 256, s, NULL), want);
        expect("head grad m", back(s, 4, 64, 256, 64, NULL, s), want);
        expect("head grad heads", back(4, s, 64, 256, 64, NULL, s), want);
        expect("head grad d", back(4, 4, s, 256, 64, NULL, s), want);
        expect("head grad ld", back(4, 4, 64, s, 64, NULL, s), want);
        expect("head grad hs", back(4, 4, 64, 256, s, NULL, s), want);
        expect("head grad ws", kq_headnorm_rope_backward_workspace_bytes(s, 64, &n), want);
        expect("head grad ws", kq_headnorm_rope_backward_workspace_bytes(64, s, &n), want);
        expect("write m", put(s, 2, 2, 64, 128, 64, NULL, 9), want);
        expect("write heads", put(4, s, 2, 64, 128, 64, NULL, 9), want);
        expect("write heads", put(4, 2, s, 64, 128, 64, NULL, 9), want);
        expect("write ld", put(4, 2, 2, 64, s, 64, NULL, 9), want);
        expect("write hs", put(4, 2, 2, 64, 128, s, NULL, 9), want);
        expect("write slots", put(4, 2, 2, 64, 128, 64, NULL, s), want);
        expect("read m", get(s, 2, 64, 128, 64, 9), want);
        expect("read heads", get(4, s, 64, 128, 64, 9), want);
        expect("read ld", get(4, 2, 64, s, 64, 9), want);
        expect("read hs", get(4, 2, 64, 128, s, 9), want);
        expect("read slots", get(4, 2, 64, 128, 64, s), want);
        expect("gated m", gated(s, 64, 256, 64, 64, 1), want);
        expect("gated n", gated(4, s, 256, s, s, 1), want);
        expect("gated ldo", gated(4, 64, 256, s, 64, 0), want);
        expect("gated ldg", gated(4, 64, 256, 64, s, 0), want);
        expect("gated grad m", gated_back(s, 64, 64, s), want);
        expect("gated grad n", gated_back(4, s, s, s), want);
        expect("gated grad ld", gated_back(4, 64, s, s), want);
        expect("gated grad ws", kq_mxfp4_gated_linear_backward_workspace_bytes(s, 64, &n), want);
        expect("gated grad ws", kq_mxfp4_gated_linear_backward_workspace_bytes(64, s, &n), want);
        /* the members of a rotation */
        kq_rope r = rope;
        r.rot = s;
        expect("rot", head(4, 4, 64, 256, 64, &r), KQ_ERR_SHAPE);
        r = rope;
        r.axes = 4;
        r.axis_pairs[i % 4] = s;
        expect("pairs", put(4, 2, 2, 64, 128, 64, &r, 9), KQ_ERR_SHAPE);
        expect("frequencies", kq_rope_frequencies(s < 0 ? s : s | 1, 1e4, KQ_ROPE_PLAIN, 1, 1, 1, 2, NULL), KQ_ERR_SHAPE);
    }
    rope.axes = INT32_MAX;
    expect("axes", head(4, 4, 64, 256, 64, &rope), KQ_ERR_UNSUPPORTED);
    rope.axes = INT32_MIN;
    expect("axes", back(4, 4, 64, 256, 64, &rope, 1 << 20), KQ_ERR_UNSUPPORTED);
    /* sizes that fit one by one and not together */
    expect("head overlap", head(big, 65536, 1024, 1024, big, NULL), KQ_ERR_SHAPE);
    expect("head groups", head(big, 65536, 32, 65536 * 32, 32, NULL), KQ_ERR_UNSUPPORTED);
    expect("head groups", head(big, 65536, 1, 65536, 1, NULL), KQ_ERR_UNSUPPORTED);
    expect("write groups", put(big, 65536, 0, 32, big, big, NULL, big), KQ_ERR_UNSUPPORTED);
    expect("write groups", put(big, 1, 65535, 1024, 0, 0, NULL, big), KQ_ERR_UNSUPPORTED);
    expect("read groups", get(big, 65536, 1024, 65536 * 1024, 1024, big), KQ_ERR_UNSUPPORTED);
    expect("head grad short", back(big, 65536, 1024, 65536 * 1024, 1024, NULL, 64), KQ_ERR_SHAPE);
    expect("gated k", gated(4, 64, big, 64, 64, 0), KQ_ERR_UNSUPPORTED);
    expect("gated scales", gated(big, 64, 8192, 64, 64, 0), KQ_ERR_UNSUPPORTED);
    expect("gated scales", gated(64, big, 8192, big, big, 0), KQ_ERR_UNSUPPORTED);
    expect("gated rows", gated(big, 64, 32, big, 64, 0), KQ_ERR_UNSUPPORTED);
    expect("gated grad short", gated_back(big, big, big, 64), KQ_ERR_SHAPE);
    /* workspaces of the largest sizes */
    expect("head ws", kq_headnorm_rope_backward_workspace_bytes(big, 1024, &n), KQ_OK);
    if (n != 256 * 2 * 1024 * 4) ++failures;
    expect("gated ws", kq_mxfp4_gated_linear_backward_workspace_bytes(big, big, &n), KQ_OK);
    if (n <= 0 || n % (8 * big) != 0) ++failures;
    expect("ws null", kq_headnorm_rope_backward_workspace_bytes(1, 1, NULL), KQ_ERR_NULL);
    expect("ws null", kq_mxfp4_gated_linear_backward_workspace_bytes(1, 1, NULL), KQ_ERR_NULL);
    /* frequencies at the ends of their range */
    double f[512];
    expect("base", kq_rope_frequencies(64, INFINITY, KQ_ROPE_PLAIN, 1, 1, 1, 2, f), KQ_ERR_SHAPE);
    expect("base", kq_rope_frequencies(64, NAN, KQ_ROPE_PLAIN, 1, 1, 1, 2, f), KQ_ERR_SHAPE);
    expect("huge base", kq_rope_frequencies(1024, 1e308, KQ_ROPE_BASE, 1e308, 1, 1, 2, f), KQ_OK);
    expect("tiny factor", kq_rope_frequencies(1024, 1e4, KQ_ROPE_LINEAR, 1e-308, 1, 1, 2, f), KQ_OK);
    expect("parts", kq_rope_frequencies(1024, 1e-308, KQ_ROPE_PARTS, 1e-308, 1e308, -1e308, 1e308, f), KQ_OK);
    /* nothing to do */
    expect("no tokens", kq_headnorm_rope(NULL, KQ_F32, 0, 4, 64, 0, 0, 1, NULL, NULL, 4, 0.f, NULL, NULL, 0, 0, NULL), KQ_OK);
    expect("no slots", kq_cache_write_mxfp4(GOOD, 64, 64, 1, NULL, 0, 0, 0, KQ_F32, 4, 64, 0, NULL, 0.f, NULL, S, 0, NULL, NULL, NULL, NULL, NULL), KQ_OK);
    expect("no tokens", kq_cache_read_mxfp4(NULL, 0, NULL, NULL, 0, 2, 64, KQ_F32, NULL, 128, 64, NULL), KQ_OK);
    expect("no rows", kq_mxfp4_gated_linear(NULL, NULL, NULL, NULL, NULL, NULL, 1, 0, 64, 256, NULL, NULL, 0, KQ_F32, NULL, 64, NULL, 0, NULL, 0, NULL), KQ_OK);
    expect("no columns", kq_mxfp4_gated_linear_backward(NULL, 0, NULL, 0, NULL, 0, KQ_F32, 4, 0, 1, NULL, 0, NULL, 0, NULL, NULL, NULL, 0, NULL), KQ_OK);
    if (failures) {
        fprintf(stderr, "%d host-check failures\n", failures);
        return 1;
    }
    printf("block host-check sanitizer driver: ok\n");
    return 0;
}
