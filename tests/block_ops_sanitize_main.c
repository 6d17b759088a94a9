/* Drives the argument checks of the block operators with fake device pointers: none of
 * these calls may reach the device.  Built against a library whose host code has
 * AddressSanitizer and UndefinedBehaviorSanitizer instrumentation
 * (tests/test_block_ops_sanitize.py); any report aborts it. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "moe_w4.h"

static int failures = 0;
#define EXPECT(call, want)                                                                        \
    do {                                                                                          \
        const int got_ = (call);                                                                  \
        if (got_ != (want)) {                                                                     \
            fprintf(stderr, "%s:%d: %s returned %d, expected %d\n", __FILE__, __LINE__, #call, got_, \
                    (int)(want));                                                                 \
            ++failures;                                                                           \
        }                                                                                         \
    } while (0)

#define P(a) ((void *)(uintptr_t)(a))
#define A P(0x100000000000)
#define B P(0x200000000000)
#define C P(0x300000000000)
#define D P(0x400000000000)
#define E P(0x500000000000)
#define F P(0x600000000000)
#define W P(0x700000000000)

static const int64_t edges[] = {INT64_MIN, -1, 0, 1, 4, 7, 8, 9, 63, 64, 65, 127, 128, 129, 1024, 1025, 32768, 32776, 65536,
                                1048576, 1048577, 4194304, 4194305, 16777216, 16777217, INT64_MAX};
#define EDGES (sizeof(edges) / sizeof(edges[0]))

int main(void) {
    /* every size at its limits and beyond, alone and in pairs: no product of sizes may overflow; a NULL output refuses what is left */
    for (size_t i = 0; i < EDGES; ++i)
        for (size_t j = 0; j < EDGES; ++j) {
            const int64_t a = edges[i], b = edges[j];
            (void)moe_w4_matvec_workspace_bytes(a, b);
            (void)moe_w4_norm_workspace_bytes(a, b);
            for (size_t k = 0; k < EDGES; ++k) (void)moe_w4_grouped_mm_dw_workspace_bytes(edges[k], a, b, b);
            if (a != 0 && b != 0) {
                EXPECT(moe_w4_grouped_mm(A, B, C, a, b, 64, 64, MOE_W4_BF16, NULL, NULL), MOE_W4_EINVAL);
                EXPECT(moe_w4_grouped_mm_dx(A, B, C, 4, 64, a, b, MOE_W4_F16, NULL, NULL), MOE_W4_EINVAL);
                EXPECT(moe_w4_grouped_mm_dw(A, B, C, a, b, 64, 64, MOE_W4_BF16, NULL, NULL, MOE_W4_F32, NULL, 0, NULL), MOE_W4_EINVAL);
                EXPECT(moe_w4_matvec(A, B, C, a, b, 128, 64, 1, MOE_W4_BF16, NULL, MOE_W4_F32, W, SIZE_MAX, NULL), MOE_W4_EINVAL);
                EXPECT(moe_w4_matvec(A, B, C, 1, a, b, 32, 1, MOE_W4_BF16, NULL, MOE_W4_F32, W, SIZE_MAX, NULL), MOE_W4_EINVAL);
                EXPECT(moe_w4_norm_residual(A, B, NULL, 0, 1.0f, NULL, NULL, 3, 0.0f, a, b, MOE_W4_F32, MOE_W4_F32, NULL, D, NULL),
                       MOE_W4_EINVAL);
                EXPECT(moe_w4_norm_residual_backward(A, B, NULL, 0, 1.0f, NULL, NULL, 3, 0.0f, a, b, MOE_W4_F32, MOE_W4_F32, NULL, C,
                                                     NULL, E, NULL, NULL, NULL, W, 1u << 30, NULL), MOE_W4_EINVAL);
            }
        }

    /* nothing to do */
    EXPECT(moe_w4_grouped_mm(NULL, NULL, NULL, 0, 5, 8, 8, MOE_W4_BF16, NULL, NULL), MOE_W4_OK);
    EXPECT(moe_w4_grouped_mm_dx(NULL, NULL, NULL, 5, 0, 8, 8, MOE_W4_BF16, NULL, NULL), MOE_W4_OK);
    EXPECT(moe_w4_grouped_mm_dw(NULL, NULL, NULL, 0, 5, 8, 8, MOE_W4_BF16, NULL, NULL, MOE_W4_F32, NULL, 0, NULL), MOE_W4_OK);
    EXPECT(moe_w4_matvec(NULL, NULL, NULL, 0, 5, 128, 64, 0, MOE_W4_F16, NULL, MOE_W4_F16, NULL, 0, NULL), MOE_W4_OK);
    EXPECT(moe_w4_norm_residual(NULL, NULL, NULL, 0, 1.0f, NULL, NULL, 2, 0.0f, 0, 64, 1, 1, NULL, NULL, NULL), MOE_W4_OK);

    /* alignment, overlaps at the far end, workspaces, types */
    const size_t big = (size_t)1048576 * 32768 * 2;
    EXPECT(moe_w4_grouped_mm(A, B, C, 4, 1048576, 64, 32768, MOE_W4_BF16, (char *)A + big - 16, NULL), MOE_W4_EINVAL);
    EXPECT(moe_w4_grouped_mm(A, B, (int32_t *)P(0x300000000002), 4, 8, 64, 64, MOE_W4_BF16, D, NULL), MOE_W4_EINVAL);
    EXPECT(moe_w4_grouped_mm(A, B, C, 4, 8, 64, 64, MOE_W4_F32, D, NULL), MOE_W4_EINVAL);
    EXPECT(moe_w4_grouped_mm_dw(A, B, C, 4, 8, 64, 64, MOE_W4_BF16, NULL, D, MOE_W4_F16, NULL, 0, NULL), MOE_W4_EINVAL);
    const size_t wdw = moe_w4_grouped_mm_dw_workspace_bytes(1, 1048576, 64, 64);
    if (wdw == 0) ++failures;
    EXPECT(moe_w4_grouped_mm_dw(A, B, C, 1, 1048576, 64, 64, MOE_W4_BF16, NULL, D, MOE_W4_F32, W, wdw - 1, NULL), MOE_W4_EWORKSPACE);
    EXPECT(moe_w4_grouped_mm_dw(A, B, C, 1, 1048576, 64, 64, MOE_W4_BF16, NULL, D, MOE_W4_F32, A, wdw, NULL), MOE_W4_EINVAL);
    const size_t wmv = moe_w4_matvec_workspace_bytes(64, 65536);
    EXPECT(moe_w4_matvec(A, B, C, 64, 16777216, 65536, 32, 1, MOE_W4_BF16, D, MOE_W4_F32, W, wmv - 1, NULL), MOE_W4_EWORKSPACE);
    EXPECT(moe_w4_matvec(A, B, C, 64, 8, 65536, 48, 1, MOE_W4_BF16, D, MOE_W4_F32, W, wmv, NULL), MOE_W4_EINVAL);
    EXPECT(moe_w4_matvec(A, B, C, 1, 8, 128, 128, 1, MOE_W4_BF16, D, 3, W, wmv, NULL), MOE_W4_EINVAL);
    const size_t wn = moe_w4_norm_workspace_bytes(4194304, 8192);
    EXPECT(moe_w4_norm_residual_backward(A, B, NULL, 0, 1.0f, NULL, NULL, 3, 0.0f, 4194304, 8192, 1, 0, NULL, C, D, E, NULL, NULL,
                                         NULL, W, wn - 1, NULL), MOE_W4_EWORKSPACE);
    EXPECT(moe_w4_norm_residual(A, B, C, 4, 1.0f, NULL, NULL, 3, 0.0f, 8, 64, 1, 0, D, E, NULL), MOE_W4_EINVAL);
    EXPECT(moe_w4_norm_residual(A, B, C, 3, 1.0f, NULL, NULL, 3, 0.0f, 8, 64, 1, 0, D, D, NULL), MOE_W4_EINVAL);
    EXPECT(moe_w4_norm_residual(A, B, NULL, 0, INFINITY, NULL, NULL, 3, 0.0f, 8, 64, 1, 0, D, E, NULL), MOE_W4_EINVAL);
    EXPECT(moe_w4_norm_residual(A, B, NULL, 0, 1.0f, NULL, NULL, 3, NAN, 8, 64, 1, 0, D, E, NULL), MOE_W4_EINVAL);
    EXPECT(moe_w4_norm_residual(A, B, NULL, 0, 1.0f, F, NULL, 2, 0.0f, 8, 64, 1, 0, D, E, NULL), MOE_W4_EINVAL);

    if (failures) {
        fprintf(stderr, "%d check(s) failed\n", failures);
        return 1;
    }
    printf("block operators under the sanitizers: ok\n");
    return 0;
}
