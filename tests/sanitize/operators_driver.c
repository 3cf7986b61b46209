/* Drives the host side of the operators around the product (argument
 * validation, workspace sizes) over valid, invalid and extreme arguments, for a
 * build with AddressSanitizer and UndefinedBehaviorSanitizer on the host code.
 * No GPU is needed and none is used: pointers are stand-ins, and calls with
 * valid arguments are made only without a GPU, where they stop at the device
 * check. Exits non-zero on an unexpected status. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "bitlinear.h"

static int fails = 0;
#define EXPECT(cond)                                                         \
    do {                                                                     \
        if (!(cond)) {                                                       \
            fprintf(stderr, "%s:%d: expected %s\n", __FILE__, __LINE__, #cond); \
            ++fails;                                                         \
        }                                                                    \
    } while (0)

int main(int argc, char **argv) {
    const int have_gpu = argc > 1 && strcmp(argv[1], "gpu") == 0;
    void *P = (void *)(uintptr_t)0x10000;
    float *F = (float *)P;
    const int64_t sizes[] = {INT64_MIN, -1, 0, 1, 7, 8, 63, 511, 512, 513, 4096, 8192, 8193, 32768, 65537,
                             (1 << 24) - 1, 1 << 24, (1 << 24) + 1, 2147483647LL, 2147483648LL, INT64_MAX};
    const int n = (int)(sizeof sizes / sizeof sizes[0]);
    const int64_t seg_ok[2] = {5, 3}, seg_big[2] = {2147483647LL, 1}, seg_zero[2] = {5, 0},
                  seg_neg[2] = {INT64_MIN, INT64_MAX};
    const int64_t *segs[] = {seg_ok, seg_big, seg_zero, seg_neg, NULL};
    const float scales[] = {1.0f, 0.0f, INFINITY, NAN};
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < n; ++j) {
            const int64_t M = sizes[i], K = sizes[j];
            const int fits = M > 0 && K > 0 && M <= 1 << 24 && K <= 1 << 24;
            EXPECT((bitlinear_epilogue_backward_workspace_bytes(M, K) > 0) == fits);
            EXPECT((bitlinear_block_norm_backward_workspace_bytes(M, K) > 0) == fits);
            for (int s = 0; s < 5; ++s)
                for (int act = -1; act < 7; act += 2)
                    for (int f = 0; f < 4; ++f) {
                        /* y misaligned: always refused, after every other check has run */
                        void *bad = (char *)P + 4;
                        bl_status a = bitlinear_forward_epilogue(P, F, P, 0, F, segs[s], 2, M, K, P, 0, act,
                                                                 P, scales[f], P, bad, 0, NULL);
                        bl_status b = bitlinear_linear_epilogue(P, 0, P, 0, F, segs[s], 2, M, K, P, 0, act,
                                                                P, scales[f], P, bad, 0, NULL);
                        EXPECT(a == BL_ERR_INVALID_ARG || (a == BL_OK && M == 0));
                        EXPECT(b == BL_ERR_INVALID_ARG || (b == BL_OK && M == 0) ||
                               (b == BL_ERR_UNSUPPORTED && M > 4));
                    }
            bl_status c = bitlinear_epilogue_backward(P, 0, P, 0, 4, 1.0f, M, K, P, 0, F, P, P, 0, NULL);
            EXPECT(c == BL_ERR_INVALID_ARG || c == BL_OK || (M == 0 && c == BL_ERR_DEVICE));
            bl_status d = bitlinear_block_norm(P, 0, P, 1, 1.0f, P, 1, 1, P, P, 1e-5f, 2, P, P, 1e-5f, 0, M, K,
                                               P, P, P, NULL, F, NULL);
            EXPECT(d == BL_ERR_INVALID_ARG || (d == BL_OK && M == 0));
            bl_status e = bitlinear_block_norm_backward(P, P, 0, P, 0, P, 1, F, 1.0f, P, 1, 1, P, P, 2, P, 0, M,
                                                        K, P, P, P, F, F, F, F, P, 0, NULL);
            EXPECT(e == BL_ERR_INVALID_ARG || (M == 0 && e == BL_ERR_DEVICE));
            if (have_gpu || !fits) continue;
            /* valid calls: the device check, before any launch */
            const size_t ws = bitlinear_block_norm_backward_workspace_bytes(M, K);
            EXPECT(bitlinear_block_norm(P, 0, P, 1, 1.0f, P, 1, 1, P, P, 1e-5f, 2, P, P, 1e-5f, 0, M,
                                        K < 16909320 ? K : 8, P, P, P, F, F, NULL) == BL_ERR_DEVICE);
            EXPECT(bitlinear_block_norm_backward(P, P, 0, P, 0, P, 1, F, 1.0f, P, 1, 1, P, P, 2, P, 0, M, K, P,
                                                 P, P, F, F, F, F, P, ws, NULL) == BL_ERR_DEVICE);
            EXPECT(bitlinear_epilogue_backward(P, 0, P, 0, 4, 1.0f, M, K, P, 0, F, P, P, SIZE_MAX, NULL) ==
                   BL_ERR_DEVICE);
        }
    for (int kind = -2; kind < 5; ++kind)
        for (int gate = -2; gate < 5; ++gate)
            for (int dt = -1; dt < 3; ++dt) {
                if (have_gpu && kind >= 0 && kind <= 2 && gate >= 0 && gate <= 2 && dt >= 0 && dt <= 1) continue;
                (void)bitlinear_block_norm(P, dt, P, dt, 1.0f, P, gate, kind, P, P, 1e-5f, kind, P, P, 1e-5f, dt,
                                           4, 64, P, P, P, F, F, NULL);
                (void)bitlinear_block_norm_backward(P, P, dt, P, dt, P, dt, F, 1.0f, P, gate, kind, P, P, kind, P,
                                                    dt, 4, 64, P, P, P, F, F, F, F, P, 1 << 24, NULL);
            }
    if (fails) return 1;
    printf("operators driver: ok\n");
    return 0;
}
