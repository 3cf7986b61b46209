/* Drives the host side of the gated products, the 8-bit checkpoints and the
 * gradients from codes and stacks (argument validation, workspace sizes and the
 * plans behind them) over valid, invalid and extreme arguments, for a build with
 * AddressSanitizer and UndefinedBehaviorSanitizer on the host code. No GPU is
 * needed and none is used: pointers are stand-ins, and calls with valid arguments
 * are made only without a GPU, where they stop at the device check. Exits non-zero
 * on an unexpected status. */
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
    void *P = (void *)(uintptr_t)0x10000, *bad = (char *)P + 4;
    float *F = (float *)P;
    const int64_t sizes[] = {INT64_MIN, -1, 0, 1, 7, 8, 63, 4096, 8193, (1 << 23) - 1, 1 << 23, (1 << 23) + 1,
                             1 << 24, (1 << 24) + 1, 1 << 30, 2147483647LL, INT64_MAX};
    const int n = (int)(sizeof sizes / sizeof sizes[0]);
    const int64_t seg_ok[2] = {5, 3}, seg_big[2] = {2147483647LL, 1}, seg_zero[2] = {5, 0},
                  seg_neg[2] = {INT64_MIN, INT64_MAX};
    const int64_t *segs[] = {seg_ok, seg_big, seg_zero, seg_neg, NULL};
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < n; ++j) {
            const int64_t M = sizes[i], N = sizes[j];
            const int half = M > 0 && N > 0 && M <= 1 << 23 && N <= 1 << 23;
            EXPECT((bitlinear_gated_backward_workspace_bytes(M, N) > 0) == (half && M > 128));
            EXPECT(bitlinear_checkpoint_groups(N) == (N < 1 ? 0 : N / 64 + (N % 64 != 0)));
            for (int k = 0; k < n; ++k) {
                const int64_t K = sizes[k];
                for (int dt = -1; dt < 3; ++dt) {
                    const size_t w = bitlinear_backward_weight_codes_workspace_bytes(M, N, K, dt);
                    const size_t x = bitlinear_backward_input_segmented_workspace_bytes(M, N, K, dt);
                    const int ok = M > 0 && N > 0 && K > 0 && M <= 1 << 24 && N <= 1 << 24 && K <= 1 << 24 &&
                                   dt >= 0 && dt < 2;
                    EXPECT(ok || w == 0);
                    EXPECT((ok && N <= 1 << 23) || x == 0);
                    bl_status a = bitlinear_backward_weight_codes(P, 0, P, F, M, N, K, bad, dt, P, SIZE_MAX, NULL);
                    EXPECT(a == BL_ERR_INVALID_ARG);
                    if (w > 0) {
                        a = bitlinear_backward_weight_codes(P, 0, P, F, M, N, K, P, dt, P, w - 1, NULL);
                        EXPECT(a == BL_ERR_INVALID_ARG);
                    }
                    if (ok && !have_gpu)
                        EXPECT(bitlinear_backward_weight_codes(P, 0, P, F, M, N, K, P, dt, P, w, NULL) ==
                               BL_ERR_DEVICE);
                }
            }
            for (int s = 0; s < 5; ++s)
                for (int act = -1; act < 7; act += 2) {
                    /* an output misaligned: always refused, after every other check has run */
                    bl_status c = bitlinear_backward_input_segmented(P, 0, P, 0, F, segs[s], 2, M, N, bad, 0, P,
                                                                     SIZE_MAX, NULL);
                    EXPECT(c == BL_ERR_INVALID_ARG || (c == BL_OK && M == 0));
                    bl_status d = bitlinear_forward_gated(P, F, P, 0, F, N, M, 64, P, 0, act, P, P, F, bad, 0, NULL);
                    EXPECT(d == BL_ERR_INVALID_ARG || (d == BL_OK && M == 0));
                    d = bitlinear_linear_gated(P, 0, P, 0, F, N, M, 64, P, 0, act, P, bad, 0, NULL);
                    EXPECT(d == BL_ERR_INVALID_ARG || (d == BL_OK && M == 0) || (d == BL_ERR_UNSUPPORTED && M > 4));
                    d = bitlinear_gated_backward(P, 0, P, 0, NULL, NULL, act, M, N, bad, 0, F, P, SIZE_MAX, NULL);
                    EXPECT(d == BL_ERR_INVALID_ARG || d == BL_OK);
                }
            bl_status e = bitlinear_checkpoint(P, 0, M, N, bad, F, NULL);
            EXPECT(e == BL_ERR_INVALID_ARG);
            e = bitlinear_checkpoint_restore(P, F, M, N, bad, 0, NULL);
            EXPECT(e == BL_ERR_INVALID_ARG);
            if (have_gpu || !half) continue;
            EXPECT(bitlinear_checkpoint(P, 0, M, N, P, F, NULL) == BL_ERR_DEVICE);
            EXPECT(bitlinear_checkpoint_restore(P, F, M, N, P, 1, NULL) == BL_ERR_DEVICE);
            EXPECT(bitlinear_gated_backward(P, 0, NULL, 0, P, F, 3, M, N, P, 0, F, P,
                                            bitlinear_gated_backward_workspace_bytes(M, N), NULL) == BL_ERR_DEVICE);
            EXPECT(bitlinear_forward_gated(P, F, P, 0, F, N, M < 8192 ? M : 8, 64, P, 0, 3, P, P, F, P, 0, NULL) ==
                   BL_ERR_DEVICE);
        }
    if (fails) return 1;
    printf("gated driver: ok\n");
    return 0;
}
