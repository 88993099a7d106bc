/* Takes every layer entry point of include/moegg.h down its refusal paths (nothing is launched).
 * Built and run under sanitizers by tests/test_host_sanitizers_layer.py; prints "ok". */
#include <limits.h>
#include <math.h>
#include <stdio.h>

#include "../include/moegg.h"

#define EXPECT(call, want)                                                        \
    do {                                                                          \
        int got_ = (int)(call);                                                   \
        if (got_ != (int)(want)) {                                                \
            printf("line %d: got %d, want %d\n", __LINE__, got_, (int)(want));    \
            return 1;                                                             \
        }                                                                         \
    } while (0)

int main(void) {
    void* p = (void*)0x100000;
    void* odd = (void*)0x100001;
    float* f = (float*)p;
    int32_t* i = (int32_t*)p;
    const int B = INT_MAX;

    EXPECT(moegg_route_workspace_bytes(-1, 8), 0);
    EXPECT(moegg_route_workspace_bytes(B, B), 0);
    EXPECT(moegg_route_workspace_bytes(16773120, 1024) > 0, 1);
    EXPECT(moegg_route(p, MOEGG_LOGITS_FP32, NULL, i, f, i, i, B, B, B, MOEGG_SCORE_SOFTMAX, 1, 1, 1, 1, 1.f, 10, 1, 0, p,
                       SIZE_MAX, NULL), MOEGG_ERR_UNSUPPORTED);
    EXPECT(moegg_route(p, MOEGG_LOGITS_FP32, NULL, i, f, i, i, 10, 8, 2, MOEGG_SCORE_SOFTMAX, 1, 1, 1, 1, NAN, 10, 1, 0, p,
                       SIZE_MAX, NULL), MOEGG_ERR_INVALID_ARG);
    EXPECT(moegg_route(p, MOEGG_LOGITS_FP32, NULL, i, f, i, i, 10, 8, 2, MOEGG_SCORE_SOFTMAX, 3, 1, 1, 1, 1.f, 10, 1, 0, p,
                       SIZE_MAX, NULL), MOEGG_ERR_INVALID_ARG);
    EXPECT(moegg_route(p, MOEGG_LOGITS_FP32, NULL, i, f, i, i, 10, 8, 2, MOEGG_SCORE_SOFTMAX, 1, 1, 1, 1, 1.f, 10, 1, 0,
                       NULL, 0, NULL), MOEGG_ERR_WORKSPACE);
    EXPECT(moegg_route(p, (moegg_logits_t)7, NULL, i, f, i, i, 10, 8, 2, MOEGG_SCORE_SOFTMAX, 1, 1, 1, 1, 1.f, 10, 1, 0, p,
                       SIZE_MAX, NULL), MOEGG_ERR_INVALID_ARG);
    EXPECT(moegg_route_backward(p, MOEGG_LOGITS_BF16, i, f, p, B, 1024, 32, MOEGG_SCORE_SIGMOID, 0, 1.f, NULL),
           MOEGG_ERR_UNSUPPORTED);
    EXPECT(moegg_route_backward(NULL, MOEGG_LOGITS_BF16, i, f, p, 1, 8, 2, MOEGG_SCORE_SIGMOID, 0, 1.f, NULL),
           MOEGG_ERR_INVALID_ARG);
    EXPECT(moegg_dispatch(p, i, p, p, B, 1, B, B, MOEGG_BF16, NULL), MOEGG_ERR_UNSUPPORTED);
    EXPECT(moegg_dispatch(p, i, p, p, 8, 2, 130, 16, MOEGG_FP8_E4M3, NULL), MOEGG_ERR_UNSUPPORTED);
    EXPECT(moegg_dispatch(p, i, p, odd, 8, 2, 128, 16, MOEGG_FP8_E4M3_E8M0, NULL), MOEGG_ERR_INVALID_ARG);
    EXPECT(moegg_dispatch(p, i, p, p, 8, 2, 128, 16, (moegg_dtype_t)99, NULL), MOEGG_ERR_INVALID_ARG);
    EXPECT(moegg_combine(p, i, NULL, p, B, 32, B, B, NULL), MOEGG_ERR_UNSUPPORTED);
    EXPECT(moegg_combine(NULL, i, NULL, p, 4, 2, 64, 8, NULL), MOEGG_ERR_INVALID_ARG);
    EXPECT(moegg_combine_backward(p, p, f, i, p, p, f, B, 32, B, B, MOEGG_BF16, NULL), MOEGG_ERR_UNSUPPORTED);
    EXPECT(moegg_combine_backward(p, p, NULL, i, p, p, f, 4, 2, 128, 8, MOEGG_BF16, NULL), MOEGG_ERR_INVALID_ARG);
    EXPECT(moegg_swiglu_checkpoint(p, i, p, p, p, f, 4096, INT64_MAX, 128, MOEGG_BF16, NULL), MOEGG_ERR_INVALID_ARG);
    EXPECT(moegg_swiglu_checkpoint(p, i, p, p, p, f, 4096, B, 1 << 30, MOEGG_BF16, NULL), MOEGG_ERR_UNSUPPORTED);
    EXPECT(moegg_swiglu_checkpoint_backward(p, i, p, f, p, NULL, 8, 100, 128, NULL), MOEGG_ERR_INVALID_ARG);
    EXPECT(moegg_swiglu_checkpoint_backward_fp8(p, i, p, f, p, f, p, p, p, p, 8, 100, 128, INT64_MIN, MOEGG_FP8_E4M3, 0,
                                                NULL), MOEGG_ERR_INVALID_ARG);
    EXPECT(moegg_swiglu_checkpoint_backward_fp8(p, i, p, f, p, f, p, p, p, p, 8, B, 1 << 24, 1, MOEGG_FP8_E4M3, 0, NULL),
           MOEGG_ERR_UNSUPPORTED);
    EXPECT(moegg_checkpoint_to_k_groups(p, f, i, p, p, 8, B, 1 << 28, 1, MOEGG_FP8_E4M3, 1, NULL), MOEGG_ERR_UNSUPPORTED);
    EXPECT(moegg_checkpoint_to_k_groups(p, NULL, i, p, p, 8, 100, 256, 1, MOEGG_FP8_E4M3, 1, NULL), MOEGG_ERR_INVALID_ARG);
    printf("ok\n");
    return 0;
}
