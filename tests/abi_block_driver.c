/* Takes every entry point of the operators around the layer down its refusal paths (nothing is launched).
 * Built and run under sanitizers by tests/test_host_sanitizers_block.py; prints "ok". */
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

    EXPECT(moegg_rms_norm_workspace_bytes(B, B), 0);
    EXPECT(moegg_rms_norm_workspace_bytes(INT_MIN, 8), 0);
    EXPECT(moegg_rms_norm_workspace_bytes(2097151, 32768) > 0, 1);
    EXPECT(moegg_rms_norm(p, p, p, MOEGG_WEIGHT_BF16, 1e-6f, p, p, p, p, f, B, 128, MOEGG_FP8_E4M3, NULL),
           MOEGG_ERR_UNSUPPORTED);
    EXPECT(moegg_rms_norm(p, p, p, MOEGG_WEIGHT_BF16, 1e-6f, p, p, p, p, f, 1, B, MOEGG_FP8_E4M3, NULL),
           MOEGG_ERR_UNSUPPORTED);
    EXPECT(moegg_rms_norm(p, p, p, (moegg_weight_t)99, 1e-6f, p, p, p, p, f, 1, 128, MOEGG_FP8_E4M3, NULL),
           MOEGG_ERR_INVALID_ARG);
    EXPECT(moegg_rms_norm(p, p, p, MOEGG_WEIGHT_FP32, NAN, p, p, p, p, f, 1, 128, MOEGG_FP8_E4M3, NULL),
           MOEGG_ERR_INVALID_ARG);
    EXPECT(moegg_rms_norm(p, p, p, MOEGG_WEIGHT_FP32, 1.f, p, p, odd, p, f, 1, 128, (moegg_dtype_t)-7, NULL),
           MOEGG_ERR_INVALID_ARG);
    EXPECT(moegg_rms_norm_backward(p, p, p, MOEGG_WEIGHT_FP32, f, p, p, f, B, B, p, SIZE_MAX, NULL),
           MOEGG_ERR_UNSUPPORTED);
    EXPECT(moegg_rms_norm_backward(p, p, p, MOEGG_WEIGHT_FP32, f, p, odd, f, 4, 128, p, SIZE_MAX, NULL),
           MOEGG_ERR_INVALID_ARG);
    EXPECT(moegg_rms_norm_backward(p, p, p, MOEGG_WEIGHT_FP32, f, p, p, f, 4, 128, NULL, 0, NULL), MOEGG_ERR_WORKSPACE);
    EXPECT(moegg_balance_loss_workspace_bytes(B, B, B), 0);
    EXPECT(moegg_balance_loss_workspace_bytes(16773120, 1024, 65536) > 0, 1);
    EXPECT(moegg_balance_loss(p, MOEGG_LOGITS_FP32, i, i, f, f, i, f, B, 1024, 32, 65536, MOEGG_SCORE_SOFTMAX, p, SIZE_MAX,
                              NULL), MOEGG_ERR_UNSUPPORTED);
    EXPECT(moegg_balance_loss(p, (moegg_logits_t)12, i, i, f, f, i, f, 8, 8, 2, 2, MOEGG_SCORE_SOFTMAX, p, SIZE_MAX, NULL),
           MOEGG_ERR_INVALID_ARG);
    EXPECT(moegg_balance_loss(p, MOEGG_LOGITS_FP32, i, i, f, f, i, f, 8, 8, 2, 2, MOEGG_SCORE_SOFTMAX, odd, SIZE_MAX, NULL),
           MOEGG_ERR_WORKSPACE);
    EXPECT(moegg_balance_loss_backward(p, MOEGG_LOGITS_BF16, i, i, f, f, p, p, B, B, B, B, MOEGG_SCORE_SOFTMAX, NULL),
           MOEGG_ERR_UNSUPPORTED);
    EXPECT(moegg_balance_loss_backward(p, MOEGG_LOGITS_BF16, i, i, f, f, odd, p, 8, 8, 2, 2, MOEGG_SCORE_SOFTMAX, NULL),
           MOEGG_ERR_INVALID_ARG);
    EXPECT(moegg_lora_workspace_bytes(B, B, B), 0);
    EXPECT(moegg_lora_workspace_bytes(1 << 24, 1 << 30, 128) > 0, 1);
    EXPECT(moegg_lora(p, p, p, f, i, p, p, B, 8, 8, 8, B, p, SIZE_MAX, NULL), MOEGG_ERR_UNSUPPORTED);
    EXPECT(moegg_lora(p, p, p, f, i, p, p, 1 << 24, 1 << 30, 1 << 30, 8, B, p, SIZE_MAX, NULL), MOEGG_ERR_UNSUPPORTED);
    EXPECT(moegg_lora(p, p, p, f, i, p, odd, 8, 8, 8, 8, 1, p, SIZE_MAX, NULL), MOEGG_ERR_INVALID_ARG);
    EXPECT(moegg_lora(p, p, p, f, i, p, p, 8, 8, 8, 8, 1, NULL, 0, NULL), MOEGG_ERR_WORKSPACE);
    printf("ok\n");
    return 0;
}
