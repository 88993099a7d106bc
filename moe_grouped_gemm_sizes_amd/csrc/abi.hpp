// abi.hpp -- what the C entry points of the layer operators share (layer_api.hip,
// block_api.hip): checks of pointers, types and operands, and status codes.
#pragma once
#include <hip/hip_runtime.h>

#include <initializer_list>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "../../include/moegg.h"
#include "layer.hpp"

namespace moegg {
namespace {

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

moegg_status_t hip_status(hipError_t e, const char* what) {
    if (e == hipSuccess) return MOEGG_OK;
    const char* v = getenv("MOEGG_DEBUG");
    if (v && v[0] == '1') fprintf(stderr, "moegg: %s failed: %s\n", what, hipGetErrorString(e));
    return MOEGG_ERR_HIP;
}

// A launch's work-items are counted in 32 bits.
const int64_t kMaxWorkItems = 0x7FFFFFFFll;

// A caller's enum as the number it is: C callers can pass any int, and reading
// one that names no enumerator as the enum is undefined.
template <typename T>
int number(const T& e) {
    static_assert(sizeof(T) == sizeof(int), "C enums are ints");
    int v;
    memcpy(&v, &e, sizeof(v));
    return v;
}

bool format_of(const moegg_dtype_t& d, OperandFormat* f) {
    switch (number(d)) {
        case MOEGG_BF16: *f = kBf16; return true;
        case MOEGG_FP8_E4M3: *f = kRows; return true;
        case MOEGG_FP8_E4M3_SCALE_KM: *f = kKm; return true;
        case MOEGG_FP8_E4M3_E8M0: *f = kE8m0; return true;
        default: return false;
    }
}

bool known(const moegg_logits_t& l, const moegg_score_t& s) {
    return (number(l) == MOEGG_LOGITS_FP32 || number(l) == MOEGG_LOGITS_BF16) &&
           (number(s) == MOEGG_SCORE_SOFTMAX || number(s) == MOEGG_SCORE_SIGMOID);
}

bool all16(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (!aligned(p, 16)) return false;
    return true;
}
bool all4(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (!aligned(p, 4)) return false;
    return true;
}
bool any_null(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (!p) return true;
    return false;
}

// An operand of `fmt` that is written, and its scales.
moegg_status_t check_operand(const void* p, const void* scale, int64_t rows, int W, OperandFormat fmt) {
    if (rows > 0 && !p) return MOEGG_ERR_INVALID_ARG;
    if (fmt == kBf16) return aligned(p, 2) ? MOEGG_OK : MOEGG_ERR_INVALID_ARG;
    if (rows > 0 && !scale) return MOEGG_ERR_INVALID_ARG;
    if (!aligned(p, 16) || !aligned(scale, 4)) return MOEGG_ERR_INVALID_ARG;
    return W % kGroup == 0 ? MOEGG_OK : MOEGG_ERR_UNSUPPORTED;
}

}  // namespace
}  // namespace moegg
