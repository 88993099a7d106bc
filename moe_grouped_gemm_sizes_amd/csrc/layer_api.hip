// layer_api.hip -- the C ABI of the layer operators declared in
// include/moegg.h (routing, token permutation, activation checkpoints):
// argument validation and launches.  No call allocates or synchronizes.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "../../include/moegg.h"
#include "layer.hpp"
#include "workspace.hpp"

using namespace moegg;

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

// T tokens of k assignments and width W against `rows` expert rows.
moegg_status_t check_permute(const int32_t* row_of, int T, int k, int W, int64_t rows) {
    if (T < 0 || k < 1 || W < 1 || rows < 0 || rows > INT32_MAX) return MOEGG_ERR_INVALID_ARG;
    if (T > 0 && !row_of) return MOEGG_ERR_INVALID_ARG;
    if (!aligned(row_of, 4)) return MOEGG_ERR_INVALID_ARG;
    // columns are 32-bit, and go up to 8191 past the width
    if (k > kRouteMaxTopK || W > 1 << 30) return MOEGG_ERR_UNSUPPORTED;
    if ((int64_t)T * k > INT32_MAX) return MOEGG_ERR_UNSUPPORTED;
    // a wave for each token and 512 columns, and up to 256 workgroups of 4 more
    if (((int64_t)T * (((int64_t)W + 511) / 512) + 1024) * 64 > kMaxWorkItems) return MOEGG_ERR_UNSUPPORTED;
    return MOEGG_OK;
}

// An operand of `fmt` that is written, and its scales.
moegg_status_t check_operand(const void* p, const void* scale, int64_t rows, int W, OperandFormat fmt) {
    if (rows > 0 && !p) return MOEGG_ERR_INVALID_ARG;
    if (fmt == kBf16) return aligned(p, 2) ? MOEGG_OK : MOEGG_ERR_INVALID_ARG;
    if (rows > 0 && !scale) return MOEGG_ERR_INVALID_ARG;
    if (!aligned(p, 16) || !aligned(scale, 4)) return MOEGG_ERR_INVALID_ARG;
    return W % kGroup == 0 ? MOEGG_OK : MOEGG_ERR_UNSUPPORTED;
}

// Shared by the checkpoint calls: counts, rows, width (a multiple of `unit`) and
// grid, `threads` work-items for each token group and unit.
moegg_status_t check_checkpoint(const int32_t* m_sizes, int G, int64_t rows, int W, int unit, int64_t threads) {
    if (!m_sizes || !aligned(m_sizes, 4) || G < 1 || G > kMaxExperts || rows < 0 || rows > INT32_MAX || W < 1)
        return MOEGG_ERR_INVALID_ARG;
    if (W % unit != 0) return MOEGG_ERR_UNSUPPORTED;
    // 128 rows of 4 W bytes are one buffer resource; the grid is rounded up by at most 1024 workgroups
    if (W > 1 << 21 || ((rows / 128 + G) * (W / unit) + 1024) * threads > kMaxWorkItems) return MOEGG_ERR_UNSUPPORTED;
    return MOEGG_OK;
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

}  // namespace

extern "C" {

size_t moegg_route_workspace_bytes(int T, int E) {
    if (T < 0 || T > kRouteMaxTokens || E < 1 || E > kRouteMaxExperts) return 0;
    const size_t tiles = std::min<size_t>(((size_t)T + 3) / 4, kRouteMaxTiles);   // of any call of up to T tokens
    return align256(std::max<size_t>(tiles, 1) * sizeof(uint16_t) * (size_t)route_count_width(E));
}

moegg_status_t moegg_route(const void* logits, moegg_logits_t logits_dtype, const float* bias, int32_t* ids,
                           float* weights, int32_t* m_sizes, int32_t* row_of, int T, int E, int k,
                           moegg_score_t score, int n_groups, int topk_groups, int group_top, int renorm, float scale,
                           int64_t rows_total, int seg_align, int cap, void* ws, size_t ws_bytes, void* stream) {
    if (T < 0 || E < 1 || k < 1 || k > E || rows_total < 0 || rows_total > INT32_MAX || seg_align < 1 || cap < 0)
        return MOEGG_ERR_INVALID_ARG;
    if (T > 0 && any_null({logits, ids, weights, row_of})) return MOEGG_ERR_INVALID_ARG;
    if (!m_sizes) return MOEGG_ERR_INVALID_ARG;
    if (!known(logits_dtype, score)) return MOEGG_ERR_INVALID_ARG;
    if (!aligned(logits, logits_dtype == MOEGG_LOGITS_BF16 ? 2 : 4) || !all4({bias, ids, weights, m_sizes, row_of}))
        return MOEGG_ERR_INVALID_ARG;
    if (n_groups < 1 || n_groups > E || E % n_groups != 0 || topk_groups < 1 || topk_groups > n_groups || group_top < 1)
        return MOEGG_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !isfinite(scale)) return MOEGG_ERR_INVALID_ARG;
    if (T > kRouteMaxTokens || E > kRouteMaxExperts || k > kRouteMaxTopK || n_groups > 64 || group_top > 2)
        return MOEGG_ERR_UNSUPPORTED;
    if (!ws || !aligned(ws, 256) || ws_bytes < moegg_route_workspace_bytes(T, E)) return MOEGG_ERR_WORKSPACE;
    RouteArgs a{};
    a.logits = logits;
    a.bias = bias;
    a.ids = ids;
    a.weights = weights;
    a.m_sizes = m_sizes;
    a.row_of = row_of;
    a.tile_counts = (uint16_t*)ws;
    a.T = T;
    a.E = E;
    a.k = k;
    a.bf16 = logits_dtype == MOEGG_LOGITS_BF16;
    a.sigmoid = score == MOEGG_SCORE_SIGMOID;
    a.renorm = renorm != 0;
    a.n_groups = n_groups;
    a.topk_groups = topk_groups;
    a.group_top = std::min(group_top, E / n_groups);
    a.scale = scale;
    a.rows_total = rows_total;
    a.seg_align = seg_align;
    a.cap = cap;
    a.tile_tokens = route_tile_tokens(T);
    return hip_status(launch_route(a, (hipStream_t)stream), "route");
}

moegg_status_t moegg_route_backward(const void* logits, moegg_logits_t logits_dtype, const int32_t* ids,
                                    const float* d_weights, void* d_logits, int T, int E, int k, moegg_score_t score,
                                    int renorm, float scale, void* stream) {
    if (T < 0 || E < 1 || k < 1 || k > E) return MOEGG_ERR_INVALID_ARG;
    if (T > 0 && any_null({logits, ids, d_weights, d_logits})) return MOEGG_ERR_INVALID_ARG;
    if (!known(logits_dtype, score)) return MOEGG_ERR_INVALID_ARG;
    const uintptr_t z = logits_dtype == MOEGG_LOGITS_BF16 ? 2 : 4;
    if (!aligned(logits, z) || !aligned(d_logits, z) || !all4({ids, d_weights})) return MOEGG_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !isfinite(scale)) return MOEGG_ERR_INVALID_ARG;
    if (T > kRouteMaxTokens || E > kRouteMaxExperts || k > kRouteMaxTopK) return MOEGG_ERR_UNSUPPORTED;
    RouteBackwardArgs a{logits, ids, d_weights, d_logits, T, E, k, logits_dtype == MOEGG_LOGITS_BF16,
                        score == MOEGG_SCORE_SIGMOID, renorm != 0, scale};
    return hip_status(launch_route_backward(a, (hipStream_t)stream), "route backward");
}

moegg_status_t moegg_dispatch(const void* x, const int32_t* row_of, void* A, void* A_scale, int T, int k, int K,
                              int64_t rows_total, moegg_dtype_t dtype, void* stream) {
    moegg_status_t st = check_permute(row_of, T, k, K, rows_total);
    if (st != MOEGG_OK) return st;
    PermuteArgs a{};
    if (!format_of(dtype, &a.fmt)) return MOEGG_ERR_INVALID_ARG;
    if ((T > 0 && !x) || !aligned(x, a.fmt == kBf16 ? 2 : 16)) return MOEGG_ERR_INVALID_ARG;
    st = check_operand(A, A_scale, rows_total, K, a.fmt);
    if (st != MOEGG_OK) return st;
    a.x = x;
    a.row_of = row_of;
    a.out = A;
    a.scale = A_scale;
    a.T = T;
    a.k = k;
    a.W = K;
    a.rows = (int)rows_total;
    return hip_status(launch_dispatch(a, (hipStream_t)stream), "dispatch");
}

moegg_status_t moegg_combine(const void* Y, const int32_t* row_of, const float* weights, void* out, int T, int k,
                             int N, int64_t rows_total, void* stream) {
    moegg_status_t st = check_permute(row_of, T, k, N, rows_total);
    if (st != MOEGG_OK) return st;
    if ((rows_total > 0 && !Y) || (T > 0 && !out)) return MOEGG_ERR_INVALID_ARG;
    if (!aligned(Y, 2) || !aligned(out, 2) || !aligned(weights, 4)) return MOEGG_ERR_INVALID_ARG;
    PermuteArgs a{};
    a.x = Y;
    a.weights = weights;
    a.row_of = row_of;
    a.out = out;
    a.T = T;
    a.k = k;
    a.W = N;
    a.rows = (int)rows_total;
    return hip_status(launch_combine(a, (hipStream_t)stream), "combine");
}

moegg_status_t moegg_combine_backward(const void* dout, const void* Y, const float* weights, const int32_t* row_of,
                                      void* dY, void* dY_scale, float* d_weights, int T, int k, int N,
                                      int64_t rows_total, moegg_dtype_t dtype, void* stream) {
    moegg_status_t st = check_permute(row_of, T, k, N, rows_total);
    if (st != MOEGG_OK) return st;
    PermuteArgs a{};
    if (!format_of(dtype, &a.fmt)) return MOEGG_ERR_INVALID_ARG;
    if (T > 0 && any_null({dout, weights, d_weights})) return MOEGG_ERR_INVALID_ARG;
    if (rows_total > 0 && !Y) return MOEGG_ERR_INVALID_ARG;
    const uintptr_t z = a.fmt == kBf16 ? 2 : 16;
    if (!aligned(dout, z) || !aligned(Y, z) || !all4({weights, d_weights})) return MOEGG_ERR_INVALID_ARG;
    st = check_operand(dY, dY_scale, rows_total, N, a.fmt);
    if (st != MOEGG_OK) return st;
    a.x = dout;
    a.Y = Y;
    a.weights = weights;
    a.row_of = row_of;
    a.out = dY;
    a.scale = dY_scale;
    a.d_weights = d_weights;
    a.T = T;
    a.k = k;
    a.W = N;
    a.rows = (int)rows_total;
    return hip_status(launch_combine_backward(a, (hipStream_t)stream), "combine backward");
}

moegg_status_t moegg_swiglu_checkpoint(const void* GU, const int32_t* m_sizes, void* H, void* H_scale, void* ckpt,
                                       float* ckpt_scale, int G, int64_t rows_total, int I, moegg_dtype_t dtype,
                                       void* stream) {
    moegg_status_t st = check_checkpoint(m_sizes, G, rows_total, I, 128, 16 * 128);
    if (st != MOEGG_OK) return st;
    CheckpointArgs a{};
    if (!format_of(dtype, &a.fmt)) return MOEGG_ERR_INVALID_ARG;
    if (a.fmt == kE8m0) return MOEGG_ERR_UNSUPPORTED;
    if (rows_total > 0 && any_null({GU, H, ckpt, ckpt_scale})) return MOEGG_ERR_INVALID_ARG;
    if (rows_total > 0 && a.fmt != kBf16 && !H_scale) return MOEGG_ERR_INVALID_ARG;
    if (!all16({GU, H, ckpt}) || !all4({H_scale, ckpt_scale})) return MOEGG_ERR_INVALID_ARG;
    a.in = GU;
    a.m_sizes = m_sizes;
    a.ckpt = (uint8_t*)ckpt;
    a.ckpt_scale = ckpt_scale;
    a.row_out = H;
    a.row_scale = H_scale;
    a.G = G;
    a.rows = (int)rows_total;
    a.W = I;
    return hip_status(launch_swiglu_checkpoint(a, (hipStream_t)stream), "SwiGLU checkpoint");
}

moegg_status_t moegg_swiglu_checkpoint_backward(const void* dH, const int32_t* m_sizes, const void* ckpt,
                                                const float* ckpt_scale, void* dGU, void* H, int G,
                                                int64_t rows_total, int I, void* stream) {
    moegg_status_t st = check_checkpoint(m_sizes, G, rows_total, I, 128, 16 * 128);
    if (st != MOEGG_OK) return st;
    if (rows_total > 0 && any_null({dH, ckpt, ckpt_scale, dGU, H})) return MOEGG_ERR_INVALID_ARG;
    if (!all16({dH, ckpt, dGU, H}) || !all4({ckpt_scale})) return MOEGG_ERR_INVALID_ARG;
    CheckpointArgs a{};
    a.in = dH;
    a.m_sizes = m_sizes;
    a.ckpt = (uint8_t*)ckpt;
    a.ckpt_scale = (float*)ckpt_scale;
    a.row_out = dGU;
    a.H = H;
    a.G = G;
    a.rows = (int)rows_total;
    a.W = I;
    return hip_status(launch_swiglu_checkpoint_backward(a, (hipStream_t)stream), "SwiGLU checkpoint backward");
}

moegg_status_t moegg_swiglu_checkpoint_backward_fp8(
    const void* dH, const int32_t* m_sizes, const void* ckpt, const float* ckpt_scale, void* dGU, float* dGU_scale,
    void* dGU_k, void* dGU_k_scale, void* H_k, void* H_k_scale, int G, int64_t rows_total, int I,
    int64_t scale_groups, moegg_dtype_t dtype, int k_e8m0, void* stream) {
    moegg_status_t st = check_checkpoint(m_sizes, G, rows_total, I, 128, 512);
    if (st != MOEGG_OK) return st;
    CheckpointArgs a{};
    if (!format_of(dtype, &a.fmt)) return MOEGG_ERR_INVALID_ARG;
    if (a.fmt != kRows && a.fmt != kKm) return MOEGG_ERR_UNSUPPORTED;
    if (scale_groups < 0) return MOEGG_ERR_INVALID_ARG;
    if (rows_total > 0 && any_null({dH, ckpt, ckpt_scale, dGU, dGU_scale, dGU_k, H_k})) return MOEGG_ERR_INVALID_ARG;
    if (rows_total > 0 && scale_groups > 0 && any_null({dGU_k_scale, H_k_scale})) return MOEGG_ERR_INVALID_ARG;
    if (!all16({dH, ckpt, dGU, dGU_k, H_k}) || !all4({ckpt_scale, dGU_scale, dGU_k_scale, H_k_scale}))
        return MOEGG_ERR_INVALID_ARG;
    a.in = dH;
    a.m_sizes = m_sizes;
    a.ckpt = (uint8_t*)ckpt;
    a.ckpt_scale = (float*)ckpt_scale;
    a.row_out = dGU;
    a.row_scale = dGU_scale;
    a.k_out = (uint8_t*)dGU_k;
    a.k_scale = dGU_k_scale;
    a.hk_out = (uint8_t*)H_k;
    a.hk_scale = H_k_scale;
    a.G = G;
    a.rows = (int)rows_total;
    a.W = I;
    a.scale_groups = scale_groups;
    a.k_e8m0 = k_e8m0 != 0;
    return hip_status(launch_swiglu_checkpoint_backward_fp8(a, (hipStream_t)stream), "SwiGLU checkpoint backward");
}

moegg_status_t moegg_checkpoint_to_k_groups(const void* X, const float* X_scale, const int32_t* m_sizes, void* X_k,
                                            void* X_k_scale, int G, int64_t rows_total, int M, int64_t scale_groups,
                                            moegg_dtype_t dtype, int k_e8m0, void* stream) {
    moegg_status_t st = check_checkpoint(m_sizes, G, rows_total, M, 256, 256);
    if (st != MOEGG_OK) return st;
    CheckpointArgs a{};
    if (!format_of(dtype, &a.fmt)) return MOEGG_ERR_INVALID_ARG;
    if (a.fmt == kE8m0) return MOEGG_ERR_UNSUPPORTED;
    if (scale_groups < 0) return MOEGG_ERR_INVALID_ARG;
    if (rows_total > 0 && any_null({X, X_k})) return MOEGG_ERR_INVALID_ARG;
    if (rows_total > 0 && ((a.fmt != kBf16 && !X_scale) || (scale_groups > 0 && !X_k_scale)))
        return MOEGG_ERR_INVALID_ARG;
    if (!all16({X, X_k}) || !all4({X_scale, X_k_scale})) return MOEGG_ERR_INVALID_ARG;
    a.in = X;
    a.in_scale = X_scale;
    a.m_sizes = m_sizes;
    a.k_out = (uint8_t*)X_k;
    a.k_scale = X_k_scale;
    a.G = G;
    a.rows = (int)rows_total;
    a.W = M;
    a.scale_groups = scale_groups;
    a.k_e8m0 = k_e8m0 != 0;
    return hip_status(launch_checkpoint_to_k_groups(a, (hipStream_t)stream), "checkpoint to token groups");
}

}  // extern "C"
