// block_api.hip -- the C ABI of the operators around the MoE layer declared in
// include/moegg.h (RMS norm, balance loss, low-rank adapters): argument
// validation and launches.  No call allocates or synchronizes.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <stdint.h>

#include "../../include/moegg.h"
#include "abi.hpp"
#include "block.hpp"
#include "workspace.hpp"

using namespace moegg;

namespace {

bool known_weight(const moegg_weight_t& w) { return number(w) == MOEGG_WEIGHT_FP32 || number(w) == MOEGG_WEIGHT_BF16; }

// T rows of K columns, a workgroup of up to 1024 threads for each.
moegg_status_t check_norm(int T, int K) {
    if (T < 0 || K < 1) return MOEGG_ERR_INVALID_ARG;
    if (K > kNormMaxWidth || (int64_t)T * 1024 > kMaxWorkItems) return MOEGG_ERR_UNSUPPORTED;
    return MOEGG_OK;
}

// Shared by both directions of the balance loss.
moegg_status_t check_balance(const moegg_logits_t& logits_dtype, const moegg_score_t& score, const void* logits,
                             const int32_t* offsets, int T, int E, int k, int S) {
    if (T < 0 || E < 1 || k < 1 || k > E || S < 1) return MOEGG_ERR_INVALID_ARG;
    if (!known(logits_dtype, score)) return MOEGG_ERR_INVALID_ARG;
    if ((T > 0 && !logits) || !aligned(logits, logits_dtype == MOEGG_LOGITS_BF16 ? 2 : 4)) return MOEGG_ERR_INVALID_ARG;
    if ((S > 1 && !offsets) || !aligned(offsets, 4)) return MOEGG_ERR_INVALID_ARG;
    if (T > kRouteMaxTokens || E > kBalanceMaxExperts || k > kRouteMaxTopK || S > kBalanceMaxSequences)
        return MOEGG_ERR_UNSUPPORTED;
    return MOEGG_OK;
}

// Rows of partial sums of any call of up to T tokens and S sequences.
size_t balance_pieces(int T, int S) { return std::min<size_t>(((size_t)T + 31) / 32, 256) + (size_t)S; }

// Workspace of the adapters' call, which serves every call of fewer rows.
struct LoraLayout {
    size_t order, tiles, total;
};
LoraLayout lora_layout(int T, int K, int R) {
    // parts of K times rows: those of 512 workgroups' tiles, or T; and no more parts than there is work for
    const size_t units = ((size_t)K + 127) / 128, rows = T;
    const size_t parts = std::max(std::min(rows * ((units + 3) / 4), (size_t)1024 * kLoraChunk), rows);
    LoraLayout l;
    l.order = align256(parts * sizeof(float) * (size_t)R);
    l.tiles = l.order + align256(rows * sizeof(int32_t));
    l.total = l.tiles + align256(std::max<size_t>(lora_tile_slots(T), 1) * sizeof(int4));
    return l;
}

}  // namespace

extern "C" {

moegg_status_t moegg_rms_norm(const void* x, const void* residual, const void* weight, moegg_weight_t weight_dtype,
                              float eps, void* sum_out, void* y, void* q, void* q_scale, float* rstd, int T, int K,
                              moegg_dtype_t q_dtype, void* stream) {
    moegg_status_t st = check_norm(T, K);
    if (st != MOEGG_OK) return st;
    NormArgs a{};
    if (!format_of(q_dtype, &a.fmt) || !known_weight(weight_dtype)) return MOEGG_ERR_INVALID_ARG;
    if (!(eps >= 0x1p-126f) || !(eps < __builtin_inff())) return MOEGG_ERR_INVALID_ARG;
    if (T > 0 && any_null({x, weight})) return MOEGG_ERR_INVALID_ARG;
    if (!residual && sum_out) return MOEGG_ERR_INVALID_ARG;
    if (a.fmt == kBf16 && (q || q_scale || (T > 0 && !y))) return MOEGG_ERR_INVALID_ARG;
    const bool bf16 = weight_dtype == MOEGG_WEIGHT_BF16;
    for (const void* p : {x, residual, (const void*)sum_out, (const void*)y})
        if (!aligned(p, a.fmt == kBf16 ? 2 : 16)) return MOEGG_ERR_INVALID_ARG;
    if (!aligned(weight, a.fmt == kBf16 ? (bf16 ? 2 : 4) : 16) || !aligned(rstd, 4)) return MOEGG_ERR_INVALID_ARG;
    if (a.fmt != kBf16) {
        st = check_operand(q, q_scale, T, K, a.fmt);
        if (st != MOEGG_OK) return st;
    }
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.sum_out = sum_out;
    a.y = y;
    a.q = q;
    a.q_scale = q_scale;
    a.rstd = rstd;
    a.T = T;
    a.K = K;
    a.weight_bf16 = bf16;
    a.eps = eps;
    return hip_status(launch_rms_norm(a, (hipStream_t)stream), "RMS norm");
}

size_t moegg_rms_norm_workspace_bytes(int T, int K) {
    if (check_norm(T, K) != MOEGG_OK) return 0;
    return align256((size_t)std::max(norm_parts(T), 1) * sizeof(float) * (size_t)K);
}

moegg_status_t moegg_rms_norm_backward(const void* dy, const void* h, const void* weight, moegg_weight_t weight_dtype,
                                       const float* rstd, const void* d_sum, void* dx, float* d_weight, int T, int K,
                                       void* ws, size_t ws_bytes, void* stream) {
    moegg_status_t st = check_norm(T, K);
    if (st != MOEGG_OK) return st;
    if (!known_weight(weight_dtype)) return MOEGG_ERR_INVALID_ARG;
    if (T > 0 && any_null({dy, h, weight, rstd, dx})) return MOEGG_ERR_INVALID_ARG;
    const bool bf16 = weight_dtype == MOEGG_WEIGHT_BF16;
    for (const void* p : {dy, h, d_sum, (const void*)dx})
        if (!aligned(p, 2)) return MOEGG_ERR_INVALID_ARG;
    if (!aligned(weight, bf16 ? 2 : 4) || !all4({rstd, d_weight})) return MOEGG_ERR_INVALID_ARG;
    if (d_weight && (!ws || !aligned(ws, 256) || ws_bytes < moegg_rms_norm_workspace_bytes(T, K)))
        return MOEGG_ERR_WORKSPACE;
    NormArgs a{};
    a.x = h;
    a.residual = d_sum;
    a.weight = weight;
    a.dy = dy;
    a.y = dx;
    a.rstd = (float*)rstd;
    a.d_weight = d_weight;
    a.parts = (float*)ws;
    a.T = T;
    a.K = K;
    a.weight_bf16 = bf16;
    return hip_status(launch_rms_norm_backward(a, (hipStream_t)stream), "RMS norm backward");
}

size_t moegg_balance_loss_workspace_bytes(int T, int E, int S) {
    if (T < 0 || T > kRouteMaxTokens || E < 1 || E > kBalanceMaxExperts || S < 1 || S > kBalanceMaxSequences) return 0;
    return align256(balance_pieces(T, S) * (8 * (size_t)E + 4));
}

moegg_status_t moegg_balance_loss(const void* logits, moegg_logits_t logits_dtype, const int32_t* ids,
                                  const int32_t* seq_offsets, float* loss, float* z_loss, int32_t* counts, float* probs,
                                  int T, int E, int k, int S, moegg_score_t score, void* ws, size_t ws_bytes,
                                  void* stream) {
    moegg_status_t st = check_balance(logits_dtype, score, logits, seq_offsets, T, E, k, S);
    if (st != MOEGG_OK) return st;
    if ((T > 0 && !ids) || any_null({loss, counts})) return MOEGG_ERR_INVALID_ARG;
    if (!all4({ids, loss, z_loss, counts, probs})) return MOEGG_ERR_INVALID_ARG;
    if (z_loss && score != MOEGG_SCORE_SOFTMAX) return MOEGG_ERR_UNSUPPORTED;
    if (!ws || !aligned(ws, 256) || ws_bytes < moegg_balance_loss_workspace_bytes(T, E, S)) return MOEGG_ERR_WORKSPACE;
    BalanceArgs a{};
    const size_t rows = balance_pieces(T, S);
    a.logits = logits;
    a.ids = ids;
    a.offsets = seq_offsets;
    a.loss = loss;
    a.z_loss = z_loss;
    a.counts = counts;
    a.probs = probs;
    a.part_p = (float*)ws;
    a.part_n = (int32_t*)(a.part_p + rows * E);
    a.part_z = (float*)(a.part_n + rows * E);
    a.T = T;
    a.E = E;
    a.k = k;
    a.S = S;
    a.bf16 = logits_dtype == MOEGG_LOGITS_BF16;
    a.sigmoid = score == MOEGG_SCORE_SIGMOID;
    a.tile_tokens = balance_tile_tokens(T);
    return hip_status(launch_balance_loss(a, (hipStream_t)stream), "balance loss");
}

moegg_status_t moegg_balance_loss_backward(const void* logits, moegg_logits_t logits_dtype, const int32_t* counts,
                                           const int32_t* seq_offsets, const float* d_loss, const float* d_z_loss,
                                           const void* before, void* d_logits, int T, int E, int k, int S,
                                           moegg_score_t score, void* stream) {
    moegg_status_t st = check_balance(logits_dtype, score, logits, seq_offsets, T, E, k, S);
    if (st != MOEGG_OK) return st;
    if (T > 0 && any_null({counts, d_loss, d_logits})) return MOEGG_ERR_INVALID_ARG;
    const uintptr_t z = logits_dtype == MOEGG_LOGITS_BF16 ? 2 : 4;
    if (!all4({counts, d_loss, d_z_loss}) || !aligned(before, z) || !aligned(d_logits, z)) return MOEGG_ERR_INVALID_ARG;
    if (d_z_loss && score != MOEGG_SCORE_SOFTMAX) return MOEGG_ERR_UNSUPPORTED;
    BalanceBackwardArgs a{logits, counts, seq_offsets, d_loss, d_z_loss, before, d_logits, T, E, k, S,
                          logits_dtype == MOEGG_LOGITS_BF16, score == MOEGG_SCORE_SIGMOID};
    return hip_status(launch_balance_loss_backward(a, (hipStream_t)stream), "balance loss backward");
}

size_t moegg_lora_workspace_bytes(int T, int K, int R) {
    if (T < 0 || T > kLoraMaxRows || K < 8 || K > 1 << 30 || K % 8 != 0 || R < 8 || R % 8 != 0 || R > kLoraMaxRank) return 0;
    return lora_layout(T, K, R).total;
}

moegg_status_t moegg_lora(const void* X, const void* A, const void* B, const float* scale, const int32_t* adapter,
                          const void* Y, void* out, int T, int K, int N, int R, int L, void* ws, size_t ws_bytes,
                          void* stream) {
    if (T < 0 || K < 1 || N < 1 || R < 1 || L < 1) return MOEGG_ERR_INVALID_ARG;
    if (T > 0 && any_null({X, A, B, adapter, Y, out})) return MOEGG_ERR_INVALID_ARG;
    if (!all16({X, A, B, Y, out}) || !all4({scale, adapter})) return MOEGG_ERR_INVALID_ARG;
    if (K % 8 != 0 || N % 8 != 0 || R % 8 != 0 || R > kLoraMaxRank || T > kLoraMaxRows) return MOEGG_ERR_UNSUPPORTED;
    const int64_t chunks = ((int64_t)T + kLoraChunk - 1) / kLoraChunk, panels = ((int64_t)N + 255) / 256;
    // columns are 32-bit, and go up to 255 past the width; up to 4096 workgroups more than one for each chunk and panel
    if (K > 1 << 30 || N > 1 << 30 || (chunks * panels + 8192) * 256 > kMaxWorkItems)
        return MOEGG_ERR_UNSUPPORTED;
    if (!ws || !aligned(ws, 256) || ws_bytes < moegg_lora_workspace_bytes(T, K, R)) return MOEGG_ERR_WORKSPACE;
    const LoraLayout at = lora_layout(T, K, R);
    unsigned char* w = (unsigned char*)ws;
    LoraArgs a{};
    a.X = X;
    a.A = A;
    a.B = B;
    a.scale = scale;
    a.adapter = adapter;
    a.Y = Y;
    a.out = out;
    a.U = (float*)w;
    a.order = (int32_t*)(w + at.order);
    a.tiles = (int4*)(w + at.tiles);
    a.T = T;
    a.K = K;
    a.N = N;
    a.R = R;
    a.L = L;
    a.splits = lora_splits(T, K, R);
    a.max_tiles = lora_max_tiles(T, L);
    return hip_status(launch_lora(a, (hipStream_t)stream), "low-rank adapters");
}

}  // extern "C"
