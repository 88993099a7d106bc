// block.hpp -- arguments and launchers of the operators of a block around the
// MoE layer: RMS norm (norm.hip), the router's balance loss (balance.hip) and
// low-rank adapters (lora.hip), which the C ABI (block_api.hip) calls.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "layer.hpp"

namespace moegg {

constexpr int kNormMaxWidth = 32768;     // columns of a row that one workgroup holds in registers
constexpr int kNormMaxParts = 256;       // partial sums of the weight's gradient
constexpr int kBalanceMaxExperts = 1024;
constexpr int kBalanceMaxSequences = 65536;
constexpr int kLoraChunk = 64;           // rows whose adapters one wave looks at together
// Rows up to which chunks are taken as they come, and sorted beyond (us, 7168 -> 16 -> 4096; rows of 64 adapters in
// any order, some of them popular: 64 rows 13.5 and 13.9 sorted, 128 18.7 and 15.3, 256 31.5 and 18.4; rank 64, 32
// adapters: 17.7 and 17.8, 23.0 and 20.8, 47.5 and 25.3; packed rows of 4 adapters: 10.7 and 14.8, 11.2 and 17.0, 13.5
// and 17.9, which 129 to 256 rows pay for those in any order).
constexpr int kLoraChunkRows = 128;
constexpr int kLoraWindow = 8192;        // rows that one workgroup sorts by adapter
constexpr int kLoraMaxSorted = 16384;    // adapters whose counts are 64 KB of LDS
constexpr int kLoraMaxRank = 128;
constexpr int kLoraMaxRows = 1 << 24;

struct NormArgs {
    const void* x;                       // forward: bf16 [T, K]; backward: h
    const void* residual;                // forward: bf16 [T, K] or NULL; backward: d_sum
    const void* weight;                  // fp32 or bf16 [K]
    const void* dy;                      // backward: bf16 [T, K]
    void* sum_out;                       // bf16 [T, K] or NULL
    void* y;                             // forward: bf16 [T, K] or NULL; backward: dx
    void* q;                             // e4m3 [T, K] or NULL
    void* q_scale;
    float* rstd;                         // [T]; forward: or NULL
    float* d_weight;                     // backward: [K] or NULL
    float* parts;                        // backward: [norm_parts(T), K]
    int T, K;
    int weight_bf16;
    float eps;
    OperandFormat fmt;                   // of q; kBf16: none
};

struct BalanceArgs {
    const void* logits;                  // fp32 or bf16 [T, E]
    const int32_t* ids;                  // [T, k]
    const int32_t* offsets;              // [S + 1] or NULL: one sequence of all tokens
    float* loss;                         // [S]
    float* z_loss;                       // [S] or NULL
    int32_t* counts;                     // [S, E]
    float* probs;                        // [S, E] or NULL
    float* part_p;                       // [pieces, E]: sums of probabilities
    int32_t* part_n;                     // [pieces, E]: assignments
    float* part_z;                       // [pieces]
    int T, E, k, S, bf16, sigmoid;
    int tile_tokens;                     // tokens of one workgroup
};

struct BalanceBackwardArgs {
    const void* logits;
    const int32_t* counts;
    const int32_t* offsets;
    const float* d_loss;                 // [S]
    const float* d_z;                    // [S] or NULL
    const void* before;                  // logits' type [T, E] or NULL
    void* d_logits;
    int T, E, k, S, bf16, sigmoid;
};

struct LoraArgs {
    const void* X;                       // bf16 [T, K]
    const void* A;                       // bf16 [L, R, K]
    const void* B;                       // bf16 [L, N, R]
    const float* scale;                  // [L] or NULL
    const int32_t* adapter;              // [T]
    const void* Y;                       // bf16 [T, N]
    void* out;                           // bf16 [T, N]
    float* U;                            // [splits, T, R]
    int32_t* order;                      // [T]: rows by adapter, window by window
    int4* tiles;                         // [windows, max_tiles]: adapter, first place in `order`, rows
                                         // (0 past the last one)
    int T, K, N, R, L;
    int splits;                          // of K
    int max_tiles;                       // of a window, or of a chunk
};

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s);
hipError_t launch_rms_norm_backward(const NormArgs& a, hipStream_t s);
hipError_t launch_balance_loss(const BalanceArgs& a, hipStream_t s);
hipError_t launch_balance_loss_backward(const BalanceBackwardArgs& a, hipStream_t s);
hipError_t launch_lora(const LoraArgs& a, hipStream_t s);

// Partial sums that the norm's backward pass leaves: one a workgroup, and no more
// workgroups than CUs.
inline int norm_parts(int T) { return T < kNormMaxParts ? T : kNormMaxParts; }

// Tokens of one workgroup of the balance loss.
inline int balance_tile_tokens(int T) {
    const int t = (T + 255) / 256;
    return t <= 32 ? 32 : (t + 15) / 16 * 16;
}

// Whether rows are sorted by adapter first, which the counts of all adapters in LDS allow.
inline bool lora_sorted(int T, int L) { return T > kLoraChunkRows && L < kLoraMaxSorted; }

// Tiles of a window or chunk at most: full ones, and one of fewer rows for each adapter
// (and for rows without one).
inline int lora_max_tiles(int T, int L) {
    const bool sorted = lora_sorted(T, L);
    const int most = sorted ? kLoraWindow : kLoraChunk, rows = T < most ? T : most;
    const int all = rows / (sorted ? kLoraChunk : 16) + (L < rows ? L + 1 : rows);
    return sorted || all < rows ? all : rows;
}

// Entries of the tile lists of any call of up to T rows.
inline int64_t lora_tile_slots(int T) {
    const int64_t windows = ((int64_t)T + kLoraWindow - 1) / kLoraWindow, rows = T < kLoraWindow ? T : kLoraWindow;
    return windows * (rows / kLoraChunk + rows);
}

// Parts of K that workgroups of the first product take: 2 units of 128 columns a wave (1 where
// rows are few), and no more of them than make 512 workgroups of full tiles, or 256 past a rank of
// 32, whose sums are more to add (8191 rows, 2048 -> 64 -> 7168: 512 90 us, 256 85 us; 4096 rows,
// 7168 -> 16 -> 4096: 40 and 42 us, 1024 45 us).  Rows in chunks are taken to share an adapter in
// pairs (96 rows of 64 adapters, ranks 16, 64 and 128: 16.5, 27.7 and 48.4 us; as if all 64 were alike
// 17.3, 26.8 and 46.2 us, none 16.8, 26.6 and 49.1 us).
inline int lora_splits(int T, int K, int R) {
    const int each = T <= kLoraChunkRows ? 2 : kLoraChunk, most = R <= 32 ? 512 : 256;
    const int tiles = (T + each - 1) / each, units = (K + 127) / 128;
    const int want = tiles > 0 ? (most + tiles - 1) / tiles : 1;
    const int share = (units + 4 * want - 1) / (4 * want);
    return (units + 4 * share - 1) / (4 * share);
}

}  // namespace moegg
