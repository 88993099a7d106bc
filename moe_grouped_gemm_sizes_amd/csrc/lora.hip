// lora.hip -- low-rank adapters of many requests, added to a projection's output:
//     out[t] = Y[t] + scale_a (X[t] A_a^T) B_a^T,   a the adapter of row t.
//
// Two products of a rank of 8 to 128, so that rows and weights are moved and little is
// computed.  The rows of one adapter are found by the kernels themselves: a wave
// looks at 64 consecutive rows, a lane each, and takes the adapters among them one
// by one; requests lie in consecutive rows, so that long prompts have one or two
// there.  Then matrix products in blocks of 16 rows.
#include <hip/hip_runtime.h>

#include "block.hpp"
#include "device.hpp"
#include "layer.hpp"
#include "rows.hpp"

namespace moegg {

constexpr int kThreads = 256;
constexpr int kBlocks = kLoraChunk / 16;  // row blocks of a chunk

// The adapters among a chunk's 64 rows, in the order of their first rows.
struct ChunkRows {
    int own;                             // this lane's adapter; -1: none, or past the last row
    uint64_t left;                       // rows whose adapter was not taken yet
    __device__ __forceinline__ ChunkRows(const LoraArgs& a, int chunk) {
        const int t = chunk * kLoraChunk + ((int)threadIdx.x & 63);
        own = t < a.T ? a.adapter[t] : -1;
        if (own >= a.L) own = -1;
        left = __ballot(own >= 0);
    }
    // The next adapter and its rows.
    __device__ __forceinline__ int next(uint64_t& rows) {
        const int adapter = __builtin_amdgcn_readlane(own, __builtin_ctzll(left));
        rows = __ballot(own == adapter);
        left &= ~rows;
        return adapter;
    }
};

// Row (within the chunk) of the i-th set bit of `rows`, for every lane's own i;
// past the last one the last one's.  Goes through LDS: lane r of the chunk says where it is.
__device__ __forceinline__ void list_rows(uint64_t rows, int* list_s) {
    const int lane = threadIdx.x & 63;
    if (rows >> lane & 1) list_s[__popcll(rows & ((1ull << lane) - 1))] = lane;
}

// ----------------------------------------------------------------- X A^T

// A workgroup takes the rows of one adapter in a chunk and a part of K, its waves
// a quarter of that each; their sums meet in LDS.  D = X A^T in blocks of 16 rows x
// 16 ranks.
template <int RT, int CT>
__device__ __forceinline__ void shrink(const LoraArgs& a, const int* list_s, int n, int adapter, int chunk, int split,
                                       float (*sum_s)[16][16]) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int l16 = lane & 15, grp = lane >> 4;
    // K in steps of 32, shared out over splits x 4 waves
    const int steps = (a.K + 31) / 32, shares = a.splits * 4, share = split * 4 + wave;
    const int s0 = (int)((int64_t)steps * share / shares), s1 = (int)((int64_t)steps * (share + 1) / shares);
    const uint16_t* x[RT];
    const uint16_t* w[CT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
        x[r] = (const uint16_t*)a.X + ((int64_t)chunk * kLoraChunk + list_s[min(r * 16 + l16, n - 1)]) * a.K + grp * 8;
#pragma unroll
    for (int c = 0; c < CT; ++c)
        w[c] = (const uint16_t*)a.A + ((int64_t)adapter * a.R + min(c * 16 + l16, a.R - 1)) * a.K + grp * 8;
    v4f acc[RT][CT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[r][c] = v4f{0, 0, 0, 0};
#pragma unroll 4
    for (int s = s0; s < s1; ++s) {
        const bool in = s * 32 + grp * 8 < a.K;              // K % 8 == 0: whole pieces
        v4i xv[RT], wv[CT];
#pragma unroll
        for (int r = 0; r < RT; ++r) xv[r] = in ? *(const v4i*)(x[r] + s * 32) : v4i{0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < CT; ++c) wv[c] = in ? *(const v4i*)(w[c] + s * 32) : v4i{0, 0, 0, 0};
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int c = 0; c < CT; ++c) acc[r][c] = mfma_bf16(xv[r], wv[c], acc[r][c]);
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            __syncthreads();
#pragma unroll
            for (int v = 0; v < 4; ++v) sum_s[wave][grp * 4 + v][l16] = acc[r][c][v];
            __syncthreads();
            const int row = threadIdx.x >> 4, rank = c * 16 + (threadIdx.x & 15);
            const float u = (sum_s[0][row][threadIdx.x & 15] + sum_s[1][row][threadIdx.x & 15]) +
                            (sum_s[2][row][threadIdx.x & 15] + sum_s[3][row][threadIdx.x & 15]);
            if (r * 16 + row < n && rank < a.R) {
                const int64_t t = (int64_t)chunk * kLoraChunk + list_s[r * 16 + row];
                a.U[((int64_t)split * a.T + t) * a.R + rank] = u;
            }
        }
    }
    __syncthreads();
}

template <int CT>
__global__ __launch_bounds__(kThreads) void lora_shrink_kernel(LoraArgs a, int slots) {
    __shared__ int list_s[kLoraChunk];
    __shared__ float sum_s[4][16][16];
    const int split = blockIdx.x % a.splits, slot = blockIdx.x / a.splits % slots, chunk = blockIdx.x / a.splits / slots;
    ChunkRows at(a, chunk);
    for (int i = 0; at.left; ++i) {
        uint64_t rows;
        const int adapter = at.next(rows);
        if (i % slots != slot) continue;
        const int n = __popcll(rows);
        if (threadIdx.x < 64) list_rows(rows, list_s);
        __syncthreads();
        if (n <= 16) shrink<1, CT>(a, list_s, n, adapter, chunk, split, sum_s);
        else shrink<kBlocks, CT>(a, list_s, n, adapter, chunk, split, sum_s);
    }
}

// ----------------------------------------------------------------- U B^T

// U in two bf16, the value and what is left of it (2^-16 of it is lost at most): one
// would put half a step of bf16, 2^-8, on every term.
__device__ __forceinline__ void split_bf16(float u, uint16_t& hi, uint16_t& lo) {
    const __bf16 h = (__bf16)u;
    const float left = u - (float)h;
    const __bf16 l = (__bf16)(left == left && fabsf(left) < __builtin_inff() ? left : 0.f);
    hi = __builtin_bit_cast(uint16_t, h);
    lo = __builtin_bit_cast(uint16_t, l);
}

// A wave takes 64 columns of out for the rows of one adapter in a chunk.  D = B U^T:
// a lane has one row of out and, with columns 16 (i / 4) + 4 b + i % 4 as row i of
// block b, 16 consecutive columns of it.
template <int RT, int RS>
__device__ __forceinline__ void expand(const LoraArgs& a, const int* list_s, const uint16_t (*u_s)[2][RS * 32 + 8], int n,
                                       int adapter, int chunk, int col) {
    const int lane = threadIdx.x & 63, l16 = lane & 15, grp = lane >> 4;
    const float scale = a.scale ? a.scale[adapter] : 1.f;
    v4f acc[RT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[r][b] = v4f{0, 0, 0, 0};
    v4i w[4][RS];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const int c = col + 16 * (l16 >> 2) + 4 * b + (l16 & 3);
        const uint16_t* p = (const uint16_t*)a.B + ((int64_t)adapter * a.N + min(c, a.N - 1)) * a.R + grp * 8;
#pragma unroll
        for (int s = 0; s < RS; ++s) w[b][s] = s * 32 + grp * 8 < a.R ? *(const v4i*)(p + s * 32) : v4i{0, 0, 0, 0};
    }
    const int c = col + 16 * grp;                            // this lane's 16 columns
    u32x4 y[RT][2];
    int64_t at[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        at[r] = ((int64_t)chunk * kLoraChunk + list_s[min(r * 16 + l16, n - 1)]) * a.N + c;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            y[r][h] = c + 8 * h < a.N ? *(const u32x4*)((const uint16_t*)a.Y + at[r] + 8 * h) : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int s = 0; s < RS; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const v4i u = *(const v4i*)&u_s[r * 16 + l16][h][s * 32 + grp * 8];
#pragma unroll
                for (int b = 0; b < 4; ++b) acc[r][b] = mfma_bf16(w[b][s], u, acc[r][b]);
            }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        if (r * 16 + l16 >= n) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (c + 8 * h >= a.N) continue;                  // N % 8 == 0
            float f[8];
            unpack8(y[r][h], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = __builtin_fmaf(scale, acc[r][2 * h + j / 4][j % 4], f[j]);
            *(u32x4*)((uint16_t*)a.out + at[r] + 8 * h) = pack8(f);
        }
    }
}

template <int RS>
__global__ __launch_bounds__(kThreads) void lora_expand_kernel(LoraArgs a, int slots, int panels) {
    __shared__ int list_s[kLoraChunk];
    __shared__ __align__(16) uint16_t u_s[kLoraChunk][2][RS * 32 + 8];   // 16 bytes more: rows on different banks
    const int panel = blockIdx.x % panels, slot = blockIdx.x / panels % slots, chunk = blockIdx.x / panels / slots;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int col = panel * 256 + wave * 64;
    ChunkRows at(a, chunk);
    const bool none = at.own < 0 && chunk * kLoraChunk + ((int)threadIdx.x & 63) < a.T;
    const uint64_t bare = __ballot(none);                    // rows without an adapter
    for (int i = 0; at.left; ++i) {
        uint64_t rows;
        const int adapter = at.next(rows);
        if (i % slots != slot) continue;
        const int n = __popcll(rows);
        __syncthreads();
        if (threadIdx.x < 64) list_rows(rows, list_s);
        __syncthreads();
        const int blocks = (n + 15) / 16;
        for (int j = threadIdx.x; j < blocks * 16 * RS * 32; j += kThreads) {
            const int row = j / (RS * 32), rank = j % (RS * 32);
            float u = 0.f;
            if (row < n && rank < a.R) {
                const int64_t t = (int64_t)chunk * kLoraChunk + list_s[row];
                for (int s = 0; s < a.splits; ++s) u += a.U[((int64_t)s * a.T + t) * a.R + rank];
            }
            split_bf16(u, u_s[row][0][rank], u_s[row][1][rank]);
        }
        __syncthreads();
        if (col < a.N) {
            if (n <= 16) expand<1, RS>(a, list_s, u_s, n, adapter, chunk, col);
            else expand<kBlocks, RS>(a, list_s, u_s, n, adapter, chunk, col);
        }
    }
    if (slot == 0 && a.out != a.Y)
        for (uint64_t left = bare; left; left &= left - 1) {
            const int64_t t = (int64_t)chunk * kLoraChunk + __builtin_ctzll(left);
            const int c = panel * 256 + (int)threadIdx.x * 8;
            if (threadIdx.x < 32 && c < a.N)
                *(u32x4*)((uint16_t*)a.out + t * a.N + c) = *(const u32x4*)((const uint16_t*)a.Y + t * a.N + c);
        }
}

// ----------------------------------------------------------------- launches

// Workgroups that share a chunk's adapters among them: no more than there can be,
// and no more than 1024 workgroups call for.
static int lora_slots(const LoraArgs& a, int64_t others) {
    int most = a.L < kLoraChunk ? a.L : kLoraChunk;
    if (a.T < most) most = a.T;
    const int64_t want = (1024 + others - 1) / others;
    return most < want ? most : (int)want;
}

hipError_t launch_lora(const LoraArgs& a, hipStream_t s) {
    if (a.T == 0) return hipSuccess;
    const int64_t chunks = (a.T + kLoraChunk - 1) / kLoraChunk;
    int slots = lora_slots(a, chunks * a.splits);
    dim3 grid((unsigned)(chunks * slots * a.splits));
    if (a.R <= 16) lora_shrink_kernel<1><<<grid, kThreads, 0, s>>>(a, slots);
    else if (a.R <= 32) lora_shrink_kernel<2><<<grid, kThreads, 0, s>>>(a, slots);
    else if (a.R <= 64) lora_shrink_kernel<4><<<grid, kThreads, 0, s>>>(a, slots);
    else lora_shrink_kernel<8><<<grid, kThreads, 0, s>>>(a, slots);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int panels = (a.N + 255) / 256;
    slots = lora_slots(a, chunks * panels);
    grid = dim3((unsigned)(chunks * slots * panels));
    if (a.R <= 32) lora_expand_kernel<1><<<grid, kThreads, 0, s>>>(a, slots, panels);
    else if (a.R <= 64) lora_expand_kernel<2><<<grid, kThreads, 0, s>>>(a, slots, panels);
    else lora_expand_kernel<4><<<grid, kThreads, 0, s>>>(a, slots, panels);
    return hipGetLastError();
}

}  // namespace moegg
