// permute.hip -- tokens into expert rows (dispatch), expert rows back into
// tokens (combine), and combine's backward pass.
//
// All three are bound by memory.  Token rows are read once, whatever k is:
// a wave holds a piece of a token in registers and writes it to the token's k
// rows, or sums the k rows' pieces.  Quantization is along the row, in groups
// of 128 = 8 lanes of 16 elements, so the amax needs three DPP steps and every
// store is 16 bytes a lane.
#include <hip/hip_runtime.h>

#include "device.hpp"
#include "layer.hpp"
#include "rows.hpp"

namespace moegg {

constexpr int kThreads = 256;

// Work item of a wave.
constexpr int kItemRun = 32;              // neighbouring workgroups on one XCD
__device__ __forceinline__ int64_t wave_item() {
    return work_position<kItemRun>() * (kThreads / 64) + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
}
static dim3 item_grid(int64_t items) { return run_grid<kItemRun>((items + kThreads / 64 - 1) / (kThreads / 64)); }

// Rows outside [0, rows) (no expert, over the capacity) are skipped.
__device__ __forceinline__ int uniform_row(const int32_t* p) { return __builtin_amdgcn_readfirstlane(*p); }

// ----------------------------------------------------------------- dispatch

// bf16: a wave copies 512 elements of a token to its k rows.  4096 tokens of
// 7168 to 8 experts each: 92 us, 5.7 TB/s of one read and 8 writes (101 us from
// HBM; 108 us with streamed loads).
__global__ __launch_bounds__(kThreads) void dispatch_bf16_kernel(PermuteArgs a, int chunks) {
    const int64_t item = wave_item();
    if (item >= (int64_t)a.T * chunks) return;
    const int lane = threadIdx.x & 63;
    const int64_t t = item / chunks;
    const int c = (int)(item % chunks) * 512 + lane * 8, n = a.W - c;
    if (n <= 0) return;
    const u32x4 v = load8<false>((const uint16_t*)a.x + t * a.W + c, n);
    for (int j = 0; j < a.k; ++j) {
        const int row = uniform_row(a.row_of + t * a.k + j);
        if ((uint32_t)row < (uint32_t)a.rows) store8((uint16_t*)a.out + (int64_t)row * a.W + c, v, n);
    }
}

// e4m3: a wave quantizes 1024 elements (8 groups) of a token, 16 a lane, and
// stores them to its k rows.  The same 4096 tokens: 46 us with row-major scales
// (6.5 TB/s), 50 us with transposed ones; 54 and 61 us with the tokens from HBM,
// 57 and 64 us with streamed loads.  Transposed scales are 4 bytes to a line each,
// 1.8 million of them; giving an XCD neighbouring tokens or neighbouring columns
// (whole lines then merge in its L2) makes no difference.
template <OperandFormat FMT>
__global__ __launch_bounds__(kThreads) void dispatch_fp8_kernel(PermuteArgs a, int chunks) {
    const int64_t item = wave_item();
    if (item >= (int64_t)a.T * chunks) return;
    const int lane = threadIdx.x & 63;
    const int64_t t = item / chunks;
    const int c = (int)(item % chunks) * 1024 + lane * 16;
    const bool in = c < a.W;                             // W % 128 == 0: whole groups
    u32x4 x0 = {0, 0, 0, 0}, x1 = {0, 0, 0, 0};
    if (in) {
        const u32x4* p = (const u32x4*)((const uint16_t*)a.x + t * a.W + c);
        x0 = p[0];                                       // halves of a line each: a streaming load fetches it twice
        x1 = p[1];
    }
    float f[16];
    unpack8(x0, f);
    unpack8(x1, f + 8);
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(f[i]));
    const GroupScale g = group_scale<FMT == kE8m0>(max8(m));
    uint32_t codes[4];
    quantize<16, FMT != kE8m0>(f, g, codes);
    const u32x4 q = {codes[0], codes[1], codes[2], codes[3]};
    const int kg = c / kGroup, groups = a.W / kGroup;
    for (int j0 = 0; j0 < a.k; j0 += 8) {
        // a group's 8 lanes store its scale to 8 rows
        const int js = j0 + (lane & 7);
        const int srow = js < a.k ? a.row_of[t * a.k + js] : -1;
        if (in && (uint32_t)srow < (uint32_t)a.rows) {
            if (FMT == kRows) ((float*)a.scale)[(int64_t)srow * groups + kg] = g.s;
            if (FMT == kKm) ((float*)a.scale)[(int64_t)kg * a.rows + srow] = g.s;
            if (FMT == kE8m0) ((uint8_t*)a.scale)[(int64_t)kg * a.rows + srow] = (uint8_t)g.byte;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int row = __builtin_amdgcn_readlane(srow, j);
            if (in && (uint32_t)row < (uint32_t)a.rows) 
                store_once((uint8_t*)a.out + (int64_t)row * a.W + c, q);
        }
    }
}

// ----------------------------------------------------------------- combine

// A wave sums 512 columns of a token's rows in fp32, in the order of its
// assignments, and rounds once.  Eight rows are in flight at a time.  32768 rows
// of 7168 into 4096 tokens: 88 us, 6.0 TB/s; with cached accesses and each XCD on
// an eighth of the tokens 107 us.
__global__ __launch_bounds__(kThreads) void combine_kernel(PermuteArgs a, int chunks) {
    const int64_t item = wave_item();
    if (item >= (int64_t)a.T * chunks) return;
    const int lane = threadIdx.x & 63;
    const int64_t t = item / chunks;
    const int c = (int)(item % chunks) * 512 + lane * 8, n = a.W - c;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    for (int j0 = 0; j0 < a.k; j0 += 8) {
        const int js = j0 + (lane & 7);
        const int srow = js < a.k ? a.row_of[t * a.k + js] : -1;
        const float sw = js < a.k && a.weights ? a.weights[t * a.k + js] : 1.f;
        u32x4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int row = __builtin_amdgcn_readlane(srow, j);
            v[j] = u32x4{0, 0, 0, 0};
            if ((uint32_t)row < (uint32_t)a.rows && n > 0)
                v[j] = load8<true>((const uint16_t*)a.x + (int64_t)row * a.W + c, n);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int row = __builtin_amdgcn_readlane(srow, j);
            if ((uint32_t)row >= (uint32_t)a.rows) continue;
            const float w = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(sw), j));
            float f[8];
            unpack8(v[j], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(w, f[i], acc[i]);
        }
    }
    if (n <= 0) return;
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(acc[2 * i], acc[2 * i + 1]);
    store8((uint16_t*)a.out + t * a.W + c, o, n);
}

// A workgroup takes a token: dY rows are weight * dout, and each weight's
// gradient is the dot product of its row of Y with dout, summed in fp32 in a
// fixed order (lane pieces, wave, waves).  dout is read once per 8 rows.  32768
// rows of 7168 in bf16: 181 us, 5.5 TB/s; with e4m3 dY 143 us (row-major scales),
// 151 us (transposed) and 146 us (E8M0), 167 to 174 us where dout comes from HBM.
// As many waves as there are 512-column pieces: 4 waves going round take 202 us.
template <OperandFormat FMT>
__global__ __launch_bounds__(1024) void combine_backward_kernel(PermuteArgs a) {
    // Rows loaded at a time.  With quantization beside them, 8 leave one workgroup a CU at 7168 columns (158 us), 2
    // leave two (144 us); in bf16 there are two either way.
    constexpr int kAhead = FMT == kBf16 ? 8 : 2;
    __shared__ float part_s[16][8];
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int groups = a.W / kGroup;
    for (int j0 = 0; j0 < a.k; j0 += 8) {
        const int js = j0 + (lane & 7);
        const int srow = js < a.k ? a.row_of[t * a.k + js] : -1;
        const float sw = js < a.k ? a.weights[t * a.k + js] : 0.f;
        float dot[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) dot[j] = 0.f;
        for (int c0 = wave * 512; c0 < a.W; c0 += (int)blockDim.x * 8) {
            const int c = c0 + lane * 8, n = a.W - c;
            u32x4 dv = {0, 0, 0, 0};
            if (n > 0) dv = load8<false>((const uint16_t*)a.x + t * a.W + c, n);
            float d[8];
            unpack8(dv, d);
            float amax = 0.f;
            if (FMT != kBf16) {
#pragma unroll
                for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(d[i]));
                amax = max16(amax);
            }
#pragma unroll
            for (int h = 0; h < 8; h += kAhead) {
                u32x4 y[kAhead];
#pragma unroll
                for (int j = h; j < h + kAhead; ++j) {
                    const int row = __builtin_amdgcn_readlane(srow, j);
                    y[j - h] = u32x4{0, 0, 0, 0};
                    if ((uint32_t)row < (uint32_t)a.rows && n > 0)
                        y[j - h] = load8<true>((const uint16_t*)a.Y + (int64_t)row * a.W + c, n);
                }
#pragma unroll
                for (int j = h; j < h + kAhead; ++j) {
                    const int row = __builtin_amdgcn_readlane(srow, j);
                    if ((uint32_t)row >= (uint32_t)a.rows) continue;
                    const float w = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(sw), j));
                    float f[8], o[8];
                    unpack8(y[j - h], f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        dot[j] = __builtin_fmaf(f[i], d[i], dot[j]);
                        o[i] = w * d[i];
                    }
                    if (FMT == kBf16) {
                        u32x4 v;
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[i] = pack_bf16x2(o[2 * i], o[2 * i + 1]);
                        if (n > 0) store8((uint16_t*)a.out + (int64_t)row * a.W + c, v, n);
                    } else {
                        // rounding keeps order: the largest |w d| is |w| times the largest |d|, rounded
                        const GroupScale g = group_scale<FMT == kE8m0>(fabsf(w * amax));
                        uint32_t codes[2];
                        quantize<8, FMT != kE8m0>(o, g, codes);
                        const u32x2 q = {codes[0], codes[1]};
                        if (n > 0) {
                            store_once((uint8_t*)a.out + (int64_t)row * a.W + c, q);
                            if ((lane & 15) == 0) {
                                const int kg = c / kGroup;
                                if (FMT == kRows) ((float*)a.scale)[(int64_t)row * groups + kg] = g.s;
                                if (FMT == kKm) ((float*)a.scale)[(int64_t)kg * a.rows + row] = g.s;
                                if (FMT == kE8m0) ((uint8_t*)a.scale)[(int64_t)kg * a.rows + row] = (uint8_t)g.byte;
                            }
                        }
                    }
                }
                __builtin_amdgcn_sched_barrier(0);       // the next rows' loads not before: their registers
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = wave_sum(dot[j]);
            if (lane == 0) part_s[wave][j] = v;
        }
        __syncthreads();
        if (threadIdx.x < 8 && j0 + (int)threadIdx.x < a.k) {
            float v = 0.f;
            for (int w = 0; w < (int)blockDim.x / 64; ++w) v += part_s[w][threadIdx.x];
            a.d_weights[t * a.k + j0 + threadIdx.x] = v;
        }
        __syncthreads();
    }
}

// ----------------------------------------------------------------- launches

hipError_t launch_dispatch(const PermuteArgs& a, hipStream_t s) {
    if (a.T == 0) return hipSuccess;
    const int chunks = a.fmt == kBf16 ? (a.W + 511) / 512 : (a.W + 1023) / 1024;
    const dim3 grid = item_grid((int64_t)a.T * chunks);
    switch (a.fmt) {
        case kBf16: dispatch_bf16_kernel<<<grid, kThreads, 0, s>>>(a, chunks); break;
        case kRows: dispatch_fp8_kernel<kRows><<<grid, kThreads, 0, s>>>(a, chunks); break;
        case kKm: dispatch_fp8_kernel<kKm><<<grid, kThreads, 0, s>>>(a, chunks); break;
        case kE8m0: dispatch_fp8_kernel<kE8m0><<<grid, kThreads, 0, s>>>(a, chunks); break;
    }
    return hipGetLastError();
}

hipError_t launch_combine(const PermuteArgs& a, hipStream_t s) {
    if (a.T == 0) return hipSuccess;
    const int chunks = (a.W + 511) / 512;
    combine_kernel<<<item_grid((int64_t)a.T * chunks), kThreads, 0, s>>>(a, chunks);
    return hipGetLastError();
}

hipError_t launch_combine_backward(const PermuteArgs& a, hipStream_t s) {
    if (a.T == 0) return hipSuccess;
    // a wave for each 512 columns, up to 16
    const int threads = 64 * (a.W >= 16 * 512 ? 16 : (a.W + 511) / 512);
    switch (a.fmt) {
        case kBf16: combine_backward_kernel<kBf16><<<a.T, threads, 0, s>>>(a); break;
        case kRows: combine_backward_kernel<kRows><<<a.T, threads, 0, s>>>(a); break;
        case kKm: combine_backward_kernel<kKm><<<a.T, threads, 0, s>>>(a); break;
        case kE8m0: combine_backward_kernel<kE8m0><<<a.T, threads, 0, s>>>(a); break;
    }
    return hipGetLastError();
}

}  // namespace moegg
