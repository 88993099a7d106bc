// norm.hip -- root-mean-square norm with the residual's addition and an e4m3
// operand as output, and its backward pass.
//
// Both are bound by memory: they move what they have to at the rate of a copy
// (5.2 TB/s), rows held in registers between the sum and what it scales.  A group of 128
// columns is 16 lanes of 8, so its amax takes four DPP steps.
#include <hip/hip_runtime.h>

#include "block.hpp"
#include "device.hpp"
#include "layer.hpp"
#include "rows.hpp"

namespace moegg {

// 8 weights from column c on, as fp32; 0 past the row's end.
__device__ __forceinline__ void load_weight8(const void* w, int bf16, int c, int n, float (&f)[8]) {
    if (bf16) {
        unpack8(load8<false>((const uint16_t*)w + c, n), f);
    } else if (n >= 8) {
        typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
        const f32x4_a4 lo = *(const f32x4_a4*)((const float*)w + c), hi = *(const f32x4_a4*)((const float*)w + c + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = lo[i];
            f[4 + i] = hi[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = i < n ? ((const float*)w)[c + i] : 0.f;
    }
}

// A row is taken by `waves` waves, 8 CH columns a thread; a workgroup takes as many rows as it
// has such groups of waves.
struct RowPart {
    int waves, group, thread;            // group: the row within the workgroup; thread: within the row

    __device__ __forceinline__ explicit RowPart(int waves_) : waves(waves_) {
        const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        group = wave / waves;
        thread = (wave - group * waves) * 64 + ((int)threadIdx.x & 63);
    }
    __device__ __forceinline__ int column(int i) const { return (i * waves * 64 + thread) * 8; }
    // Sum over the row in a fixed order, in every thread of it.  Rows of one wave need no barrier.
    // part_s: one float a wave, free again after the workgroup's next barrier.
    __device__ __forceinline__ float sum(float v, float* part_s) const {
        v = wave_sum(v);
        if (waves == 1) return v;
        if ((threadIdx.x & 63) == 0) part_s[threadIdx.x >> 6] = v;
        lds_barrier();
        // 16 lanes read the waves' sums and add them
        const int l16 = threadIdx.x & 15;
        float s = l16 < waves ? part_s[group * waves + l16] : 0.f;
        s += __uint_as_float(lane_of<DPP_XOR1>(__float_as_uint(s)));
        s += __uint_as_float(lane_of<DPP_XOR2>(__float_as_uint(s)));
        s += __uint_as_float(lane_of<DPP_HALF_MIRROR>(__float_as_uint(s)));
        return s + __uint_as_float(lane_of<DPP_MIRROR>(__float_as_uint(s)));
    }
};

// 1 / sqrt(x): the hardware's (1 ulp) and one Newton step.
__device__ __forceinline__ float rsqrt_f32(float x) {
    const float r = __builtin_amdgcn_rsqf(x);
    if (!(r > 0.f) || !(r < __builtin_inff())) return r;
    return __builtin_fmaf(0.5f * r, __builtin_fmaf(-x * r, r, 1.f), r);
}

// ----------------------------------------------------------------- forward

// A row is held in registers, so that it is read once: h = bf16(x + r), the sum of h^2 in fp32,
// then h rstd w.  4096 rows of 7168 with a residual, into bf16 and e4m3 with transposed scales: 49 us,
// 5.4 TB/s (stores through the caches: 52 us), with E8M0 scales alike; of 12288, 16384 and 32768: 83,
// 110 and 234 us, 5.2 to 5.5 TB/s.  One row 3.3 us, a launch and a chain of load, sum and store (of
// 32768 columns 7.2 us).
template <OperandFormat FMT, int CH>
__global__ __launch_bounds__(1024) void rms_norm_kernel(NormArgs a, int waves) {
    __shared__ float part_s[2][16];
    const RowPart part(waves);
    const int64_t t = (int64_t)blockIdx.x * (blockDim.x / 64 / waves) + part.group, at = t * a.K;
    const int width = t < a.T ? a.K : 0;                     // of this row
    u32x4 h[CH], r[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = part.column(i), n = width - c;
        h[i] = r[i] = u32x4{0, 0, 0, 0};
        if (n > 0) h[i] = load8<false>((const uint16_t*)a.x + at + c, n);
        if (n > 0 && a.residual) r[i] = load8<false>((const uint16_t*)a.residual + at + c, n);
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = part.column(i), n = width - c;
        float f[8];
        unpack8(h[i], f);
        if (a.residual) {
            float g[8];
            unpack8(r[i], g);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] += g[j];
            h[i] = pack8(f);
            if (n > 0 && a.sum_out) store8((uint16_t*)a.sum_out + at + c, h[i], n);
            unpack8(h[i], f);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(f[j], f[j], sum);
    }
    sum = part.sum(sum, part_s[0]);
    // some row's squares past fp32's range, by themselves or with eps, or an infinity or NaN in it: with rows of
    // several waves all of the workgroup's take part in a second sum
    const float square = sum / (float)a.K + a.eps;
    bool far = !(square < __builtin_inff());
    if (waves > 1 && (int)blockDim.x > waves * 64) {
        float all = a.eps;
        for (int w = 0; w < (int)blockDim.x / 64; ++w) all += part_s[0][w];
        far = !(all < 0x1p127f);                             // another order of sums than a row's: not to the last bit
    }
    float rstd = rsqrt_f32(square);
    if (far) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            float f[8];
            unpack8(h[i], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float v = f[j] * 0x1p-80f;
                s = __builtin_fmaf(v, v, s);
            }
        }
        s = part.sum(s, part_s[1]);
        // an eps that is lost at this scale is nothing beside the squares
        if (!(square < __builtin_inff())) rstd = rsqrt_f32(s / (float)a.K + a.eps * 0x1p-80f * 0x1p-80f) * 0x1p-80f;
    }
    if (width == 0) return;
    if (a.rstd && part.thread == 0) a.rstd[t] = rstd;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = part.column(i), n = width - c;
        float f[8], w[8];
        unpack8(h[i], f);
        load_weight8(a.weight, a.weight_bf16, c, n, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = f[j] * rstd * w[j];
        if (n > 0 && a.y) store8((uint16_t*)a.y + at + c, pack8(f), n);
        if (FMT != kBf16) {
            const GroupScale g = group_scale<FMT == kE8m0>(max16(amax8(f, 0.f)));
            uint32_t codes[2];
            quantize<8, FMT != kE8m0>(f, g, codes);   // bf16 values times rstd and a weight: the rounded quotient
            if (n > 0) {
                *(u32x2*)((uint8_t*)a.q + at + c) = u32x2{codes[0], codes[1]};
                if ((threadIdx.x & 15) == 0) {
                    const int kg = c / kGroup;
                    if (FMT == kRows) ((float*)a.q_scale)[t * (a.K / kGroup) + kg] = g.s;
                    if (FMT == kKm) ((float*)a.q_scale)[(int64_t)kg * a.T + t] = g.s;
                    if (FMT == kE8m0) ((uint8_t*)a.q_scale)[(int64_t)kg * a.T + t] = (uint8_t)g.byte;
                }
            }
        }
    }
}

// ----------------------------------------------------------------- backward

// With xhat = h rstd and g = dy w:  dx = d_sum + rstd (g - xhat mean(g xhat)),
// dw = sum over rows of dy xhat.  A workgroup goes through rows, as many at a time as it has groups
// of waves, the next two on their way, and sums its share of dw in registers: one
// partial row a workgroup, which a second launch adds in order.
struct BackwardPiece {
    u32x4 h, dy, d_sum;
    float rstd;

    __device__ __forceinline__ void load(const NormArgs& a, int64_t t, int c) {
        const int n = t < a.T ? a.K - c : 0;
        h = dy = d_sum = u32x4{0, 0, 0, 0};
        rstd = t < a.T ? a.rstd[t] : 0.f;
        if (n > 0) {
            const int64_t at = t * a.K + c;
            h = load8<false>((const uint16_t*)a.x + at, n);
            dy = load8<false>((const uint16_t*)a.dy + at, n);
            if (a.residual) d_sum = load8<false>((const uint16_t*)a.residual + at, n);
        }
    }
    // This piece's share of the sum of g xhat, and dy xhat on top of acc.
    __device__ __forceinline__ float dot(const float (&w)[8], float (&acc)[8]) const {
        float f[8], g[8], d = 0.f;
        unpack8(h, f);
        unpack8(dy, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float xhat = f[j] * rstd;
            d = __builtin_fmaf(g[j] * w[j], xhat, d);
            acc[j] = __builtin_fmaf(g[j], xhat, acc[j]);
        }
        return d;
    }
    __device__ __forceinline__ void store(const NormArgs& a, const float (&w)[8], float mean, int64_t t, int c) const {
        const int n = t < a.T ? a.K - c : 0;
        float f[8], g[8], s[8];
        unpack8(h, f);
        unpack8(dy, g);
        unpack8(d_sum, s);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] = __builtin_fmaf(rstd, __builtin_fmaf(-f[j] * rstd, mean, g[j] * w[j]), s[j]);
        if (n > 0) store8((uint16_t*)a.y + t * a.K + c, pack8(s), n);
    }
};

// 4096 rows of 7168 with d_sum: 46 us, 5.1 TB/s, and 4.5 us for the partial rows (58 us for both
// with each row loaded after the one before it, 57 us with one row ahead, 51 us with two).  Rows past
// 8192 columns are read twice, one at a time: 4096 of 12288, 16384 and 32768 take 111, 130 and 477 us
// with the partial rows, 3.6, 4.1 and 2.3 TB/s of what has to move, the last with 83 registers spilled;
// one row 12.5, 15 and 40 us.
template <int CH>
__global__ __launch_bounds__(1024) void rms_norm_backward_kernel(NormArgs a, int waves) {
    // what the workgroup's groups of waves add up to: of rows of up to 8192 columns, which may have several groups
    __shared__ float acc_s[CH == 1 ? 1024 * 8 : 1];
    __shared__ float part_s[2][16];
    const RowPart part(waves);
    const int groups = (int)blockDim.x / 64 / waves;
    const int64_t step = (int64_t)gridDim.x * groups;
    int64_t t = (int64_t)blockIdx.x * groups + part.group;
    float w[8], acc[CH][8];
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
    auto weights = [&](int i) { load_weight8(a.weight, a.weight_bf16, part.column(i), a.K - part.column(i), w); };
    // every group goes round as often as the first, whose row is the lowest
    if (CH == 1) {
        const int c = part.column(0);
        BackwardPiece now, next, after;
        now.load(a, t, c);
        next.load(a, t + step, c);
        weights(0);
        for (int turn = 0; t - part.group < a.T; t += step, turn ^= 1) {
            after.load(a, t + 2 * step, c);
            const float mean = part.sum(now.dot(w, acc[0]), part_s[turn]) / (float)a.K;
            now.store(a, w, mean, t, c);
            now = next;
            next = after;
        }
    } else {
        // no registers for a row of more than 8192 columns beside its sums: read again from the cache
        for (int turn = 0; t - part.group < a.T; t += step, turn ^= 1) {
            BackwardPiece piece;
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                piece.load(a, t, part.column(i));
                weights(i);
                dot += piece.dot(w, acc[i]);
            }
            const float mean = part.sum(dot, part_s[turn]) / (float)a.K;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                piece.load(a, t, part.column(i));
                weights(i);
                piece.store(a, w, mean, t, part.column(i));
            }
        }
    }
    if (!a.d_weight) return;
    if (CH == 1 && groups > 1) {
        const int row = waves * 512;                         // columns that a group holds, the row's and up to 511 more
#pragma unroll
        for (int j = 0; j < 8; ++j) acc_s[part.group * row + part.thread * 8 + j] = acc[0][j];
        __syncthreads();
        if (part.group != 0) return;
        for (int g = 1; g < groups; ++g)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[0][j] += acc_s[g * row + part.thread * 8 + j];
    }
    if (part.group != 0) return;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = part.column(i);
        float* p = a.parts + (int64_t)blockIdx.x * a.K + c;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < a.K) p[j] = acc[i][j];
    }
}

// d_weight: 64 columns a workgroup, its 16 waves on every 16th partial row.
__global__ __launch_bounds__(1024) void norm_parts_kernel(NormArgs a, int parts) {
    __shared__ float sum_s[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = (int)blockIdx.x * 64 + lane;
    constexpr int kEach = kNormMaxParts / 16;                // all of a wave's rows are loaded together
    float v[kEach], s = 0.f;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int p = wave + 16 * i;
        v[i] = c < a.K && p < parts ? a.parts[(int64_t)p * a.K + c] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) s += v[i];
    sum_s[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < a.K) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) s += sum_s[i][lane];
        a.d_weight[c] = s;
    }
}

// ----------------------------------------------------------------- launches

// Waves that take a row, at 8 CH columns a thread.
static int row_waves(int K, int ch) { return (K + 512 * ch - 1) / (512 * ch); }

// Columns of a thread: 8, or 16 where many rows are wide (us at 7168 columns and 8 or 16: 256 rows 4.7 and 5.2, 1024
// rows 13.4 and 11.9; at 4096 columns 7.5 and 8.0, 4096 rows 24.3 and 24.6) or not aligned (8191 rows of 2047: 16.5
// and 14.9), and past what 16 waves hold.
static int row_chunks(int T, int K) {
    if (K > 8192) return K <= 16384 ? 2 : 4;
    return T > 512 && (K > 4096 || (K % 8 != 0 && K > 1024)) ? 2 : 1;
}

template <OperandFormat FMT>
static void rms_norm_as(const NormArgs& a, hipStream_t s) {
    const int ch = row_chunks(a.T, a.K), waves = row_waves(a.K, ch);
    const int rows = waves >= 4 ? 1 : 4 / waves;             // of a workgroup
    const dim3 grid((a.T + rows - 1) / rows), threads(64 * waves * rows);
    if (ch == 1) rms_norm_kernel<FMT, 1><<<grid, threads, 0, s>>>(a, waves);
    else if (ch == 2) rms_norm_kernel<FMT, 2><<<grid, threads, 0, s>>>(a, waves);
    else rms_norm_kernel<FMT, 4><<<grid, threads, 0, s>>>(a, waves);
}

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s) {
    if (a.T == 0) return hipSuccess;
    switch (a.fmt) {
        case kBf16: rms_norm_as<kBf16>(a, s); break;
        case kRows: rms_norm_as<kRows>(a, s); break;
        case kKm: rms_norm_as<kKm>(a, s); break;
        case kE8m0: rms_norm_as<kE8m0>(a, s); break;
    }
    return hipGetLastError();
}

hipError_t launch_rms_norm_backward(const NormArgs& a, hipStream_t s) {
    const int ch = a.K <= 8192 ? 1 : (a.K <= 16384 ? 2 : 4), waves = row_waves(a.K, ch), groups = 16 / waves;
    const int parts = norm_parts((a.T + groups - 1) / groups);
    if (a.T > 0) {
        const dim3 threads(64 * waves * groups);
        if (ch == 1) rms_norm_backward_kernel<1><<<parts, threads, 0, s>>>(a, waves);
        else if (ch == 2) rms_norm_backward_kernel<2><<<parts, threads, 0, s>>>(a, waves);
        else rms_norm_backward_kernel<4><<<parts, threads, 0, s>>>(a, waves);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.d_weight) norm_parts_kernel<<<(a.K + 63) / 64, 1024, 0, s>>>(a, parts);
    return hipGetLastError();
}

}  // namespace moegg
