// norm.hip -- root-mean-square norm with the residual's addition and an e4m3
// operand as output, and its backward pass.
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

// Sum over the workgroup in a fixed order, in every thread.
__device__ __forceinline__ float block_sum(float v, float* part_s) {
    v = wave_sum(v);
    const int waves = (int)blockDim.x / 64;
    if (waves == 1) return v;
    if ((threadIdx.x & 63) == 0) part_s[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.f;
    for (int w = 0; w < waves; ++w) s += part_s[w];
    __syncthreads();
    return s;
}

// 1 / sqrt(x): the hardware's (1 ulp) and one Newton step.
__device__ __forceinline__ float rsqrt_f32(float x) {
    const float r = __builtin_amdgcn_rsqf(x);
    if (!(r > 0.f) || !(r < __builtin_inff())) return r;
    return __builtin_fmaf(0.5f * r, __builtin_fmaf(-x * r, r, 1.f), r);
}

// ----------------------------------------------------------------- forward

// A workgroup takes a row and holds it in registers, 8 CH columns a thread, so
// that it is read once: h = bf16(x + r), the sum of h^2 in fp32, then h rstd w.
template <OperandFormat FMT, int CH>
__global__ __launch_bounds__(1024) void rms_norm_kernel(NormArgs a) {
    __shared__ float part_s[16];
    const int64_t t = blockIdx.x, at = t * a.K;
    u32x4 h[CH], r[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = (i * (int)blockDim.x + (int)threadIdx.x) * 8, n = a.K - c;
        h[i] = r[i] = u32x4{0, 0, 0, 0};
        if (n > 0) h[i] = load8<false>((const uint16_t*)a.x + at + c, n);
        if (n > 0 && a.residual) r[i] = load8<false>((const uint16_t*)a.residual + at + c, n);
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = (i * (int)blockDim.x + (int)threadIdx.x) * 8, n = a.K - c;
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
    sum = block_sum(sum, part_s);
    float rstd;
    if (sum < __builtin_inff()) {
        rstd = rsqrt_f32(sum / (float)a.K + a.eps);
    } else {                             // squares past fp32's range, or an infinity or NaN in the row
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
        rstd = rsqrt_f32(block_sum(s, part_s) / (float)a.K) * 0x1p-80f;
    }
    if (a.rstd && threadIdx.x == 0) a.rstd[t] = rstd;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = (i * (int)blockDim.x + (int)threadIdx.x) * 8, n = a.K - c;
        float f[8], w[8];
        unpack8(h[i], f);
        load_weight8(a.weight, a.weight_bf16, c, n, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = f[j] * rstd * w[j];
        if (n > 0 && a.y) store8((uint16_t*)a.y + at + c, pack8(f), n);
        if (FMT != kBf16) {
            const GroupScale g = group_scale<FMT == kE8m0>(max16(amax8(f, 0.f)));
            uint32_t codes[2];
            quantize<8>(f, g, codes);
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
// dw = sum over rows of dy xhat.  A workgroup takes every parts-th row and sums
// its share of dw in registers, one partial row a workgroup; a second launch
// adds those in order.
template <int CH>
__global__ __launch_bounds__(1024) void rms_norm_backward_kernel(NormArgs a) {
    __shared__ float part_s[16];
    float w[CH][8], acc[CH][8];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = (i * (int)blockDim.x + (int)threadIdx.x) * 8;
        load_weight8(a.weight, a.weight_bf16, c, a.K - c, w[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
    }
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const int64_t at = t * a.K;
        const float rstd = a.rstd[t];
        u32x4 h[CH], d[CH], r[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = (i * (int)blockDim.x + (int)threadIdx.x) * 8, n = a.K - c;
            h[i] = d[i] = r[i] = u32x4{0, 0, 0, 0};
            if (n > 0) {
                h[i] = load8<false>((const uint16_t*)a.x + at + c, n);
                d[i] = load8<false>((const uint16_t*)a.dy + at + c, n);
                if (a.residual) r[i] = load8<false>((const uint16_t*)a.residual + at + c, n);
            }
        }
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            float f[8], g[8];
            unpack8(h[i], f);
            unpack8(d[i], g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float xhat = f[j] * rstd;
                dot = __builtin_fmaf(g[j] * w[i][j], xhat, dot);
                acc[i][j] = __builtin_fmaf(g[j], xhat, acc[i][j]);
            }
        }
        const float mean = block_sum(dot, part_s) / (float)a.K;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = (i * (int)blockDim.x + (int)threadIdx.x) * 8, n = a.K - c;
            float f[8], g[8], s[8];
            unpack8(h[i], f);
            unpack8(d[i], g);
            unpack8(r[i], s);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s[j] = __builtin_fmaf(rstd, __builtin_fmaf(-f[j] * rstd, mean, g[j] * w[i][j]), s[j]);
            if (n > 0) store8((uint16_t*)a.y + at + c, pack8(s), n);
        }
    }
    if (!a.d_weight) return;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = (i * (int)blockDim.x + (int)threadIdx.x) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < a.K) a.parts[(int64_t)blockIdx.x * a.K + c + j] = acc[i][j];
    }
}

// d_weight: 64 columns a workgroup, its 16 waves on every 16th partial row.
__global__ __launch_bounds__(1024) void norm_parts_kernel(NormArgs a, int parts) {
    __shared__ float sum_s[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = (int)blockIdx.x * 64 + lane;
    float v = 0.f;
    if (c < a.K)
        for (int p = wave; p < parts; p += 16) v += a.parts[(int64_t)p * a.K + c];
    sum_s[wave][lane] = v;
    __syncthreads();
    if (wave == 0 && c < a.K) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) s += sum_s[i][lane];
        a.d_weight[c] = s;
    }
}

// ----------------------------------------------------------------- launches

static int norm_threads(int K, int ch) { return 64 * ((K + 512 * ch - 1) / (512 * ch)); }

template <OperandFormat FMT>
static void rms_norm_as(const NormArgs& a, hipStream_t s) {
    if (a.K <= 8192) rms_norm_kernel<FMT, 1><<<a.T, norm_threads(a.K, 1), 0, s>>>(a);
    else if (a.K <= 16384) rms_norm_kernel<FMT, 2><<<a.T, norm_threads(a.K, 2), 0, s>>>(a);
    else rms_norm_kernel<FMT, 4><<<a.T, norm_threads(a.K, 4), 0, s>>>(a);
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
    const int parts = norm_parts(a.T);
    if (a.T > 0) {
        if (a.K <= 8192) rms_norm_backward_kernel<1><<<parts, norm_threads(a.K, 1), 0, s>>>(a);
        else if (a.K <= 16384) rms_norm_backward_kernel<2><<<parts, norm_threads(a.K, 2), 0, s>>>(a);
        else rms_norm_backward_kernel<4><<<parts, norm_threads(a.K, 4), 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.d_weight) norm_parts_kernel<<<(a.K + 63) / 64, 1024, 0, s>>>(a, parts);
    return hipGetLastError();
}

}  // namespace moegg
