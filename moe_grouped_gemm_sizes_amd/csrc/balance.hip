// balance.hip -- the router's balance loss and z loss of every sequence, the
// counts of its experts, and their gradient.
//
// For a sequence of n tokens with k assignments each, p a token's softmax (or
// its sigmoids over their sum), c_e the assignments of expert e and P_e the mean
// of p_e over the tokens:
//     loss = E / (k n) sum_e c_e P_e,    z = mean of (ln sum_e e^logit)^2.
#include <hip/hip_runtime.h>

#include "block.hpp"
#include "layer.hpp"
#include "logits.hpp"

namespace moegg {

// ----------------------------------------------------------------- one token

// A group of LPT lanes takes a token, VPL neighbouring experts a lane.
template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
    v += __uint_as_float(lane_of<DPP_XOR1>(__float_as_uint(v)));
    v += __uint_as_float(lane_of<DPP_XOR2>(__float_as_uint(v)));
    if (LPT >= 8) v += __uint_as_float(lane_of<DPP_HALF_MIRROR>(__float_as_uint(v)));
    if (LPT >= 16) v += __uint_as_float(lane_of<DPP_MIRROR>(__float_as_uint(v)));
    if (LPT >= 32) v += __shfl_xor(v, 16, 64);
    if (LPT >= 64) v += __shfl_xor(v, 32, 64);
    return v;
}
template <int LPT>
__device__ __forceinline__ float group_max(float v) {
    v = fmaxf(v, __uint_as_float(lane_of<DPP_XOR1>(__float_as_uint(v))));
    v = fmaxf(v, __uint_as_float(lane_of<DPP_XOR2>(__float_as_uint(v))));
    if (LPT >= 8) v = fmaxf(v, __uint_as_float(lane_of<DPP_HALF_MIRROR>(__float_as_uint(v))));
    if (LPT >= 16) v = fmaxf(v, __uint_as_float(lane_of<DPP_MIRROR>(__float_as_uint(v))));
    if (LPT >= 32) v = fmaxf(v, __shfl_xor(v, 16, 64));
    if (LPT >= 64) v = fmaxf(v, __shfl_xor(v, 32, 64));
    return v;
}

// p of the lane's experts from their logits (-inf: none, p 0); returns the
// logits' log-sum-exp, 0 for a token without experts (sigmoid: not computed).
template <int VPL, int LPT>
__device__ __forceinline__ float probabilities(const float (&l)[VPL], bool sigmoid, float (&p)[VPL]) {
    constexpr float ninf = -__builtin_inff();
    float m = l[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = fmaxf(m, l[i]);
    m = group_max<LPT>(m);
    // what is taken out of every exponential: the largest one's, and of sigmoids no more than 1
    const float top = !(m > ninf) || (sigmoid && m > 0.f) ? 0.f : m;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        if (sigmoid) p[i] = l[i] > ninf ? expf(fminf(l[i], 0.f) - top) / (1.f + expf(-fabsf(l[i]))) : 0.f;
        else p[i] = expf(l[i] - top);
        sum += p[i];
    }
    sum = group_sum<LPT>(sum);
    const float r = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) p[i] *= r;
    return sigmoid || !(sum > 0.f) ? 0.f : top + logf(sum);
}

// The sequence that holds token t: the last one that starts at or before it (0 if none does).
__device__ __forceinline__ int sequence_of(const int32_t* offsets, int S, int t) {
    int lo = 0, hi = S;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (offsets[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}
// Bounds of sequence s, within [0, T] whatever the offsets are.
__device__ __forceinline__ void bounds_of(const int32_t* offsets, int s, int T, int& start, int& end) {
    start = 0;
    end = T;
    if (offsets) {
        start = min(max(offsets[s], 0), T);
        end = min(max(offsets[s + 1], start), T);
    }
}

// ----------------------------------------------------------------- forward

// Sums over tokens [t0, t1) of one sequence, left in LDS.
template <int WAVES, int VPL, int LPT>
struct Piece {
    static constexpr int kExperts = VPL * LPT, kTokens = 64 / LPT;
    float p[WAVES][kExperts];
    int n[kExperts];
    float z[WAVES];

    __device__ __forceinline__ void add(const BalanceArgs& a, int t0, int t1) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane % LPT;
        for (int e = threadIdx.x; e < kExperts; e += WAVES * 64) n[e] = 0;
        __syncthreads();
        for (int64_t i = (int64_t)t0 * a.k + threadIdx.x; i < (int64_t)t1 * a.k; i += WAVES * 64) {
            const int id = a.ids[i];
            if (id >= 0 && id < a.E) atomicAdd(&n[id], 1);       // whole numbers: any order
        }
        float acc[VPL], zs = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) acc[i] = 0.f;
        for (int tw = t0 + wave * kTokens; tw < t1; tw += WAVES * kTokens) {
            const int t = tw + lane / LPT;
            const bool there = t < t1;
            float l[VPL], v[VPL];
            load_logits<VPL>(a.logits, min(t, t1 - 1), a.E, a.bf16, sub, l);
            const float lse = probabilities<VPL, LPT>(l, a.sigmoid, v);
#pragma unroll
            for (int i = 0; i < VPL; ++i) acc[i] += there ? v[i] : 0.f;
            zs += there ? lse * lse : 0.f;
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
#pragma unroll
            for (int off = LPT; off < 64; off <<= 1) acc[i] += __shfl_xor(acc[i], off, 64);
            if (lane < LPT) p[wave][sub * VPL + i] = acc[i];
        }
#pragma unroll
        for (int off = LPT; off < 64; off <<= 1) zs += __shfl_xor(zs, off, 64);
        if (lane == 0) z[wave] = zs;
        __syncthreads();
    }
    __device__ __forceinline__ float sum_p(int e) const {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) s += p[w][e];
        return s;
    }
    __device__ __forceinline__ float sum_z() const {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) s += z[w];
        return s;
    }
};

// Sum of 64-bit terms over the workgroup in a fixed order, in thread 0.
__device__ __forceinline__ double block_sum_f64(double v, double* part_s) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    if ((threadIdx.x & 63) == 0) part_s[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0.;
    if (threadIdx.x == 0)
        for (int w = 0; w < (int)blockDim.x / 64; ++w) s += part_s[w];
    return s;
}

// A sequence's outputs from the sums of expert threadIdx.x (threads past E: of none).
__device__ __forceinline__ void finish(const BalanceArgs& a, int s, int n, double p, int count, double z, double* part_s) {
    const int e = threadIdx.x;
    const double mean = n > 0 ? p / n : 0.;
    if (e < a.E) {
        a.counts[(int64_t)s * a.E + e] = count;
        if (a.probs) a.probs[(int64_t)s * a.E + e] = (float)mean;
    }
    const double loss = block_sum_f64(e < a.E ? count * mean : 0., part_s);
    if (threadIdx.x == 0) {
        a.loss[s] = n > 0 ? (float)(loss * a.E / ((double)a.k * n)) : 0.f;
        if (a.z_loss) a.z_loss[s] = n > 0 ? (float)(z / n) : 0.f;
    }
}

// Sums of a tile of tokens, one row of them for each sequence that it meets.
// Tiles and sequences both go up along the tokens, so tile + sequence tells these
// rows apart.
template <int VPL, int LPT>
__global__ __launch_bounds__(256) void balance_tile_kernel(BalanceArgs a) {
    __shared__ Piece<4, VPL, LPT> piece;
    const int t0 = (int)blockIdx.x * a.tile_tokens, t1 = min(t0 + a.tile_tokens, a.T);
    for (int s = a.offsets ? sequence_of(a.offsets, a.S, t0) : 0; s < a.S; ++s) {
        int start, end;
        bounds_of(a.offsets, s, a.T, start, end);
        if (start >= t1) break;
        start = max(start, t0);
        end = min(end, t1);
        if (start >= end) continue;
        piece.add(a, start, end);
        const int64_t row = (int64_t)blockIdx.x + s;
        for (int e = threadIdx.x; e < a.E; e += 256) {
            a.part_p[row * a.E + e] = piece.sum_p(e);
            a.part_n[row * a.E + e] = piece.n[e];
        }
        if (threadIdx.x == 0) a.part_z[row] = piece.sum_z();
        __syncthreads();
    }
}

// A workgroup adds a sequence's rows in order: experts along the threads, and
// every (1024 / experts)-th row a group of threads.
__global__ __launch_bounds__(1024) void balance_finish_kernel(BalanceArgs a) {
    __shared__ double p_s[1024], part_s[16];
    __shared__ int n_s[1024];
    const int s = blockIdx.x;
    int start, end;
    bounds_of(a.offsets, s, a.T, start, end);
    int width = 64;
    while (width < a.E) width <<= 1;
    const int e = threadIdx.x & (width - 1), part = threadIdx.x / width, parts = 1024 / width;
    double p = 0., z = 0.;
    int n = 0;
    if (start < end) {
        const int first = start / a.tile_tokens, last = (end - 1) / a.tile_tokens;
        if (e < a.E)
            for (int c = first + part; c <= last; c += parts) {
                p += a.part_p[((int64_t)c + s) * a.E + e];
                n += a.part_n[((int64_t)c + s) * a.E + e];
            }
        if (a.z_loss)
            for (int c = first + (int)threadIdx.x; c <= last; c += 1024) z += a.part_z[(int64_t)c + s];
    }
    p_s[threadIdx.x] = p;
    n_s[threadIdx.x] = n;
    z = block_sum_f64(z, part_s);
    __syncthreads();
    if (part == 0)
        for (int i = 1; i < parts; ++i) {
            p += p_s[i * width + e];
            n += n_s[i * width + e];
        }
    finish(a, s, end - start, p, n, z, part_s);          // E <= width: threads of part 0 hold all experts
}

// ----------------------------------------------------------------- backward

// g_e = d_loss E c_e / (k n^2); softmax: p (g - <p, g>) + d_z 2 lse / n p;
// sigmoids: p (1 - sigmoid) (g - <p, g>).
template <int VPL, int LPT>
__global__ __launch_bounds__(256) void balance_backward_kernel(BalanceBackwardArgs a) {
    constexpr int kTokens = 64 / LPT;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane % LPT;
    const int64_t t = ((int64_t)blockIdx.x * 4 + wave) * kTokens + lane / LPT;
    const int64_t row = t < a.T ? t : a.T - 1;
    float l[VPL], p[VPL], o[VPL];
    load_logits<VPL>(a.logits, row, a.E, a.bf16, sub, l);
    const int s = a.offsets ? sequence_of(a.offsets, a.S, (int)row) : 0;
    int start, end;
    bounds_of(a.offsets, s, a.T, start, end);
    const bool in = row >= start && row < end;
    const float n = (float)max(end - start, 1);
    const float c = in ? a.d_loss[s] * ((float)a.E / (float)a.k) / n / n : 0.f;
    const float dz = in && a.d_z ? 2.f * a.d_z[s] / n : 0.f;
    const float lse = probabilities<VPL, LPT>(l, a.sigmoid, p);
    float d = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = sub * VPL + i;
        o[i] = e < a.E ? c * (float)a.counts[(int64_t)s * a.E + e] : 0.f;
        d = __builtin_fmaf(p[i], o[i], d);
    }
    d = group_sum<LPT>(d);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        o[i] = p[i] * (o[i] - d);
        // 1 - sigmoid(x) = sigmoid(-x), without the subtraction
        if (a.sigmoid) o[i] = p[i] > 0.f ? o[i] / (1.f + expf(l[i])) : 0.f;
        else o[i] = __builtin_fmaf(p[i], dz * lse, o[i]);
    }
    if (t >= a.T) return;
    if (a.bf16) {
        __bf16 r[VPL];
        if (a.before) {
            uint16_t b[VPL];
            load_row<uint16_t, VPL>((const uint16_t*)a.before + t * a.E, a.E, sub, b);
#pragma unroll
            for (int i = 0; i < VPL; ++i) o[i] += __uint_as_float((uint32_t)b[i] << 16);
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) r[i] = (__bf16)o[i];
        store_row<__bf16, VPL>((__bf16*)a.d_logits + t * a.E, a.E, sub, r);
    } else {
        if (a.before) {
            float b[VPL];
            load_row<float, VPL>((const float*)a.before + t * a.E, a.E, sub, b);
#pragma unroll
            for (int i = 0; i < VPL; ++i) o[i] += b[i];
        }
        store_row<float, VPL>((float*)a.d_logits + t * a.E, a.E, sub, o);
    }
}

// ----------------------------------------------------------------- launches

template <int VPL, int LPT>
static hipError_t balance_as(const BalanceArgs& a, hipStream_t s) {
    if (a.T > 0) {
        balance_tile_kernel<VPL, LPT><<<(a.T + a.tile_tokens - 1) / a.tile_tokens, 256, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    balance_finish_kernel<<<a.S, 1024, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_balance_loss(const BalanceArgs& a, hipStream_t s) {
    if (a.E <= 64) return balance_as<4, 16>(a, s);
    if (a.E <= 128) return balance_as<4, 32>(a, s);
    if (a.E <= 256) return balance_as<4, 64>(a, s);
    if (a.E <= 512) return balance_as<8, 64>(a, s);
    return balance_as<16, 64>(a, s);
}

template <int VPL, int LPT>
static hipError_t balance_backward_as(const BalanceBackwardArgs& a, hipStream_t s) {
    constexpr int tokens = 4 * (64 / LPT);
    balance_backward_kernel<VPL, LPT><<<(a.T + tokens - 1) / tokens, 256, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_balance_loss_backward(const BalanceBackwardArgs& a, hipStream_t s) {
    if (a.T == 0) return hipSuccess;
    if (a.E <= 64) return balance_backward_as<4, 16>(a, s);
    if (a.E <= 128) return balance_backward_as<4, 32>(a, s);
    if (a.E <= 256) return balance_backward_as<4, 64>(a, s);
    if (a.E <= 512) return balance_backward_as<8, 64>(a, s);
    return balance_backward_as<16, 64>(a, s);
}

}  // namespace moegg
