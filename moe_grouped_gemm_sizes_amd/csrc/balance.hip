// balance.hip -- the router's balance loss and z loss of every sequence, the
// counts of its experts, and their gradient.
//
// For a sequence of n tokens with k assignments each, p a token's softmax (or
// its sigmoids over their sum), c_e the assignments of expert e and P_e the mean
// of p_e over the tokens:
//     loss = E / (k n) sum_e c_e P_e,    z = mean of (ln sum_e e^logit)^2.
//
// Logits are few bytes (8191 tokens over 256 experts: 8 MB, 1.6 us): launches and chains
// of dependent loads bound these calls, so loads are sent as early as they can be.
#include <hip/hip_runtime.h>

#include "block.hpp"
#include "layer.hpp"
#include "logits.hpp"

namespace moegg {

// ----------------------------------------------------------------- one token

// A group of LPT lanes takes a token, VPL neighbouring experts a lane.  Steps of 16
// and 32 lanes swap rows of lanes in registers.
template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
    v += __uint_as_float(lane_of<DPP_XOR1>(__float_as_uint(v)));
    v += __uint_as_float(lane_of<DPP_XOR2>(__float_as_uint(v)));
    v += __uint_as_float(lane_of<DPP_HALF_MIRROR>(__float_as_uint(v)));
    v += __uint_as_float(lane_of<DPP_MIRROR>(__float_as_uint(v)));
    if (LPT >= 32) {
        const auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(x[0]) + __uint_as_float(x[1]);
    }
    if (LPT >= 64) {
        const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(x[0]) + __uint_as_float(x[1]);
    }
    return v;
}
template <int LPT>
__device__ __forceinline__ float group_max(float v) {
    v = fmaxf(v, __uint_as_float(lane_of<DPP_XOR1>(__float_as_uint(v))));
    v = fmaxf(v, __uint_as_float(lane_of<DPP_XOR2>(__float_as_uint(v))));
    v = fmaxf(v, __uint_as_float(lane_of<DPP_HALF_MIRROR>(__float_as_uint(v))));
    v = fmaxf(v, __uint_as_float(lane_of<DPP_MIRROR>(__float_as_uint(v))));
    if (LPT >= 32) {
        const auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
    }
    if (LPT >= 64) {
        const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
    }
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

// The sequence that holds token t, the same for the whole wave: the last one that starts at or
// before it (0 if none does).  64 offsets a step, one load up to 64 sequences.
__device__ __forceinline__ int sequence_of(const int32_t* offsets, int S, int t) {
    int lo = 0, n = S;
    while (n > 1) {
        const int step = (n + 63) / 64, i = ((int)threadIdx.x & 63) * step;
        const uint64_t before = __ballot(i < n && offsets[lo + min(i, n - 1)] <= t);
        const int last = max((int)__popcll(before) - 1, 0) * step;
        lo += last;
        n = min(step, n - last);
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

// Sum of 64-bit terms over the workgroup in a fixed order, in thread 0.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xF, false);
    return v + __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
__device__ __forceinline__ double block_sum_f64(double v, double* part_s) {
    v = dpp_add<DPP_SHR + 1, 0xF>(v);
    v = dpp_add<DPP_SHR + 2, 0xF>(v);
    v = dpp_add<DPP_SHR + 4, 0xF>(v);
    v = dpp_add<DPP_SHR + 8, 0xF>(v);
    v = dpp_add<DPP_BCAST15, 0xA>(v);
    v = dpp_add<DPP_BCAST31, 0xC>(v);
    if ((threadIdx.x & 63) == 63) part_s[threadIdx.x >> 6] = v;
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

// Bounds of sequences from one on, a lane each.
struct Bounds {
    int base, at;                        // first sequence held; this lane's offset

    __device__ __forceinline__ void hold(const BalanceArgs& a, int s) {
        base = s;
        at = min(max(a.offsets[min(s + ((int)threadIdx.x & 63), a.S)], 0), a.T);
    }
    __device__ __forceinline__ void of(const BalanceArgs& a, int s, int& start, int& end) {
        if (!a.offsets) {
            start = 0;
            end = a.T;
            return;
        }
        if (s - base > 62) hold(a, s);
        start = __builtin_amdgcn_readlane(at, s - base);
        end = max(__builtin_amdgcn_readlane(at, s - base + 1), start);
    }
};

// Sums of a tile of tokens, one row of them for each sequence that it meets.
// Tiles and sequences both go up along the tokens, so tile + sequence tells these
// rows apart.  32 tokens at a time, whose logits and assignments are on their way
// while their sequences are looked up; a sequence's sums are in registers until it
// ends.  8191 tokens over 256 experts in 16 sequences: 7 us, of which a launch is 1.75 and
// three loads one after the other most of the rest (11 us with the sequences looked up first, in 4
// waves of 8 tokens); over 1024 experts 16 us.  Sequences of a tile come one after the other, 0.6 us
// each with their two barriers: 32 tokens in one 4.4 us, in 16 of them 13 us; 4096 tokens over 64
// experts in one 4.1 us, in 1000 of them 15 to 18 us.
constexpr int kTileStep = 32;
template <int VPL, int LPT>
constexpr int kTileWaves = VPL == 16 || LPT == 16 ? 8 : 16;  // LDS for 1024 experts; 4 tokens a wave up to 64

template <int VPL, int LPT>
__global__ __launch_bounds__((kTileWaves<VPL, LPT> * 64)) void balance_tile_kernel(BalanceArgs a) {
    constexpr int kWaves = kTileWaves<VPL, LPT>, kThreads = kWaves * 64, kExperts = VPL * LPT, kTokens = 64 / LPT;
    constexpr int kTurns = kTileStep / (kWaves * kTokens), kIds = kTileStep * kRouteMaxTopK / kThreads;
    __shared__ float p_s[kWaves][kExperts], z_s[kWaves];
    __shared__ int n_s[kExperts];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane % LPT, token = wave * kTokens + lane / LPT;
    const int t0 = (int)blockIdx.x * a.tile_tokens, t1 = min(t0 + a.tile_tokens, a.T);
    float acc[VPL], zs = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) acc[i] = 0.f;
    Bounds bounds{};
    int s = 0, start = 0, end = 0;
    for (int t = t0; t < t1; t += kTileStep) {
        const int last = min(t + kTileStep, t1);
        float p[kTurns][VPL], z[kTurns];
        int id[kIds], of[kIds];                              // an assignment and its token
#pragma unroll
        for (int r = 0; r < kTurns; ++r)
            load_logits<VPL>(a.logits, min(t + token + r * kWaves * kTokens, last - 1), a.E, a.bf16, sub, p[r]);
#pragma unroll
        for (int i = 0; i < kIds; ++i) {
            const int j = i * kThreads + (int)threadIdx.x;
            id[i] = j < (last - t) * a.k ? a.ids[(int64_t)t * a.k + j] : -1;
            if (id[i] >= a.E) id[i] = -1;
            of[i] = t + j / a.k;
        }
        if (t == t0) {
            if (a.offsets) {
                s = sequence_of(a.offsets, a.S, t0);
                bounds.hold(a, s);
            }
            bounds.of(a, s, start, end);
            for (int e = threadIdx.x; e < kExperts; e += kThreads) n_s[e] = 0;
            lds_barrier();
        }
#pragma unroll
        for (int r = 0; r < kTurns; ++r) {
            const float lse = probabilities<VPL, LPT>(p[r], a.sigmoid, p[r]);
            z[r] = lse * lse;
        }
        for (;;) {                                           // the sequences that these tokens are of
            const int from = max(start, t), to = min(end, last);
#pragma unroll
            for (int r = 0; r < kTurns; ++r) {
                const int at = t + token + r * kWaves * kTokens;
                const bool in = at >= from && at < to;
#pragma unroll
                for (int i = 0; i < VPL; ++i) acc[i] += in ? p[r][i] : 0.f;
                zs += in ? z[r] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < kIds; ++i)
                if (id[i] >= 0 && of[i] >= from && of[i] < to) atomicAdd(&n_s[id[i]], 1);   // whole numbers: any order
            if (end > last && last < t1) break;              // the sequence goes on in the tile's next step
            // the sequence's sums in this tile, if it has any tokens there
            if (max(start, t0) < min(end, t1)) {
#pragma unroll
                for (int i = 0; i < VPL; ++i) {
#pragma unroll
                    for (int off = LPT; off < 64; off <<= 1) acc[i] += __shfl_xor(acc[i], off, 64);
                    if (lane < LPT) p_s[wave][sub * VPL + i] = acc[i];
                    acc[i] = 0.f;
                }
#pragma unroll
                for (int off = LPT; off < 64; off <<= 1) zs += __shfl_xor(zs, off, 64);
                if (lane == 0) z_s[wave] = zs;
                zs = 0.f;
                lds_barrier();
                const int64_t row = (int64_t)blockIdx.x + s;
                for (int e = threadIdx.x; e < kExperts; e += kThreads) {
                    float sum = 0.f;
#pragma unroll
                    for (int w = 0; w < kWaves; ++w) sum += p_s[w][e];
                    if (e < a.E) {
                        a.part_p[row * a.E + e] = sum;
                        a.part_n[row * a.E + e] = n_s[e];
                    }
                    n_s[e] = 0;
                }
                if (threadIdx.x == 0) {
                    float sum = 0.f;
#pragma unroll
                    for (int w = 0; w < kWaves; ++w) sum += z_s[w];
                    a.part_z[row] = sum;
                }
                lds_barrier();
            }
            if (end > last) break;                           // or in the next tile
            if (s + 1 >= a.S) {
                start = end = a.T;                           // tokens past the last sequence
                break;
            }
            bounds.of(a, ++s, start, end);
            if (start >= last) break;
        }
    }
}

// A workgroup adds a sequence's rows in order: experts along the threads, and
// every (1024 / experts)-th row a group of threads, four rows on their way at a time.  A turn of
// these is a trip to what other XCDs wrote, and one sequence of 8191 tokens has 256 rows: 4.9 us over
// 64 experts (4 turns), 11 us over 256 (16), 21 over 512 and 38 over 1024 (64).  In 16
// sequences over 256 experts 4.2 to 5.7 us (8.4 us with the rows one by one and 64-bit sums through
// LDS).
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
            for (int c = first + part; c <= last; c += 4 * parts) {
                float v[4];
                int m[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {                    // four rows on their way together
                    const int64_t at = ((int64_t)min(c + i * parts, last) + s) * a.E + e;
                    v[i] = a.part_p[at];
                    m[i] = a.part_n[at];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    p += c + i * parts <= last ? v[i] : 0.f;
                    n += c + i * parts <= last ? m[i] : 0;
                }
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
// sigmoids: p (1 - sigmoid) (g - <p, g>).  A token a group of lanes and no loop: 8191 tokens over 160
// experts on top of what was there, in 1 or 5 sequences, 7 us, 1.75 of them a launch (in 1000: 8.7 us).
template <int VPL, int LPT>
__global__ __launch_bounds__(256) void balance_backward_kernel(BalanceBackwardArgs a) {
    constexpr int kTokens = 64 / LPT;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane % LPT;
    const int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * kTokens, t = t0 + lane / LPT;
    if (t0 >= a.T) return;
    const int64_t row = t < a.T ? t : a.T - 1;
    float l[VPL], p[VPL], o[VPL], before[VPL];
    load_logits<VPL>(a.logits, row, a.E, a.bf16, sub, l);
#pragma unroll
    for (int i = 0; i < VPL; ++i) before[i] = 0.f;
    if (a.before) {
        if (a.bf16) {
            uint16_t b[VPL];
            load_row<uint16_t, VPL>((const uint16_t*)a.before + row * a.E, a.E, sub, b);
#pragma unroll
            for (int i = 0; i < VPL; ++i) before[i] = __uint_as_float((uint32_t)b[i] << 16);
        } else {
            load_row<float, VPL>((const float*)a.before + row * a.E, a.E, sub, before);
        }
    }
    // the wave's first token's sequence, and from there on to this one's
    int s = a.offsets ? sequence_of(a.offsets, a.S, (int)t0) : 0, start, end;
    bounds_of(a.offsets, s, a.T, start, end);
    while (row >= end && s + 1 < a.S) bounds_of(a.offsets, ++s, a.T, start, end);
    const bool in = row >= start && row < end;
    const float n = (float)max(end - start, 1);
    const float c = in ? a.d_loss[s] * ((float)a.E / (float)a.k) / n / n : 0.f;
    const float dz = in && a.d_z ? a.d_z[s] / n : 0.f;
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
        else o[i] = __builtin_fmaf(2.f, p[i] * dz * lse, o[i]);   // p first: 0 beside an infinite logit's lse
    }
    if (t >= a.T) return;
#pragma unroll
    for (int i = 0; i < VPL; ++i) o[i] += before[i];
    if (a.bf16) {
        __bf16 r[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) r[i] = (__bf16)o[i];
        store_row<__bf16, VPL>((__bf16*)a.d_logits + t * a.E, a.E, sub, r);
    } else {
        store_row<float, VPL>((float*)a.d_logits + t * a.E, a.E, sub, o);
    }
}

// ----------------------------------------------------------------- launches

template <int VPL, int LPT>
static hipError_t balance_as(const BalanceArgs& a, hipStream_t s) {
    if (a.T > 0) {
        balance_tile_kernel<VPL, LPT><<<(a.T + a.tile_tokens - 1) / a.tile_tokens, kTileWaves<VPL, LPT> * 64, 0, s>>>(a);
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
