// route.hip -- router logits -> expert ids, weights, counts and the row of
// every assignment, and the gradient of the logits.
//
// One wave takes one token: lane l holds the logits of experts l, l + 64, ...
// in registers.  A key is a 32-bit logit (softmax and sigmoid are monotone, so
// without a bias the logits themselves order the experts), or score + bias in
// 64 bits, mapped to unsigned integers of the same order.  Each of the k picks
// is a wave-wide maximum by DPP and a ballot that finds its lowest holder.
//
// The row of assignment (t, j) is its expert's segment start plus the number
// of earlier tokens with the same expert.  No order of atomics enters: inside
// a 64-token step each expert has a 64-bit mask of its tokens (set by OR), and
// a rank is a popcount of the bits below; steps add up in LDS, token tiles
// through a [tiles, E] table of 16-bit counts.  Up to 64 tokens, one workgroup
// does everything in one launch; beyond, route_kernel leaves ranks inside the
// tile in row_of, and route_rows_kernel, whose every workgroup sums the table,
// adds the segment start and the earlier tiles.
//
// What bounds it: launches and the VALU.  One token over 256 experts takes 7 us,
// 4096 tokens over 64 experts 6 + 4 us.  8191 tokens over 256 experts in groups
// with a bias take 21 + 6 us: 7 us for launch and loads, then 970 instructions a
// token (140 for the 64-bit sigmoids, 280 for the picks).  Sixteen lanes a token
// need 510 in 32 bits, but then some token of a call this size always has two
// values too near to tell apart, and the 64-bit repeat costs more than is won.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "layer.hpp"

namespace moegg {

constexpr int kStep = 64;                 // tokens that share one round of masks
constexpr float kFltMax = 3.402823466e+38f;

// What routing reads as a logit: NaN is no expert, +inf the largest number.
// -0 becomes +0, so that equal logits have equal keys.
__device__ __forceinline__ float clean_logit(float l) {
    return l != l ? -__builtin_inff() : fminf(l, kFltMax) + 0.f;
}

__device__ __forceinline__ float load_logit(const void* p, int64_t i, int bf16) {
    return bf16 ? __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16) : ((const float*)p)[i];
}

// The lane's logits of token t, -inf past the experts.  All loads are issued
// before any is used: no branch between them (lanes past the end read the last one).
template <int VPL>
__device__ __forceinline__ void load_logits(const void* logits, int64_t t, int E, int bf16, int lane, float (&l)[VPL]) {
    if (bf16) {
        const uint16_t* p = (const uint16_t*)logits + t * E;
        uint16_t r[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) r[i] = p[min(lane + 64 * i, E - 1)];
#pragma unroll
        for (int i = 0; i < VPL; ++i) l[i] = __uint_as_float((uint32_t)r[i] << 16);
    } else {
        const float* p = (const float*)logits + t * E;
#pragma unroll
        for (int i = 0; i < VPL; ++i) l[i] = p[min(lane + 64 * i, E - 1)];
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] = lane + 64 * i < E ? clean_logit(l[i]) : -__builtin_inff();
}

// Unsigned integers in the order of the floats.
__device__ __forceinline__ uint32_t key32(float f) {
    const uint32_t b = __float_as_uint(f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint64_t key64(double d) {
    const uint64_t b = (uint64_t)__double_as_longlong(d);
    return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}

__device__ __forceinline__ float unkey32(uint32_t k) {
    return __uint_as_float(k ^ (~(uint32_t)((int32_t)k >> 31) | 0x80000000u));
}
template <typename T>
__device__ __forceinline__ void swap_if(bool c, T& a, T& b) {
    const T x = c ? b : a, y = c ? a : b;
    a = x;
    b = y;
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}

__device__ __forceinline__ float sigmoid_f32(float x) { return 1.f / (1.f + expf(-x)); }

// Scores in 64 bits: their users compare sums of them, and two of a token's
// may be nearer to each other than 32 bits tell apart.
template <int VPL>
__device__ __forceinline__ void scores64(const float (&l)[VPL], int sigmoid, double (&s)[VPL]) {
    if (sigmoid) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) s[i] = 1.0 / (1.0 + exp(-(double)l[i]));
        return;
    }
    float m = l[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = fmaxf(m, l[i]);
    m = wave_max(m);
    const double top = m > -__builtin_inff() ? (double)m : 0.0;
    double z = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        s[i] = exp((double)l[i] - top);
        z += s[i];
    }
    z = wave_sum_f64(z);
    const double r = z > 0 ? 1.0 / z : 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) s[i] *= r;
}

// Weights of the k chosen experts; lane j < k holds the j-th one's
// logit (-inf where there is none).  A softmax over all experts brings its
// maximum and sum of exponentials (top, z).
__device__ __forceinline__ float route_weight(float got, int sigmoid, int renorm, float scale, float top, float z) {
    const bool there = got > -__builtin_inff();
    if (!renorm) {
        if (!there) return 0.f;
        return scale * (sigmoid ? sigmoid_f32(got) : expf(got - top) / z);
    }
    const float m = wave_max(got);
    float t = 0.f;
    if (!sigmoid) {
        if (there) t = expf(got - m);
    } else if (there) {
        // the ratio of sigmoids with e^min(m, 0) taken out of both, so that far negative
        // logits keep their ratio: sigma(x) = e^x / (1 + e^x)
        const float low = fminf(m, 0.f);
        t = got > 0.f ? sigmoid_f32(got) : expf(got - low) / (1.f + expf(got));
    }
    const float sum = wave_sum(t);
    return sum > 0.f ? scale * t / sum : 0.f;
}

// One token: picks into lane j's `id` (-1: none) and weight.
// MODE 0: 32-bit keys, no 64-bit scores; 1: 32-bit keys, groups by 64-bit
// scores; 2: 64-bit keys (bias).  gbuf: E doubles of this wave (n_groups > 1).
template <int VPL, int MODE>
__device__ __forceinline__ void route_token(const RouteArgs& a, int t, int lane, double* gbuf, uint32_t gs_magic,
                                            int lanes_lg, int& id, float& weight) {
    const int E = a.E, k = a.k;
    constexpr float ninf = -__builtin_inff();
    float l[VPL], bias[VPL];
    if constexpr (MODE == 2) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) bias[i] = a.bias[min(lane + 64 * i, E - 1)];
    }
    load_logits<VPL>(a.logits, t, E, a.bf16, lane, l);
    double s[MODE ? VPL : 1];
    if constexpr (MODE != 0) scores64<VPL>(l, a.sigmoid, s);
    uint32_t hi[VPL], lo[MODE == 2 ? VPL : 1];       // keys, 0: not to be picked
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        if constexpr (MODE == 2) {
            const float b = clean_logit(bias[i]);        // NaN, -inf: not to be chosen
            const bool there = l[i] > ninf && b > ninf;
            s[i] = there ? s[i] + (double)b : -__builtin_inf();
            const uint64_t key = there ? key64(s[i]) : 0;
            hi[i] = (uint32_t)(key >> 32);
            lo[i] = (uint32_t)key;
        } else {
            hi[i] = l[i] > ninf ? key32(l[i]) : 0u;
            if constexpr (MODE == 1) s[i] = l[i] > ninf ? s[i] : -__builtin_inf();
        }
    }
    if (a.n_groups > 1) {
        // 2^lanes_lg lanes share a group; each keeps the two best of its part
        const int gs = E / a.n_groups, L = 1 << lanes_lg;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = lane + 64 * i;
            if (e < E) {
                if constexpr (MODE == 0) gbuf[e] = (double)l[i];
                else gbuf[e] = s[i];
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        const int g = lane >> lanes_lg, r = lane & (L - 1);
        double t1 = -__builtin_inf(), t2 = -__builtin_inf();
        if (g < a.n_groups)
            for (int i = r; i < gs; i += L) {
                const double v = gbuf[g * gs + i];
                t2 = fmax(t2, fmin(t1, v));
                t1 = fmax(t1, v);
            }
        __builtin_amdgcn_wave_barrier();
        for (int off = 1; off < L; off <<= 1) {
            const double o1 = __shfl_xor(t1, off, 64), o2 = __shfl_xor(t2, off, 64);
            t2 = fmax(fmax(t2, o2), fmin(t1, o1));
            t1 = fmax(t1, o1);
        }
        const double score = a.group_top == 2 ? t1 + t2 : t1;
        int rank = 0;
        for (int o = 0; o < a.n_groups; ++o) {
            const double v = __shfl(score, o << lanes_lg, 64);
            rank += v > score || (v == score && o < g);
        }
        const uint64_t keep = __ballot(rank < a.topk_groups);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = lane + 64 * i;
            const int eg = gs_magic ? (int)__umulhi((uint32_t)e, gs_magic) : e;
            if (e >= E || !((keep >> ((eg << lanes_lg) & 63)) & 1)) {
                hi[i] = 0;
                if constexpr (MODE == 2) lo[i] = 0;
            }
        }
    }
    id = -1;
    float got = ninf;
    if constexpr (VPL <= 4) {
        // The lane's keys in descending order (equal ones by id: only strictly smaller keys move back), so that a
        // pick looks at one key a lane and its holder moves up the others.
        typedef typename std::conditional<MODE == 2, uint64_t, uint32_t>::type Key;
        Key key[VPL];
        int e[VPL], left = 0;                            // left: experts that can be picked
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            e[i] = lane + 64 * i;
            if constexpr (MODE == 2) key[i] = (uint64_t)hi[i] << 32 | lo[i];
            else key[i] = hi[i];
            left += __popcll(__ballot(hi[i] != 0));
        }
#pragma unroll
        for (int n = VPL - 1; n > 0; --n) {
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const bool less = key[i] < key[i + 1];
                swap_if(less, key[i], key[i + 1]);
                swap_if(less, e[i], e[i + 1]);
            }
        }
        const int picks = min(k, left);
        for (int j = 0; j < picks; ++j) {
            const uint32_t top = (uint32_t)(key[0] >> (MODE == 2 ? 32 : 0));
            const uint32_t m = wave_max_u32(top);
            uint64_t who = __ballot(top == m);
            if constexpr (MODE == 2) {
                if (who & (who - 1)) {
                    const uint32_t low = wave_max_u32(top == m ? (uint32_t)key[0] : 0u);
                    who = __ballot(top == m && (uint32_t)key[0] == low);
                }
            }
            int src = __builtin_ctzll(who);
            if constexpr (VPL > 1) {
                if (who & (who - 1))                     // equal keys: the lowest id
                    src = (int)(~wave_max_u32((who >> lane) & 1 ? ~(uint32_t)e[0] : 0u) & 63u);
            }
            const int ej = VPL > 1 ? __builtin_amdgcn_readlane(e[0], src) : src;
            id = lane == j ? ej : id;
            if constexpr (MODE != 2) got = lane == j ? unkey32(m) : got;
            if (lane == src) {
#pragma unroll
                for (int i = 0; i + 1 < VPL; ++i) {
                    key[i] = key[i + 1];
                    e[i] = e[i + 1];
                }
                key[VPL - 1] = 0;
            }
        }
        if constexpr (MODE == 2) {
            if (id >= 0) got = clean_logit(load_logit(a.logits, (int64_t)t * E + id, a.bf16));
        }
    } else {
        for (int j = 0; j < k; ++j) {
            uint32_t m = hi[0];
#pragma unroll
            for (int i = 1; i < VPL; ++i) m = max(m, hi[i]);
            m = wave_max_u32(m);
            if (m == 0) break;                               // nothing left: the same for every lane
            uint32_t ml = 0;
            if constexpr (MODE == 2) {
#pragma unroll
                for (int i = 0; i < VPL; ++i) ml = max(ml, hi[i] == m ? lo[i] : 0u);
                ml = wave_max_u32(ml);
            }
            bool found = false;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                bool mine = hi[i] == m;
                if constexpr (MODE == 2) mine = mine && lo[i] == ml;
                const uint64_t who = __ballot(mine);
                if (!found && who) {
                    found = true;
                    const int src = __builtin_ctzll(who);
                    const float gv = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(l[i]), src));
                    if (lane == j) { id = src + 64 * i; got = gv; }
                    if (lane == src) hi[i] = 0;
                }
            }
        }
    }
    float top = 0.f, z = 1.f;
    if (!a.sigmoid && !a.renorm) {
        float m = l[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i) m = fmaxf(m, l[i]);
        m = wave_max(m);
        top = m > ninf ? m : 0.f;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) sum += expf(l[i] - top);
        z = wave_sum(sum);
    }
    weight = route_weight(got, a.sigmoid, a.renorm, a.scale, top, z);
}

// Exclusive scan of the experts' aligned counts by one wave: total[e] -> start[e].
// Sums stop at 2^31 - 1, which no row reaches.
constexpr uint32_t kNoRow = 0x7FFFFFFFu;
__device__ __forceinline__ uint32_t sum_rows(uint32_t a, uint32_t b) { return min(a + b, kNoRow); }
__device__ void segment_starts(const int32_t* total, uint32_t* start, int E, int seg_align, int cap, int lane) {
    uint32_t before = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
        const int e = e0 + lane;
        uint32_t m = e < E ? (uint32_t)total[e] : 0u;
        if (cap) m = e < E ? (uint32_t)cap : 0u;
        else if (seg_align > 1)
            m = (uint32_t)min((uint64_t)kNoRow,
                              (uint64_t)((m + (uint32_t)seg_align - 1) / (uint32_t)seg_align) * (uint32_t)seg_align);
        uint32_t end = m;
        end = sum_rows(end, dpp<DPP_SHR + 1>(0, end));
        end = sum_rows(end, dpp<DPP_SHR + 2>(0, end));
        end = sum_rows(end, dpp<DPP_SHR + 4>(0, end));
        end = sum_rows(end, dpp<DPP_SHR + 8>(0, end));
        end = sum_rows(end, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)end, DPP_BCAST15, 0xA, 0xF, false));
        end = sum_rows(end, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)end, DPP_BCAST31, 0xC, 0xF, false));
        const uint32_t above = (uint32_t)__shfl_up((int)end, 1, 64);
        if (e < E) start[e] = sum_rows(before, lane ? above : 0u);
        before = sum_rows(before, (uint32_t)__builtin_amdgcn_readlane((int)end, 63));
    }
}

__device__ __forceinline__ int32_t final_row(uint32_t start, uint32_t rank, int cap, int64_t rows_total) {
    if (cap && rank >= (uint32_t)cap) return -1;
    return start + rank < (uint32_t)rows_total ? (int32_t)(start + rank) : -1;   // both below 2^31
}

// Workgroup b routes tokens [b * tile_tokens, ...).  ONE: the only workgroup;
// it also writes m_sizes and final rows.
template <int VPL, int MODE, bool ONE>
__global__ __launch_bounds__(1024) void route_kernel(RouteArgs a, uint32_t gs_magic, int lanes_lg) {
    extern __shared__ double gbuf_all[];                 // groups only: E per wave
    __shared__ unsigned long long mask_s[kRouteMaxExperts];
    __shared__ int32_t count_s[kRouteMaxExperts];
    __shared__ int16_t ids_s[kStep * kRouteMaxTopK];
    __shared__ uint32_t start_s[ONE ? kRouteMaxExperts : 1];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int waves = blockDim.x >> 6, E = a.E, k = a.k;
    const int t0 = ONE ? 0 : blockIdx.x * a.tile_tokens, t1 = ONE ? a.T : min(a.T, t0 + a.tile_tokens);
    double* gbuf = gbuf_all + (a.n_groups > 1 ? wave * E : 0);
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        mask_s[e] = 0;
        count_s[e] = 0;
    }
    lds_barrier();
    for (int ts = t0; ts < t1; ts += kStep) {
        const int n = min(kStep, t1 - ts);
        for (int i = wave; i < n; i += waves) {
            int id;
            float w;
            route_token<VPL, MODE>(a, ts + i, lane, gbuf, gs_magic, lanes_lg, id, w);
            if (lane < k) {
                const int64_t at = (int64_t)(ts + i) * k + lane;
                a.ids[at] = id;
                a.weights[at] = w;
                ids_s[i * k + lane] = (int16_t)id;
                if (id >= 0) atomicOr(&mask_s[id], 1ull << i);
            }
        }
        lds_barrier();
        if constexpr (ONE) {                             // one step holds every token
            for (int e = threadIdx.x; e < E; e += blockDim.x) count_s[e] = __popcll(mask_s[e]);
            lds_barrier();
            break;
        }
        for (int x = threadIdx.x; x < n * k; x += blockDim.x) {
            const int id = ids_s[x], i = x / k;
            if (id >= 0)
                a.row_of[(int64_t)ts * k + x] = count_s[id] + __popcll(mask_s[id] & ((1ull << i) - 1));
        }
        lds_barrier();
        for (int e = threadIdx.x; e < E; e += blockDim.x) {
            count_s[e] += __popcll(mask_s[e]);
            mask_s[e] = 0;
        }
        lds_barrier();
    }
    if constexpr (ONE) {
        if (wave == 0) segment_starts(count_s, start_s, E, a.seg_align, a.cap, lane);
        for (int e = threadIdx.x; e < E; e += blockDim.x) a.m_sizes[e] = count_s[e];
        lds_barrier();
        for (int x = threadIdx.x; x < a.T * k; x += blockDim.x) {
            const int id = ids_s[x], i = x / k;
            a.row_of[x] = id < 0 ? -1
                                 : final_row(start_s[id], (uint32_t)__popcll(mask_s[id] & ((1ull << i) - 1)), a.cap,
                                             a.rows_total);
        }
    } else {
        uint32_t* out = (uint32_t*)(a.tile_counts + (int64_t)blockIdx.x * ((E + 1) & ~1));
        for (int e = threadIdx.x; e < (E + 1) / 2; e += blockDim.x)
            out[e] = (uint32_t)count_s[2 * e] | (2 * e + 1 < E ? (uint32_t)count_s[2 * e + 1] << 16 : 0u);
    }
}

constexpr int kRowsThreads = 1024;

// Ranks inside a tile -> rows: every workgroup sums the table of tile counts
// (64 KB at 128 tiles of 256 experts, from L2), scans the segments and
// finishes its own tile.
__global__ __launch_bounds__(kRowsThreads) void route_rows_kernel(RouteArgs a, int tiles) {
    __shared__ int32_t total_s[kRouteMaxExperts];
    __shared__ int32_t before_s[kRouteMaxExperts];
    __shared__ uint32_t start_s[kRouteMaxExperts];
    const int E = a.E, pairs = (E + 1) / 2, b = blockIdx.x, k = a.k;
    for (int e = threadIdx.x; e < 2 * pairs; e += kRowsThreads) {
        total_s[e] = 0;
        before_s[e] = 0;
    }
    __syncthreads();
    // `parts` threads share a pair of experts, each summing every parts-th tile
    const int parts = max(1, kRowsThreads / pairs);
    const int part = threadIdx.x / pairs, p = threadIdx.x % pairs;
    if (part < parts) {
        const uint32_t* in = (const uint32_t*)a.tile_counts + p;
        uint32_t tl = 0, th = 0, bl = 0, bh = 0;
#pragma unroll 8
        for (int i = part; i < tiles; i += parts) {
            const uint32_t v = in[(int64_t)i * pairs];
            tl += v & 0xFFFFu;
            th += v >> 16;
            bl += i < b ? v & 0xFFFFu : 0u;
            bh += i < b ? v >> 16 : 0u;
        }
        // sums of whole numbers: the atomics' order does not matter
        atomicAdd(&total_s[2 * p], (int)tl);
        atomicAdd(&total_s[2 * p + 1], (int)th);
        atomicAdd(&before_s[2 * p], (int)bl);
        atomicAdd(&before_s[2 * p + 1], (int)bh);
    }
    __syncthreads();
    if (threadIdx.x < 64) segment_starts(total_s, start_s, E, a.seg_align, a.cap, threadIdx.x);
    if (b == 0)
        for (int e = threadIdx.x; e < E; e += kRowsThreads) a.m_sizes[e] = total_s[e];
    __syncthreads();
    const int64_t x0 = (int64_t)b * a.tile_tokens * k, x1 = min((int64_t)a.T * k, x0 + (int64_t)a.tile_tokens * k);
    for (int64_t x = x0 + threadIdx.x; x < x1; x += kRowsThreads) {
        const int id = a.ids[x];
        a.row_of[x] = id < 0 ? -1 : final_row(start_s[id], (uint32_t)before_s[id] + (uint32_t)a.row_of[x], a.cap, a.rows_total);
    }
}

// Gradient of the logits, one wave a token.  With p the scores, w the weights
// and dw their gradients (over the chosen experts c):
//   softmax            scale * p_e * (dw_e [e chosen] - sum_c dw_c p_c)
//   softmax, renorm    w_c * (dw_c - sum dw w / scale)
//   sigmoid            scale * p_c (1 - p_c) dw_c
//   sigmoid, renorm    (1 - p_c) w_c * (dw_c - sum dw w / scale)
// and 0 for the other experts.  8191 tokens over 160 experts: 7 us, most of it
// launch and latency (10 MB).
template <int VPL>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteBackwardArgs a) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * 4 + wave;
    if (t >= a.T) return;
    constexpr float ninf = -__builtin_inff();
    const int E = a.E, k = a.k;
    const int id = lane < k ? a.ids[t * k + lane] : -1;
    const bool there = id >= 0 && id < E;
    const float got = there ? clean_logit(load_logit(a.logits, t * E + id, a.bf16)) : ninf;
    const float dw = there ? a.d_weights[t * k + lane] : 0.f;
    const bool full = !a.sigmoid && !a.renorm;
    float p[VPL], top = 0.f, z = 1.f;
    if (full) {
        float m = ninf;
        load_logits<VPL>(a.logits, t, E, a.bf16, lane, p);
#pragma unroll
        for (int i = 0; i < VPL; ++i) m = fmaxf(m, p[i]);
        m = wave_max(m);
        top = m > ninf ? m : 0.f;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            p[i] = expf(p[i] - top);
            sum += p[i];
        }
        z = wave_sum(sum);
        const float r = z > 0.f ? 1.f / z : 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) p[i] *= r;
    }
    float g, d = 0.f;                                    // g: gradient of the lane's chosen logit
    if (full) {
        g = dw;
        d = wave_sum(there && z > 0.f ? dw * (expf(got - top) / z) : 0.f);
    } else {
        const float w = route_weight(got, a.sigmoid, a.renorm, a.scale, 0.f, 1.f);
        g = a.renorm ? w * (dw - wave_sum(dw * w) / a.scale) : w * dw;
        // 1 - sigma(x) = sigma(-x), without the subtraction
        if (a.sigmoid) g = there ? g * sigmoid_f32(-got) : 0.f;
    }
    float o[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) o[i] = 0.f;
    for (int j = 0; j < k; ++j) {
        const int ej = __builtin_amdgcn_readlane(there ? id : -1, j);
        const float gj = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(g), j));
#pragma unroll
        for (int i = 0; i < VPL; ++i) o[i] += ej == lane + 64 * i ? gj : 0.f;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = lane + 64 * i;
        if (e >= E) continue;
        const float v = full ? a.scale * p[i] * (o[i] - d) : o[i];
        if (a.bf16) ((__bf16*)a.d_logits)[t * E + e] = (__bf16)v;
        else ((float*)a.d_logits)[t * E + e] = v;
    }
}

// ----------------------------------------------------------------- launches

template <int VPL, int MODE>
static hipError_t route_as(const RouteArgs& a, hipStream_t s) {
    uint32_t magic = 0;
    int lg = 0;
    if (a.n_groups > 1) {
        // e / gs for e < 1024 as the high half of e * magic (0 stands for groups of one)
        magic = (uint32_t)(0xFFFFFFFFull / (uint32_t)(a.E / a.n_groups)) + 1u;
        while ((a.n_groups << (lg + 1)) <= 64) ++lg;
    }
    // with groups, a wave has E doubles of LDS: at most 32 KB for all of them
    const int most = a.n_groups == 1 || a.E <= 256 ? 16 : (a.E <= 512 ? 8 : 4);
    if (a.T <= kStep) {
        const int waves = a.T < 4 ? 4 : (a.T < most ? a.T : most);
        route_kernel<VPL, MODE, true>
            <<<1, waves * 64, a.n_groups > 1 ? sizeof(double) * (size_t)a.E * waves : 0, s>>>(a, magic, lg);
        return hipGetLastError();
    }
    const int tiles = (a.T + a.tile_tokens - 1) / a.tile_tokens;
    const int tokens = a.tile_tokens < kStep ? a.tile_tokens : kStep;
    const int waves = std::min(tokens, most);
    const size_t lds = a.n_groups > 1 ? sizeof(double) * (size_t)a.E * waves : 0;
    route_kernel<VPL, MODE, false><<<tiles, waves * 64, lds, s>>>(a, magic, lg);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    route_rows_kernel<<<tiles, kRowsThreads, 0, s>>>(a, tiles);
    return hipGetLastError();
}

template <int VPL>
static hipError_t route_mode(const RouteArgs& a, hipStream_t s) {
    if (a.bias) return route_as<VPL, 2>(a, s);
    if (a.n_groups > 1 && a.group_top == 2) return route_as<VPL, 1>(a, s);
    return route_as<VPL, 0>(a, s);
}

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
    if (a.E <= 64) return route_mode<1>(a, s);
    if (a.E <= 128) return route_mode<2>(a, s);
    if (a.E <= 256) return route_mode<4>(a, s);
    if (a.E <= 512) return route_mode<8>(a, s);
    return route_mode<16>(a, s);
}

template <int VPL>
static hipError_t route_backward_as(const RouteBackwardArgs& a, hipStream_t s) {
    route_backward_kernel<VPL><<<(a.T + 3) / 4, 256, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_route_backward(const RouteBackwardArgs& a, hipStream_t s) {
    if (a.T == 0) return hipSuccess;
    if (a.E <= 64) return route_backward_as<1>(a, s);
    if (a.E <= 128) return route_backward_as<2>(a, s);
    if (a.E <= 192) return route_backward_as<3>(a, s);
    if (a.E <= 256) return route_backward_as<4>(a, s);
    if (a.E <= 512) return route_backward_as<8>(a, s);
    return route_backward_as<16>(a, s);
}

}  // namespace moegg
