// route.hip -- router logits -> expert ids, weights, counts and the row of
// every assignment, and the gradient of the logits.
//
// One wave takes one token: lane l holds the logits of VPL neighbouring experts
// from l VPL on in registers, so that equal keys go to the lowest lane, and most
// groups are whole runs of lanes.  A key is a 32-bit logit (softmax and sigmoid are
// monotone, so without a bias the logits themselves order the experts), or score +
// bias in 64 bits, mapped to unsigned integers of the same order.  Each of the k
// picks is a wave-wide maximum by DPP and a ballot that finds its holder.
//
// The row of assignment (t, j) is its expert's segment start plus the number
// of earlier tokens with the same expert.  No order of atomics enters: inside
// a 64-token step each expert has a 64-bit mask of its tokens (set by OR), and
// a rank is a popcount of the bits below; steps add up in LDS, token tiles
// through a [tiles, E] table of 16-bit counts.  For a few tokens, one workgroup
// does everything in one launch; beyond, route_kernel leaves ranks inside the
// tile in row_of, and route_rows_kernel, whose every workgroup sums the table,
// adds the segment start and the earlier tiles.
//
// What bounds it: launches and the VALU.  One token over 256 experts in groups
// with a bias takes 5.7 us, 4096 tokens over 64 experts 5.3 + 2.7 us, 8191 tokens
// over 256 experts in groups with a bias 17 + 3.8 us: 3 us of the first to launch and
// load, then 740 instructions a token (150 for the 64-bit sigmoids, 190 for eight
// picks, 90 for the weights).  Sixteen lanes a token need 510 in 32 bits, but then
// some token of a call this size always has two values too near to tell apart, and
// the 64-bit repeat costs more than is won.
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
    return l != l ? -__builtin_inff() : __builtin_amdgcn_fmed3f(l, -__builtin_inff(), kFltMax) + 0.f;
}

__device__ __forceinline__ float load_logit(const void* p, int64_t i, int bf16) {
    return bf16 ? __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16) : ((const float*)p)[i];
}

// VPL consecutive elements of a row of E that lane `lane` holds; what it gets
// past the row's end is of no meaning, and read within it.  One vector load if
// VPL divides E, else no branch between the loads.
template <typename T, int VPL>
__device__ __forceinline__ void load_row(const T* p, int E, int lane, T (&r)[VPL]) {
    if (VPL > 1 && E % VPL == 0) {
        typedef T Vec __attribute__((ext_vector_type(VPL), aligned(sizeof(T))));
        const Vec v = *(const Vec*)(p + min(lane * VPL, E - VPL));
#pragma unroll
        for (int i = 0; i < VPL; ++i) r[i] = v[i];
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) r[i] = p[min(lane * VPL + i, E - 1)];
    }
}
template <typename T, int VPL>
__device__ __forceinline__ void store_row(T* p, int E, int lane, const T (&r)[VPL]) {
    if (VPL > 1 && E % VPL == 0) {
        typedef T Vec __attribute__((ext_vector_type(VPL), aligned(sizeof(T))));
        Vec v;
#pragma unroll
        for (int i = 0; i < VPL; ++i) v[i] = r[i];
        if (lane * VPL < E) *(Vec*)(p + lane * VPL) = v;
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (lane * VPL + i < E) p[lane * VPL + i] = r[i];
    }
}
template <int VPL>
__device__ __forceinline__ void load_logits(const void* logits, int64_t t, int E, int bf16, int lane, float (&l)[VPL]) {
    if (bf16) {
        uint16_t r[VPL];
        load_row<uint16_t, VPL>((const uint16_t*)logits + t * E, E, lane, r);
#pragma unroll
        for (int i = 0; i < VPL; ++i) l[i] = __uint_as_float((uint32_t)r[i] << 16);
    } else {
        load_row<float, VPL>((const float*)logits + t * E, E, lane, l);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] = lane * VPL + i < E ? clean_logit(l[i]) : -__builtin_inff();
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

// Maximum of floats that are not NaN, by the integers of their order.
__device__ __forceinline__ float wave_max_ordered(float v) { return unkey32(wave_max_u32(key32(v))); }

// e^x for x in [-750, 0], to 1 ulp or so: x = n ln 2 + r with |r| <= ln 2 / 2, and
// the series of e^r up to r^13 (the next term is 4e-18 of it).
__device__ __forceinline__ double exp_f64(double x) {
    const double n = __builtin_rint(x * 1.4426950408889634);
    double r = __builtin_fma(n, -0x1.62e42fefa0000p-1, x);          // ln 2 to 41 bits: the product is exact
    r = __builtin_fma(n, -0x1.cf79abc9e3b3ap-40, r);                // and the rest of it
    double p = 1.0 / 6227020800.0;
    p = __builtin_fma(p, r, 1.0 / 479001600.0);
    p = __builtin_fma(p, r, 1.0 / 39916800.0);
    p = __builtin_fma(p, r, 1.0 / 3628800.0);
    p = __builtin_fma(p, r, 1.0 / 362880.0);
    p = __builtin_fma(p, r, 1.0 / 40320.0);
    p = __builtin_fma(p, r, 1.0 / 5040.0);
    p = __builtin_fma(p, r, 1.0 / 720.0);
    p = __builtin_fma(p, r, 1.0 / 120.0);
    p = __builtin_fma(p, r, 1.0 / 24.0);
    p = __builtin_fma(p, r, 1.0 / 6.0);
    p = __builtin_fma(p, r, 0.5);
    p = __builtin_fma(p, r, 1.0);
    p = __builtin_fma(p, r, 1.0);
    return __builtin_amdgcn_ldexp(p, (int)n);
}

// 1 / (1 + e^-x), x not NaN: with e = e^-|x| it is 1 / (1 + e) or e / (1 + e); the
// reciprocal of 1 + e in [1, 2] by two Newton steps.
__device__ __forceinline__ double sigmoid_f64(float x) {
    const double e = exp_f64((double)__builtin_amdgcn_fmed3f(-fabsf(x), -750.f, 0.f)), d = 1.0 + e;
    double r = __builtin_amdgcn_rcp(d);
    r = __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
    r = __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
    return x < 0.f ? e * r : r;
}

// Scores in 64 bits: their users compare sums of them, and two of a token's
// may be nearer to each other than 32 bits tell apart.
template <int VPL>
__device__ __forceinline__ void scores64(const float (&l)[VPL], int sigmoid, double (&s)[VPL]) {
    if (sigmoid) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) s[i] = sigmoid_f64(l[i]);
        return;
    }
    float m = l[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = fmaxf(m, l[i]);
    m = wave_max_ordered(m);
    const double top = m > -__builtin_inff() ? (double)m : 0.0;
    double z = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const double x = (double)l[i] - top;
        s[i] = exp_f64(x > -750.0 ? x : -750.0);         // e^-750 is 0
        z += s[i];
    }
    z = wave_sum_f64(z);
    const double r = z > 0 ? 1.0 / z : 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) s[i] *= r;
}

// The two largest of a group's scores, of which this lane and o's lane saw different parts.
template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    return __longlong_as_double((long long)((uint64_t)lane_of<CTRL>((uint32_t)(b >> 32)) << 32 | lane_of<CTRL>((uint32_t)b)));
}
__device__ __forceinline__ void merge_best(double o1, double o2, double& t1, double& t2) {
    t2 = fmax(fmax(t2, o2), fmin(t1, o1));
    t1 = fmax(t1, o1);
}
// Over aligned runs of 2^lg lanes, lg <= 5.
__device__ __forceinline__ void merge_lanes(int lg, double& t1, double& t2) {
    if (lg > 0) merge_best(dpp_f64<DPP_XOR1>(t1), dpp_f64<DPP_XOR1>(t2), t1, t2);
    if (lg > 1) merge_best(dpp_f64<DPP_XOR2>(t1), dpp_f64<DPP_XOR2>(t2), t1, t2);
    if (lg > 2) merge_best(dpp_f64<DPP_HALF_MIRROR>(t1), dpp_f64<DPP_HALF_MIRROR>(t2), t1, t2);
    if (lg > 3) merge_best(dpp_f64<DPP_MIRROR>(t1), dpp_f64<DPP_MIRROR>(t2), t1, t2);
    if (lg > 4) merge_best(__shfl_xor(t1, 16, 64), __shfl_xor(t2, 16, 64), t1, t2);
}

// Where a wave keeps a token's groups.
struct Groups {
    int in_lanes;                                        // group g: the experts of lanes g 2^lg .. (g + 1) 2^lg - 1
    int lg;                                              // lanes that share a group's work: 2^lg, at most 64 / n_groups
    uint32_t magic;                                      // e / group size = umulhi(e, magic); 0: groups of one
};

// Weights of the k chosen experts; lane j < k holds the j-th one's
// logit (-inf where there is none).  A softmax over all experts brings its
// maximum and sum of exponentials (top, z).
__device__ __forceinline__ float route_weight(float got, int sigmoid, int renorm, float scale, float top, float z) {
    const bool there = got > -__builtin_inff();
    if (!renorm) {
        if (!there) return 0.f;
        return scale * (sigmoid ? sigmoid_f32(got) : expf(got - top) / z);
    }
    const float m = wave_max_ordered(got);
    float t = 0.f;
    if (!sigmoid) {
        if (there) t = expf(got - m);
    } else if (there) {
        // the ratio of sigmoids with e^min(m, 0) taken out of both, so that far negative logits keep
        // their ratio: sigma(x) = e^min(x, 0) / (1 + e^-|x|)
        t = expf(fminf(got, 0.f) - fminf(m, 0.f)) / (1.f + expf(-fabsf(got)));
    }
    const float sum = wave_sum(t);
    return sum > 0.f ? scale * t / sum : 0.f;
}

// One token: picks into lane j's `id` (-1: none) and weight.
// MODE 0: 32-bit keys, no 64-bit scores; 1: 32-bit keys, groups by 64-bit
// scores; 2: 64-bit keys (bias).  gbuf: E doubles of this wave, where groups do
// not lie on whole runs of lanes.
template <int VPL, int MODE>
__device__ __forceinline__ void route_token(const RouteArgs& a, const Groups& gr, int t, int lane, double* gbuf, int& id,
                                            float& weight) {
    typedef typename std::conditional<MODE == 2, uint64_t, uint32_t>::type Key;
    const int E = a.E, k = a.k;
    constexpr float ninf = -__builtin_inff();
    float l[VPL], bias[VPL];
    if constexpr (MODE == 2) load_row<float, VPL>(a.bias, E, lane, bias);
    load_logits<VPL>(a.logits, t, E, a.bf16, lane, l);
    double s[MODE ? VPL : 1];
    if constexpr (MODE != 0) scores64<VPL>(l, a.sigmoid, s);
    Key key[VPL];                                        // 0: not to be picked
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        if constexpr (MODE == 2) {
            const float b = clean_logit(bias[i]);        // NaN, -inf: not to be chosen
            const bool there = l[i] > ninf && b > ninf;
            s[i] = there ? s[i] + (double)b : -__builtin_inf();
            key[i] = there ? key64(s[i]) : 0;
        } else {
            key[i] = l[i] > ninf ? key32(l[i]) : 0u;
            if constexpr (MODE == 1) s[i] = l[i] > ninf ? s[i] : -__builtin_inf();
        }
    }
    if (a.n_groups > 1) {
        // 2^lg lanes have a group; each keeps the two best of its part
        const int L = 1 << gr.lg, g = lane >> gr.lg, r = lane & (L - 1);
        double t1 = -__builtin_inf(), t2 = -__builtin_inf();
        if (gr.in_lanes) {                               // its own experts
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const double v = MODE == 0 ? (double)l[i] : s[MODE ? i : 0];
                t2 = fmax(t2, fmin(t1, v));
                t1 = fmax(t1, v);
            }
        } else {
            const int gs = E / a.n_groups;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const int e = lane * VPL + i;
                if (e < E) gbuf[e] = MODE == 0 ? (double)l[i] : s[MODE ? i : 0];
            }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
            if (g < a.n_groups)
                for (int i = r; i < gs; i += L) {
                    const double v = gbuf[g * gs + i];
                    t2 = fmax(t2, fmin(t1, v));
                    t1 = fmax(t1, v);
                }
            __builtin_amdgcn_wave_barrier();
        }
        merge_lanes(gr.lg, t1, t2);
        // of the scores that there are: a group with one has that one, a group with none -inf, which no other has
        const double score = a.group_top == 2 && t2 > -__builtin_inf() ? t1 + t2 : t1;
        // A group's lanes compare it with L groups at a time: its rank is the number of better ones.
        int rank = 0;
        for (int o0 = 0; o0 < a.n_groups; o0 += L) {
            const int o = o0 + r;
            const double v = __shfl(score, o << gr.lg, 64);
            const uint64_t better = __ballot(o < a.n_groups && (v > score || (v == score && o < g)));
            rank += __popcll((better >> (g << gr.lg)) & ((1ull << L) - 1));
        }
        if (gr.in_lanes) {
            if (rank >= a.topk_groups) {
#pragma unroll
                for (int i = 0; i < VPL; ++i) key[i] = 0;
            }
        } else {
            const uint64_t keep = __ballot(rank < a.topk_groups);
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const int e = lane * VPL + i;
                const int eg = gr.magic ? (int)__umulhi((uint32_t)e, gr.magic) : e;
                if (e >= E || !((keep >> ((eg << gr.lg) & 63)) & 1)) key[i] = 0;
            }
        }
    }
    float top = 0.f, z = 1.f;
    if (!a.sigmoid && !a.renorm) {
        float m = l[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i) m = fmaxf(m, l[i]);
        m = wave_max_ordered(m);
        top = m > ninf ? m : 0.f;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) sum += expf(l[i] - top);
        z = wave_sum(sum);
    }
    // A pick looks at one key a lane, its largest: key[0], of its expert at[0].  Up to four, the lane's keys are
    // sorted and its holder moves up the others; beyond, it looks for its next one.  Equal keys: the lowest id, which
    // the lowest lane has; in a lane they keep their order.
    constexpr bool SORT = VPL <= 4;
    Key rest[VPL];                                       // SORT: key itself
    int at[VPL];
    if constexpr (SORT) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) at[i] = i;
#pragma unroll
        for (int n = VPL - 1; n > 0; --n) {
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const bool less = key[i] < key[i + 1];
                swap_if(less, key[i], key[i + 1]);
                swap_if(less, at[i], at[i + 1]);
            }
        }
    }
    auto find_largest = [&]() {
        key[0] = rest[0];
        at[0] = 0;
#pragma unroll
        for (int i = 1; i < VPL; ++i) {
            const bool more = rest[i] > key[0];
            key[0] = more ? rest[i] : key[0];
            at[0] = more ? i : at[0];
        }
    };
    if constexpr (!SORT) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) rest[i] = key[i];
        find_largest();
    }
    int picks = 0;                                       // experts that can be picked, at most k
#pragma unroll
    for (int i = 0; i < VPL; ++i) picks += __popcll(__ballot(SORT ? key[i] != 0 : rest[i] != 0));
    picks = min(picks, k);
    id = -1;
    float got = ninf;
    for (int j = 0; j < picks; ++j) {
        const uint32_t hi = (uint32_t)(key[0] >> (MODE == 2 ? 32 : 0));
        const uint32_t m = wave_max_u32(hi);
        uint64_t who = __ballot(hi == m);
        if constexpr (MODE == 2) {
            if (who & (who - 1)) {
                const uint32_t low = wave_max_u32(hi == m ? (uint32_t)key[0] : 0u);
                who = __ballot(hi == m && (uint32_t)key[0] == low);
            }
        }
        const int src = __builtin_ctzll(who);
        const int ej = VPL > 1 ? src * VPL + __builtin_amdgcn_readlane(at[0], src) : src;
        id = lane == j ? ej : id;
        if constexpr (MODE != 2) got = lane == j ? unkey32(m) : got;
        if (lane == src) {
            if constexpr (SORT) {
#pragma unroll
                for (int i = 0; i + 1 < VPL; ++i) {
                    key[i] = key[i + 1];
                    at[i] = at[i + 1];
                }
                key[VPL - 1] = 0;
            } else {
#pragma unroll
                for (int i = 0; i < VPL; ++i) rest[i] = i == at[0] ? 0 : rest[i];
                find_largest();
            }
        }
    }
    if constexpr (MODE == 2) {
        if constexpr (SORT) {                            // from the lane that has it
            const int from = id < 0 ? 0 : id / VPL, i = id & (VPL - 1);
            float v = __shfl(l[0], from, 64);
#pragma unroll
            for (int n = 1; n < VPL; ++n) {
                const float x = __shfl(l[n], from, 64);
                v = i == n ? x : v;
            }
            got = id < 0 ? ninf : v;
        } else if (id >= 0) {
            got = clean_logit(load_logit(a.logits, (int64_t)t * E + id, a.bf16));
        }
    }
    weight = route_weight(got, a.sigmoid, a.renorm, a.scale, top, z);
}

// Rows of an expert's segment, and sums of them, stop at 2^31 - 1, which no row reaches.
constexpr uint32_t kNoRow = 0x7FFFFFFFu;
__device__ __forceinline__ uint32_t sum_rows(uint32_t a, uint32_t b) { return min(a + b, kNoRow); }
__device__ __forceinline__ uint32_t segment_rows(uint32_t m, int seg_align, int cap) {
    if (cap) return (uint32_t)cap;
    if (seg_align == 1) return m;
    return (uint32_t)min((uint64_t)kNoRow,
                         (uint64_t)((m + (uint32_t)seg_align - 1) / (uint32_t)seg_align) * (uint32_t)seg_align);
}
// Segment rows of E experts -> where the segments start, by one wave: a run of experts a lane.
__device__ void segment_starts(uint32_t* seg, int E, int lane) {
    const int run = (E + 63) / 64, e0 = min(lane * run, E), e1 = min(e0 + run, E);
    uint32_t sum = 0;
#pragma unroll 4
    for (int e = e0; e < e1; ++e) sum = sum_rows(sum, seg[e]);
    uint32_t end = sum;
    end = sum_rows(end, dpp<DPP_SHR + 1>(0, end));
    end = sum_rows(end, dpp<DPP_SHR + 2>(0, end));
    end = sum_rows(end, dpp<DPP_SHR + 4>(0, end));
    end = sum_rows(end, dpp<DPP_SHR + 8>(0, end));
    end = sum_rows(end, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)end, DPP_BCAST15, 0xA, 0xF, false));
    end = sum_rows(end, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)end, DPP_BCAST31, 0xC, 0xF, false));
    uint32_t start = (uint32_t)__shfl_up((int)end, 1, 64);
    if (lane == 0) start = 0;
#pragma unroll 4
    for (int e = e0; e < e1; ++e) {
        const uint32_t rows = seg[e];
        seg[e] = start;
        start = sum_rows(start, rows);
    }
}

__device__ __forceinline__ int32_t final_row(uint32_t start, uint32_t rank, int cap, int64_t rows_total) {
    if (cap && rank >= (uint32_t)cap) return -1;
    return start + rank < (uint32_t)rows_total ? (int32_t)(start + rank) : -1;   // both below 2^31
}

// Workgroup b routes tokens [b * tile_tokens, ...).  ONE: the only workgroup;
// it also writes m_sizes and final rows.
constexpr int route_threads(int vpl) { return vpl > 8 ? 512 : 1024; }   // 16 experts a lane need over 128 registers
template <int VPL, int MODE, bool ONE>
__global__ __launch_bounds__(route_threads(VPL)) void route_kernel(RouteArgs a, Groups gr) {
    extern __shared__ double gbuf_all[];                 // groups off whole lanes: E per wave
    __shared__ unsigned long long mask_s[kRouteMaxExperts];
    __shared__ int32_t count_s[kRouteMaxExperts];
    __shared__ int16_t ids_s[kStep * kRouteMaxTopK];
    __shared__ uint32_t start_s[ONE ? kRouteMaxExperts : 1];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int waves = blockDim.x >> 6, E = a.E, k = a.k;
    const int t0 = ONE ? 0 : blockIdx.x * a.tile_tokens, t1 = ONE ? a.T : min(a.T, t0 + a.tile_tokens);
    double* gbuf = gbuf_all + (gr.in_lanes ? 0 : wave * E);
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
            route_token<VPL, MODE>(a, gr, ts + i, lane, gbuf, id, w);
            if (lane < k) {
                const int64_t at = (int64_t)(ts + i) * k + lane;
                a.ids[at] = id;
                a.weights[at] = w;
                ids_s[i * k + lane] = (int16_t)id;
                if (id >= 0) atomicOr(&mask_s[id], 1ull << i);
            }
        }
        lds_barrier();
        if constexpr (ONE) break;                        // one step holds every token
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
        for (int e = threadIdx.x; e < E; e += blockDim.x) {
            const int m = __popcll(mask_s[e]);
            a.m_sizes[e] = m;
            start_s[e] = segment_rows(m, a.seg_align, a.cap);
        }
        lds_barrier();
        if (wave == 0) segment_starts(start_s, E, lane);
        lds_barrier();
        for (int x = threadIdx.x; x < a.T * k; x += blockDim.x) {
            const int id = ids_s[x], i = x / k;
            a.row_of[x] = id < 0 ? -1
                                 : final_row(start_s[id], (uint32_t)__popcll(mask_s[id] & ((1ull << i) - 1)), a.cap,
                                             a.rows_total);
        }
    } else {
        const int width = route_count_width(E);
        uint32_t* out = (uint32_t*)(a.tile_counts + (int64_t)blockIdx.x * width);
        for (int e = threadIdx.x; e < width / 2; e += blockDim.x)
            out[e] = (2 * e < E ? (uint32_t)count_s[2 * e] : 0u) | (2 * e + 1 < E ? (uint32_t)count_s[2 * e + 1] << 16 : 0u);
    }
}

constexpr int kRowsThreads = 1024;

// Ranks inside a tile -> rows: every workgroup sums the table of tile counts
// (128 KB at 256 tiles of 256 experts, from L2), scans the segments and
// finishes its own tile.  That shape takes 3.8 us, most of it launch and
// latency (4 bytes a load and 32-bit sums: 6.2 us).
// PAIRS (fewer than 2^16 tokens): counts are summed two to a word.
template <bool PAIRS>
__global__ __launch_bounds__(kRowsThreads) void route_rows_kernel(RouteArgs a, int tiles, int lg) {
    // Sums of all assignments, and above them those of earlier tiles: of experts 8 p + 2 n and 8 p + 2 n + 1 at
    // n * eights + p (PAIRS), or of expert 8 p + n there; neighbouring threads add to neighbouring words.
    __shared__ unsigned long long sum_s[PAIRS ? kRouteMaxExperts / 2 : kRouteMaxExperts];
    __shared__ uint32_t before_s[kRouteMaxExperts], start_s[kRouteMaxExperts];
    constexpr int N = PAIRS ? 4 : 8;
    const int E = a.E, b = blockIdx.x, k = a.k;
    const int eights = (E + 7) / 8;                      // 16 bytes of a tile's counts
    for (int e = threadIdx.x; e < N * eights; e += kRowsThreads) sum_s[e] = 0;
    lds_barrier();
    // its own assignments, on their way while the table is summed
    const int64_t x0 = (int64_t)b * a.tile_tokens * k, x1 = min((int64_t)a.T * k, x0 + (int64_t)a.tile_tokens * k);
    const int64_t xf = min(x0 + threadIdx.x, x1 - 1);
    const int first_id = a.ids[xf], first_rank = a.row_of[xf];
    // `parts` threads share 8 experts (2^lg >= eights threads a part), each summing every parts-th tile, 8 loads at a time
    const int parts = min(min(kRowsThreads >> lg, 32), tiles);
    const int part = threadIdx.x >> lg, p = threadIdx.x & ((1 << lg) - 1);
    if (part < parts && p < eights) {
        const u32x4* in = (const u32x4*)a.tile_counts + p;
        uint32_t total[N] = {0}, before[N] = {0};
        for (int i0 = part; i0 < tiles; i0 += 8 * parts) {
            u32x4 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = in[min(i0 + j * parts, tiles - 1) * eights];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int i = i0 + j * parts;
                const bool in_all = i < tiles, in_before = i < b;
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const uint32_t c = PAIRS ? v[j][n % 4] : (n & 1 ? v[j][n / 2] >> 16 : v[j][n / 2] & 0xFFFFu);
                    total[n] += in_all ? c : 0u;
                    before[n] += in_before ? c : 0u;
                }
            }
        }
        // sums of whole numbers: the atomics' order does not matter
#pragma unroll
        for (int n = 0; n < N; ++n)
            atomicAdd(&sum_s[n * eights + p], (unsigned long long)before[n] << 32 | total[n]);
    }
    lds_barrier();
    for (int e = threadIdx.x; e < E; e += kRowsThreads) {
        const int n = PAIRS ? (e & 7) >> 1 : e & 7;
        const uint64_t v = sum_s[n * eights + (e >> 3)];
        uint32_t m = (uint32_t)v, bef = (uint32_t)(v >> 32);
        if (PAIRS) {
            m = e & 1 ? m >> 16 : m & 0xFFFFu;
            bef = e & 1 ? bef >> 16 : bef & 0xFFFFu;
        }
        before_s[e] = bef;
        start_s[e] = segment_rows(m, a.seg_align, a.cap);
        if (b == 0) a.m_sizes[e] = (int32_t)m;
    }
    lds_barrier();
    if (threadIdx.x < 64) segment_starts(start_s, E, threadIdx.x);
    lds_barrier();
    for (int64_t x = x0 + threadIdx.x; x < x1; x += kRowsThreads) {
        const bool first = x == x0 + threadIdx.x;
        const int id = first ? first_id : a.ids[x];
        const uint32_t rank = (uint32_t)(first ? first_rank : a.row_of[x]);
        a.row_of[x] = id < 0 ? -1 : final_row(start_s[id], before_s[id] + rank, a.cap, a.rows_total);
    }
}

// Gradient of the logits, one wave a token.  With p the scores, w the weights
// and dw their gradients (over the chosen experts c):
//   softmax            scale * p_e * (dw_e [e chosen] - sum_c dw_c p_c)
//   softmax, renorm    w_c * (dw_c - sum dw w / scale)
//   sigmoid            scale * p_c (1 - p_c) dw_c
//   sigmoid, renorm    (1 - p_c) w_c * (dw_c - sum dw w / scale)
// and 0 for the other experts.  8191 tokens over 160 experts: 6 us, most of it
// launch and latency (10 MB).
template <int VPL>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteBackwardArgs a) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * 4 + wave;
    if (t >= a.T) return;
    constexpr float ninf = -__builtin_inff();
    const int E = a.E, k = a.k;
    const bool full = !a.sigmoid && !a.renorm;           // every logit has a gradient
    float p[VPL];
    if (full) load_logits<VPL>(a.logits, t, E, a.bf16, lane, p);
    const int id = lane < k ? a.ids[t * k + lane] : -1;
    const float dw_in = lane < k ? a.d_weights[t * k + lane] : 0.f;
    const bool there = id >= 0 && id < E;
    const float dw = there ? dw_in : 0.f;
    float g = dw;                                        // gradient of the lane's chosen logit, or of its score
    if (!full) {
        const float got = there ? clean_logit(load_logit(a.logits, t * E + id, a.bf16)) : ninf;
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
        for (int i = 0; i < VPL; ++i) o[i] += ej == lane * VPL + i ? gj : 0.f;
    }
    if (full) {
        float m = p[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i) m = fmaxf(m, p[i]);
        m = wave_max_ordered(m);
        const float top = m > ninf ? m : 0.f;
        float sum = 0.f, d = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            p[i] = expf(p[i] - top);
            sum += p[i];
        }
        sum = wave_sum(sum);
        const float r = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            p[i] *= r;
            d = __builtin_fmaf(o[i], p[i], d);
        }
        d = wave_sum(d);
#pragma unroll
        for (int i = 0; i < VPL; ++i) o[i] = a.scale * p[i] * (o[i] - d);
    }
    if (a.bf16) {
        __bf16 r[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) r[i] = (__bf16)o[i];
        store_row<__bf16, VPL>((__bf16*)a.d_logits + t * E, E, lane, r);
    } else {
        store_row<float, VPL>((float*)a.d_logits + t * E, E, lane, o);
    }
}

// ----------------------------------------------------------------- launches

// Tokens that one workgroup does by itself, a wave for each at first.  In one and in
// two launches (us, k = 8): 64 experts 24 tokens 5.3 and 6.6, 32 tokens 6.3 and 6.6,
// 48 tokens 8.0 and 6.6; 256 experts 32 tokens 8.3 and 7.4, but a second launch costs
// the host 2.2; with a bias 64 experts 24 tokens 6.3 and 7.1, 32 tokens 7.8 and 7.1,
// 256 experts 20 tokens 9.0 and 8.7; in groups 16 tokens 9.0 and 9.6, 17 tokens 9.3.
template <int VPL, int MODE>
static int one_launch_tokens(const RouteArgs& a) {
    if (a.n_groups > 1 || VPL > 4) return 16;
    return MODE == 0 ? 32 : (VPL <= 2 ? 24 : 16);
}

template <int VPL, int MODE>
static hipError_t route_as(const RouteArgs& a, hipStream_t s) {
    Groups gr{1, 0, 0};
    if (a.n_groups > 1) {
        const int gs = a.E / a.n_groups, lanes = gs / VPL;
        gr.in_lanes = gs % VPL == 0 && (lanes & (lanes - 1)) == 0;
        // e / gs for e < 1024 as the high half of e * magic (0 stands for groups of one)
        gr.magic = (uint32_t)(0xFFFFFFFFull / (uint32_t)gs) + 1u;
        while ((gr.in_lanes ? 2 << gr.lg <= lanes : a.n_groups << (gr.lg + 1) <= 64)) ++gr.lg;
    }
    // groups off whole lanes: a wave has E doubles of LDS, at most 32 KB for all of them
    const int most = std::min(route_threads(VPL) / 64, gr.in_lanes || a.E <= 256 ? 16 : (a.E <= 512 ? 8 : 4));
    const size_t lds = gr.in_lanes ? 0 : sizeof(double) * (size_t)a.E;
    if (a.T <= one_launch_tokens<VPL, MODE>(a)) {        // at most kStep
        const int waves = a.T < 4 ? 4 : (a.T < most ? a.T : most);
        route_kernel<VPL, MODE, true><<<1, waves * 64, lds * waves, s>>>(a, gr);
        return hipGetLastError();
    }
    const int tiles = (a.T + a.tile_tokens - 1) / a.tile_tokens;
    const int waves = std::min(a.tile_tokens < kStep ? a.tile_tokens : kStep, most);
    route_kernel<VPL, MODE, false><<<tiles, waves * 64, lds * waves, s>>>(a, gr);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    int rows_lg = 0;
    while (1 << rows_lg < route_count_width(a.E) / 8) ++rows_lg;
    if (a.T < 1 << 16) route_rows_kernel<true><<<tiles, kRowsThreads, 0, s>>>(a, tiles, rows_lg);
    else route_rows_kernel<false><<<tiles, kRowsThreads, 0, s>>>(a, tiles, rows_lg);
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
    if (a.E <= 256) return route_backward_as<4>(a, s);
    if (a.E <= 512) return route_backward_as<8>(a, s);
    return route_backward_as<16>(a, s);
}

}  // namespace moegg
