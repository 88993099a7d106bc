// layer.hpp -- what the layer operators around the grouped GEMMs share: wave
// reductions, e4m3 quantization by groups, and the launchers that the C ABI
// (layer_api.hip) calls (route.hip, permute.hip, checkpoint.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moegg.h"

namespace moegg {

constexpr int kRouteMaxExperts = 1024;   // experts a wave holds in registers, 16 a lane
constexpr int kRouteMaxTopK = 32;
constexpr int kRouteMaxTiles = 256;      // token tiles of a routing call (one workgroup each)
constexpr int kRouteMaxTokens = kRouteMaxTiles * 65520;   // a tile's counts are 16 bits
constexpr int kGroup = 128;              // elements of one quantization group

struct RouteArgs {
    const void* logits;                  // fp32 or bf16 [T, E]
    const float* bias;                   // [E] or NULL
    int32_t* ids;                        // [T, k]
    float* weights;                      // [T, k]
    int32_t* m_sizes;                    // [E]
    int32_t* row_of;                     // [T, k]
    uint16_t* tile_counts;               // [tiles, route_count_width(E)]: assignments of each token tile
    int T, E, k;
    int bf16;                            // logits' type
    int sigmoid, renorm;
    int n_groups, topk_groups, group_top;
    float scale;
    int64_t rows_total;
    int seg_align, cap;
    int tile_tokens;                     // tokens of one workgroup
};

struct RouteBackwardArgs {
    const void* logits;
    const int32_t* ids;
    const float* d_weights;
    void* d_logits;                      // logits' type
    int T, E, k, bf16, sigmoid, renorm;
    float scale;
};

// How a row-major operand is stored (moegg_dtype_t of the call that will read it).
enum OperandFormat { kBf16 = 0, kRows = 1, kKm = 2, kE8m0 = 3 };

struct PermuteArgs {
    const void* x;                       // dispatch: bf16 [T, W]; combine: Y bf16 [rows, W]; backward: dout [T, W]
    const void* Y;                       // combine backward: bf16 [rows, W]
    const float* weights;                // [T, k] or NULL
    const int32_t* row_of;               // [T, k]
    void* out;                           // dispatch: A; combine: out; backward: dY
    void* scale;                         // of an e4m3 output
    float* d_weights;                    // combine backward: [T, k]
    int T, k, W;
    int rows;                            // rows of the expert side
    OperandFormat fmt;
};

struct CheckpointArgs {
    const void* in;                      // forward: GU bf16; backward: dH bf16; k groups: X
    const float* in_scale;               // k groups: scales of X (NULL: bf16)
    const int32_t* m_sizes;              // [G]
    uint8_t* ckpt;                       // e4m3 [rows, 2I]
    float* ckpt_scale;                   // [rows, 2I / 128]
    void* row_out;                       // forward: H; backward: dGU
    void* row_scale;
    void* H;                             // bf16 backward: H
    uint8_t* k_out;                      // dGU or X by token groups
    void* k_scale;
    uint8_t* hk_out;                     // H by token groups
    void* hk_scale;
    int G, rows, W;                      // W: I, or the width of X
    int64_t scale_groups;
    OperandFormat fmt;                   // of row_out; k groups: of X
    int k_e8m0;                          // token-group scales are E8M0 bytes
};

hipError_t launch_route(const RouteArgs& a, hipStream_t s);
hipError_t launch_route_backward(const RouteBackwardArgs& a, hipStream_t s);
hipError_t launch_dispatch(const PermuteArgs& a, hipStream_t s);
hipError_t launch_combine(const PermuteArgs& a, hipStream_t s);
hipError_t launch_combine_backward(const PermuteArgs& a, hipStream_t s);
hipError_t launch_swiglu_checkpoint(const CheckpointArgs& a, hipStream_t s);
hipError_t launch_swiglu_checkpoint_backward(const CheckpointArgs& a, hipStream_t s);
hipError_t launch_swiglu_checkpoint_backward_fp8(const CheckpointArgs& a, hipStream_t s);
hipError_t launch_checkpoint_to_k_groups(const CheckpointArgs& a, hipStream_t s);

// Tokens of one workgroup of a routing call: 4 (a wave on each SIMD) as long as
// that makes at most 256 workgroups, then in steps of 4 up to a wave each, then of
// 16.  64 tokens over 256 experts in groups: 10.5 us in tiles of 4, 14 us in tiles of 16.
inline int route_tile_tokens(int T) {
    const int t = (T + kRouteMaxTiles - 1) / kRouteMaxTiles;
    return t <= 4 ? 4 : (t <= 16 ? (t + 3) / 4 * 4 : (t + 15) / 16 * 16);
}

// Counts of one tile: 16 bits for every expert, in whole 16 bytes.
constexpr int route_count_width(int E) { return (E + 7) & ~7; }

#ifdef __HIPCC__

// ----------------------------------------------------------------- order of work

constexpr int kXcds = 8;

// Position of this workgroup's work: consecutive workgroups go to the 8 XCDs in
// turn, and RUN neighbouring pieces of work to one XCD, so that all of the chip
// works on one stretch of memory at a time and lines that neighbours share meet
// in one L2.  The grid is a multiple of 8 RUN.
template <int RUN>
__device__ __forceinline__ int64_t work_position() {
    const int order = blockIdx.x / kXcds;
    return ((int64_t)(order / RUN) * kXcds + blockIdx.x % kXcds) * RUN + order % RUN;
}
template <int RUN>
static dim3 run_grid(int64_t pieces) {
    constexpr int64_t round = kXcds * RUN;
    return dim3((unsigned)((pieces + round - 1) / round * round));
}

// ----------------------------------------------------------------- cross-lane

// Lane exchange by DPP: CTRL is quad_perm, row_shr, row_ror, row_bcast, ...
// (16-lane rows); lanes with no source get `old`.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t old, uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)x, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ float dpp_f(float old, float x) {
    return __uint_as_float(dpp<CTRL>(__float_as_uint(old), __float_as_uint(x)));
}
constexpr int DPP_XOR1 = 0xB1;            // quad_perm [1,0,3,2]
constexpr int DPP_XOR2 = 0x4E;            // quad_perm [2,3,0,1]
constexpr int DPP_HALF_MIRROR = 0x141;    // lane i of 8 <-> 7 - i
constexpr int DPP_MIRROR = 0x140;         // lane i of 16 <-> 15 - i
constexpr int DPP_ROR4 = 0x124, DPP_ROR8 = 0x128;   // lane i of 16 <- i - 4, i - 8 mod 16
constexpr int DPP_SHR = 0x110;            // + n: row_shr by n
constexpr int DPP_BCAST15 = 0x142, DPP_BCAST31 = 0x143;

// Lane exchange in which every lane has a source.
template <int CTRL>
__device__ __forceinline__ uint32_t lane_of(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, CTRL, 0xF, 0xF, true);
}
// Maximum over each aligned group of 8 or 16 lanes, in every lane of it, of
// floats that are not negative and not NaN: their bits compare as integers,
// which needs no NaN handling and folds the lane exchange into the maximum.
__device__ __forceinline__ float max8(float f) {
    uint32_t v = __float_as_uint(f);
    v = max(v, lane_of<DPP_XOR1>(v));
    v = max(v, lane_of<DPP_XOR2>(v));
    return __uint_as_float(max(v, lane_of<DPP_HALF_MIRROR>(v)));
}
__device__ __forceinline__ float max16(float f) {
    const uint32_t v = __float_as_uint(max8(f));
    return __uint_as_float(max(v, lane_of<DPP_MIRROR>(v)));
}

// Wave-wide reductions: an inclusive scan by DPP whose last lane holds the
// result, handed to every lane as a scalar.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    v = max(v, dpp<DPP_SHR + 1>(0, v));
    v = max(v, dpp<DPP_SHR + 2>(0, v));
    v = max(v, dpp<DPP_SHR + 4>(0, v));
    v = max(v, dpp<DPP_SHR + 8>(0, v));
    v = max(v, dpp<DPP_BCAST15>(0, v));
    v = max(v, dpp<DPP_BCAST31>(0, v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
// row_bcast hands a row's sum to the next rows only: with bound lanes reading
// 0, lane 63 sums rows 0..3 in a fixed order.
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp_f<DPP_SHR + 1>(0.f, v);
    v += dpp_f<DPP_SHR + 2>(0.f, v);
    v += dpp_f<DPP_SHR + 4>(0.f, v);
    v += dpp_f<DPP_SHR + 8>(0.f, v);
    v += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), DPP_BCAST15, 0xA, 0xF, false));
    v += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), DPP_BCAST31, 0xC, 0xF, false));
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// A barrier for what the workgroup shares in LDS: global accesses stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// ----------------------------------------------------------------- streams

// Accesses to data that this kernel does not touch again: marked so that
// caches let go of them first.
template <typename T>
__device__ __forceinline__ T load_once(const T* p) {
    return __builtin_nontemporal_load(p);
}
template <typename T>
__device__ __forceinline__ void store_once(void* p, T v) {
    __builtin_nontemporal_store(v, (T*)p);
}

// ----------------------------------------------------------------- numbers

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
// the same, at any even address (rows of odd width); one load or store all the same
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// 1 / (1 + e^-x) by the hardware's exp2 and reciprocal (1 ulp each).  The
// rounded product x log2 e costs |x| 2^-24 relative at most, and the constant,
// 0.22 2^-24 off, a quarter of that: 1.2e-6 at |x| = 16; its users round the
// result to 8 or 4 bits.  Below 2^-126 the reciprocal is 0.
__device__ __forceinline__ float sigmoid_fast(float x) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x * -1.44269504f));
}

// Four fp32 -> four e4m3 codes, round to nearest even, |x| <= 448 (NaN: code 0x7F).
__device__ __forceinline__ uint32_t e4m3_x4(float a, float b, float c, float d) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}
// Four e4m3 codes -> fp32.
__device__ __forceinline__ void e4m3_to_f32(uint32_t v, float* f) {
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)v, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)v, true);
    f[0] = lo.x;
    f[1] = lo.y;
    f[2] = hi.x;
    f[3] = hi.y;
}

// One group's scale amax / 448 (1 where that is 0; POW2: the smallest power of
// two that is at least it, from 2^-126 up, as value and E8M0 byte) and what turns
// values into codes: pre, which is 1 but for scales whose reciprocal may
// overflow, the reciprocal inv of the divisor s * pre, and what that is short of it.
struct GroupScale {
    float s, pre, inv, low;
    uint32_t byte;
};
constexpr float kTinyScale = 0x1p-100f;
template <bool POW2>
__device__ __forceinline__ GroupScale group_scale(float amax) {
    GroupScale g;
    // amax / 448 correctly rounded: the product with the rounded reciprocal, and its remainder
    const float q = amax * (1.f / 448.f);
    g.s = __builtin_fmaf(__builtin_fmaf(-448.f, q, amax), 1.f / 448.f, q);
    if (!(g.s >= kTinyScale)) {                          // 0, tiny, or NaN of an infinite amax
        g.s = amax / 448.f;
        if (!(g.s > 0.f)) g.s = 1.f;
    }
    g.pre = 1.f;
    g.byte = 0;
    if (POW2) {
        const uint32_t b = __float_as_uint(g.s);
        const uint32_t e = max((b >> 23) + ((b & 0x7FFFFFu) != 0u), 1u);   // amax finite: at most 247; inf: 255
        g.byte = e;
        g.s = __uint_as_float(e << 23);
        g.inv = e == 255u ? 0.f : __uint_as_float((254u - e) << 23);
        g.low = 0.f;
    } else {
        if (g.s < kTinyScale) g.pre = 0x1p+100f;
        const float d = g.s * g.pre;
        g.inv = __builtin_amdgcn_rcpf(d);
        g.low = d < __builtin_inff() ? __builtin_fmaf(-d, g.inv, 1.f) * g.inv : 0.f;
    }
    return g;
}

// x / s.  The product with the hardware's reciprocal (1 ulp) is within 2 ulp;
// EXACT adds the rest of the reciprocal before it rounds, which leaves 2^-45: in
// effect the rounded quotient.  bf16 values against a bf16 maximum meet e4m3's
// rounding borders exactly (one value in two hundred of normal data), both times a
// weight within an ulp, and there the last bit decides the code: dispatch, combine's
// backward pass, the SwiGLU checkpoint, the norm and bf16 rows into token groups take EXACT.
// Values that have no such common factor do so once in 2^20, and take the product.
template <bool EXACT>
__device__ __forceinline__ float quotient(float x, float inv, float low) {
    return EXACT ? __builtin_fmaf(x, inv, x * low) : x * inv;
}

// Quotient where pre is not 1: a scale down there may itself be rounded so
// coarsely (subnormals) that its largest value is past 448 times it.
template <bool EXACT = false>
__device__ __forceinline__ float tiny_quotient(float x, float pre, float inv, float low = 0.f) {
    const float q = quotient<EXACT>(x * pre, inv, low);
    return q != q ? q : fminf(fmaxf(q, -448.f), 448.f);
}

// N values of one group -> their codes, four to a word.
template <int N, bool EXACT = false>
__device__ __forceinline__ void quantize(const float* v, const GroupScale& g, uint32_t* q) {
    if (g.pre == 1.f) {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            q[i / 4] = e4m3_x4(quotient<EXACT>(v[i], g.inv, g.low), quotient<EXACT>(v[i + 1], g.inv, g.low),
                               quotient<EXACT>(v[i + 2], g.inv, g.low), quotient<EXACT>(v[i + 3], g.inv, g.low));
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            q[i / 4] = e4m3_x4(tiny_quotient<EXACT>(v[i], g.pre, g.inv, g.low),
                               tiny_quotient<EXACT>(v[i + 1], g.pre, g.inv, g.low),
                               tiny_quotient<EXACT>(v[i + 2], g.pre, g.inv, g.low),
                               tiny_quotient<EXACT>(v[i + 3], g.pre, g.inv, g.low));
    }
}

#endif  // __HIPCC__

}  // namespace moegg
