// logits.hpp -- rows of router logits: how they are read, a few neighbouring
// experts a lane, and how rows of their type are stored.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moegg {

constexpr float kFltMax = 3.402823466e+38f;

// What routing reads as a logit: NaN is no expert, +inf the largest number.
// -0 becomes +0, so that equal logits have equal keys.
__device__ __forceinline__ float clean_logit(float l) {
    return l != l ? -__builtin_inff() : __builtin_amdgcn_fmed3f(l, -__builtin_inff(), kFltMax) + 0.f;
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

}  // namespace moegg
