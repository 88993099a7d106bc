// rows.hpp -- pieces of 8 bf16 of a row: loads and stores at any even address,
// and to and from fp32.
#pragma once
#include <hip/hip_runtime.h>

#include "device.hpp"
#include "layer.hpp"

namespace moegg {

// Up to 8 bf16 of a row piece: one 16-byte load where all 8 are there.  Expert
// rows are streamed (ONCE).  Tokens and their gradients are not: they are small
// beside them and mostly just written, so that they come from the memory-side
// cache, which streaming loads do without.
template <bool ONCE>
__device__ __forceinline__ u32x4 load8(const uint16_t* p, int n) {
    if (n >= 8) return ONCE ? __builtin_nontemporal_load((const u32x4_a2*)p) : *(const u32x4_a2*)p;
    uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < n) v[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
    return u32x4{v[0], v[1], v[2], v[3]};
}
__device__ __forceinline__ void store8(uint16_t* p, u32x4 v, int n) {
    if (n >= 8) {
        __builtin_nontemporal_store(v, (u32x4_a2*)p);
        return;
    }
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < n) p[i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
}
__device__ __forceinline__ void unpack8(u32x4 v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(v[i]);
        f[2 * i + 1] = bf16_hi(v[i]);
    }
}

__device__ __forceinline__ u32x4 pack8(const float* f) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    return v;
}
__device__ __forceinline__ float amax8(const float* f, float m) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
    return m;
}

}  // namespace moegg
