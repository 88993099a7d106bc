// rows.hpp -- pieces of 8 bf16 of a row: loads and stores at any even address,
// and to and from fp32.
#pragma once
#include <hip/hip_runtime.h>

#include "device.hpp"
#include "layer.hpp"

namespace moegg {

typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef uint32_t u32_a2 __attribute__((aligned(2)));

// Up to 8 bf16 of a row piece: one 16-byte load where all 8 are there, else pieces of
// 4, 2 and 1 (a row's last lane waits once then, not for each of up to 7).  Expert
// rows are streamed (ONCE).  Tokens and their gradients are not: they are small
// beside them and mostly just written, so that they come from the memory-side
// cache, which streaming loads do without.
template <bool ONCE>
__device__ __forceinline__ u32x4 load8(const uint16_t* p, int n) {
    if (n >= 8) return ONCE ? __builtin_nontemporal_load((const u32x4_a2*)p) : *(const u32x4_a2*)p;
    u32x4 v = {0, 0, 0, 0};
    if (n <= 0) return v;
    u32x2_a2 four = {0, 0};
    u32_a2 two = 0;
    uint16_t one = 0;
    if (n & 4) four = *(const u32x2_a2*)p;
    if (n & 2) two = *(const u32_a2*)(p + (n & 4));
    if (n & 1) one = p[n & 6];
    // 4, then 2, then 1 of them in a row: the later ones start at word 0 or 2, and one after that
    const uint32_t tail = n & 2 ? (uint32_t)two : (uint32_t)one, last = n & 2 ? (uint32_t)one : 0u;
    return n & 4 ? u32x4{four.x, four.y, tail, last} : u32x4{tail, last, 0, 0};
}
__device__ __forceinline__ void store8(uint16_t* p, u32x4 v, int n) {
    if (n >= 8) {
        __builtin_nontemporal_store(v, (u32x4_a2*)p);
        return;
    }
    if (n <= 0) return;
    if (n & 4) *(u32x2_a2*)p = u32x2{v.x, v.y};
    const uint32_t tail = n & 4 ? v.z : v.x, last = n & 4 ? v.w : v.y;
    if (n & 2) *(u32_a2*)(p + (n & 4)) = tail;
    if (n & 1) p[n & 6] = (uint16_t)(n & 2 ? last : tail);
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
