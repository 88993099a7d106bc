// checkpoint.hip -- 8-bit activation checkpoints of the expert MLP: SwiGLU
// whose gate/up input is kept as e4m3 with fp32 1x128 scales, the backward
// pass that reads it, and the change from row scales to the token-group scales
// of the K-grouped weight gradient.
//
// All are bound by memory.  Gate and up columns alternate in blocks of 16 (the
// row order of W1), so 16 lanes take one row's unit of 256 gate/up columns =
// 128 columns of H: lane 2q + h has gate columns 32q + 8h .. + 7, the up columns
// 16 further on, and columns 16q + 8h .. + 7 of H.  A 128-column group of the
// checkpoint is 8 lanes and a group of H all 16, so each amax is three or four
// DPP steps; codes of neighbouring lanes are exchanged so that each lane stores
// 16 contiguous bytes.
#include <hip/hip_runtime.h>

#include "device.hpp"
#include "layer.hpp"

namespace moegg {

constexpr int kThreads = 256;
constexpr int kXcds = 8;
constexpr int kUnit = 256;                // gate/up columns of 16 lanes

// Codes of 8 gate and 8 up columns <-> 16 contiguous codes of a unit at lane * 16.
__device__ __forceinline__ u32x4 join_codes(u32x2 g, u32x2 u, bool odd) {
    const u32x2 send = odd ? g : u;
    u32x2 got;
    got.x = dpp<DPP_XOR1>(0, send.x);
    got.y = dpp<DPP_XOR1>(0, send.y);
    return odd ? u32x4{got.x, got.y, u.x, u.y} : u32x4{g.x, g.y, got.x, got.y};
}
__device__ __forceinline__ void split_codes(u32x4 c, bool odd, u32x2& g, u32x2& u) {
    const u32x2 lo = {c.x, c.y}, hi = {c.z, c.w};
    const u32x2 send = odd ? lo : hi;
    u32x2 got;
    got.x = dpp<DPP_XOR1>(0, send.x);
    got.y = dpp<DPP_XOR1>(0, send.y);
    g = odd ? got : lo;
    u = odd ? hi : got;
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
__device__ __forceinline__ u32x2 quantize8(const float* f, const GroupScale& g) {
    return u32x2{quantize_x4(f[0], f[1], f[2], f[3], g), quantize_x4(f[4], f[5], f[6], f[7], g)};
}
__device__ __forceinline__ float amax8(const float* f, float m) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
    return m;
}

// One scale of a row-major operand: group kg of row `row`.
template <OperandFormat FMT>
__device__ __forceinline__ void store_scale(void* p, int64_t row, int kg, int groups, int rows, float s) {
    if (FMT == kRows) ((float*)p)[row * groups + kg] = s;
    if (FMT == kKm) ((float*)p)[(int64_t)kg * rows + row] = s;
}

// Rows of all experts: the sum of the counts, negative ones read as 0, at most `rows`.
__device__ __forceinline__ int valid_rows(const int32_t* m_sizes, int G, int rows) {
    const int lane = threadIdx.x & 63;
    uint32_t sum = 0;                                    // sum <= rows < 2^31 and a count < 2^31: no overflow
    for (int e = lane; e < G; e += 64) sum = min(sum + (uint32_t)max(m_sizes[e], 0), (uint32_t)rows);
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) sum = min(sum + (uint32_t)__shfl_xor((int)sum, off, 64), (uint32_t)rows);
    return __builtin_amdgcn_readfirstlane((int)sum);
}

// Units of this workgroup: XCD x works on the x-th eighth of the rows, each of
// its workgroups on a run of them.
struct UnitRange {
    int64_t at, end;
};
__device__ __forceinline__ UnitRange unit_range(int64_t units) {
    const int64_t order = (int64_t)(blockIdx.x % kXcds) * (gridDim.x / kXcds) + blockIdx.x / kXcds;
    const int64_t per = ((units + gridDim.x - 1) / gridDim.x + 15) / 16 * 16;
    return {min(units, order * per) + (threadIdx.x >> 4), min(units, (order + 1) * per)};
}

// ----------------------------------------------------------------- forward

template <OperandFormat FMT>
__global__ __launch_bounds__(kThreads) void swiglu_checkpoint_kernel(CheckpointArgs a) {
    const int upr = a.W / 128;                           // units of a row
    const UnitRange r = unit_range((int64_t)valid_rows(a.m_sizes, a.G, a.rows) * upr);
    const int l16 = threadIdx.x & 15;
    const bool odd = l16 & 1;
    for (int64_t u = r.at; u < r.end; u += kThreads / 16) {
        const uint16_t* p = (const uint16_t*)a.in + u * kUnit + 32 * (l16 >> 1) + 8 * odd;
        float g[8], v[8], h[8];
        unpack8(*(const u32x4*)p, g);
        unpack8(*(const u32x4*)(p + 16), v);
        const GroupScale cs = group_scale<false>(max8(amax8(v, amax8(g, 0.f))));
        *(u32x4*)(a.ckpt + u * kUnit + l16 * 16) = join_codes(quantize8(g, cs), quantize8(v, cs), odd);
        if ((l16 & 7) == 0) a.ckpt_scale[u * 2 + (l16 >> 3)] = cs.s;
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = g[i] * sigmoid_fast(g[i]) * v[i];
        if (FMT == kBf16) {
            *(u32x4*)((uint16_t*)a.row_out + u * 128 + l16 * 8) = pack8(h);
        } else {
            const GroupScale hs = group_scale<false>(max16(amax8(h, 0.f)));
            *(u32x2*)((uint8_t*)a.row_out + u * 128 + l16 * 8) = quantize8(h, hs);
            if (l16 == 0) {
                const int64_t row = u / upr;
                store_scale<FMT>(a.row_scale, row, (int)(u - row * upr), upr, a.rows, hs.s);
            }
        }
    }
}

// ----------------------------------------------------------------- backward

// One lane's 8 columns: gradients of gate and up, and H again, from the
// checkpoint's values and dH.  With s = sigmoid(g):
//   du = dh g s,   dg = dh u (s + g s (1 - s)),   h = g s u.
__device__ __forceinline__ void swiglu_grad8(u32x4 codes, float scale, u32x4 dh, bool odd, float* dg, float* du,
                                             float* h) {
    u32x2 gc, uc;
    split_codes(codes, odd, gc, uc);
    float g[8], u[8], d[8];
    e4m3_to_f32(gc.x, g);
    e4m3_to_f32(gc.y, g + 4);
    e4m3_to_f32(uc.x, u);
    e4m3_to_f32(uc.y, u + 4);
    unpack8(dh, d);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float gv = g[i] * scale, uv = u[i] * scale;
        const float s = sigmoid_fast(gv), gs = gv * s;
        du[i] = d[i] * gs;
        dg[i] = d[i] * uv * (s + __builtin_fmaf(-gs, s, gs));
        h[i] = gs * uv;
    }
}

__global__ __launch_bounds__(kThreads) void swiglu_backward_kernel(CheckpointArgs a) {
    const int upr = a.W / 128;
    const UnitRange r = unit_range((int64_t)valid_rows(a.m_sizes, a.G, a.rows) * upr);
    const int l16 = threadIdx.x & 15;
    const bool odd = l16 & 1;
    for (int64_t u = r.at; u < r.end; u += kThreads / 16) {
        const u32x4 codes = *(const u32x4*)(a.ckpt + u * kUnit + l16 * 16);
        const u32x4 dh = *(const u32x4*)((const uint16_t*)a.in + u * 128 + l16 * 8);
        const float scale = a.ckpt_scale[u * 2 + (l16 >> 3)];
        float dg[8], du[8], h[8];
        swiglu_grad8(codes, scale, dh, odd, dg, du, h);
        uint16_t* p = (uint16_t*)a.row_out + u * kUnit + 32 * (l16 >> 1) + 8 * odd;
        *(u32x4*)p = pack8(dg);
        *(u32x4*)(p + 16) = pack8(du);
        *(u32x4*)((uint16_t*)a.H + u * 128 + l16 * 8) = pack8(h);
    }
}

// ----------------------------------------------------------------- token groups

// The token group (up to 128 consecutive rows of one expert) with index `want`,
// numbered across experts in order as the K-grouped weight gradient numbers
// them.  Every wave finds it for itself: prefix sums of 64 experts at a time.
struct TokenGroup {
    int row, n;                                          // n = 0: there is no such group
};
__device__ __forceinline__ TokenGroup token_group(const int32_t* m_sizes, int G, int rows, int want) {
    const int lane = threadIdx.x & 63;
    uint32_t off = 0;
    int groups = 0;
    for (int e0 = 0; e0 < G; e0 += 64) {
        const uint32_t m = e0 + lane < G ? (uint32_t)max(m_sizes[e0 + lane], 0) : 0u;
        uint32_t end = m;                                // saturating: ends stay within [0, rows]
        end = min(end, (uint32_t)rows);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t o = (uint32_t)__shfl_up((int)end, d, 64);
            if (lane >= d) end = min(end + o, (uint32_t)rows);
        }
        end = min(end + off, (uint32_t)rows);
        uint32_t start = (uint32_t)__shfl_up((int)end, 1, 64);
        if (lane == 0) start = off;
        const int n = (int)(end - start + 127) / 128;
        int gend = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(gend, d, 64);
            if (lane >= d) gend += o;
        }
        gend += groups;
        const uint64_t who = __ballot(want < gend);
        if (who) {
            const int src = __builtin_ctzll(who);
            const int s = __builtin_amdgcn_readlane((int)start, src), e = __builtin_amdgcn_readlane((int)end, src);
            const int first = __builtin_amdgcn_readlane(gend - n, src);
            const int row = s + (want - first) * 128;
            return {row, min(128, e - row)};
        }
        off = (uint32_t)__builtin_amdgcn_readlane((int)end, 63);
        groups = __builtin_amdgcn_readlane(gend, 63);
    }
    return {0, 0};
}

// Column maxima of the wave's four 16-lane rows: N values a lane (columns
// i of the lane's own N) -> N / 4, of column 4i + {0, 2, 1, 3}[lane / 16].
template <int N>
__device__ __forceinline__ void reduce_rows(const float (&v)[N], float (&out)[N / 4]) {
    float r[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[2 * i]), __float_as_uint(v[2 * i + 1]), false, false);
        r[i] = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
    }
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(r[2 * i]), __float_as_uint(r[2 * i + 1]), false, false);
        out[i] = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
    }
}

// Column scales of a tile: maxima of WAVES waves in red -> scale and inverse in
// LDS, scale stored to k_scale.  tiny: some scale needs tiny_quotient.
template <bool E8M0>
__device__ __forceinline__ void column_scale(float amax, float* s_out, float* inv_out, int* tiny, void* k_scale,
                                             int64_t at, bool store) {
    const GroupScale g = group_scale<E8M0>(amax);
    *s_out = g.s;
    *inv_out = g.inv;
    if (g.s < kTinyScale) *tiny = 1;
    if (store) {
        if (E8M0) ((uint8_t*)k_scale)[at] = (uint8_t)g.byte;
        else ((float*)k_scale)[at] = g.s;
    }
}

template <int N>
__device__ __forceinline__ void quantize_columns(const float* v, const float* s, const float* inv, bool tiny,
                                                 uint32_t (&q)[N / 4]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        if (tiny) {
            q[i / 4] = e4m3_x4(tiny_quotient(v[i], s[i]), tiny_quotient(v[i + 1], s[i + 1]),
                               tiny_quotient(v[i + 2], s[i + 2]), tiny_quotient(v[i + 3], s[i + 3]));
        } else {
            q[i / 4] = e4m3_x4(v[i] * inv[i], v[i + 1] * inv[i + 1], v[i + 2] * inv[i + 2], v[i + 3] * inv[i + 3]);
        }
    }
}

// ----------------------------------------------------------------- fp8 backward

// A workgroup takes a token group x 256 gate/up columns: 8 waves, 32 rows at
// a time, 4 times.  The gradients stay in registers in fp32 between the row
// scales (DPP) and the column scales (registers, lane swaps, LDS), so that the
// checkpoint and dH are read and SwiGLU is evaluated once.
constexpr int kBwdThreads = 512, kBwdWaves = kBwdThreads / 64, kBwdPasses = 128 / (kBwdThreads / 16);

template <OperandFormat FMT, bool E8M0>
__global__ __launch_bounds__(kBwdThreads, 2) void swiglu_backward_fp8_kernel(CheckpointArgs a) {
    constexpr int C = kUnit + 128;                       // columns of dGU (in lane order), then of H
    __shared__ float red_s[kBwdWaves][C];
    __shared__ float s_s[C], inv_s[C];
    __shared__ int tiny_s;
    const int upr = a.W / 128;
    const int want = blockIdx.x / upr, unit = blockIdx.x % upr;
    const TokenGroup tg = token_group(a.m_sizes, a.G, a.rows, want);
    if (tg.n <= 0) return;
    const int lane = threadIdx.x & 63, l16 = lane & 15, wave = threadIdx.x >> 6;
    const bool odd = l16 & 1;
    if (threadIdx.x == 0) tiny_s = 0;
    float v[kBwdPasses][24];                             // 8 of gate, 8 of up, 8 of H
    const int r0 = wave * 4 + (lane >> 4);
#pragma unroll
    for (int p = 0; p < kBwdPasses; ++p) {
        const int r = r0 + p * (kBwdThreads / 16);
        const bool in = r < tg.n;
        const int64_t row = tg.row + r, u = row * upr + unit;
        u32x4 codes = {0, 0, 0, 0}, dh = {0, 0, 0, 0};
        float scale = 0.f;
        if (in) {
            codes = *(const u32x4*)(a.ckpt + u * kUnit + l16 * 16);
            dh = *(const u32x4*)((const uint16_t*)a.in + u * 128 + l16 * 8);
            scale = a.ckpt_scale[u * 2 + (l16 >> 3)];
        }
        swiglu_grad8(codes, scale, dh, odd, v[p], v[p] + 8, v[p] + 16);
        const GroupScale g = group_scale<false>(max8(amax8(v[p] + 8, amax8(v[p], 0.f))));
        const u32x4 q = join_codes(quantize8(v[p], g), quantize8(v[p] + 8, g), odd);
        if (in) {
            *(u32x4*)((uint8_t*)a.row_out + u * kUnit + l16 * 16) = q;
            if ((l16 & 7) == 0) store_scale<FMT>(a.row_scale, row, unit * 2 + (l16 >> 3), upr * 2, a.rows, g.s);
        }
    }
    float m[24], red[6];
#pragma unroll
    for (int i = 0; i < 24; ++i) {
        m[i] = 0.f;
#pragma unroll
        for (int p = 0; p < kBwdPasses; ++p) m[i] = fmaxf(m[i], fabsf(v[p][i]));
    }
    reduce_rows<24>(m, red);
    const int sub = lane >> 4, perm = sub == 1 ? 2 : (sub == 2 ? 1 : sub);
#pragma unroll
    for (int i = 0; i < 4; ++i) red_s[wave][l16 * 16 + 4 * i + perm] = red[i];
#pragma unroll
    for (int i = 0; i < 2; ++i) red_s[wave][kUnit + l16 * 8 + 4 * i + perm] = red[4 + i];
    __syncthreads();
    if (threadIdx.x < C) {
        const int c = threadIdx.x;
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < kBwdWaves; ++w) x = fmaxf(x, red_s[w][c]);
        const bool store = want < a.scale_groups;
        if (c < kUnit) {
            const int l = c >> 4, i = c & 15;            // lane l: 8 gate columns, then the 8 up columns 16 further on
            const int col = 32 * (l >> 1) + 8 * (l & 1) + (i < 8 ? i : i + 8);
            column_scale<E8M0>(x, &s_s[c], &inv_s[c], &tiny_s, a.k_scale,
                               (int64_t)want * (2 * a.W) + unit * kUnit + col, store);
        } else {
            column_scale<E8M0>(x, &s_s[c], &inv_s[c], &tiny_s, a.hk_scale, (int64_t)want * a.W + unit * 128 + c - kUnit,
                               store);
        }
    }
    __syncthreads();
    const bool tiny = tiny_s;
#pragma unroll
    for (int p = 0; p < kBwdPasses; ++p) {
        const int r = r0 + p * (kBwdThreads / 16);
        const int64_t u = (int64_t)(tg.row + r) * upr + unit;
        uint32_t q[4], qh[2];
        quantize_columns<16>(v[p], s_s + l16 * 16, inv_s + l16 * 16, tiny, q);
        quantize_columns<8>(v[p] + 16, s_s + kUnit + l16 * 8, inv_s + kUnit + l16 * 8, tiny, qh);
        const u32x4 c = join_codes(u32x2{q[0], q[1]}, u32x2{q[2], q[3]}, odd);
        if (r < tg.n) {
            *(u32x4*)(a.k_out + u * kUnit + l16 * 16) = c;
            *(u32x2*)(a.hk_out + u * 128 + l16 * 8) = u32x2{qh[0], qh[1]};
        }
    }
}

// ----------------------------------------------------------------- row scales -> token groups

// A workgroup takes a token group x 256 columns: 4 waves, 16 rows at a time, 8
// times.  The codes (or bf16 values) stay in registers as they were read, and
// are scaled twice: for the columns' maxima and for the new codes.
constexpr int kKgPasses = 128 / (kThreads / 16);

template <OperandFormat FMT, bool E8M0>
__global__ __launch_bounds__(kThreads) void k_groups_kernel(CheckpointArgs a) {
    __shared__ float red_s[kThreads / 64][kUnit];
    __shared__ float s_s[kUnit], inv_s[kUnit];
    __shared__ int tiny_s;
    constexpr int RAW = FMT == kBf16 ? 2 : 1;
    const int upr = a.W / kUnit, groups = a.W / kGroup;
    const int want = blockIdx.x / upr, unit = blockIdx.x % upr;
    const TokenGroup tg = token_group(a.m_sizes, a.G, a.rows, want);
    if (tg.n <= 0) return;
    const int lane = threadIdx.x & 63, l16 = lane & 15, wave = threadIdx.x >> 6;
    if (threadIdx.x == 0) tiny_s = 0;
    const int r0 = wave * 4 + (lane >> 4), kg = unit * 2 + (l16 >> 3);
    u32x4 raw[kKgPasses][RAW];
    float scale[kKgPasses];
#pragma unroll
    for (int p = 0; p < kKgPasses; ++p) {
        const int r = r0 + p * (kThreads / 16);
        const int64_t row = tg.row + r;
#pragma unroll
        for (int i = 0; i < RAW; ++i) raw[p][i] = u32x4{0, 0, 0, 0};
        scale[p] = 0.f;
        if (r < tg.n) {
            if (FMT == kBf16) {
                const u32x4* q = (const u32x4*)((const uint16_t*)a.in + row * a.W + unit * kUnit + l16 * 16);
                raw[p][0] = q[0];
                raw[p][RAW - 1] = q[1];
            } else {
                raw[p][0] = *(const u32x4*)((const uint8_t*)a.in + row * a.W + unit * kUnit + l16 * 16);
                scale[p] = FMT == kRows ? a.in_scale[row * groups + kg] : a.in_scale[(int64_t)kg * a.rows + row];
            }
        }
    }
    auto values = [&](int p, float (&v)[16]) {
        if (FMT == kBf16) {
            unpack8(raw[p][0], v);
            unpack8(raw[p][RAW - 1], v + 8);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) e4m3_to_f32(raw[p][0][i], v + 4 * i);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] *= scale[p];
        }
    };
    float m[16], red[4];
#pragma unroll
    for (int i = 0; i < 16; ++i) m[i] = 0.f;
#pragma unroll
    for (int p = 0; p < kKgPasses; ++p) {
        float v[16];
        values(p, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) m[i] = fmaxf(m[i], fabsf(v[i]));
    }
    reduce_rows<16>(m, red);
    const int sub = lane >> 4, perm = sub == 1 ? 2 : (sub == 2 ? 1 : sub);
#pragma unroll
    for (int i = 0; i < 4; ++i) red_s[wave][l16 * 16 + 4 * i + perm] = red[i];
    __syncthreads();
    {
        const int c = threadIdx.x;
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < kThreads / 64; ++w) x = fmaxf(x, red_s[w][c]);
        column_scale<E8M0>(x, &s_s[c], &inv_s[c], &tiny_s, a.k_scale, (int64_t)want * a.W + unit * kUnit + c,
                           want < a.scale_groups);
    }
    __syncthreads();
    const bool tiny = tiny_s;
#pragma unroll
    for (int p = 0; p < kKgPasses; ++p) {
        const int r = r0 + p * (kThreads / 16);
        float v[16];
        uint32_t q[4];
        values(p, v);
        quantize_columns<16>(v, s_s + l16 * 16, inv_s + l16 * 16, tiny, q);
        if (r < tg.n)
            *(u32x4*)(a.k_out + (int64_t)(tg.row + r) * a.W + unit * kUnit + l16 * 16) = u32x4{q[0], q[1], q[2], q[3]};
    }
}

// ----------------------------------------------------------------- launches

// Workgroups of the row-wise kernels: 8 a CU, fewer where there are not that many units.
static dim3 row_grid(const CheckpointArgs& a) {
    const int64_t units = (int64_t)a.rows * (a.W / 128), blocks = (units + 15) / 16;
    return dim3((unsigned)(blocks >= 2048 ? 2048 : (blocks + kXcds - 1) / kXcds * kXcds));
}

// Token groups of any histogram: each expert can leave one short group.
static int64_t most_groups(const CheckpointArgs& a) {
    const int64_t n = (int64_t)a.rows / 128 + a.G;
    return n < a.rows ? n : a.rows;
}

hipError_t launch_swiglu_checkpoint(const CheckpointArgs& a, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    if (a.fmt == kBf16) swiglu_checkpoint_kernel<kBf16><<<row_grid(a), kThreads, 0, s>>>(a);
    else if (a.fmt == kRows) swiglu_checkpoint_kernel<kRows><<<row_grid(a), kThreads, 0, s>>>(a);
    else swiglu_checkpoint_kernel<kKm><<<row_grid(a), kThreads, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_swiglu_checkpoint_backward(const CheckpointArgs& a, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    swiglu_backward_kernel<<<row_grid(a), kThreads, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_swiglu_checkpoint_backward_fp8(const CheckpointArgs& a, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    const dim3 grid((unsigned)(most_groups(a) * (a.W / 128)));
    if (a.fmt == kRows) {
        if (a.k_e8m0) swiglu_backward_fp8_kernel<kRows, true><<<grid, kBwdThreads, 0, s>>>(a);
        else swiglu_backward_fp8_kernel<kRows, false><<<grid, kBwdThreads, 0, s>>>(a);
    } else {
        if (a.k_e8m0) swiglu_backward_fp8_kernel<kKm, true><<<grid, kBwdThreads, 0, s>>>(a);
        else swiglu_backward_fp8_kernel<kKm, false><<<grid, kBwdThreads, 0, s>>>(a);
    }
    return hipGetLastError();
}

template <OperandFormat FMT>
static void k_groups_as(const CheckpointArgs& a, dim3 grid, hipStream_t s) {
    if (a.k_e8m0) k_groups_kernel<FMT, true><<<grid, kThreads, 0, s>>>(a);
    else k_groups_kernel<FMT, false><<<grid, kThreads, 0, s>>>(a);
}

hipError_t launch_checkpoint_to_k_groups(const CheckpointArgs& a, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    const dim3 grid((unsigned)(most_groups(a) * (a.W / kUnit)));
    if (a.fmt == kBf16) k_groups_as<kBf16>(a, grid, s);
    else if (a.fmt == kRows) k_groups_as<kRows>(a, grid, s);
    else k_groups_as<kKm>(a, grid, s);
    return hipGetLastError();
}

}  // namespace moegg
