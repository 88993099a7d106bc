// checkpoint.hip -- 8-bit activation checkpoints of the expert MLP: SwiGLU
// whose gate/up input is kept as e4m3 with fp32 1x128 scales, the backward
// pass that reads it, and the change from row scales to the token-group scales
// of the K-grouped weight gradient.
//
// All are bound by memory.  Gate and up columns alternate in blocks of 16 (the
// row order of W1).  A lane computes 8 columns of H from 8 gate columns and the
// 8 up columns 16 further on; lanes exchange halves by DPP so that every load
// and store is 16 contiguous bytes a lane and whole lines an instruction.
#include <hip/hip_runtime.h>

#include "device.hpp"
#include "layer.hpp"
#include "rows.hpp"

namespace moegg {

constexpr int kThreads = 256;
constexpr int kUnit = 256;                // gate/up columns of 16 lanes

// Codes of 8 gate and 8 up columns <-> 16 contiguous codes of a unit at lane * 16.
__device__ __forceinline__ u32x4 join_codes(u32x2 g, u32x2 u, bool odd) {
    const u32x2 send = odd ? g : u;
    const u32x2 got = {lane_of<DPP_XOR1>(send.x), lane_of<DPP_XOR1>(send.y)};
    return odd ? u32x4{got.x, got.y, u.x, u.y} : u32x4{g.x, g.y, got.x, got.y};
}
__device__ __forceinline__ void split_codes(u32x4 c, bool odd, u32x2& g, u32x2& u) {
    const u32x2 lo = {c.x, c.y}, hi = {c.z, c.w};
    const u32x2 send = odd ? lo : hi;
    const u32x2 got = {lane_of<DPP_XOR1>(send.x), lane_of<DPP_XOR1>(send.y)};
    g = odd ? got : lo;
    u = odd ? hi : got;
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

// Runs of the row-wise kernels, which take 16 units a workgroup: 32 of them are
// the 32 rows that share a line of transposed scales at 2048 columns of H.  Runs
// of 1 to 1024 are within 1 %; a workgroup that loops over its share of the
// rows instead of taking one piece needs 103 us where this takes 82.
constexpr int kRowRun = 32;

// ----------------------------------------------------------------- forward

// A lane's part of a unit of 256 gate/up columns: half `odd` (8 gate and 8 up
// columns) of its 32-column block `block`.  Lanes 4q .. 4q + 3 have blocks q and
// q + 4, one in each 128-column half of the unit.
struct UnitLane {
    int l16;
    bool odd, upper;                                     // upper: block q + 4
    int block;
    __device__ __forceinline__ UnitLane()
        : l16(threadIdx.x & 15), odd(l16 & 1), upper(l16 & 2), block((upper ? 4 : 0) + (l16 >> 2)) {}
    __device__ __forceinline__ int codes() const { return block * 32 + odd * 16; }   // 16 bytes of the unit
    __device__ __forceinline__ int h() const { return block * 16 + odd * 8; }         // 8 columns of H
};
// 16-byte pieces l16 of a unit's two halves <-> gate and up columns of the lane's block (bf16).
__device__ __forceinline__ u32x4 from_lane2(u32x4 v) {
    return u32x4{lane_of<DPP_XOR2>(v.x), lane_of<DPP_XOR2>(v.y), lane_of<DPP_XOR2>(v.z), lane_of<DPP_XOR2>(v.w)};
}
__device__ __forceinline__ void split_halves(u32x4 first, u32x4 second, bool upper, u32x4& gate, u32x4& up) {
    const u32x4 got = from_lane2(upper ? first : second);
    gate = upper ? got : first;
    up = upper ? second : got;
}
__device__ __forceinline__ void join_halves(u32x4 gate, u32x4 up, bool upper, u32x4& first, u32x4& second) {
    const u32x4 got = from_lane2(upper ? gate : up);
    first = upper ? got : gate;
    second = upper ? up : got;
}
// Maximum over the 8 lanes that share a 128-column half, of a float that is not negative.
__device__ __forceinline__ float max_half(float f) {
    uint32_t v = __float_as_uint(f);
    v = max(v, lane_of<DPP_XOR1>(v));
    v = max(v, lane_of<DPP_ROR4>(v));
    return __uint_as_float(max(v, lane_of<DPP_ROR8>(v)));
}

// 32768 rows of 4096 gate/up columns, H in e4m3: 82 us, 5.8 TB/s of the bytes it
// has to move (80 us with the checkpoint's quotients 2 ulp off).
template <OperandFormat FMT>
__global__ __launch_bounds__(kThreads) void swiglu_checkpoint_kernel(CheckpointArgs a) {
    const int upr = a.W / 128;                           // units of a row
    const UnitLane at;
    const int64_t u = work_position<kRowRun>() * (kThreads / 16) + (threadIdx.x >> 4);
    if (u < (int64_t)valid_rows(a.m_sizes, a.G, a.rows) * upr) {
        const uint16_t* p = (const uint16_t*)a.in + u * kUnit + at.l16 * 8;
        u32x4 gate, up;
        split_halves(load_once((const u32x4*)p), load_once((const u32x4*)(p + 128)), at.upper, gate, up);
        float gu[16], h[8];                              // 8 of gate, 8 of up
        unpack8(gate, gu);
        unpack8(up, gu + 8);
        const GroupScale cs = group_scale<false>(max_half(amax8(gu + 8, amax8(gu, 0.f))));
        uint32_t q[4];
        quantize<16, true>(gu, cs, q);                   // bf16 values: the rounded quotient
        store_once(a.ckpt + u * kUnit + at.codes(), join_codes(u32x2{q[0], q[1]}, u32x2{q[2], q[3]}, at.odd));
        if ((at.l16 & 13) == 0) a.ckpt_scale[u * 2 + at.upper] = cs.s;
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = gu[i] * sigmoid_fast(gu[i]) * gu[8 + i];
        if (FMT == kBf16) {
            store_once((uint16_t*)a.row_out + u * 128 + at.h(), pack8(h));
        } else {
            const GroupScale hs = group_scale<false>(max16(amax8(h, 0.f)));
            uint32_t hq[2];
            quantize<8>(h, hs, hq);
            store_once((uint8_t*)a.row_out + u * 128 + at.h(), u32x2{hq[0], hq[1]});
            if (at.l16 == 0) {
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

// 8048 rows of 4096 gate/up columns: 29 us, 5.7 TB/s.
__global__ __launch_bounds__(kThreads) void swiglu_backward_kernel(CheckpointArgs a) {
    const int upr = a.W / 128;
    const UnitLane at;
    const int64_t u = work_position<kRowRun>() * (kThreads / 16) + (threadIdx.x >> 4);
    if (u < (int64_t)valid_rows(a.m_sizes, a.G, a.rows) * upr) {
        const u32x4 codes = load_once((const u32x4*)(a.ckpt + u * kUnit + at.codes()));
        const u32x4 dh = load_once((const u32x4*)((const uint16_t*)a.in + u * 128 + at.h()));
        const float scale = a.ckpt_scale[u * 2 + at.upper];
        float dg[8], du[8], h[8];
        swiglu_grad8(codes, scale, dh, at.odd, dg, du, h);
        u32x4 first, second;
        join_halves(pack8(dg), pack8(du), at.upper, first, second);
        uint16_t* p = (uint16_t*)a.row_out + u * kUnit + at.l16 * 8;
        store_once(p, first);
        store_once(p + 128, second);
        store_once((uint16_t*)a.H + u * 128 + at.h(), pack8(h));
    }
}

// ----------------------------------------------------------------- token groups

// The token group (up to 128 consecutive rows of one expert) with index `want`,
// numbered across experts in order as the K-grouped weight gradient numbers
// them.  Every wave finds it for itself: prefix sums of 64 experts at a time, which
// few experts hide; the same 32768 rows over 64, 256 and 1024 experts take the fp8
// backward 114, 168 and 620 us and the token-group scales 85, 105 and 367 us.
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

// A column's scale: pre, inverse and (not NULL) what that is short into LDS, the scale itself to k_scale.
// tiny: some column has a pre that is not 1.
template <bool E8M0>
__device__ __forceinline__ void column_scale(float amax, float* pre, float* inv, float* low, int* tiny, void* k_scale,
                                             int64_t at, bool store) {
    const GroupScale g = group_scale<E8M0>(amax);
    *pre = g.pre;
    *inv = g.inv;
    if (low) *low = g.low;
    if (g.pre != 1.f) *tiny = 1;
    if (store) {
        if (E8M0) ((uint8_t*)k_scale)[at] = (uint8_t)g.byte;
        else ((float*)k_scale)[at] = g.s;
    }
}

// low: what the inverses are short of (EXACT: the rounded quotient), else not of use.
template <int N, bool EXACT>
__device__ __forceinline__ void quantize_columns(const float* v, const float* pre, const float* inv, const float* low,
                                                 bool tiny, uint32_t (&q)[N / 4]) {
    if (!tiny) {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            q[i / 4] = e4m3_x4(quotient<EXACT>(v[i], inv[i], low[i]), quotient<EXACT>(v[i + 1], inv[i + 1], low[i + 1]),
                               quotient<EXACT>(v[i + 2], inv[i + 2], low[i + 2]),
                               quotient<EXACT>(v[i + 3], inv[i + 3], low[i + 3]));
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            q[i / 4] = e4m3_x4(tiny_quotient<EXACT>(v[i], pre[i], inv[i], low[i]),
                               tiny_quotient<EXACT>(v[i + 1], pre[i + 1], inv[i + 1], low[i + 1]),
                               tiny_quotient<EXACT>(v[i + 2], pre[i + 2], inv[i + 2], low[i + 2]),
                               tiny_quotient<EXACT>(v[i + 3], pre[i + 3], inv[i + 3], low[i + 3]));
    }
}

// ----------------------------------------------------------------- fp8 backward

// A workgroup takes a token group x 128 gate/up columns (8 lanes a row): 4
// waves, 32 rows at a time, 4 times.  The gradients stay in registers in fp32
// between the row scales (DPP) and the column scales (registers, lane swaps,
// LDS), so that the checkpoint and dH are read and SwiGLU is evaluated once.
// Rows past the group are out of their buffers' range: they read as 0 and
// their stores are dropped.
// 32768 rows of 4096 columns: 114 us, 5.4 TB/s, with the VALU busy for two
// thirds of that.  148 registers hold three workgroups a CU.  What counts besides
// is where the chip works at one time: runs of 2, 16, 17 and 64 neighbouring units
// to an XCD take 139, 121, 114 and 129 us (odd runs of 11 to 21 are alike, even ones
// put the XCDs at equal distances in powers of two), cached instead of streaming
// accesses 132 us.  Only H_k's stores are cached: a unit writes half lines of it,
// which meet their other halves in L2 (streamed: 3 us more).
// Earlier forms: SwiGLU evaluated again for the columns, in 121 registers, 166 us
// (the VALU was the limit); 256 columns and 512 threads 187 us (one workgroup a
// CU); 512 threads of half the registers 135 us; workgroups that go on to further
// tiles and load them ahead 167 us.
constexpr int kBwdCols = 128, kBwdRows = kThreads / 8, kBwdPasses = 128 / kBwdRows;
constexpr int kBwdRun = 17;

template <bool ONCE = true>
__device__ __forceinline__ u32x4 buffer_load16(__amdgpu_buffer_rsrc_t rs, uint32_t off, uint32_t soff) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, (int)off, (int)soff, ONCE ? CP_NT : 0));
}

// Past the end of every buffer here (2^31 bytes at most), and no step added to it wraps.
constexpr uint32_t kOutOfRange = 0x80000000u;

template <OperandFormat FMT, bool E8M0>
__global__ __launch_bounds__(kThreads) void swiglu_backward_fp8_kernel(CheckpointArgs a) {
    constexpr int C = kBwdCols + kBwdCols / 2;           // columns of dGU (in lane order), then of H
    __shared__ float red_s[kThreads / 64][C];
    __shared__ float pre_s[C], inv_s[C];
    __shared__ int tiny_s;
    const int upr = a.W / 64;                            // units of a row
    const int64_t tile = work_position<kBwdRun>();
    const int want = (int)(tile / upr), unit = (int)(tile - (int64_t)want * upr);
    const TokenGroup tg = token_group(a.m_sizes, a.G, a.rows, want);
    if (tg.n <= 0) return;
    const int lane = threadIdx.x & 63, l8 = lane & 7;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const bool odd = l8 & 1;
    if (threadIdx.x == 0) tiny_s = 0;
    const int64_t u = (int64_t)tg.row * upr + unit;      // units before the tile's first
    const uint32_t units = (uint32_t)tg.n * upr - unit;  // from there to the group's end
    const int r0 = wave * 8 + (lane >> 3);
    const uint32_t at = (uint32_t)(r0 * upr);
    u32x4 codes[kBwdPasses], dh[kBwdPasses];
    float scale[kBwdPasses];
    {
        auto ck = make_rsrc(a.ckpt + u * kBwdCols, units * kBwdCols);
        auto in = make_rsrc((const uint16_t*)a.in + u * 64, units * 128);
        auto sc = make_rsrc(a.ckpt_scale + u, units * 4);
#pragma unroll
        for (int p = 0; p < kBwdPasses; ++p) {
            const uint32_t step = (uint32_t)(p * kBwdRows * upr);
            codes[p] = buffer_load16(ck, at * kBwdCols + l8 * 16, step * kBwdCols);
            dh[p] = buffer_load16(in, at * 128 + l8 * 16, step * 128);
            scale[p] = __uint_as_float(
                (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(sc, (int)(at * 4), (int)(step * 4), 0));
        }
    }
    float v[kBwdPasses][24];                             // 8 of gate, 8 of up, 8 of H
    {
        auto out = make_rsrc((const uint8_t*)a.row_out + u * kBwdCols, units * kBwdCols);
        auto out_scale = FMT == kRows ? make_rsrc((const float*)a.row_scale + u, units * 4)
                                      : make_rsrc((const float*)a.row_scale + (int64_t)unit * a.rows + tg.row, tg.n * 4);
        const uint32_t scale_at = l8 ? kOutOfRange : (FMT == kRows ? at * 4 : (uint32_t)r0 * 4);
        const int scale_step = FMT == kRows ? upr * 4 : 4;
#pragma unroll
        for (int p = 0; p < kBwdPasses; ++p) {
            swiglu_grad8(codes[p], scale[p], dh[p], odd, v[p], v[p] + 8, v[p] + 16);
            const GroupScale g = group_scale<false>(max8(amax8(v[p] + 8, amax8(v[p], 0.f))));
            uint32_t q[4];
            quantize<16>(v[p], g, q);
            __builtin_amdgcn_raw_buffer_store_b128(join_codes(u32x2{q[0], q[1]}, u32x2{q[2], q[3]}, odd), out,
                                                   (int)(at * kBwdCols + l8 * 16), p * kBwdRows * upr * kBwdCols, CP_NT);
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(g.s), out_scale, (int)scale_at, p * kBwdRows * scale_step, 0);
            __builtin_amdgcn_sched_barrier(0);           // one pass's temporaries at a time
        }
    }
    const int sub = lane >> 4, perm = sub == 1 ? 2 : (sub == 2 ? 1 : sub);
#pragma unroll
    for (int part = 0; part < 3; ++part) {               // gate, up, H: few registers beside v
        float m[8], red[2];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float y = 0.f;
#pragma unroll
            for (int p = 0; p < kBwdPasses; ++p) y = fmaxf(y, fabsf(v[p][part * 8 + i]));
            // the two rows of a 16-lane row
            m[i] = __uint_as_float(max(__float_as_uint(y), lane_of<DPP_ROR8>(__float_as_uint(y))));
        }
        reduce_rows<8>(m, red);
        float* to = red_s[wave] + (part < 2 ? l8 * 16 + part * 8 : kBwdCols + l8 * 8) + perm;
        to[0] = red[0];                                  // the 16-lane row's halves hold the same
        to[4] = red[1];
        __builtin_amdgcn_sched_barrier(0);
    }
    __syncthreads();
    if (threadIdx.x < C) {
        const int c = threadIdx.x;
        float y = 0.f;
#pragma unroll
        for (int w = 0; w < kThreads / 64; ++w) y = fmaxf(y, red_s[w][c]);
        const bool store = want < a.scale_groups;
        if (c < kBwdCols) {
            const int l = c >> 4, i = c & 15;            // lane l: 8 gate columns, then the 8 up columns 16 further on
            const int col = 32 * (l >> 1) + 8 * (l & 1) + (i < 8 ? i : i + 8);
            column_scale<E8M0>(y, &pre_s[c], &inv_s[c], nullptr, &tiny_s, a.k_scale,
                               (int64_t)want * (2 * a.W) + unit * kBwdCols + col, store);
        } else {
            column_scale<E8M0>(y, &pre_s[c], &inv_s[c], nullptr, &tiny_s, a.hk_scale,
                               (int64_t)want * a.W + unit * 64 + c - kBwdCols, store);
        }
    }
    __syncthreads();
    const bool tiny = tiny_s;
    auto k_out = make_rsrc(a.k_out + u * kBwdCols, units * kBwdCols);
    auto hk_out = make_rsrc(a.hk_out + u * 64, units * 64);
#pragma unroll
    for (int p = 0; p < kBwdPasses; ++p) {
        uint32_t q[4], qh[2];
        asm volatile("" ::: "memory");                   // 24 inverses from LDS again, not in registers beside v
        quantize_columns<16, false>(v[p], pre_s + l8 * 16, inv_s + l8 * 16, inv_s, tiny, q);
        quantize_columns<8, false>(v[p] + 16, pre_s + kBwdCols + l8 * 8, inv_s + kBwdCols + l8 * 8, inv_s, tiny, qh);
        const uint32_t step = (uint32_t)(p * kBwdRows * upr);
        __builtin_amdgcn_raw_buffer_store_b128(join_codes(u32x2{q[0], q[1]}, u32x2{q[2], q[3]}, odd), k_out,
                                               (int)(at * kBwdCols + l8 * 16), (int)(step * kBwdCols), CP_NT);
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{qh[0], qh[1]}, hk_out, (int)(at * 64 + l8 * 8), (int)(step * 64), 0);
    }
}

// ----------------------------------------------------------------- row scales -> token groups

// A workgroup takes a token group x 256 columns: 4 waves, 16 rows at a time, 8
// times.  The codes (or bf16 values) stay in registers as they were read, and
// are scaled twice: for the columns' maxima and for the new codes.  32768 rows of
// 7168 columns: 85 us, 5.7 TB/s, in runs of 11 units to an XCD (of 8: 89 us, of 16:
// 90 us; odd runs from 3 to 13 within 2 us).  In runs of 8, cached accesses took
// 94 us and values kept in fp32 between the two 100 us.  bf16 loads are not
// streamed: each takes the halves of lines, which would then be fetched twice (4096
// columns: 74 us, 82 us streamed).  bf16 rows take the rounded quotient, at no cost
// that shows; e4m3 rows would take 92 us with it.
constexpr int kKgRows = kThreads / 16, kKgPasses = 128 / kKgRows, kKgRun = 11;

template <OperandFormat FMT, bool E8M0>
__global__ __launch_bounds__(kThreads) void k_groups_kernel(CheckpointArgs a) {
    __shared__ float red_s[kThreads / 64][kUnit];
    constexpr bool EXACT = FMT == kBf16 && !E8M0;        // bf16 values: the rounded quotient (by a power of two it is)
    __shared__ float pre_s[kUnit], inv_s[kUnit], low_s[EXACT ? kUnit : 1];
    __shared__ int tiny_s;
    constexpr int RAW = FMT == kBf16 ? 2 : 1;
    const int upr = a.W / kUnit;                         // units of a row
    const int64_t tile = work_position<kKgRun>();
    const int want = (int)(tile / upr), unit = (int)(tile - (int64_t)want * upr);
    const TokenGroup tg = token_group(a.m_sizes, a.G, a.rows, want);
    if (tg.n <= 0) return;
    const int lane = threadIdx.x & 63, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    if (threadIdx.x == 0) tiny_s = 0;
    const int64_t u = (int64_t)tg.row * upr + unit;      // units before the tile's first
    const uint32_t units = (uint32_t)tg.n * upr - unit;  // from there to the group's end
    const int r0 = wave * 4 + (lane >> 4);
    const uint32_t at = (uint32_t)(r0 * upr);
    u32x4 raw[kKgPasses][RAW];
    float scale[kKgPasses];
    {
        auto in = make_rsrc((const uint8_t*)a.in + u * kUnit * RAW, units * kUnit * RAW);
        auto sc = make_rsrc(FMT == kRows ? a.in_scale + u * 2 : nullptr, units * 8);
        const int half = l16 >> 3;                       // the row's 128-column half
#pragma unroll
        for (int p = 0; p < kKgPasses; ++p) {
            const uint32_t step = (uint32_t)(p * kKgRows);
#pragma unroll
            for (int i = 0; i < RAW; ++i)
                raw[p][i] = buffer_load16<FMT != kBf16>(in, (at * kUnit + l16 * 16) * RAW + i * 16, step * upr * kUnit * RAW);
            scale[p] = 0.f;
            if (FMT == kRows)
                scale[p] = __uint_as_float((uint32_t)__builtin_amdgcn_raw_buffer_load_b32(
                    sc, (int)(at * 8 + half * 4), (int)(step * upr * 8), 0));
            if (FMT == kKm) {
                const int r = r0 + (int)step;            // rows of other groups follow: not out of range
                const float x = a.in_scale[(int64_t)(unit * 2 + half) * a.rows + min(tg.row + r, a.rows - 1)];
                scale[p] = r < tg.n ? x : 0.f;
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
    for (int p = 0; p < kKgPasses; p += 2) {
        float v[16], w[16];
        values(p, v);
        values(p + 1, w);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            m[i] = fmaxf(fmaxf(m[i], fabsf(v[i])), fabsf(w[i]));
            asm volatile("" : "+v"(m[i]));               // now, not when all values are there
        }
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
        column_scale<E8M0>(x, &pre_s[c], &inv_s[c], EXACT ? &low_s[c] : nullptr, &tiny_s, a.k_scale,
                           (int64_t)want * a.W + unit * kUnit + c, want < a.scale_groups);
    }
    __syncthreads();
    const bool tiny = tiny_s;
    // EXACT's 32 numbers of a lane's columns stay in registers (512 columns: 11.2 us, read in each pass 13.2 us)
    float inv[16], low[16];
    if (EXACT) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            inv[i] = inv_s[l16 * 16 + i];
            low[i] = low_s[l16 * 16 + i];
        }
    }
    auto k_out = make_rsrc(a.k_out + u * kUnit, units * kUnit);
#pragma unroll
    for (int p = 0; p < kKgPasses; ++p) {
        float v[16];
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < RAW; ++i) asm volatile("" : "+v"(raw[p][i]));   // scaled anew, not kept in fp32
        values(p, v);
        if (EXACT) quantize_columns<16, true>(v, pre_s + l16 * 16, inv, low, tiny, q);
        else quantize_columns<16, false>(v, pre_s + l16 * 16, inv_s + l16 * 16, inv_s, tiny, q);
        __builtin_amdgcn_raw_buffer_store_b128(u32x4{q[0], q[1], q[2], q[3]}, k_out, (int)(at * kUnit + l16 * 16),
                                               (int)(p * kKgRows * upr * kUnit), CP_NT);
    }
}

// ----------------------------------------------------------------- launches

static dim3 row_grid(const CheckpointArgs& a) {
    return run_grid<kRowRun>(((int64_t)a.rows * (a.W / 128) + 15) / 16);
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
    const dim3 grid = run_grid<kBwdRun>(most_groups(a) * (a.W / 64));
    if (a.fmt == kRows) {
        if (a.k_e8m0) swiglu_backward_fp8_kernel<kRows, true><<<grid, kThreads, 0, s>>>(a);
        else swiglu_backward_fp8_kernel<kRows, false><<<grid, kThreads, 0, s>>>(a);
    } else {
        if (a.k_e8m0) swiglu_backward_fp8_kernel<kKm, true><<<grid, kThreads, 0, s>>>(a);
        else swiglu_backward_fp8_kernel<kKm, false><<<grid, kThreads, 0, s>>>(a);
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
    const dim3 grid = run_grid<kKgRun>(most_groups(a) * (a.W / kUnit));
    if (a.fmt == kBf16) k_groups_as<kBf16>(a, grid, s);
    else if (a.fmt == kRows) k_groups_as<kRows>(a, grid, s);
    else k_groups_as<kKm>(a, grid, s);
    return hipGetLastError();
}

}  // namespace moegg
