// lora.hip -- low-rank adapters of many requests, added to a projection's output:
//     out[t] = Y[t] + scale_a (X[t] A_a^T) B_a^T,   a the adapter of row t.
//
// Two products with a rank of 8 to 128, so that rows and weights are moved and little
// is computed.  Both take tiles of rows with one adapter.  Up to 128 rows the kernels
// find these by themselves: a wave looks at a chunk of 64 consecutive rows, a lane
// each, counts for all of them at once the earlier rows with the same adapter, and has
// a tile start at every 16th of these.  Beyond, a first launch sorts windows of 8192
// rows by their adapters, so that an adapter's weights are read for 64 rows together
// whatever the order of the rows; with more adapters than LDS counts any number of rows
// goes in chunks.
#include <hip/hip_runtime.h>

#include "block.hpp"
#include "device.hpp"
#include "layer.hpp"
#include "rows.hpp"

namespace moegg {

constexpr int kThreads = 256;             // and columns of out that a workgroup of the second product takes
constexpr int kTile = kLoraChunk;         // rows of a tile
constexpr int kChunkTile = 16;            // and of one that was not sorted

// ----------------------------------------------------------------- tiles

// Rows of a window in the order of their adapters, and its tiles.  Rows with one
// adapter come in any order (an LDS atomic gives them their places): a row's result
// does not depend on its place.  One workgroup's latencies: 3.1 us for 256 rows, 4.6 for
// 4096, 6.9 for 8191.
__global__ __launch_bounds__(1024) void lora_sort_kernel(LoraArgs a, int copy) {
    extern __shared__ int count_s[];                         // [L + 1]: rows of each adapter, then their first place
    __shared__ uint32_t both_s[16];
    __shared__ int all_tiles_s;
    constexpr int kEach = kLoraWindow / 1024;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, first = (int)blockIdx.x * kLoraWindow;
    int4* tiles = a.tiles + (int64_t)blockIdx.x * a.max_tiles;
    int key[kEach], rank[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int t = first + i * 1024 + (int)threadIdx.x;
        key[i] = t < a.T ? a.adapter[t] : -2;
        if (key[i] != -2 || t < a.T) key[i] = (uint32_t)key[i] < (uint32_t)a.L ? key[i] : a.L;
    }
    for (int k = threadIdx.x; k <= a.L; k += 1024) count_s[k] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        // a wave of one adapter (the rows of a long prompt) adds once
        const int k0 = __builtin_amdgcn_readfirstlane(key[i]);
        if (__all(key[i] == k0)) {
            int base = 0;
            if (lane == 0 && k0 >= 0) base = atomicAdd(&count_s[k0], 64);
            rank[i] = __builtin_amdgcn_readfirstlane(base) + lane;
        } else if (key[i] >= 0) {
            rank[i] = atomicAdd(&count_s[key[i]], 1);
        }
    }
    __syncthreads();
    // places and tiles before each adapter: a run of adapters a thread, rows and tiles as the
    // halves of a word (8192 and 8320 at most)
    const int per = (a.L + 1024) / 1024, k0 = min((int)threadIdx.x * per, a.L + 1), k1 = min(k0 + per, a.L + 1);
    uint32_t both = 0;
    for (int k = k0; k < k1; ++k) {
        const uint32_t c = count_s[k], n = k < a.L || copy ? (c + kTile - 1) / kTile : 0;
        both += n << 16 | c;
    }
    uint32_t end = both;
    end += dpp<DPP_SHR + 1>(0, end);
    end += dpp<DPP_SHR + 2>(0, end);
    end += dpp<DPP_SHR + 4>(0, end);
    end += dpp<DPP_SHR + 8>(0, end);
    end += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)end, DPP_BCAST15, 0xA, 0xF, false);
    end += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)end, DPP_BCAST31, 0xC, 0xF, false);
    if (lane == 63) both_s[wave] = end;
    __syncthreads();
    end -= both;
#pragma unroll
    for (int w = 0; w < 15; ++w) end += w < wave ? both_s[w] : 0u;
    int place = (int)(end & 0xFFFFu), tile = (int)(end >> 16);
    for (int k = k0; k < k1; ++k) {
        const int c = count_s[k];
        count_s[k] = place;
        if (k < a.L || copy)
            for (int b = 0; b < c; b += kTile) tiles[tile++] = int4{k < a.L ? k : -1, first + place + b, min(kTile, c - b), 0};
        place += c;
    }
    if (threadIdx.x == 1023) all_tiles_s = tile;             // a word of its own: both_s is still being read
    __syncthreads();
    for (int i = all_tiles_s + (int)threadIdx.x; i < a.max_tiles; i += 1024) tiles[i] = int4{-1, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kEach; ++i)
        if (key[i] >= 0) a.order[first + count_s[key[i]] + rank[i]] = first + i * 1024 + (int)threadIdx.x;
}

// The tiles that a workgroup takes: every slots-th one of its chunk or window,
// their rows listed in LDS.
template <bool SORTED>
struct Tiles {
    int at, slots, unit;
    int own, rank;                       // chunk: this lane's adapter (-1: none, -2: no row), earlier rows with the same
    uint64_t starts;                     // chunk: first rows of tiles

    // A row starts a tile if the number of earlier rows with its adapter is a multiple of
    // 16: counted for all rows at once, one comparison with each row.  Taking adapter
    // after adapter instead costs a late tile of 40 adapters 1 us.
    __device__ __forceinline__ Tiles(const LoraArgs& a, int unit_, int slot, int slots_, bool bare)
        : at(slot), slots(slots_), unit(unit_) {
        if (!SORTED) {
            const int lane = threadIdx.x & 63, first = unit * kLoraChunk, rows = min(a.T - first, kLoraChunk);
            own = lane < rows ? a.adapter[first + lane] : -2;
            if (lane < rows) own = (uint32_t)own < (uint32_t)a.L ? own : -1;
            rank = 0;
            for (int i = 0; i < rows; i += 8)
#pragma unroll
                for (int j = 0; j < 8; ++j) rank += (__builtin_amdgcn_readlane(own, i + j) == own) & (i + j < lane);
            starts = __ballot(rank % kChunkTile == 0 && (own >= 0 || (bare && own == -1)));
        }
    }
    // The next tile's adapter (-1: rows without one) and number of rows; false: there is none.
    __device__ __forceinline__ bool next(const LoraArgs& a, int* list_s, int& adapter, int& n) {
        const int lane = threadIdx.x & 63;
        if (SORTED) {
            if (at >= a.max_tiles) return false;
            const int4 tile = a.tiles[(int64_t)unit * a.max_tiles + at];
            adapter = __builtin_amdgcn_readfirstlane(tile.x);
            n = __builtin_amdgcn_readfirstlane(tile.z);
            if (n == 0) return false;
            if (threadIdx.x < 64) list_s[lane] = a.order[tile.y + min(lane, n - 1)];
        } else {
            const uint64_t before = (1ull << lane) - 1;
            const uint64_t it = __ballot((starts >> lane & 1) && __popcll(starts & before) == at);
            if (!it) return false;
            const int src = __builtin_ctzll(it);
            adapter = __builtin_amdgcn_readlane(own, src);
            const uint32_t place = (uint32_t)(rank - __builtin_amdgcn_readlane(rank, src));
            const bool mine = own == adapter && place < kChunkTile;
            n = __popcll(__ballot(mine));
            if (threadIdx.x < 64 && mine) list_s[place] = unit * kLoraChunk + lane;
        }
        at += slots;
        __syncthreads();
        return true;
    }
};

// ----------------------------------------------------------------- X A^T

// A workgroup takes a tile and a part of K, its waves a share of that each; their
// sums meet in LDS.  D = X A^T in blocks of 16 rows x 16 ranks.  K goes in units of 128
// columns, whole lines, all of whose loads are in flight together.  4096 rows of 7168 to a rank of
// 16: 15 us for 59 MB; 8 waves a workgroup (22 us: one of them a CU) and loads of half a unit
// ahead of the products (15 us) do not pay.  Rank 64, 8191 rows of 2048: 16 to 21 us; rank 128
// in 194 registers, two waves a SIMD: 4096 rows of 7168 in 56 us.
constexpr int kUnit = 128;

template <int RT, int CT>
__device__ __forceinline__ void shrink(const LoraArgs& a, const int* list_s, int n, int adapter, int split,
                                       float (*sum_s)[16][CT * 16 + 4]) {
    constexpr int kSteps = CT <= 2 ? kUnit / 32 : kUnit / 64;    // loaded together; higher ranks: half a unit
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int l16 = lane & 15, grp = lane >> 4;
    const int units = (a.K + kUnit - 1) / kUnit, shares = a.splits * 4, share = split * 4 + wave;
    const int u0 = (int)((int64_t)units * share / shares), u1 = (int)((int64_t)units * (share + 1) / shares);
    const uint16_t* x[RT];
    const uint16_t* w[CT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
        x[r] = (const uint16_t*)a.X + (int64_t)list_s[min(r * 16 + l16, n - 1)] * a.K + grp * 8;
#pragma unroll
    for (int c = 0; c < CT; ++c)
        w[c] = (const uint16_t*)a.A + ((int64_t)adapter * a.R + min(c * 16 + l16, a.R - 1)) * a.K + grp * 8;
    v4f acc[RT][CT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[r][c] = v4f{0, 0, 0, 0};
    for (int k = u0 * kUnit; k < u1 * kUnit; k += kSteps * 32) {
        v4i xv[kSteps][RT], wv[kSteps][CT];
        if (k + kSteps * 32 <= a.K) {
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
#pragma unroll
                for (int r = 0; r < RT; ++r) xv[s][r] = *(const v4i*)(x[r] + k + s * 32);
#pragma unroll
                for (int c = 0; c < CT; ++c) wv[s][c] = *(const v4i*)(w[c] + k + s * 32);
            }
        } else {
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const bool in = k + s * 32 + grp * 8 < a.K;      // K % 8 == 0: whole pieces
#pragma unroll
                for (int r = 0; r < RT; ++r) xv[s][r] = in ? *(const v4i*)(x[r] + k + s * 32) : v4i{0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < CT; ++c) wv[s][c] = in ? *(const v4i*)(w[c] + k + s * 32) : v4i{0, 0, 0, 0};
            }
        }
        __builtin_amdgcn_sched_barrier(0);                       // no product before the last load is sent
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int c = 0; c < CT; ++c) acc[r][c] = mfma_bf16(xv[s][r], wv[s][c], acc[r][c]);
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        if (r) __syncthreads();
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int v = 0; v < 4; ++v) sum_s[wave][grp * 4 + v][c * 16 + l16] = acc[r][c][v];
        __syncthreads();
        for (int i = threadIdx.x; i < 16 * CT * 4; i += kThreads) {
            const int row = i / (CT * 4), rank = i % (CT * 4) * 4;
            if (r * 16 + row >= n || rank >= a.R) continue;      // R % 8 == 0
            v4f s = *(const v4f*)&sum_s[0][row][rank];
#pragma unroll
            for (int m = 1; m < 4; ++m) s += *(const v4f*)&sum_s[m][row][rank];
            *(v4f*)(a.U + ((int64_t)split * a.T + list_s[r * 16 + row]) * a.R + rank) = s;
        }
    }
    __syncthreads();
}

template <int CT, bool SORTED>
__global__ __launch_bounds__(kThreads) void lora_shrink_kernel(LoraArgs a, int slots) {
    __shared__ int list_s[kTile];
    __shared__ __align__(16) float sum_s[4][16][CT * 16 + 4];
    const int split = blockIdx.x % a.splits, slot = blockIdx.x / a.splits % slots, unit = blockIdx.x / a.splits / slots;
    Tiles<SORTED> tiles(a, unit, slot, slots, false);
    int adapter, n;
    while (tiles.next(a, list_s, adapter, n)) {
        if (SORTED && adapter < 0) break;                    // rows without an adapter come last
        if (!SORTED || n <= 16) shrink<1, CT>(a, list_s, n, adapter, split, sum_s);
        else if (n <= 32) shrink<2, CT>(a, list_s, n, adapter, split, sum_s);
        else shrink<4, CT>(a, list_s, n, adapter, split, sum_s);
    }
}

// ----------------------------------------------------------------- U B^T

// U in two bf16, the value and what is left of it (2^-16 of it is lost at most): one
// would put half a step of bf16, 2^-8, on every term.  The first is a number, so that fp32
// past bf16's last one has its rest in the second, as have infinities and NaN.
__device__ __forceinline__ void split_bf16(float u, uint16_t& hi, uint16_t& lo) {
    constexpr float most = 0x1.FEp+127f;
    const __bf16 h = (__bf16)__builtin_amdgcn_fmed3f(u, -most, most);
    const __bf16 l = (__bf16)(u - (float)h);
    hi = __builtin_bit_cast(uint16_t, h);
    lo = __builtin_bit_cast(uint16_t, l);
}

// A wave takes 64 columns of out at a time for a tile.  D = B U^T: a lane has one row of out
// and, with columns 32 (b / 2) + 8 (i / 4) + 4 (b % 2) + i % 4 as row i of block b, twice 8
// consecutive columns of it.  Neighbouring lanes exchange one of the two, so that a load
// or store moves 8 rows of 128 bytes, whole lines, and not halves of 16.
__device__ __forceinline__ void swap_halves(u32x4& first, u32x4& second) {
    const bool odd = threadIdx.x & 1;
    const u32x4 send = odd ? first : second;
    const u32x4 got = {lane_of<DPP_XOR1>(send.x), lane_of<DPP_XOR1>(send.y), lane_of<DPP_XOR1>(send.z),
                       lane_of<DPP_XOR1>(send.w)};
    if (odd) first = got;
    else second = got;
}

// Y and B are on their way while U's parts are added.  4096 rows, rank 16, 4096 columns: 17 us for 67 MB
// of Y and out; 8191 rows, rank 64, 7168 columns: 60 us for 235 MB, 8 of which B's fragments
// and 14 U's parts cost beside them (both without any stores 10).  Accesses in halves of lines
// cost 2 us of the first, two panels of columns a workgroup or 512 threads nothing of either; fewer
// registers (128) a third of the second.  Rank 128 takes 252 registers: 4096 rows of 4096 columns
// 35 us, 8191 of 7168 87 us.
template <int RT, int RS>
__device__ __forceinline__ void expand(const LoraArgs& a, const int* list_s, uint16_t (*u_s)[RS * 64 + 8], int n,
                                       int adapter, int col) {
    const int lane = threadIdx.x & 63, l16 = lane & 15, grp = lane >> 4;
    // U: four ranks a thread at a time, summed over the parts of K in order.  Loads return in the
    // order in which they were sent: the last of U's go before those of Y and B.
    constexpr int kItems = RT * 16 * RS * 8, kEach = (kItems + kThreads - 1) / kThreads;
    constexpr int kParts = RT == 1 ? 8 : (RT == 2 ? 4 : 2);      // loaded together
    v4f u[kEach], p[kParts][kEach];
    const int64_t step = (int64_t)a.T * a.R;
    auto part = [&](int j, int s) {
        const int i = j * kThreads + (int)threadIdx.x, row = i / (RS * 8), rank = i % (RS * 8) * 4;
        return row < n && rank < a.R && s < a.splits ? *(const v4f*)(a.U + s * step + (int64_t)list_s[row] * a.R + rank)
                                                    : v4f{0, 0, 0, 0};
    };
#pragma unroll
    for (int j = 0; j < kEach; ++j) u[j] = v4f{0, 0, 0, 0};
    int s0 = 0;
    auto parts = [&]() {
#pragma unroll
        for (int s = 0; s < kParts; ++s)
#pragma unroll
            for (int j = 0; j < kEach; ++j) p[s][j] = part(j, s0 + s);
    };
    auto add = [&]() {
#pragma unroll
        for (int s = 0; s < kParts; ++s)
#pragma unroll
            for (int j = 0; j < kEach; ++j) u[j] += p[s][j];
    };
    for (; s0 + kParts < a.splits; s0 += kParts) {
        parts();
        add();
    }
    parts();
    __builtin_amdgcn_sched_barrier(0);
    v4i w[4][RS];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const int c = col + 32 * (b >> 1) + 8 * (l16 >> 2) + 4 * (b & 1) + (l16 & 3);
        const uint16_t* p = (const uint16_t*)a.B + ((int64_t)adapter * a.N + min(c, a.N - 1)) * a.R + grp * 8;
#pragma unroll
        for (int s = 0; s < RS; ++s) w[b][s] = s * 32 + grp * 8 < a.R ? *(const v4i*)(p + s * 32) : v4i{0, 0, 0, 0};
    }
    // the lane's place in its i-th access to row block r: of an even row, or of the odd one after it
    const int c = col + 8 * grp + 32 * (l16 & 1);            // N % 8 == 0: whole pieces
    auto place = [&](int r, int i) { return (int64_t)list_s[min(r * 16 + (l16 & 14) + i, n - 1)] * a.N + c; };
    u32x4 y[RT][2];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            y[r][i] = c < a.N ? *(const u32x4*)((const uint16_t*)a.Y + place(r, i)) : u32x4{0, 0, 0, 0};
    const float scale = a.scale ? a.scale[adapter] : 1.f;
    __builtin_amdgcn_sched_barrier(0);
    add();
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int i = j * kThreads + (int)threadIdx.x, row = i / (RS * 8), rank = i % (RS * 8) * 4;
        if (i >= kItems) break;
        uint16_t hi[4], lo[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) split_bf16(u[j][m], hi[m], lo[m]);
        *(u32x2*)&u_s[row][rank] = u32x2{hi[0] | (uint32_t)hi[1] << 16, hi[2] | (uint32_t)hi[3] << 16};
        *(u32x2*)&u_s[row][RS * 32 + rank] = u32x2{lo[0] | (uint32_t)lo[1] << 16, lo[2] | (uint32_t)lo[3] << 16};
    }
    lds_barrier();
    if (col >= a.N) return;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        v4f acc[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[b] = v4f{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < RS; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const v4i u = lds_read_b128(&u_s[r * 16 + l16][(h * RS + s) * 32 + grp * 8]);
#pragma unroll
                for (int b = 0; b < 4; ++b) acc[b] = mfma_bf16(w[b][s], u, acc[b]);
            }
        swap_halves(y[r][0], y[r][1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float f[8];
            unpack8(y[r][h], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = __builtin_fmaf(scale, acc[2 * h + j / 4][j % 4], f[j]);
            y[r][h] = pack8(f);
        }
        swap_halves(y[r][0], y[r][1]);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (r * 16 + (l16 & 14) + i < n && c < a.N) store_once((uint16_t*)a.out + place(r, i), y[r][i]);
    }
}

template <int RS, bool SORTED>
__global__ __launch_bounds__(kThreads, 2) void lora_expand_kernel(LoraArgs a, int slots, int panels) {
    __shared__ int list_s[kTile];
    __shared__ __align__(16) uint16_t u_s[kTile][RS * 64 + 8];   // 16 bytes more: 16 rows' pieces on all banks
    const int panel = blockIdx.x % panels, slot = blockIdx.x / panels % slots, unit = blockIdx.x / panels / slots;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    Tiles<SORTED> tiles(a, unit, slot, slots, a.out != a.Y);
    int adapter, n;
    while (tiles.next(a, list_s, adapter, n)) {
        if (adapter < 0) {                                   // copied: 8 columns a thread, 8 rows together
            const int c = panel * kThreads + (int)threadIdx.x % (kThreads / 8) * 8;
            for (int i = (int)threadIdx.x / (kThreads / 8); i < n; i += 8) {
                const int64_t at = (int64_t)list_s[i] * a.N + c;
                if (c < a.N) *(u32x4*)((uint16_t*)a.out + at) = *(const u32x4*)((const uint16_t*)a.Y + at);
            }
        } else if (!SORTED || n <= 16) {
            expand<1, RS>(a, list_s, u_s, n, adapter, panel * kThreads + wave * 64);
        } else if (n <= 32) {
            expand<2, RS>(a, list_s, u_s, n, adapter, panel * kThreads + wave * 64);
        } else {
            expand<4, RS>(a, list_s, u_s, n, adapter, panel * kThreads + wave * 64);
        }
        __syncthreads();
    }
}

// ----------------------------------------------------------------- launches

// Workgroups that share the tiles of a chunk or window: no more than there can be
// tiles, and no more than `goal` workgroups call for.
static int lora_slots(int most, int64_t others, int goal) {
    const int64_t want = (goal + others - 1) / others;
    return most < want ? most : (int)want;
}

template <int CT, int RS, bool SORTED>
static hipError_t lora_as(const LoraArgs& a, hipStream_t s) {
    const int64_t units = SORTED ? (a.T + kLoraWindow - 1) / kLoraWindow : (a.T + kLoraChunk - 1) / kLoraChunk;
    const int panels = (a.N + kThreads - 1) / kThreads;
    int slots = lora_slots(a.max_tiles, units * a.splits, 2048);
    lora_shrink_kernel<CT, SORTED><<<(unsigned)(units * slots * a.splits), kThreads, 0, s>>>(a, slots);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    slots = lora_slots(a.max_tiles, units * panels, 4096);
    lora_expand_kernel<RS, SORTED><<<(unsigned)(units * slots * panels), kThreads, 0, s>>>(a, slots, panels);
    return hipGetLastError();
}

template <bool SORTED>
static hipError_t lora_with(const LoraArgs& a, hipStream_t s) {
    if (a.R <= 16) return lora_as<1, 1, SORTED>(a, s);
    if (a.R <= 32) return lora_as<2, 1, SORTED>(a, s);
    if (a.R <= 64) return lora_as<4, 2, SORTED>(a, s);
    return lora_as<8, 4, SORTED>(a, s);
}

hipError_t launch_lora(const LoraArgs& a, hipStream_t s) {
    if (a.T == 0) return hipSuccess;
    if (!lora_sorted(a.T, a.L)) return lora_with<false>(a, s);
    const unsigned windows = (unsigned)((a.T + kLoraWindow - 1) / kLoraWindow);
    lora_sort_kernel<<<windows, 1024, (a.L + 1) * sizeof(int), s>>>(a, a.out != a.Y);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : lora_with<true>(a, s);
}

}  // namespace moegg
