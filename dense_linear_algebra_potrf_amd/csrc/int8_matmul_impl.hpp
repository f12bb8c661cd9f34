// Products of rows of 8-bit integers on the matrix cores, y = (x W^T) xs ws.
//
// Sums are 32-bit integers, so their order does not count: K may be split and joined
// as it suits, and lanes may hold columns in any order that x and W agree on.
//
// Both operands go from memory into LDS by themselves (no registers in between), in
// tiles of 16 rows and 128 columns, 2 KB.  A product of 16 x 16 x 64 wants 16
// columns of row lane % 16 of lane / 16's quarter: line l of a tile holds row
// l / 2 + 8 (l % 2), and the 16-byte pieces of a line are permuted by l / 2, so that
// any 16 neighbouring lanes read all banks once.  What a lane loads is a piece of a
// whole 128-byte line of memory.
//
// W is the product's first operand, so that a lane's four sums are neighbouring
// columns of y, and the rows of W are dealt to a wavefront's NI tiles by fours, so
// that its 4 NI sums of a row of x are.
//
// Columns past k are masked in x alone: zero times whatever W's padding holds is
// zero in integers.  Rows past the end are those of the last one, not stored.
#pragma once

#include "integer_impl.hpp"

namespace bl {
namespace int8_matmul_detail {

using namespace layer;

using i32x4 = int __attribute__((ext_vector_type(4)));

constexpr int kStep = 128;               // columns of a tile
constexpr int kTile = 16 * kStep;        // bytes of one

// The row of a tile that its line has.
__device__ __forceinline__ constexpr int row_of_line(int l) { return (l >> 1) + 8 * (l & 1); }

// 16 bytes from memory to LDS: lane i's at `to` + 16 i.
__device__ __forceinline__ void load_to_lds(const int8_t* from, uint32_t offset, int8_t* to) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(from + offset),
                                     (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}

// What lane r + 16 g of a wavefront multiplies: 16 columns from 64 s + 16 g on, of a tile's row r.
__device__ __forceinline__ i32x4 fragment(const int8_t* tile, int r, int g, int s) {
    const int line = (r & 7) * 2 + (r >> 3), piece = (4 * s + g) ^ (r & 7);
    return *reinterpret_cast<const i32x4*>(tile + line * kStep + piece * 16);
}

// The first `left` bytes of 16.
__device__ __forceinline__ i32x4 masked(i32x4 v, int left) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int b = left - 4 * i;
        v[i] = b >= 4 ? v[i] : b <= 0 ? 0 : int(uint32_t(v[i]) & ((1u << (8 * b)) - 1));
    }
    return v;
}

// Columns c .. c + COUNT - 1 of a row of y from their sums: `left` of them, times the row's
// scale and theirs.  Where the scales' product is not a normal number it says nothing of
// theirs with the sum, which is then taken in 64 bits.
template <typename T, int COUNT>
__device__ __forceinline__ void store_scaled(T* y, const int (&sum)[COUNT], float xs, const float (&ws)[COUNT], int left) {
    float v[COUNT];
    bool odd = false;
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
        const float f = xs * ws[i];
        odd = odd || !__builtin_amdgcn_classf(f, 0x108);        // a normal number, either sign
        v[i] = float(sum[i]) * f;
    }
    if (odd) {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) v[i] = float(double(sum[i]) * double(xs) * double(ws[i]));
    }
    T t[COUNT];
#pragma unroll
    for (int i = 0; i < COUNT; ++i) t[i] = T(v[i]);
    if (left >= COUNT) {
        __builtin_memcpy(y, t, sizeof(t));
    } else {
#pragma unroll
        for (int i = 0; i < COUNT; ++i)
            if (i < left) y[i] = t[i];
    }
}

// ---------------------------------------------------------------- tiles
// A workgroup takes 16 MI WM rows of x and 16 NI WN rows of W, its WM x WN wavefronts
// 16 MI and 16 NI of them each.  The next step's tiles are on their way while this
// one's are multiplied.
template <typename T, int MI, int NI, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void int8_tiles_kernel(Int8MatmulArgs a) {
    constexpr int WAVES = WM * WN, XT = MI * WM, WT = NI * WN;  // tiles of x and W
    constexpr int LOADS = 2 * (XT + WT) / WAVES;                // a wavefront's, half a tile each
    static_assert(2 * (XT + WT) % WAVES == 0);
    __shared__ __attribute__((aligned(16))) int8_t lds[2][(XT + WT) * kTile];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4, wm = wave / WN, wn = wave % WN;
    // workgroups of one XCD take neighbouring tiles, columns of tiles in groups of 8 rows
    const int tiles_m = int((a.m + 16 * XT - 1) / (16 * XT)), tiles_n = int((a.n + 16 * WT - 1) / (16 * WT));
    int tm, tn;
    {
        const int64_t total = int64_t(tiles_m) * tiles_n, each = total / 8, more = total % 8, x = blockIdx.x % 8;
        const int64_t id = x * each + (x < more ? x : more) + blockIdx.x / 8;
        const int64_t group = 8 * int64_t(tiles_n), first = id / group * 8;
        const int64_t rows = tiles_m - first < 8 ? tiles_m - first : 8, in = id % group;
        tm = int(first + in % rows), tn = int(in / rows);
    }
    const int64_t m0 = int64_t(tm) * 16 * XT, n0 = int64_t(tn) * 16 * WT;
    const int8_t* x = a.x + m0 * a.ldx;
    const int8_t* w = a.w + n0 * a.ldw;

    // where this lane's pieces of each load come from: loads 0 .. 2 XT - 1 are x's
    uint32_t offset[LOADS];
    const int k16 = int((a.k + 15) / 16 * 16), steps = int((a.k + kStep - 1) / kStep);
    uint32_t column[2];                                         // of a first and a second half
#pragma unroll
    for (int h = 0; h < 2; ++h) column[h] = 16 * ((lane & 7) ^ (row_of_line(8 * h + (lane >> 3)) & 7));
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int load = wave * LOADS + i, half = load & 1, tile = load >> 1;
        const int row = row_of_line(8 * half + (lane >> 3));
        if (tile < XT) {
            const int64_t at = 16 * tile + row, most = a.m - 1 - m0;
            offset[i] = uint32_t((at < most ? at : most) * a.ldx) + column[half];
        } else {
            const int t = tile - XT;
            const int64_t at = t / NI * 16 * NI + 4 * NI * (row >> 2) + 4 * (t % NI) + (row & 3), most = a.n - 1 - n0;
            offset[i] = uint32_t((at < most ? at : most) * a.ldw) + column[half];
        }
    }
    auto load = [&](int step, int8_t* to) {
        const int from = step * kStep, left = k16 - from;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int load = wave * LOADS + i;
            const uint32_t c = column[load & 1];
            // pieces past the row's end: the first one again, masked in x
            const uint32_t off = int(c) < left ? offset[i] : offset[i] - c;
            load_to_lds((load >> 1 < XT ? x : w) + from, off, to + load * (kTile / 2));
        }
    };

    i32x4 acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    auto multiply = [&](const int8_t* tiles, int left, auto tail) {
        const int8_t* xt = tiles + wm * MI * kTile;
        const int8_t* wt = tiles + (XT + wn * NI) * kTile;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            i32x4 xf[MI], wf[NI];
#pragma unroll
            for (int j = 0; j < NI; ++j) wf[j] = fragment(wt + j * kTile, r, g, s);
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                xf[i] = fragment(xt + i * kTile, r, g, s);
                if constexpr (decltype(tail)::value) xf[i] = masked(xf[i], left - 64 * s - 16 * g);
            }
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[j], xf[i], acc[i][j], 0, 0, 0);
        }
    };
    load(0, lds[0]);
    for (int s = 0; s + 1 < steps; ++s) {
        __syncthreads();                                        // step s is there, step s - 1 has been read
        load(s + 1, lds[(s + 1) & 1]);
        multiply(lds[s & 1], kStep, std::false_type{});
    }
    __syncthreads();
    multiply(lds[(steps - 1) & 1], int(a.k) - (steps - 1) * kStep, std::true_type{});

    const int64_t n = n0 + wn * 16 * NI + 4 * NI * g;
    const int left = a.n - n < 4 * NI ? int(a.n - n) : 4 * NI;
    if (left <= 0) return;
    float ws[4 * NI];
#pragma unroll
    for (int j = 0; j < 4 * NI; ++j) ws[j] = a.ws[j < left ? n + j : n];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int64_t m = m0 + (wm * MI + i) * 16 + r;
        if (m >= a.m) continue;
        int sum[4 * NI];
#pragma unroll
        for (int j = 0; j < 4 * NI; ++j) sum[j] = acc[i][j / 4][j % 4];
        store_scaled(static_cast<T*>(a.y) + m * a.ldy + n, sum, a.xs[m], ws, left);
    }
}

// ---------------------------------------------------------------- few rows of x
// A workgroup takes 16 NB rows of W and 16 MB of x; its wavefronts take every WAVES-th
// step of the columns, each through DEPTH tiles of its own in LDS, so that they wait
// for nobody until they join their sums.
template <typename T, int MB, int NB, int WAVES, int DEPTH>
__global__ __launch_bounds__(64 * WAVES) void int8_few_kernel(Int8MatmulArgs a) {
    constexpr int TILES = MB + NB, LOADS = 2 * TILES;
    constexpr int JOIN = WAVES * MB * NB * 64 * 16, RING = WAVES * DEPTH * TILES * kTile;
    __shared__ __attribute__((aligned(16))) int8_t lds[JOIN > RING ? JOIN : RING];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t n0 = int64_t(blockIdx.x) * 16 * NB, m0 = int64_t(blockIdx.y) * 16 * MB;
    const int8_t* x = a.x + m0 * a.ldx;
    const int8_t* w = a.w + n0 * a.ldw;
    uint32_t offset[LOADS], column[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) column[h] = 16 * ((lane & 7) ^ (row_of_line(8 * h + (lane >> 3)) & 7));
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int row = row_of_line(8 * (i & 1) + (lane >> 3)), tile = i >> 1;
        if (tile < MB) {
            const int64_t at = 16 * tile + row, most = a.m - 1 - m0;
            offset[i] = uint32_t((at < most ? at : most) * a.ldx) + column[i & 1];
        } else {
            const int64_t at = 4 * NB * (row >> 2) + 4 * (tile - MB) + (row & 3), most = a.n - 1 - n0;
            offset[i] = uint32_t((at < most ? at : most) * a.ldw) + column[i & 1];
        }
    }
    const int k16 = int((a.k + 15) / 16 * 16), steps = int((a.k + kStep - 1) / kStep);
    const int mine = steps > wave ? (steps - wave + WAVES - 1) / WAVES : 0;    // this wavefront's
    int8_t* const ring = lds + wave * DEPTH * TILES * kTile;
    auto load = [&](int i) {                                    // its i-th; past the last one, that again
        const int from = (wave + (i < mine ? i : mine - 1) * WAVES) * kStep, left = k16 - from;
        int8_t* to = ring + i % DEPTH * TILES * kTile;
#pragma unroll
        for (int l = 0; l < LOADS; ++l) {
            const uint32_t c = column[l & 1];
            load_to_lds((l >> 1 < MB ? x : w) + from, int(c) < left ? offset[l] : offset[l] - c, to + l * (kTile / 2));
        }
    };

    i32x4 acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    if (mine) {
#pragma unroll
        for (int i = 0; i + 1 < DEPTH; ++i) load(i);
        for (int i = 0; i < mine; ++i) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the place of the next has been read
            load(i + DEPTH - 1);
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LOADS * (DEPTH - 1)) : "memory");
            const int8_t* tiles = ring + i % DEPTH * TILES * kTile;
            const int left = int(a.k) - (wave + i * WAVES) * kStep;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                i32x4 xf[MB], wf[NB];
#pragma unroll
                for (int j = 0; j < NB; ++j) wf[j] = fragment(tiles + (MB + j) * kTile, r, g, s);
#pragma unroll
                for (int j = 0; j < MB; ++j) {
                    xf[j] = fragment(tiles + j * kTile, r, g, s);
                    if (left < kStep) xf[j] = masked(xf[j], left - 64 * s - 16 * g);
                }
#pragma unroll
                for (int q = 0; q < MB; ++q)
#pragma unroll
                    for (int j = 0; j < NB; ++j) acc[q][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[j], xf[q], acc[q][j], 0, 0, 0);
            }
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    // join: a lane's four sums of each tile, then a thread's tile and lane
    __syncthreads();
    i32x4* const sums = reinterpret_cast<i32x4*>(lds);
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) sums[(wave * MB * NB + i * NB + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    for (int e = threadIdx.x; e < MB * NB * 64; e += 64 * WAVES) {
        const int from = e & 63, tile = e >> 6;
        const int64_t m = m0 + 16 * (tile / NB) + (from & 15), n = n0 + 4 * NB * (from >> 4) + 4 * (tile % NB);
        if (m >= a.m || n >= a.n) continue;
        int sum[4] = {0, 0, 0, 0};
#pragma unroll
        for (int v = 0; v < WAVES; ++v) {
            const i32x4 s = sums[v * MB * NB * 64 + e];
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[j] += s[j];
        }
        const int left = a.n - n < 4 ? int(a.n - n) : 4;
        float ws[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) ws[j] = a.ws[j < left ? n + j : n];
        store_scaled(static_cast<T*>(a.y) + m * a.ldy + n, sum, a.xs[m], ws, left);
    }
}

template <typename T, int MI, int NI, int WM, int WN>
inline hipError_t tiles(const Int8MatmulArgs& a, hipStream_t s) {
    const int64_t tm = (a.m + 16 * MI * WM - 1) / (16 * MI * WM), tn = (a.n + 16 * NI * WN - 1) / (16 * NI * WN);
    return launch(int8_tiles_kernel<T, MI, NI, WM, WN>, dim3(uint32_t(tm * tn)), dim3(64 * WM * WN), 0, s, a);
}

template <typename T, int MB, int NB, int WAVES, int DEPTH>
inline hipError_t few(const Int8MatmulArgs& a, hipStream_t s) {
    const dim3 grid(uint32_t((a.n + 16 * NB - 1) / (16 * NB)), uint32_t((a.m + 16 * MB - 1) / (16 * MB)));
    return launch(int8_few_kernel<T, MB, NB, WAVES, DEPTH>, grid, dim3(64 * WAVES), 0, s, a);
}

template <typename T>
inline hipError_t int8_matmul_t(const Int8MatmulArgs& a, hipStream_t s) {
    if (a.m <= 16) return a.n >= 256 * 32 ? few<T, 1, 2, 8, 3>(a, s) : few<T, 1, 1, 8, 4>(a, s);
    if (a.m <= 32) return few<T, 2, 2, 4, 3>(a, s);
    if (a.m <= 64) return few<T, 4, 2, 4, 3>(a, s);
    const int64_t big = ((a.m + 255) / 256) * ((a.n + 255) / 256);
    if (big >= 200) return tiles<T, 8, 4, 2, 4>(a, s);
    return tiles<T, 4, 4, 2, 2>(a, s);
}

}  // namespace int8_matmul_detail
}  // namespace bl
