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
// columns of y.  In 16 bits, and in the kernel for few rows, the rows of W are dealt to a
// wavefront's NI tiles by fours, so that its 4 NI sums of a row of x are.
//
// Columns past k are masked in x alone: zero times whatever W's padding holds is
// zero in integers.  Rows past the end are those of the last one, not stored.
//
// Few rows are bound by W's bytes, and run at or above a large copy's rate (5.1 TB/s;
// several of these sizes stay in the last-level cache): 16 x 28672 x 8192 42.1 us a call,
// 5.6 TB/s; 64 x 8192 x 8192 12.9, 5.3.  1 x 4096 x 4096 takes 4.5 in the kernel, 6.7 a call.
// Many rows are bound by what a compute unit gets from the caches: 8192 x 8192 x 8192 454 us,
// 2420 TOP/s, where without its loads the kernel took 360 and without its products 430, and the
// matrix cores alone 233.  The clock goes by the codes and by what ran before: beside each other
// on the same normal codes this takes 422 and the library's product of these integers (without
// scales) 451; on codes uniform within -127..127 463, and launches apart, in a profile, 502 on average.
// Measured there and not kept: half-width steps, four of them in LDS (500 us: half lines
// load at half the rate); the two wavefronts of a SIMD in turns of reading and
// multiplying (485); loads as whole-address loads, which the compiler lets every LDS
// read wait for (510); loads after all products or before them (492, 462).
// 517 x 5003 x 2500 in 32 bits takes 17.6, with rows of 2512 bytes, so that every piece of 128
// columns lies in two cache lines; with rows of 2560 it takes 16.3.
#pragma once

#include "integer_impl.hpp"

namespace bl {
namespace int8_matmul_detail {

using namespace layer;

using i32x4 = int __attribute__((ext_vector_type(4)));

constexpr int kStep = 128;               // columns of a tile
constexpr int kTile = 16 * kStep;        // bytes of one

// Row and column (within 128) of the 16 bytes that lane i loads of a half tile.
__device__ __forceinline__ int row_of(int half, int lane) {
    const int line = 8 * half + (lane >> 3);
    return (line >> 1) + 8 * (line & 1);
}
__device__ __forceinline__ int column_of(int half, int lane) { return 16 * ((lane & 7) ^ (row_of(half, lane) & 7)); }

// 16 bytes from memory to LDS: lane i's, `offset` bytes of its own and `step` of all lanes from a
// tile's first, at `to` + 16 i.  As buffer loads: the compiler takes the form without a buffer
// for one that LDS reads have to wait for.
using Rows = __amdgpu_buffer_rsrc_t;
__device__ __forceinline__ Rows rows_at(const int8_t* p, bool any) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(p), 0, __builtin_amdgcn_readfirstlane(any ? -1 : 0), 0x00027000);
}
// A pointer that is the same for all lanes, where the compiler does not see it.
__device__ __forceinline__ const int8_t* scalar(const int8_t* p) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(v)), hi = __builtin_amdgcn_readfirstlane(uint32_t(v >> 32));
    return reinterpret_cast<const int8_t*>(uint64_t(hi) << 32 | lo);
}
__device__ __forceinline__ void load_to_lds(Rows rows, uint32_t offset, int step, int8_t* to) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rows, (__attribute__((address_space(3))) void*)to, 16, int(offset), step, 0, 0);
}

// What lane r + 16 g of a wavefront multiplies: 16 columns from 64 s + 16 g on, of a tile's row r.
__device__ __forceinline__ i32x4 fragment(const int8_t* tile, int r, int g, int s) {
    const int line = (r & 7) * 2 + (r >> 3), piece = (4 * s + g) ^ (r & 7);
    return *reinterpret_cast<const i32x4*>(tile + line * kStep + piece * 16);
}

// Waits until at most COUNT of this wavefront's loads are on their way, and until what it
// has read from LDS is there.
template <int COUNT>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(COUNT) : "memory");
}

// Waits for the workgroup; nothing that follows is read or sent for before it.
__device__ __forceinline__ void barrier() {
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Ones in the first `left` bytes of 16.
__device__ __forceinline__ i32x4 first_bytes(int left) {
    i32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int b = left - 4 * i;
        v[i] = b >= 4 ? -1 : b <= 0 ? 0 : int((1u << (8 * b)) - 1);
    }
    return v;
}

// COUNT columns of a row of y from their sums, times the row's scale and theirs.  Where the
// scales' product is not a normal number it says nothing of theirs with the sum, which
// is then taken in 64 bits.
template <typename T, int COUNT>
__device__ __forceinline__ void scaled(T (&t)[COUNT], const int (&sum)[COUNT], float xs, const float (&ws)[COUNT]) {
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
#pragma unroll
    for (int i = 0; i < COUNT; ++i) t[i] = T(v[i]);
}

// The first `left` of COUNT neighbouring columns, past the caches where PAST.
template <bool PAST, typename T, int COUNT>
__device__ __forceinline__ void store_columns(T* y, const T (&t)[COUNT], int left) {
    if (left >= COUNT) {
        if constexpr (PAST) store_past(y, t);
        else __builtin_memcpy(y, t, sizeof(t));
    } else {
#pragma unroll
        for (int i = 0; i < COUNT; ++i)
            if (i < left) y[i] = t[i];
    }
}

// ---------------------------------------------------------------- tiles
// A workgroup takes 16 MI WM rows of x and 16 NI WN rows of W, its WM x WN wavefronts
// 16 MI and 16 NI of them each.  DEPTH steps are in LDS or on their way there: while
// one is multiplied, the loads of the DEPTH - 1 after it are on their way.
//
// A barrier a step: by it step s is there (each wavefront has waited for its own loads
// of it) and step s - 1 has been read (each has waited for its reads), so that the loads
// of step s + DEPTH - 1 may go to the place of step s - 1.
template <typename T, int MI, int NI, int WM, int WN, int DEPTH>
__global__ __launch_bounds__(64 * WM * WN) void int8_tiles_kernel(Int8MatmulArgs a) {
    constexpr int WAVES = WM * WN, XT = MI * WM, WT = NI * WN;  // tiles of x and W
    constexpr int XLOADS = 2 * XT / WAVES, LOADS = XLOADS + 2 * WT / WAVES;     // a wavefront's, half a tile each
    constexpr int DEAL = sizeof(T) == 2 ? NI : 1;               // tiles that rows of W are dealt to
    static_assert(2 * XT % WAVES == 0 && 2 * WT % WAVES == 0 && DEPTH >= 2);
    __shared__ __attribute__((aligned(16))) int8_t lds[DEPTH][(XT + WT) * kTile];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4, wm = wave / WN, wn = wave % WN;
    // workgroups of one XCD take neighbouring tiles, columns of tiles in groups of 8 rows
    const uint32_t tiles_m = uint32_t((a.m + 16 * XT - 1) / (16 * XT)), tiles_n = uint32_t((a.n + 16 * WT - 1) / (16 * WT));
    const uint32_t total = tiles_m * tiles_n, xcd = blockIdx.x % 8;
    const uint32_t id = xcd * (total / 8) + (xcd < total % 8 ? xcd : total % 8) + blockIdx.x / 8;
    const uint32_t group = 8 * tiles_n, first = id / group * 8, rows = tiles_m - first < 8 ? tiles_m - first : 8;
    const int64_t m0 = int64_t(first + id % group % rows) * 16 * XT, n0 = int64_t(id % group / rows) * 16 * WT;
    const int8_t* const x = scalar(a.x + m0 * a.ldx);
    const int8_t* const w = scalar(a.w + n0 * a.ldw);

    // which KB of a step's tiles each load fills (x's first), and where this lane's piece comes from
    auto place = [&](int i) { return i < XLOADS ? wave * XLOADS + i : 2 * XT + wave * (LOADS - XLOADS) + i - XLOADS; };
    auto piece = [&](int i) { return column_of(place(i) & 1, lane); };
    const int k16 = int((a.k + 15) / 16 * 16), steps = int((a.k + kStep - 1) / kStep), tail = int(a.k % kStep);
    uint32_t offset[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int row = row_of(place(i) & 1, lane), tile = place(i) >> 1;
        if (i < XLOADS) {
            const int64_t at = 16 * tile + row, most = a.m - 1 - m0;
            offset[i] = uint32_t((at < most ? at : most) * a.ldx) + piece(i);
        } else {
            const int t = tile - XT;
            const int64_t at = t / DEAL * 16 * DEAL + 4 * DEAL * (row >> 2) + 4 * (t % DEAL) + (row & 3), most = a.n - 1 - n0;
            offset[i] = uint32_t((at < most ? at : most) * a.ldw) + piece(i);
        }
    }
    // Pieces past the row's end are the first one again.  Steps past the last one load nothing
    // (from no rows), so that the loads on their way can be counted.
    auto load = [&](int step, int8_t* to, int i) {
        const int c = piece(i), from = step * kStep;
        const bool whole = from + kStep <= k16;
        load_to_lds(rows_at(i < XLOADS ? x : w, step < steps), whole || c < k16 - from ? offset[i] : offset[i] - c, from, to + place(i) * 1024);
    };

    i32x4 acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i + 1 < DEPTH; ++i)
#pragma unroll
        for (int l = 0; l < LOADS; ++l) load(i, lds[i], l);
    int at = 0;                                                 // step s is in lds[at]
    for (int s = 0; s < steps; ++s) {
        wait_loads<LOADS * (DEPTH - 2)>();
        if (s == steps - 1 && tail) {                           // columns past k of x are cleared by whoever loaded them
#pragma unroll
            for (int i = 0; i < XLOADS; ++i) {
                i32x4* p = reinterpret_cast<i32x4*>(lds[at] + place(i) * 1024 + 16 * lane);
                if (piece(i) + 16 > tail) *p &= first_bytes(tail - piece(i));
            }
            wait_loads<LOADS * (DEPTH - 2)>();
        }
        barrier();
        int8_t* const to = lds[at == 0 ? DEPTH - 1 : at - 1];
        const int8_t* const xt = lds[at] + wm * MI * kTile;
        const int8_t* const wt = lds[at] + (XT + wn * NI) * kTile;
        // NI products at a time, what they need read two such groups ahead; the loads go between
        // the groups of the first half, so that their addresses do not hold all products up
        constexpr int GROUPS = 2 * MI, AHEAD = 2;
        i32x4 xf[GROUPS], wf[2][NI];
        auto read_w = [&](int q) {
#pragma unroll
            for (int j = 0; j < NI; ++j) wf[q][j] = fragment(wt + j * kTile, r, g, q);
        };
        auto read_x = [&](int q) { xf[q] = fragment(xt + q % MI * kTile, r, g, q / MI); };
        read_w(0);
#pragma unroll
        for (int q = 0; q < AHEAD; ++q) read_x(q);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int q = 0; q < GROUPS; ++q) {
            if (q == (MI > AHEAD ? MI - AHEAD : 0)) read_w(1);
            if (q + AHEAD < GROUPS) read_x(q + AHEAD);
            if (q < MI) {
#pragma unroll
                for (int i = q * LOADS / MI; i < (q + 1) * LOADS / MI; ++i) load(s + DEPTH - 1, to, i);
            }
#pragma unroll
            for (int j = 0; j < NI; ++j)
                acc[q % MI][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[q / MI][j], xf[q], acc[q % MI][j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
        at = at + 1 == DEPTH ? 0 : at + 1;
    }
    wait_loads<0>();

    // In 16 bits a lane's columns are neighbours; in 32 those of a row's four lanes are, 64 bytes a
    // store: 717 x 14784 x 82 takes 15.1 us, with a lane's 64 bytes in four stores 26.8.
    // All stores go past the caches, which keep more of x and W that way: 8192 x 28672 x 1024 in bf16
    // takes 302 us in place of 363, 1024 x 8192 x 8192 73 (80).  A row's follow one another, so that
    // they fill whole lines before these are sent on.
    constexpr int COUNT = 4 * DEAL;                             // neighbouring columns
    const int64_t n = n0 + wn * 16 * NI + COUNT * g;
    const int left = a.n - n < 16 * NI ? int(a.n - n) : 16 * NI;
    if (left <= 0) return;
    auto column = [](int c) { return c / COUNT * 4 * COUNT + c % COUNT; };
    float ws[4 * NI];
#pragma unroll
    for (int c = 0; c < 4 * NI; ++c) ws[c] = a.ws[column(c) < left ? n + column(c) : n];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int64_t m = m0 + (wm * MI + i) * 16 + r;
        if (m >= a.m) continue;
        int sum[4 * NI];
#pragma unroll
        for (int c = 0; c < 4 * NI; ++c) sum[c] = acc[i][c / 4][c % 4];
        __builtin_amdgcn_sched_barrier(0);                      // row by row, for the registers
        T t[NI / DEAL][COUNT];
        scaled(reinterpret_cast<T (&)[4 * NI]>(t), sum, a.xs[m], ws);
        T* const y = static_cast<T*>(a.y) + m * a.ldy + n;
        if constexpr (DEAL == NI) {
            store_columns<true>(y, t[0], left);
        } else if (left > column(4 * NI - 1)) {
#pragma unroll
            for (int j = 0; j < NI / DEAL; ++j) store_past(y + 4 * COUNT * j, t[j]);
        } else {
#pragma unroll
            for (int c = 0; c < 4 * NI; ++c)
                if (column(c) < left) y[column(c)] = t[c / COUNT][c % COUNT];
        }
    }
}

// ---------------------------------------------------------------- few rows of x
// A workgroup takes 16 NB rows of W and 16 MB of x; its wavefronts take every WAVES-th
// step of the columns, each through DEPTH tiles of its own in LDS, so that they wait
// for nobody until they join their sums.
template <typename T, int MB, int NB, int WAVES, int DEPTH>
__global__ __launch_bounds__(64 * WAVES) void int8_few_kernel(Int8MatmulArgs a) {
    static_assert(DEPTH >= 2 && DEPTH <= 4, "the waits at a wavefront's last steps");
    constexpr int TILES = MB + NB, LOADS = 2 * TILES;
    constexpr int JOIN = WAVES * MB * NB * 64 * 16, RING = WAVES * DEPTH * TILES * kTile;
    __shared__ __attribute__((aligned(16))) int8_t lds[JOIN > RING ? JOIN : RING];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t n0 = int64_t(blockIdx.x) * 16 * NB, m0 = int64_t(blockIdx.y) * 16 * MB;
    const int8_t* const x = scalar(a.x + m0 * a.ldx);
    const int8_t* const w = scalar(a.w + n0 * a.ldw);
    uint32_t offset[LOADS], column[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) column[h] = column_of(h, lane);
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int row = row_of(i & 1, lane), tile = i >> 1;
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
    // Rows are often a power of two apart, so that all their steps' bytes lie in few of the memory's
    // channels: neighbouring workgroups begin at neighbouring steps.
    const int rot = int(blockIdx.x % uint32_t(steps));
    auto step_of = [&](int i) {
        const int s = wave + i * WAVES + rot;
        return s < steps ? s : s - steps;
    };
    int8_t* const ring = lds + wave * DEPTH * TILES * kTile;
    auto load = [&](int i, int place) {                         // its i-th
        const int from = step_of(i) * kStep, left = k16 - from;
        int8_t* to = ring + place * TILES * kTile;
#pragma unroll
        for (int l = 0; l < LOADS; ++l) {
            const uint32_t c = column[l & 1];
            load_to_lds(rows_at(l >> 1 < MB ? x : w, true), int(c) < left ? offset[l] : offset[l] - c, from, to + l * (kTile / 2));
        }
    };

    i32x4 acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    auto multiply = [&](int i, int place) {
        const int8_t* tiles = ring + place * TILES * kTile;
        const int left = int(a.k) - step_of(i) * kStep;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            i32x4 xf[MB], wf[NB];
#pragma unroll
            for (int j = 0; j < NB; ++j) wf[j] = fragment(tiles + (MB + j) * kTile, r, g, s);
#pragma unroll
            for (int j = 0; j < MB; ++j) xf[j] = fragment(tiles + j * kTile, r, g, s);
            if (left < kStep) {
                const i32x4 mask = first_bytes(left - 64 * s - 16 * g);
#pragma unroll
                for (int j = 0; j < MB; ++j) xf[j] &= mask;
            }
#pragma unroll
            for (int q = 0; q < MB; ++q)
#pragma unroll
                for (int j = 0; j < NB; ++j) acc[q][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[j], xf[q], acc[q][j], 0, 0, 0);
        }
    };
#pragma unroll
    for (int i = 0; i + 1 < DEPTH; ++i)
        if (i < mine) load(i, i);
    int at = 0;
    for (int i = 0; i < mine; ++i) {
        const int after = mine - 1 - i;
        if (after >= DEPTH - 2) wait_loads<LOADS * (DEPTH - 2)>();      // its i-th is there, what was before has been read
        else if (DEPTH > 3 && after == 1) wait_loads<LOADS>();
        else wait_loads<0>();
        if (after >= DEPTH - 1) load(i + DEPTH - 1, at == 0 ? DEPTH - 1 : at - 1);
        multiply(i, at);
        at = at + 1 == DEPTH ? 0 : at + 1;
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
        T t[4];
        scaled(t, sum, a.xs[m], ws);
        store_columns<false>(static_cast<T*>(a.y) + m * a.ldy + n, t, left);
    }
}

template <typename T, int MI, int NI, int WM, int WN, int DEPTH>
inline hipError_t tiles(const Int8MatmulArgs& a, hipStream_t s) {
    const int64_t tm = (a.m + 16 * MI * WM - 1) / (16 * MI * WM), tn = (a.n + 16 * NI * WN - 1) / (16 * NI * WN);
    return launch(int8_tiles_kernel<T, MI, NI, WM, WN, DEPTH>, dim3(uint32_t(tm * tn)), dim3(64 * WM * WN), 0, s, a);
}

template <typename T, int MB, int NB, int WAVES, int DEPTH>
inline hipError_t few(const Int8MatmulArgs& a, hipStream_t s) {
    const dim3 grid(uint32_t((a.n + 16 * NB - 1) / (16 * NB)), uint32_t((a.m + 16 * MB - 1) / (16 * MB)));
    return launch(int8_few_kernel<T, MB, NB, WAVES, DEPTH>, grid, dim3(64 * WAVES), 0, s, a);
}

// ---------------------------------------------------------------- selection
// The variant with the least estimated time: `fixed` + rounds (`round` + steps `step`) us,
// the rounds those in which its workgroups go over the 256 compute units and the steps
// those of 128 columns.  The constants are fitted to each variant's times at 190 sizes
// from 1 x 64 x 64 to 8192 x 28672 x 16384 (within 8 to 16% on average); what was
// chosen took 1.8% more than the best of them on average, at most 1.5 times.  That was to bf16
// and through the caches (past them the larger ones take 1 to 8% less), before 32-bit outputs were
// dealt to lanes as they are; y's type is not in the estimate.  In us, as measured then:
//     1 x 4096 x 4096        1 x 1 tiles 4.5, 1 x 2 4.6, 1 x 4 5.6
//     1 x 28672 x 8192       1 x 1 45.0, 1 x 2 50.2, 1 x 4 40.9
//     32 x 8192 x 8192       2 x 2 11.8, 2 x 4 12.5, 4 x 2 12.0
//     32 x 28672 x 8192      2 x 2 59.4, 2 x 4 45.0, 4 x 2 61.5
//     64 x 8192 x 8192       2 x 2 22.0, 4 x 2 12.8, 4 x 4 16.3, 64 x 128 25.5
//     64 x 16384 x 8192      4 x 2 39.8, 4 x 4 29.4, 64 x 128 40.7
//     512 x 4096 x 4096      64 x 128 16.4, 128 x 128 of 8 wavefronts 20.6, of 4 27.6
//     512 x 8192 x 4096      64 x 128 31.0, 128 x 128 of 8 wavefronts 23.4, of 4 30.2
//     1024 x 8192 x 8192     128 x 128 of 8 wavefronts 82.2, of 4 72.0, 256 x 256 96.8
//     8192 x 8192 x 8192     128 x 128 of 4 wavefronts 572, 256 x 256 463
struct Variant {
    int rows, columns;                   // of y in a workgroup
    float fixed, round, step;
};
constexpr Variant kVariants[] = {
    {16, 16, 1.00f, 1.28f, 0.06f},  {16, 32, 0.92f, 1.40f, 0.08f},   {16, 64, 0.87f, 1.51f, 0.14f},   {32, 32, 0.73f, 1.74f, 0.09f},
    {32, 64, 0.61f, 2.20f, 0.16f},  {64, 32, 0.52f, 2.26f, 0.13f},   {64, 64, 0.00f, 3.30f, 0.20f},   {64, 128, 0.00f, 3.59f, 0.37f},
    {128, 128, 0.00f, 4.31f, 0.48f}, {128, 128, 1.36f, 2.84f, 0.76f}, {256, 256, 0.00f, 5.33f, 1.26f},
};
constexpr int kFew = 7;                  // of them are for few rows: rows of workgroups in a grid's second dimension

inline int choose(const Int8MatmulArgs& a) {
    const float steps = float((a.k + kStep - 1) / kStep);
    int best = 0;
    float least = 0;
    for (int i = 0; i < int(sizeof(kVariants) / sizeof(Variant)); ++i) {
        const Variant& v = kVariants[i];
        const int64_t down = (a.m + v.rows - 1) / v.rows, blocks = down * ((a.n + v.columns - 1) / v.columns);
        if (i < kFew && down > 65535) continue;
        const float time = v.fixed + float((blocks + 255) / 256) * (v.round + steps * v.step);
        if (least == 0 || time < least) best = i, least = time;
    }
    return best;
}

template <typename T>
inline hipError_t int8_matmul_t(const Int8MatmulArgs& a, hipStream_t s) {
    switch (choose(a)) {
    case 0: return few<T, 1, 1, 8, 4>(a, s);
    case 1: return few<T, 1, 2, 8, 3>(a, s);
    case 2: return few<T, 1, 4, 4, 3>(a, s);
    case 3: return few<T, 2, 2, 8, 2>(a, s);
    case 4: return few<T, 2, 4, 4, 3>(a, s);
    case 5: return few<T, 4, 2, 6, 2>(a, s);
    case 6: return few<T, 4, 4, 4, 2>(a, s);
    case 7: return tiles<T, 2, 2, 2, 4, 4>(a, s);
    case 8: return tiles<T, 4, 2, 2, 4, 4>(a, s);
    case 9: return tiles<T, 4, 4, 2, 2, 2>(a, s);
    default: return tiles<T, 8, 4, 2, 4, 2>(a, s);
    }
}

}  // namespace int8_matmul_detail
}  // namespace bl
