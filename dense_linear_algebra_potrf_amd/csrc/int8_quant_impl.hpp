// Rounding of rows to 8-bit integers with one scale a row.
//
//     scale = max |x| / 127,  q = rint(x / scale)
//
// A row is read once: it stays in the registers of the TPR threads that share it
// (VPT vectors of 8 elements each), from the search for its largest magnitude to the
// stores.  Rows that do not fit are read twice, the second time mostly from the
// cache.  Under given scales nothing is searched and every vector is on its own.
//
// HBM bounds it: an element's size and a byte for its code.  8192 rows of 8192 in bf16 take
// 39 us (a copy of as many bytes 39); 5003 of 4099 in f32 with values 36 (36), with the
// values stored through the caches 43.  Rows too long for registers are read twice with one load
// a thread on its way: 300 of 100000 in bf16 38 (18).  Under given scales 8192 of 8192 in bf16
// take 48 (39), 5003 of 4099 in f32 with values 35 (36), 200000 of 128 in bf16 18.7 (15.1).
#pragma once

#include "integer_impl.hpp"

namespace bl {
namespace int8_quant_detail {

using namespace layer;

constexpr int kThreads = 256;

// The codes, and what they stand for, of eight elements from column c on.
template <bool GIVEN, typename T>
__device__ __forceinline__ void round_store(const Int8QuantArgs& a, int64_t row, int64_t c, const Raw8<T>& x, float scale,
                                            float inverse, int left) {
    float v[8], q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = !GIVEN || x[j] == x[j] ? x[j] : 0.0f;
    Codes codes = to_codes(v, scale, inverse, q);
    if (!(inverse > 0)) {                                       // no codes under this scale
        codes = Codes{{0, 0}};
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = 0;
    }
    store_codes(a.q + row * a.ldq + c, codes, left);
    if (a.values) {
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] *= scale;
        store8_past(static_cast<T*>(a.values) + row * a.ldv + c, q, left);
    }
}

template <typename T, int TPR, int VPT>
__global__ __launch_bounds__(TPR < kThreads ? kThreads : TPR) void int8_quant_kernel(Int8QuantArgs a) {
    constexpr int ROWS = TPR < kThreads ? kThreads / TPR : 1, WAVES = TPR < 64 ? 1 : TPR / 64;
    __shared__ uint32_t tops[ROWS][WAVES];
    const int t = threadIdx.x % TPR, r = threadIdx.x / TPR, n = int(a.n);
    for (int64_t row = int64_t(blockIdx.x) * ROWS + r; row < a.rows; row += int64_t(gridDim.x) * ROWS) {
        const T* x = static_cast<const T*>(a.x) + row * a.ldx;
        Raw8<T> v[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) v[i] = load8(x + 8 * (i * TPR + t), n - 8 * (i * TPR + t));
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) top = Max{}(top, magnitude(v[i][j]));
        const float scale = code_scale(block_reduce<TPR>(top, Max{}, tops[r]));
        if (t == 0) a.scales[row] = scale;
        const float inverse = 1.0f / scale;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 8 * (i * TPR + t), left = n - c;
            if (left > 0) round_store<false>(a, row, c, v[i], scale, inverse, left);
        }
        if constexpr (WAVES > 1) __syncthreads();               // the next row's maximum
    }
}

// Rows of any length: a workgroup takes a row's vectors in turn, twice.
template <typename T>
__global__ __launch_bounds__(512) void int8_quant_long_kernel(Int8QuantArgs a) {
    __shared__ uint32_t tops[8];
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + row * a.ldx;
        uint32_t top = 0;
        for (int64_t c = 8 * threadIdx.x; c < a.n; c += 8 * 512) {
            const Raw8<T> v = load8(x + c, a.n - c < 8 ? int(a.n - c) : 8);
#pragma unroll
            for (int j = 0; j < 8; ++j) top = Max{}(top, magnitude(v[j]));
        }
        const float scale = code_scale(block_reduce<512>(top, Max{}, tops));
        if (threadIdx.x == 0) a.scales[row] = scale;
        const float inverse = 1.0f / scale;
        for (int64_t c = 8 * threadIdx.x; c < a.n; c += 8 * 512) {
            const int left = a.n - c < 8 ? int(a.n - c) : 8;
            round_store<false>(a, row, c, load8(x + c, left), scale, inverse, left);
        }
        __syncthreads();                                        // the next row's maximum
    }
}

// Given scales: 2^across threads share a row (or a part of it), 8 columns each.
template <typename T>
__global__ __launch_bounds__(kThreads) void int8_quant_given_kernel(Int8QuantArgs a, int across) {
    const int64_t c = 8 * ((int64_t(blockIdx.x) << across) + (threadIdx.x & ((1 << across) - 1)));
    if (c >= a.n) return;
    const int left = a.n - c < 8 ? int(a.n - c) : 8, down = kThreads >> across;
    for (int64_t row = int64_t(blockIdx.y) * down + (threadIdx.x >> across); row < a.rows; row += int64_t(gridDim.y) * down) {
        const float scale = a.given[row];
        const bool usable = scale >= kTiny && magnitude(scale) < kInfBits;
        round_store<true>(a, row, c, load8(static_cast<const T*>(a.x) + row * a.ldx + c, left), scale,
                          usable ? 1.0f / scale : 0.0f, left);
    }
}

constexpr int64_t kMostGroups = 1 << 20;    // workgroups of a launch; rows beyond it loop

template <typename T>
inline hipError_t int8_quant_t(const Int8QuantArgs& a, hipStream_t s) {
    auto go = [&](auto tpr, auto vpt) {
        constexpr int TPR = decltype(tpr)::value, VPT = decltype(vpt)::value, ROWS = TPR < kThreads ? kThreads / TPR : 1;
        const int64_t need = (a.rows + ROWS - 1) / ROWS;
        return launch(int8_quant_kernel<T, TPR, VPT>, dim3(uint32_t(need < kMostGroups ? need : kMostGroups)),
                      dim3(TPR < kThreads ? kThreads : TPR), 0, s, a);
    };
    const int64_t v = (a.n + 7) / 8;
    if (a.given) {
        int across = 2;
        while (across < 8 && (1 << across) < v) ++across;
        const int64_t wide = (v + (1 << across) - 1) >> across, down = (a.rows + (kThreads >> across) - 1) / (kThreads >> across);
        return launch(int8_quant_given_kernel<T>, dim3(uint32_t(wide), uint32_t(down < 65535 ? down : 65535)), dim3(kThreads), 0,
                      s, a, across);
    }
    if (v > 4096)
        return launch(int8_quant_long_kernel<T>, dim3(uint32_t(a.rows < kMostGroups ? a.rows : kMostGroups)), dim3(512), 0, s, a);
    if (v <= 16) return go(ic<16>{}, ic<1>{});
    if (v <= 32) return go(ic<32>{}, ic<1>{});
    if (v <= 64) return go(ic<64>{}, ic<1>{});
    if (v <= 128) return go(ic<64>{}, ic<2>{});
    if (v <= 256) return go(ic<256>{}, ic<1>{});
    if (v <= 512) return go(ic<256>{}, ic<2>{});
    if (v <= 768) return go(ic<256>{}, ic<3>{});
    if (v <= 1024) return go(ic<256>{}, ic<4>{});
    if (v <= 1536) return go(ic<512>{}, ic<3>{});
    if (v <= 2048) return go(ic<512>{}, ic<4>{});
    return go(ic<512>{}, ic<8>{});
}

}  // namespace int8_quant_detail
}  // namespace bl
