// Device helpers shared by the low-bit layer operators (gfx950).
#pragma once

#include "common.hpp"
#include "layer.hpp"

namespace bl {
namespace layer {

using bf16 = __bf16;
using f16 = _Float16;

constexpr float kE4M3Max = 448.0f, kE2M1Max = 6.0f;
constexpr float kTiny = 0x1p-126f;              // smallest scale that is stored
constexpr uint32_t kInfBits = 0x7f800000u;      // bits of |v| at or above it: not finite

// ---------------------------------------------------------------- eight elements
// Rows may start at any multiple of the element size: the 16-byte accesses
// below carry no alignment, which the hardware's global loads and stores accept.
// They are held as they come, two 16-bit elements to a register.
template <typename T> struct Raw8 {
    uint32_t word[2 * sizeof(T)];
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (sizeof(T) == 4) {
            return __builtin_bit_cast(float, word[i]);
        } else if constexpr (std::is_same_v<T, bf16>) {
            return __builtin_bit_cast(float, i & 1 ? word[i / 2] & 0xffff0000u : word[i / 2] << 16);
        } else {
            return float(__builtin_bit_cast(f16, uint16_t(word[i / 2] >> (16 * (i & 1)))));
        }
    }
    // Keeps the compiler from carrying the converted elements over this point
    // (twice the registers); they are converted again after it.
    __device__ __forceinline__ void keep_packed() {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (uint32_t& w : word) asm volatile("" : "+v"(w));
        }
    }
};

// `count` of 8 elements at p; the missing ones are zero.
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p, int count) {
    Raw8<T> r;
    if (count >= 8) {
        __builtin_memcpy(&r, p, sizeof(r));
    } else {
        T v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < count ? p[i] : T(0.0f);
        __builtin_memcpy(&r, v, sizeof(r));
    }
    return r;
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8], int count) {
    T v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = T(f[i]);
    if (count >= 8) {
        __builtin_memcpy(p, v, sizeof(v));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < count) p[i] = v[i];
    }
}

// ---------------------------------------------------------------- lane exchange
// Butterflies over the 4, 8 or 16 lanes of a row by DPP (quad permutes, then
// mirrors: after the quads agree, lane 7 - i of a half row and lane 15 - i of a
// row hold the other half's value), and over the four rows of the wavefront by
// the permlane swaps.  Every lane gets the result, in a fixed order.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return uint32_t(__builtin_amdgcn_mov_dpp(int(v), CTRL, 0xf, 0xf, true));
}
template <int CTRL>
__device__ __forceinline__ float dppf(float v) {
    return __builtin_bit_cast(float, dpp<CTRL>(__builtin_bit_cast(uint32_t, v)));
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

template <int LANES, typename T, typename F>
__device__ __forceinline__ T row_reduce(T v, F&& f) {
    auto step = [&](auto ctrl) {
        if constexpr (sizeof(T) == 4 && std::is_same_v<T, float>) v = f(v, dppf<decltype(ctrl)::value>(v));
        else v = f(v, T(dpp<decltype(ctrl)::value>(uint32_t(v))));
    };
    if constexpr (LANES >= 2) step(ic<kXor1>{});
    if constexpr (LANES >= 4) step(ic<kXor2>{});
    if constexpr (LANES >= 8) step(ic<kHalfMirror>{});
    if constexpr (LANES >= 16) step(ic<kMirror>{});
    return v;
}

// The same over LANES = 16, 32 or 64 neighbouring lanes.
template <int LANES, typename T, typename F>
__device__ __forceinline__ T wave_reduce(T v, F&& f) {
    v = row_reduce<16>(v, f);
    if constexpr (LANES >= 32) {
        const uint32_t u = __builtin_bit_cast(uint32_t, v);
        auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        v = f(__builtin_bit_cast(T, uint32_t(a[0])), __builtin_bit_cast(T, uint32_t(a[1])));
    }
    if constexpr (LANES >= 64) {
        const uint32_t u = __builtin_bit_cast(uint32_t, v);
        auto b = __builtin_amdgcn_permlane32_swap(u, u, false, false);
        v = f(__builtin_bit_cast(T, uint32_t(b[0])), __builtin_bit_cast(T, uint32_t(b[1])));
    }
    return v;
}

struct Add { __device__ __forceinline__ float operator()(float a, float b) const { return a + b; } };
struct Max {   // on the bits of magnitudes: a NaN is the largest
    __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; }
};

// The same over THREADS threads: part of a wavefront, one, or all of a workgroup.
// `slot` is this reduction's own LDS (an entry per wavefront), so that one barrier
// is enough.
template <int THREADS, typename T, typename F>
__device__ __forceinline__ T block_reduce(T v, F&& f, T* slot) {
    v = wave_reduce<(THREADS < 64 ? THREADS : 64)>(v, f);
    if constexpr (THREADS > 64) {
        if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
        __syncthreads();
        v = slot[0];
#pragma unroll
        for (int i = 1; i < THREADS / 64; ++i) v = f(v, slot[i]);
    }
    return v;
}

__device__ __forceinline__ uint32_t magnitude(float v) {
    return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu;
}

// ---------------------------------------------------------------- power-of-two scales
// The byte e + 127 of the least e in -127..127 with max <= MOST * 2^e, from the
// bits of the finite max: MOST = (1 + f) 2^p, so e is the exponent of max less
// p, one more where the fraction of max exceeds f (the addition carries into
// the exponent).  255 (NaN) where max is not finite.
template <int P, uint32_t FRACTION>
__device__ __forceinline__ uint32_t scale_byte(uint32_t max_bits) {
    if (max_bits >= kInfBits) return 255;
    const int e = int((max_bits + (0x7fffffu - FRACTION)) >> 23) - P;
    return uint32_t(e > 0 ? e : 0);
}
__device__ __forceinline__ uint32_t e4m3_scale_byte(uint32_t m) { return scale_byte<8, 0x600000u>(m); }
__device__ __forceinline__ uint32_t e2m1_scale_byte(uint32_t m) { return scale_byte<2, 0x400000u>(m); }

// 2^(b - 127) as a float (subnormal for 0), NaN for 255.
__device__ __forceinline__ float power_of(uint32_t b) {
    return __builtin_bit_cast(float, b == 255 ? 0x7fc00000u : b ? b << 23 : 0x00400000u);
}

// ---------------------------------------------------------------- e4m3
// Eight values times `factor`, rounded to nearest even; |value| is at most 448
// (plus a rounding error that still rounds to 448) or NaN.
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float (&v)[8], float factor, int count) {
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * factor, v[1] * factor, 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * factor, v[3] * factor, lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * factor, v[5] * factor, 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6] * factor, v[7] * factor, hi, true);
    const uint64_t all = uint64_t(uint32_t(hi)) << 32 | uint32_t(lo);
    if (count >= 8) {
        __builtin_memcpy(p, &all, 8);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < count) p[i] = uint8_t(all >> (8 * i));
    }
}

}  // namespace layer
}  // namespace bl
