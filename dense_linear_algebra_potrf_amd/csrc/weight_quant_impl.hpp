// Rounding of weights to 4-bit codes with group scales.
//
// A thread holds 8 neighbouring columns of a row (one dword of codes), so a
// group of 32, 64 or 128 columns is held by 4, 8 or 16 neighbouring lanes of a
// DPP row, and its largest magnitude (or least and largest value) takes two to
// four lane exchanges.  One pass: W is read once, the codes and values written
// once.
//
//     float:    scale 2^e, the least e with max |w| <= 6 2^e;  code = e2m1(w / scale)
//     integer:  scale = bf16(max |w| / 7);                    u = rint(w / scale) + 8
//       zeros:  scale = bf16((max - min) / 15), both with 0;  u = rint(w / scale) + z
//
// HBM bounds it.  16384 x 8192 bf16 to e2m1 with the rounded values: 120 us, 5.1
// TB/s, a large copy's rate (131 us with comparisons and selects in place of the
// conversion instructions); 4096 x 4096 f32 to integers with zero points and values:
// 32.8 us, 4.4 TB/s.  The grid is one thread for every 8 columns: with four rows to a
// thread the second took 35.1 us, and 33.0 with a product with the reciprocal in place
// of the division, and the division only next to a half.
#pragma once

#include "layer_impl.hpp"

namespace bl {
namespace weight_quant_detail {

using namespace layer;

// Eight floats of |t| <= 6 to the codes of the e2m1 floats next to them, ties to the
// even mantissa (0.25 -> 0, 0.75 -> 1, ..., 5 -> 4), the first in the low half byte;
// and back.  The conversion instructions' own scale stays 1: theirs is not defined
// for a subnormal power of two.
__device__ __forceinline__ uint32_t to_e2m1(const float (&t)[8]) {
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, t[0], t[1], 1.0f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, t[2], t[3], 1.0f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, t[4], t[5], 1.0f, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, t[6], t[7], 1.0f, 3);
}
__device__ __forceinline__ void from_e2m1(uint32_t c, float (&v)[8]) {
    using pair = float __attribute__((ext_vector_type(2)));
    const pair a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
    const pair d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2), e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y, v[4] = d.x, v[5] = d.y, v[6] = e.x, v[7] = e.y;
}

template <typename T, Format F, int GROUP, bool ZEROS>
__global__ __launch_bounds__(256) void weight_quant_kernel(WeightQuantArgs a, int across) {
    constexpr int LANES = GROUP / 8;
    // 2^across threads along a row, at least a DPP row's 16; the others down the rows
    const int64_t step = int64_t(gridDim.y) << (8 - across);
    const int c = int((blockIdx.x << across) + (threadIdx.x & ((1 << across) - 1))) * 8;
    const int left = int(a.k) - c;
    for (int64_t row = (int64_t(blockIdx.y) << (8 - across)) + (threadIdx.x >> across); row < a.n; row += step) {
        const Raw8<T> wr = load8(static_cast<const T*>(a.W) + row * a.ldw + c, left);
        float w[8], value[8];
        // the largest magnitude, or those of the values above and below zero, as bits
        // (a NaN is larger than all): one instruction a step
        uint32_t top = 0, low = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            w[j] = wr[j];
            const int32_t bits = __builtin_bit_cast(int32_t, w[j]), other = bits ^ INT32_MIN;
            top = Max{}(top, ZEROS ? uint32_t(bits > 0 ? bits : 0) : magnitude(w[j]));
            if constexpr (ZEROS) low = Max{}(low, uint32_t(other > 0 ? other : 0));
        }
        top = row_reduce<LANES>(top, Max{});
        if constexpr (ZEROS) low = row_reduce<LANES>(low, Max{});
        bool finite = top < kInfBits && low < kInfBits;
        uint32_t codes = 0;
        const int64_t g = c / GROUP;
        const bool head = (threadIdx.x & (LANES - 1)) == 0 && left > 0;
        if constexpr (F == Format::FLOAT) {
            const uint32_t b = e2m1_scale_byte(top);
            const float up = power_of(b), down = power_of(b == 255 ? 255 : 254 - b);
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] *= down;
            codes = finite ? to_e2m1(w) : 0;
            from_e2m1(codes, value);
#pragma unroll
            for (int j = 0; j < 8; ++j) value[j] *= up;
            if (head) static_cast<uint8_t*>(a.scales)[row * a.lds + g] = uint8_t(b);
        } else {
            float span, z = 8;
            [[maybe_unused]] const float least = -__builtin_bit_cast(float, low);
            if constexpr (ZEROS) {
                const float most = __builtin_bit_cast(float, top);
                span = (most - least) / 15.0f;
                finite = finite && magnitude(span) < kInfBits;
            } else {
                span = __builtin_bit_cast(float, top) / 7.0f;
            }
            const bf16 stored = bf16(finite ? fmaxf(float(bf16(span)), kTiny) : __builtin_nanf(""));
            const float scale = float(stored);
            if constexpr (ZEROS)
                if (finite) z = fminf(fmaxf(rintf(-least / scale), 0.0f), 15.0f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float q = ZEROS ? fminf(fmaxf(rintf(w[j] / scale) + z, 0.0f), 15.0f)
                                      : fminf(fmaxf(rintf(w[j] / scale), -8.0f), 7.0f) + 8.0f;
                codes |= (finite ? uint32_t(q) : 0u) << (4 * j);
                value[j] = (q - z) * scale;
            }
            if (head) {
                static_cast<bf16*>(a.scales)[row * a.lds + g] = stored;
                if constexpr (ZEROS) a.zeros[row * a.ldz + g] = uint8_t(z);
            }
        }
        const bool whole = c / 2 < a.held;                      // what has no codes is written too
        if (left <= 0 && !whole) continue;
        if (left < 8) codes &= left > 0 ? (1u << (4 * left)) - 1 : 0;   // the half byte past an odd k, and the padding
        uint8_t* out = a.codes + row * a.ldc + c / 2;
        if (left >= 7 || whole) {
            *reinterpret_cast<uint32_t*>(out) = codes;
        } else {
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if (2 * j < left) out[j] = uint8_t(codes >> (8 * j));
        }
        if (a.values) store8(static_cast<T*>(a.values) + row * a.ldv + c, value, left);
    }
}

template <typename T>
inline hipError_t weight_quant_t(Format f, int group, const WeightQuantArgs& a, hipStream_t s) {
    const int64_t threads = (a.k + 7) / 8;                     // of a row
    int across = 4;
    while (across < 8 && (1 << across) < threads) ++across;
    const int64_t down = (a.n + (256 >> across) - 1) >> (8 - across);
    const dim3 grid(uint32_t((threads + (1 << across) - 1) >> across), uint32_t(down < 65535 ? down : 65535)), block(256);
    auto go = [&](auto fmt, auto size, auto zeros) {
        return launch(weight_quant_kernel<T, decltype(fmt)::value, decltype(size)::value, decltype(zeros)::value>,
                      grid, block, 0, s, a, across);
    };
    using I = std::integral_constant<Format, Format::INTEGER>;
    if (f == Format::FLOAT) return go(std::integral_constant<Format, Format::FLOAT>{}, ic<32>{}, std::false_type{});
    if (a.zeros)
        return group == 32   ? go(I{}, ic<32>{}, std::true_type{})
               : group == 64 ? go(I{}, ic<64>{}, std::true_type{})
                             : go(I{}, ic<128>{}, std::true_type{});
    return group == 32   ? go(I{}, ic<32>{}, std::false_type{})
           : group == 64 ? go(I{}, ic<64>{}, std::false_type{})
                         : go(I{}, ic<128>{}, std::false_type{});
}

}  // namespace weight_quant_detail
}  // namespace bl
