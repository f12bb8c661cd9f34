// Products of a few rows with 4-bit weights, y = x W^T, on the matrix cores.
//
// A wavefront multiplies 16 MB rows of x with 16 NB rows of W over chunks of
// 128 columns; the wavefronts of a workgroup take every WAVES-th chunk and join
// their sums in LDS, in a fixed order.
//
// Codes come as they lie in memory, 16 bytes (32 columns) a lane: lane (r, g),
// r = lane % 16 the row of W and g = lane / 16, holds dwords 4 g .. 4 g + 3 of
// the chunk.  A product of 16 x 16 x 32 wants 32 neighbouring columns over the
// four g, so the dwords are transposed over g and register by the permlane
// swaps (four instructions for 32 codes a lane); then product t covers columns
// 32 t .. 32 t + 31, one group of scales (or a part of one), and x is read in
// its natural order.
//
// Integer codes become 16-bit floats through the 8-bit conversion: the byte
// 0000uuuu read as e4m3 is u 2^-9 for every u in 0..15, subnormal or not.  For
// half-precision x the zero point is subtracted there (exact); bfloat16 has no
// packed subtraction, so the product takes u as it is and z times the sum of x
// over the group, from a product with ones, is taken off afterwards.  Scales are
// applied to the sums in 32 bits.
//
// The detours (codes without their scale, codes without their zero point) give
// the definition's result wherever they are finite.  Where they are not, the
// element is computed again from the definition in 64 bits.
#pragma once

#include "layer_impl.hpp"

namespace bl {
namespace weight_matvec_detail {

using namespace layer;

using bf16x8 = bf16 __attribute__((ext_vector_type(8)));
using f16x8 = f16 __attribute__((ext_vector_type(8)));
using bf16x2 = bf16 __attribute__((ext_vector_type(2)));
using f16x2 = f16 __attribute__((ext_vector_type(2)));
using f32x4 = float __attribute__((ext_vector_type(4)));
using u32x4 = uint32_t __attribute__((ext_vector_type(4)));

// How x comes, and the type it is multiplied in: e4m3 values with a power of
// two per block are exact in bfloat16, without it in half precision.
enum class X : int { BF16, F16, F8_BLOCK, F8_ROW };
constexpr bool in_half(X x) { return x == X::F16 || x == X::F8_ROW; }
constexpr bool is_eight(X x) { return x == X::F8_BLOCK || x == X::F8_ROW; }

constexpr int kChunk = 128;       // columns a wavefront takes at a time
constexpr int kWaves = 8;         // wavefronts of a workgroup, at most
constexpr int kGroups = 256;      // groups of a row whose scales are in LDS at a time

// Eight columns of a row as the matrix cores take them: words of two 16-bit floats.
struct Frag { uint32_t word[4]; };

template <bool HALF>
__device__ __forceinline__ f32x4 product(const Frag& a, const Frag& b, f32x4 c) {
    if constexpr (HALF)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

template <bool HALF>
__device__ __forceinline__ Frag from_e4m3(uint32_t lo, uint32_t hi, float scale) {
    Frag f;
    if constexpr (HALF) {
        f.word[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, scale, false));
        f.word[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, scale, true));
        f.word[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, scale, false));
        f.word[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, scale, true));
    } else {
        f.word[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false));
        f.word[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true));
        f.word[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false));
        f.word[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true));
    }
    return f;
}

// Codes of 8 columns (a dword) as floats; integers less `zero` (packed halves)
// for half precision, and as they are for bfloat16.
template <bool HALF, Format F>
__device__ __forceinline__ Frag unpack(uint32_t w, [[maybe_unused]] f16x2 zero) {
    Frag f;
    if constexpr (F == Format::FLOAT) {
        if constexpr (HALF) {
            f.word[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0));
            f.word[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1));
            f.word[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2));
            f.word[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3));
        } else {
            f.word[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 0));
            f.word[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 1));
            f.word[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 2));
            f.word[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 3));
        }
    } else {
        const uint32_t even = w & 0x0f0f0f0fu, odd = w >> 4 & 0x0f0f0f0fu;
        f = from_e4m3<HALF>(__builtin_amdgcn_perm(odd, even, 0x05010400u),
                            __builtin_amdgcn_perm(odd, even, 0x07030602u), 512.0f);
        if constexpr (HALF) {
#pragma unroll
            for (uint32_t& v : f.word) v = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, v) - zero);
        }
    }
    return f;
}

// What a lane holds of x for a chunk: 8 columns of its rows for each of the
// chunk's four products.
template <X XT, int MB>
struct Rows {
    uint32_t x[MB][4][is_eight(XT) ? 2 : 4];
    uint8_t scale[MB][4];
};

// One element from the definition, in 64 bits.
__device__ __forceinline__ double by_definition(const MatvecArgs& a, X xt, Format f, int group, int64_t m, int64_t n) {
    double sum = 0;
    for (int64_t k = 0; k < a.k; ++k) {
        const uint32_t u = a.codes[n * a.ldc + k / 2] >> (4 * (k & 1)) & 15;
        const int64_t g = k / group;
        double w, x;
        if (f == Format::FLOAT) {
            const uint32_t c = u & 7;
            w = c < 2 ? 0.5 * c : ldexp(2.0 + (c & 1), int(c >> 1) - 2);
            w = (u & 8 ? -w : w) * double(power_of(static_cast<const uint8_t*>(a.scales)[n * a.lds + g]));
        } else {
            w = (double(u) - (a.zeros ? double(a.zeros[n * a.ldz + g]) : 8.0)) *
                double(float(static_cast<const bf16*>(a.scales)[n * a.lds + g]));
        }
        if (xt == X::BF16) x = double(float(static_cast<const bf16*>(a.x)[m * a.ldx + k]));
        else if (xt == X::F16) x = double(static_cast<const f16*>(a.x)[m * a.ldx + k]);
        else x = double(__builtin_amdgcn_cvt_f32_fp8(int(static_cast<const uint8_t*>(a.x)[m * a.ldx + k]), 0));
        if (xt == X::F8_BLOCK)
            x *= double(power_of(static_cast<const uint8_t*>(a.xscales)[m * a.ldxs + k / kScaleBlock]));
        sum = fmadd(w, x, sum);
    }
    return sum;
}

template <X XT, Format F, int GROUP, int MB, int NB>
__global__ __launch_bounds__(64 * kWaves) void weight_matvec_kernel(MatvecArgs a, Type yt) {
    constexpr bool HALF = in_half(XT), EIGHT = is_eight(XT);
    constexpr bool OFFSET = F == Format::INTEGER && !HALF;      // zero points are taken off the sums
    constexpr int GROUPS = kChunk / GROUP, STEPS = GROUP / 32;  // groups of a chunk, products of a group
    constexpr int TILE = 16 * NB;                               // rows of W
    __shared__ union {
        uint32_t scales[kGroups][TILE];                         // of the groups at hand, as `scale_of` reads them
        float sums[kWaves][MB * NB * 4][64];
    } lds;

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int r = lane & 15, g = lane >> 4;
    const int64_t n0 = int64_t(blockIdx.x) * TILE, m0 = int64_t(blockIdx.y) * (16 * MB);
    const int64_t chunks = (a.k + kChunk - 1) / kChunk, whole = a.k / kChunk;
    const int64_t groups = (a.k + GROUP - 1) / GROUP;

    // rows past the end read the last one; their results are not stored
    int64_t row_n[NB], row_m[MB];
#pragma unroll
    for (int i = 0; i < NB; ++i) row_n[i] = n0 + 16 * i + r < a.n ? n0 + 16 * i + r : a.n - 1;
#pragma unroll
    for (int i = 0; i < MB; ++i) row_m[i] = m0 + 16 * i + r < a.m ? m0 + 16 * i + r : a.m - 1;

    // Scales of the groups from `first` on, to LDS: a float's upper half and, for
    // integers, the zero point in the lower.  Neighbouring lanes take neighbouring
    // rows and 8 groups each, so that the writes spread over the banks.  Groups
    // that the last chunk lacks get a finite scale; their products are zero.
    auto stage = [&](int64_t first, int count) {
        const int rounded = (count + GROUPS - 1) / GROUPS * GROUPS, octets = (rounded + 7) / 8;
        for (int e = threadIdx.x; e < octets * TILE; e += blockDim.x) {
            const int row = e % TILE, at = e / TILE * 8, left = count - at;
            const int64_t n = n0 + row < a.n ? n0 + row : a.n - 1, s0 = n * a.lds + first + at;
            uint32_t v[8];
            if constexpr (F == Format::FLOAT) {
                const uint8_t* p = static_cast<const uint8_t*>(a.scales) + s0;
                uint8_t s[8] = {};
                if (left >= 8) __builtin_memcpy(s, p, 8);
                else
                    for (int j = 0; j < 7; ++j) s[j] = j < left ? p[j] : 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = __builtin_bit_cast(uint32_t, power_of(s[j]));
            } else {
                const uint16_t* p = static_cast<const uint16_t*>(a.scales) + s0;
                const uint8_t* q = a.zeros + n * a.ldz + first + at;
                uint16_t s[8] = {};
                uint8_t z[8] = {8, 8, 8, 8, 8, 8, 8, 8};
                if (left >= 8) {
                    __builtin_memcpy(s, p, 16);
                    if (a.zeros) __builtin_memcpy(z, q, 8);
                } else {
                    for (int j = 0; j < 7; ++j) {
                        s[j] = j < left ? p[j] : 0;
                        if (a.zeros) z[j] = j < left ? q[j] : 0;
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = uint32_t(s[j]) << 16 | z[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (at + j < rounded) lds.scales[at + j][row] = v[j];
        }
    };

    // TAIL: the last chunk, which ends inside; what is past the row's end is zero.
    auto load = [&](auto tail, int64_t c, uint32_t (&d)[NB][4]) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int64_t at = c * (kChunk / 2) + 16 * g;
            u32x4 w = {0, 0, 0, 0};
            if (!decltype(tail)::value || at < (a.k + 1) / 2)
                w = *reinterpret_cast<const u32x4*>(a.codes + row_n[i] * a.ldc + at);
#pragma unroll
            for (int j = 0; j < 4; ++j) d[i][j] = w[j];
        }
    };
    auto load_x = [&](auto tail, int64_t c, int t, Rows<XT, MB>& d) {
        constexpr bool TAIL = decltype(tail)::value;
        const int64_t k = c * kChunk + 32 * t + 8 * g;
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            if constexpr (EIGHT) {
                const uint8_t* p = static_cast<const uint8_t*>(a.x) + row_m[i] * a.ldx + k;
                uint64_t v = 0;
                if (!TAIL || k + 8 <= a.k) {
                    __builtin_memcpy(&v, p, 8);
                } else {
                    for (int j = 0; j < 8; ++j)
                        if (k + j < a.k) v |= uint64_t(p[j]) << (8 * j);
                }
                d.x[i][t][0] = uint32_t(v);
                d.x[i][t][1] = uint32_t(v >> 32);
                if constexpr (XT == X::F8_BLOCK) {
                    const int64_t b = c * 4 + t;
                    d.scale[i][t] = !TAIL || b * kScaleBlock < a.k
                                        ? static_cast<const uint8_t*>(a.xscales)[row_m[i] * a.ldxs + b] : 127;
                }
            } else {
                const uint16_t* p = static_cast<const uint16_t*>(a.x) + row_m[i] * a.ldx + k;
                if (!TAIL || k + 8 <= a.k) {
                    __builtin_memcpy(d.x[i][t], p, 16);
                } else {
                    uint16_t v[8] = {};
                    for (int j = 0; j < 8; ++j)
                        if (k + j < a.k) v[j] = p[j];
                    __builtin_memcpy(d.x[i][t], v, 16);
                }
            }
        }
    };

    f32x4 acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    // Multiplies a chunk whose first group is `group` of those in LDS; MORE: and
    // loads x of chunk `next` in the place of what has been multiplied.
    auto multiply = [&](auto more, uint32_t (&d)[NB][4], int group, Rows<XT, MB>& xr, int64_t next) {
#pragma unroll
        for (int j = 0; j < NB; ++j) {                          // dword (g, register) -> (register, g)
            uint32_t(&w)[4] = d[j];
            auto p = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
            auto q = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
            auto u = __builtin_amdgcn_permlane16_swap(p[0], q[0], false, false);
            auto v = __builtin_amdgcn_permlane16_swap(p[1], q[1], false, false);
            w[0] = u[0], w[1] = u[1], w[2] = v[0], w[3] = v[1];
        }
#pragma unroll
        for (int s = 0; s < GROUPS; ++s) {
            f32x4 part[MB][NB], ones[MB];
            float scale[NB], zero[NB];
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const uint32_t v = lds.scales[group + s][16 * j + r];
                scale[j] = __builtin_bit_cast(float, F == Format::FLOAT ? v : v & 0xffff0000u);
                zero[j] = float(v & 0xffu);
            }
#pragma unroll
            for (int i = 0; i < MB; ++i) {
                ones[i] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < NB; ++j) part[i][j] = f32x4{0, 0, 0, 0};
            }
#pragma unroll
            for (int q = 0; q < STEPS; ++q) {
                const int t = s * STEPS + q;
                Frag x[MB];
#pragma unroll
                for (int i = 0; i < MB; ++i) {
                    if constexpr (EIGHT)
                        x[i] = from_e4m3<HALF>(xr.x[i][t][0], xr.x[i][t][1], XT == X::F8_BLOCK ? power_of(xr.scale[i][t]) : 1.0f);
                    else
                        x[i] = Frag{{xr.x[i][t][0], xr.x[i][t][1], xr.x[i][t][2], xr.x[i][t][3]}};
                    if constexpr (OFFSET)
                        ones[i] = product<HALF>(x[i], Frag{{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u}}, ones[i]);
                }
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    const f16 z = f16(zero[j]);
                    const Frag w = unpack<HALF, F>(d[j][t], f16x2{z, z});
#pragma unroll
                    for (int i = 0; i < MB; ++i) part[i][j] = product<HALF>(x[i], w, part[i][j]);
                }
                if constexpr (decltype(more)::value) {
                    // not earlier: x would be held twice
                    __builtin_amdgcn_sched_barrier(0);
                    load_x(std::false_type{}, next, t, xr);
                }
            }
#pragma unroll
            for (int j = 0; j < NB; ++j) {
#pragma unroll
                for (int i = 0; i < MB; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float p = OFFSET ? fmadd(-zero[j], ones[i][e], part[i][j][e]) : part[i][j][e];
                        acc[i][j][e] = fmadd(scale[j], p, acc[i][j][e]);
                    }
            }
        }
    };

    constexpr int PHASE = kGroups / GROUPS;                     // chunks whose scales fit
    uint32_t now[NB][4];
    Rows<XT, MB> xr;
    for (int64_t base = 0; base < chunks; base += PHASE) {
        const int64_t end = base + PHASE < chunks ? base + PHASE : chunks;
        const int64_t full = end < whole ? end : whole;         // of them, those that lie inside the row
        int64_t c = base + wave;
        bool any = c < full;
        if (any) load(std::false_type{}, c, now);               // on its way while the scales are staged
        const int64_t g0 = base * GROUPS, count = end * GROUPS < groups ? end * GROUPS - g0 : groups - g0;
        if (base) __syncthreads();
        stage(g0, int(count));
        if (any) {
#pragma unroll
            for (int t = 0; t < 4; ++t) load_x(std::false_type{}, c, t, xr);
        }
        __syncthreads();
        if (any) {
            for (c += waves; c < full; c += waves) {
                uint32_t next[NB][4];
                load(std::false_type{}, c, next);
                multiply(std::true_type{}, now, int(c - waves - base) * GROUPS, xr, c);
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) now[i][j] = next[i][j];
            }
        }
        // the last whole chunk of this wavefront, then the partial one if its turn comes to it
        int64_t at = c - waves;
        while (any || c < end) {
            if (!any) {
                load(std::true_type{}, c, now);
#pragma unroll
                for (int t = 0; t < 4; ++t) load_x(std::true_type{}, c, t, xr);
                at = c;
                c = end;
            }
            any = false;
            multiply(std::false_type{}, now, int(at - base) * GROUPS, xr, 0);
        }
    }

    __syncthreads();                                            // the scales' LDS is free
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) lds.sums[wave][(i * NB + j) * 4 + e][lane] = acc[i][j][e];
    __syncthreads();

    const int64_t rows = a.m - m0 < 16 * MB ? a.m - m0 : 16 * MB;
    for (int e = threadIdx.x; e < int(rows) * TILE; e += blockDim.x) {
        const int ml = e / TILE, nl = e % TILE;       // y's row and column in the tile
        const int64_t m = m0 + ml, n = n0 + nl;
        if (n >= a.n) continue;
        const int slot = (ml / 16 * NB + nl / 16) * 4 + ml % 4, from = ml % 16 / 4 * 16 + nl % 16;
        float v = 0;
        for (int w = 0; w < waves; ++w) v += lds.sums[w][slot][from];
        if (magnitude(v) >= kInfBits) {
            const double s = by_definition(a, XT, F, GROUP, m, n);
            v = XT == X::F8_ROW ? float(s * double(static_cast<const float*>(a.xscales)[m])) : float(s);
        } else if (XT == X::F8_ROW) {
            v *= static_cast<const float*>(a.xscales)[m];
        }
        const int64_t at = m * a.ldy + n;
        if (yt == Type::F32) static_cast<float*>(a.y)[at] = v;
        else if (yt == Type::F16) static_cast<f16*>(a.y)[at] = f16(v);
        else static_cast<bf16*>(a.y)[at] = bf16(v);
    }
}

template <X XT>
inline hipError_t weight_matvec_t(Type yt, Format f, int group, const MatvecArgs& a, hipStream_t s) {
    const int64_t chunks = (a.k + kChunk - 1) / kChunk;
    const dim3 block(uint32_t(64 * (chunks < kWaves ? chunks : kWaves)));
    auto tile = [&](auto fmt, auto size, auto mb, auto nb) {
        constexpr int MB = decltype(mb)::value, NB = decltype(nb)::value;
        const dim3 grid(uint32_t((a.n + 16 * NB - 1) / (16 * NB)), uint32_t((a.m + 16 * MB - 1) / (16 * MB)));
        return launch(weight_matvec_kernel<XT, decltype(fmt)::value, decltype(size)::value, MB, NB>, grid, block, 0, s, a, yt);
    };
    auto shape = [&](auto fmt, auto size) {
        const bool wide = a.n >= 256 * 32;                      // enough rows for every compute unit at 32 each
        if (a.m <= 16) return wide ? tile(fmt, size, ic<1>{}, ic<2>{}) : tile(fmt, size, ic<1>{}, ic<1>{});
        return wide ? tile(fmt, size, ic<2>{}, ic<2>{}) : tile(fmt, size, ic<2>{}, ic<1>{});
    };
    if (f == Format::FLOAT) return shape(std::integral_constant<Format, Format::FLOAT>{}, ic<32>{});
    using I = std::integral_constant<Format, Format::INTEGER>;
    return group == 32 ? shape(I{}, ic<32>{}) : group == 64 ? shape(I{}, ic<64>{}) : shape(I{}, ic<128>{});
}

}  // namespace weight_matvec_detail
}  // namespace bl
