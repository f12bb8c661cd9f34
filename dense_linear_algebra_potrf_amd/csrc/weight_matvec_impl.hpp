// Products of a few rows with 4-bit weights, y = x W^T, on the matrix cores:
//     y[m, n] = sum over groups g of scale[n, g] sum_k x (u - z[n, g]).
//
// HBM bounds it: the codes are read once, 1/4 of the bytes of 16-bit weights.  Up to
// 16 rows of x cost what one does as long as the codes' stream hides the arithmetic,
// which is why even one row goes over the matrix cores: on the vector units, with a
// conversion, a scale and a multiplication per code and row, 1 x 28672 x 8192 took
// 412 us.  Measured, with what a copy of those bytes would take:
//     1 x 28672 x 8192, half precision, groups of 64, zero points  29.4 us (25.2)
//     1 x 16384 x 8192, bfloat16, groups of 128                    16.5    (13.6)
//     4 x 16384 x 4096, e4m3 blocks, e2m1 weights                   9.1    (7.0)
//     16 x 8192 x 8192, bfloat16, groups of 128                    12.5    (6.9)
//     1 x 4096 x 4096: 5.0 to 5.4 us in the kernel, 7.2 a call
//
// A wavefront multiplies 16 MB rows of x with 16 NB rows of W over chunks of
// 128 columns; the wavefronts of a workgroup take every WAVES-th chunk and join
// their sums in LDS, in a fixed order.
//
// A product of 16 x 16 x 32 wants of lane (r, g), r = lane % 16 the row and g =
// lane / 16, the columns 8 g .. 8 g + 7 of 32: product t of a chunk covers its
// columns 32 t .. 32 t + 31, one group of scales or a part of one.
//
// An integer code is put, where it lies, into the bits of a half-precision float
// 1024 + u or 64 + u, two at a time, and the float less 1024 + z or 64 + z is u - z:
// packed in half precision, for bfloat16 (which has no packed sums) by an fma from
// half precision to 32 bits each.  All of it is exact, so the zero point is off
// before the product.  Taken off the sums instead (z times the sum of x) it costs
// less (1 x 16384 x 8192 13.6 us in bfloat16, 16.5 as here; 13.6 and 13.9 in half
// precision), but a large x whose weight is zero then stands in both sums and takes
// the bits of the others with it.  Scales are applied to the sums in 32 bits.
//
// The codes go without their scale, so a sum may leave the range of 32 bits where
// the definition's does not.  What is not finite is computed again from the
// definition in 64 bits, an element at a time: one NaN in x takes 1 x 28672 x 8192
// from 29 us to 1.7 ms, one in 64 rows 64 x 8192 x 8192 from 23 us to 0.5 ms.
#pragma once

#include "layer_impl.hpp"

namespace bl {
namespace weight_matvec_detail {

using namespace layer;

using bf16x8 = bf16 __attribute__((ext_vector_type(8)));
using f16x8 = f16 __attribute__((ext_vector_type(8)));
using f16x2 = f16 __attribute__((ext_vector_type(2)));
using f32x4 = float __attribute__((ext_vector_type(4)));
using u32x4 = uint32_t __attribute__((ext_vector_type(4)));

// How x comes, and the type it is multiplied in: e4m3 values with a power of
// two per block are exact in bfloat16, without it in half precision.
enum class X : int { BF16, F16, F8_BLOCK, F8_ROW };
constexpr bool in_half(X x) { return x == X::F16 || x == X::F8_ROW; }
constexpr bool is_eight(X x) { return x == X::F8_BLOCK || x == X::F8_ROW; }
inline X kind_of(Type xt, Scale xs) {
    return xt == Type::BF16 ? X::BF16 : xt == Type::F16 ? X::F16 : xs == Scale::BLOCK ? X::F8_BLOCK : X::F8_ROW;
}

constexpr int kChunk = 128;       // columns a wavefront takes at a time
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

// What makes u - z of a code's float: less 1024 + z, or 64 + z; z is a byte.  In
// bfloat16 the integers are kept as halves (an fma with a factor of one would become
// a conversion and a sum).
template <bool HALF> struct Zero {
    f16x2 low, high;
    __device__ __forceinline__ explicit Zero(uint32_t z)
        : low(__builtin_bit_cast(f16x2, (z | z << 16) + 0x64006400u)), high(low - f16x2{f16(960.0f), f16(960.0f)}) {}
};
template <> struct Zero<false> {
    float low, high;
    __device__ __forceinline__ explicit Zero(uint32_t z) : low(-0.5f * float(z) - 512.0f), high(low + 480.0f) {}
};
// The scale of a block of 8-bit x, times 8, so that the smallest value of the smallest
// scale, 2^-9 2^-127, is a multiple of bfloat16's smallest step (2^-133), and the
// conversion instruction gets no subnormal scale; NaN where that is beyond 2^127, so
// that the element is computed again in 64 bits, and for a byte of 255.
__device__ __forceinline__ float block_power(uint32_t b) {
    return __builtin_bit_cast(float, b < 252 ? (b + 3) << 23 : 0x7fc00000u);
}
// What the sums are multiplied by: integers in bfloat16 are halves, block-scaled x is
// eight times what it stands for.
template <X XT, Format F>
constexpr float kUnit = (!in_half(XT) && F == Format::INTEGER ? 2.0f : 1.0f) * (XT == X::F8_BLOCK ? 0.125f : 1.0f);

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

// Codes of 8 columns (a dword) as floats, integers less their zero point (in
// bfloat16 half of that) and in the order in which they come apart: 0 4 1 5 2 6 3 7.
template <bool HALF, Format F>
__device__ __forceinline__ Frag unpack(uint32_t w, [[maybe_unused]] const Zero<HALF>& zero) {
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
        // half bytes 0 and 4 (1 and 5) of v: a step of the float 1024 is 1, of 64 it is 1 / 16
        uint32_t low = 0x64006400u, high = 0x54005400u, low_bits = 0x000f000fu, high_bits = 0x00f000f0u;
        asm("" : "+v"(low), "+v"(high), "+s"(low_bits), "+s"(high_bits));   // in registers: the mask and the float in one instruction
        auto pair = [&](uint32_t v, bool is_high) {
            const f16x2 u = __builtin_bit_cast(f16x2, is_high ? (v & high_bits) | high : (v & low_bits) | low);
            if constexpr (HALF) {
                return __builtin_bit_cast(uint32_t, u - (is_high ? zero.high : zero.low));
            } else {
                // small integers: the upper halves of their floats are all of them
                const float off = is_high ? zero.high : zero.low, a = fmadd(float(u.x), 0.5f, off), b = fmadd(float(u.y), 0.5f, off);
                return uint32_t(__builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, a), 0x07060302u));
            }
        };
        f.word[0] = pair(w, false), f.word[1] = pair(w, true);
        f.word[2] = pair(w >> 8, false), f.word[3] = pair(w >> 8, true);
    }
    return f;
}

// Columns 0..7 in the order 0 4 1 5 2 6 3 7, for each 8 of a piece.
template <bool EIGHT>
__device__ __forceinline__ u32x4 mixed(u32x4 v) {
    constexpr uint32_t LO = EIGHT ? 0x05010400u : 0x05040100u, HI = EIGHT ? 0x07030602u : 0x07060302u;
    auto perm = [](uint32_t a, uint32_t b, uint32_t s) { return uint32_t(__builtin_amdgcn_perm(a, b, s)); };
    if constexpr (EIGHT) return u32x4{perm(v[1], v[0], LO), perm(v[1], v[0], HI), perm(v[3], v[2], LO), perm(v[3], v[2], HI)};
    else return u32x4{perm(v[2], v[0], LO), perm(v[2], v[0], HI), perm(v[3], v[1], LO), perm(v[3], v[1], HI)};
}

// `bytes` (of elements of ES bytes) of 16 at p, the others zero: of a row that is
// shorter than 16 bytes.
template <int ES>
__device__ __forceinline__ u32x4 load_short(const uint8_t* p, int bytes) {
    uint64_t lo = 0, hi = 0;
#pragma unroll 1
    for (int j = 0; j < bytes; j += ES) {
        uint64_t e = p[j];
        if constexpr (ES == 2) e |= uint64_t(p[j + 1]) << 8;
        if (j < 8) lo |= e << (8 * j);
        else hi |= e << (8 * j - 64);
    }
    return u32x4{uint32_t(lo), uint32_t(lo >> 32), uint32_t(hi), uint32_t(hi >> 32)};
}
// The last `bytes` of 16, moved to the front; zeros after them.
__device__ __forceinline__ u32x4 to_front(u32x4 v, int bytes) {
    const uint64_t lo = uint64_t(v[1]) << 32 | v[0], hi = uint64_t(v[3]) << 32 | v[2];
    const int cut = 8 * (16 - bytes);                           // 0..120 bits
    const uint64_t a = cut == 0 ? lo : cut < 64 ? lo >> cut | hi << (64 - cut) : hi >> (cut - 64);
    const uint64_t b = cut < 64 ? hi >> cut : 0;
    return u32x4{uint32_t(a), uint32_t(a >> 32), uint32_t(b), uint32_t(b >> 32)};
}

// What a lane loads of a chunk: 16 bytes of a row of W per 16 rows, and of x in
// PIECES loads, neighbouring lanes neighbouring columns.
template <X XT, int MT, int NB>
struct Held {
    static constexpr int BYTES = MT * kChunk * (is_eight(XT) ? 1 : 2), PIECES = (BYTES + 1023) / 1024;
    u32x4 codes[NB];
    u32x4 x[PIECES];
    uint32_t xscale[(MT + 15) / 16];   // bytes of the chunk's four blocks, of row lane % 16
};

// One element from the definition, in 64 bits, by a whole wavefront.
__device__ __forceinline__ double by_definition(const MatvecArgs& a, X xt, Format f, int group, int64_t m, int64_t n) {
    double sum = 0;
#pragma unroll 1
    for (int64_t k = threadIdx.x & 63; k < a.k; k += 64) {
        const uint32_t u = a.codes[n * a.ldc + k / 2] >> (4 * (k & 1)) & 15;
        const int64_t g = k / group;
        double w, x;
        if (f == Format::FLOAT) {
            const uint32_t c = u & 7;
            const float v = c < 2 ? 0.5f * float(c) : __builtin_bit_cast(float, (126 + (c >> 1)) << 23 | (c & 1) << 22);
            w = double(u & 8 ? -v : v) * double(power_of(static_cast<const uint8_t*>(a.scales)[n * a.lds + g]));
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
    if (xt == X::F8_ROW) sum *= double(static_cast<const float*>(a.xscales)[m]);
#pragma unroll
    for (int step = 1; step < 64; step *= 2) sum += __shfl_xor(sum, step);
    return sum;
}

// Scales and zero points of kGroups groups of TILE rows of W, in LDS as they lie
// in memory; rows are padded so that 16 of them spread over the banks.  A chunk
// has GROUPS groups.  Read from memory where they are used (two bytes of each of 16
// rows a time) they cost more than the codes: 1 x 28672 x 8192 took 56 us, and 29
// with no scales at all.
template <Format F, int GROUPS, int TILE>
struct Scales {
    static constexpr int SB = F == Format::FLOAT ? 1 : 2;       // bytes of a scale
    alignas(8) uint8_t scale[TILE][kGroups * SB + 4 * SB];
    alignas(4) uint8_t zero[F == Format::FLOAT ? 1 : TILE][kGroups + 4];

    // `count` groups from `first` on, of the rows from n0 on.  Groups that the last
    // chunk lacks get zeros; their products are zero.
    __device__ __forceinline__ void stage(const MatvecArgs& a, int64_t n0, int first, int count) {
        const int octets = ((count + GROUPS - 1) / GROUPS * GROUPS + 7) / 8;
        for (int e = threadIdx.x; e < octets * TILE; e += blockDim.x) {
            const int row = e / octets, at = e % octets * 8, left = count - at;
            const int64_t n = n0 + row < a.n ? n0 + row : a.n - 1;
            const uint8_t* p = static_cast<const uint8_t*>(a.scales) + (n * a.lds + first + at) * SB;
            const uint8_t* q = a.zeros + n * a.ldz + first + at;
            uint8_t s[8 * SB] = {};
            uint64_t z = 0x0808080808080808u;
            if (left >= 8) {
                __builtin_memcpy(s, p, 8 * SB);
                if (SB == 2 && a.zeros) __builtin_memcpy(&z, q, 8);
            } else {
#pragma unroll
                for (int j = 0; j < 7; ++j)
                    if (j < left) {
#pragma unroll
                        for (int i = 0; i < SB; ++i) s[j * SB + i] = p[j * SB + i];
                        if (SB == 2 && a.zeros) z = (z & ~(0xffull << (8 * j))) | uint64_t(q[j]) << (8 * j);
                    }
            }
            // the padding takes what a row's last octet has over
#pragma unroll
            for (int i = 0; i < SB; ++i) __builtin_memcpy(&scale[row][at * SB + 8 * i], s + 8 * i, 8);
            if constexpr (SB == 2) {
                __builtin_memcpy(&zero[row][at], &z, 4);
                __builtin_memcpy(&zero[row][at + 4], reinterpret_cast<const uint8_t*>(&z) + 4, 4);
            }
        }
    }

    // Those of a row's groups from `group` on, a multiple of GROUPS.
    __device__ __forceinline__ void get(int row, int group, float (&s)[GROUPS], uint32_t (&z)[GROUPS]) const {
        uint64_t v = 0;
        __builtin_memcpy(&v, __builtin_assume_aligned(&scale[row][group * SB], GROUPS * SB), GROUPS * SB);
        uint32_t w = 0;
        if constexpr (SB == 2) __builtin_memcpy(&w, __builtin_assume_aligned(&zero[row][group], GROUPS), GROUPS);
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) {
            if constexpr (SB == 2) {
                const uint32_t half = uint32_t(v >> (32 * (i / 2)));
                s[i] = __builtin_bit_cast(float, i & 1 ? half & 0xffff0000u : half << 16);
                z[i] = w >> (8 * i) & 255u;
            } else {
                // 2^128, infinity, for a byte of 255: the sum is then not finite, and NaN by the definition
                s[i] = __builtin_amdgcn_ldexpf(1.0f, int(uint32_t(v) >> (8 * i) & 255u) - 127);
                z[i] = 0;
            }
        }
    }
};

// Joins the wavefronts' sums (slot of four rows by lane), times `unit` and the scale
// of x's row if there is one, and stores the tile's y.
template <Format F, int GROUP, int MB, int NB>
__device__ __forceinline__ void store_sums(const MatvecArgs& a, X xt, Type yt, int64_t m0, int64_t n0, int rows_m, int rows_n,
                                           int waves, const float (*sums)[MB * NB * 4][64], float unit, const float* row_scale) {
    constexpr int TILE = 16 * NB;
    const int lane = threadIdx.x & 63;
    // whole wavefronts: the detour below takes all lanes
    for (int e0 = threadIdx.x & ~63; e0 < rows_m * TILE; e0 += blockDim.x) {
        const int e = e0 + lane, ml = e / TILE, nl = e % TILE;  // y's row and column in the tile
        const int64_t m = m0 + ml, n = n0 + nl;
        const bool in = ml < rows_m && nl < rows_n;
        const int slot = (ml / 16 * NB + nl / 16) * 4 + ml % 4, from = ml % 16 / 4 * 16 + nl % 16;
        float v = 0;
        if (in) {
            for (int w = 0; w < waves; ++w) v += sums[w][slot][from];
            v *= unit;
            if (row_scale) v *= row_scale[m];
        }
        for (uint64_t odd = __ballot(magnitude(v) >= kInfBits); odd; odd &= odd - 1) {
            const int at = __builtin_ctzll(odd);
            const double d = by_definition(a, xt, F, GROUP, m0 + (e0 + at) / TILE, n0 + (e0 + at) % TILE);
            if (lane == at) v = float(d);
        }
        if (!in) continue;
        const int64_t to = m * a.ldy + n;
        if (yt == Type::F32) static_cast<float*>(a.y)[to] = v;
        else if (yt == Type::F16) static_cast<f16*>(a.y)[to] = f16(v);
        else static_cast<bf16*>(a.y)[to] = bf16(v);
    }
}

template <X XT, Format F, int GROUP, int MT, int NB, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void weight_matvec_kernel(MatvecArgs a, Type yt) {
    constexpr bool EIGHT = is_eight(XT);
    // Integers come apart with half as much work in half precision, which holds block-scaled
    // x exactly where its scales are within 2^-15 to 1.  A chunk of such x is multiplied
    // there: 1 x 28672 x 8192 in groups of 64 31.8 us, 36.0 in bfloat16; 16 x 16384 x 4096
    // 11.7 and 12.6.  For x in bfloat16 the search for its range takes half of the gain (1 x
    // 16384 x 8192 in groups of 128 15.6 and 16.5, 1 x 4096 x 14336 9.5 and 9.2): not done.
    constexpr bool EITHER = F == Format::INTEGER && XT == X::F8_BLOCK;
    constexpr int MB = (MT + 15) / 16;                          // tiles of 16 rows of x, the last partly empty
    constexpr int GROUPS = kChunk / GROUP, STEPS = GROUP / 32;  // groups of a chunk, products of a group
    constexpr int TILE = 16 * NB;                               // rows of W
    constexpr int ES = EIGHT ? 1 : 2, ROW = kChunk * ES;        // bytes of an element and a chunk's row of x
    constexpr int SLOTS = ROW / 16;                             // of 16 bytes
    using H = Held<XT, MT, NB>;
    constexpr bool MIXED = F == Format::INTEGER;                // x as the codes come apart, on its way into LDS
    constexpr int SUMS = MT < 4 ? MT : 4;                       // of a lane's four sums, those of rows of x
    __shared__ Scales<F, GROUPS, TILE> scales;                  // of the groups at hand
    __shared__ union {
        struct { u32x4 codes[NB * 64]; u32x4 x[MT * SLOTS]; } of[WAVES];
        float sums[WAVES][MB * NB * 4][64];
    } lds;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6, r = lane & 15, g = lane >> 4;
    const int64_t n0 = int64_t(blockIdx.x) * TILE, m0 = int64_t(blockIdx.y) * MT;
    const int chunks = int((a.k + kChunk - 1) / kChunk), whole = int(a.k / kChunk);
    const int groups = int((a.k + GROUP - 1) / GROUP);
    const int rows_n = a.n - n0 < TILE ? int(a.n - n0) : TILE, rows_m = a.m - m0 < MT ? int(a.m - m0) : MT;

    // Loads a chunk that lies inside the row.  Codes: lane / 4 is the row, lane % 4
    // the 16 bytes of it, so that a load takes whole lines; the transposition to the
    // matrix cores' layout goes through LDS (16 x 8192 x 8192 took 11 us then, 14 with loads in
    // that layout and the swaps of lanes).  x: 64 / PER rows a load, PER lanes a row.
    // Rows past the end are not read: their results are not stored.  One chunk ahead:
    // two and four took 9.0 and 9.5 us for 1 x 16384 x 4096 when one took 8.0 (the
    // wavefronts of a compute unit are enough loads on their way, and registers fewer).
    constexpr int PER = ROW / 16, STEP = 64 / PER;
    const uint32_t code_at = uint32_t(lane >> 2) * uint32_t(a.ldc) + 16 * (lane & 3);
    const uint32_t x_at = uint32_t(lane / PER) * uint32_t(a.ldx * ES) + 16 * (lane % PER);
    const uint8_t* const codes0 = a.codes + n0 * a.ldc;
    const uint8_t* const x0 = static_cast<const uint8_t*>(a.x) + m0 * a.ldx * ES;
    const int64_t codes_step = 16 * a.ldc, x_step = STEP * a.ldx * ES;
    auto load = [&](int c, H& d) {
        const uint8_t* codes = codes0 + int64_t(c) * (kChunk / 2);
#pragma unroll
        for (int i = 0; i < NB; ++i, codes += codes_step)
            if (16 * i + (lane >> 2) < rows_n) d.codes[i] = *reinterpret_cast<const u32x4*>(codes + code_at);
        const uint8_t* x = x0 + int64_t(c) * ROW;
#pragma unroll
        for (int q = 0; q < H::PIECES; ++q, x += x_step)
            if (STEP * q + lane / PER < rows_m) __builtin_memcpy(&d.x[q], x + x_at, 16);
        if constexpr (XT == X::F8_BLOCK) {
#pragma unroll
            for (int i = 0; i < MB; ++i)
                if (16 * i + r < rows_m)
                    __builtin_memcpy(&d.xscale[i], static_cast<const uint8_t*>(a.xscales) + (m0 + 16 * i + r) * a.ldxs + c * 4, 4);
        }
    };

    // Loads the last chunk, which ends inside: what is past the row's end is zero.
    const int left = int(a.k - int64_t(whole) * kChunk);        // columns of it
    auto load_partial = [&](H& d) {
        const uint8_t* codes = codes0 + int64_t(whole) * (kChunk / 2);
#pragma unroll
        for (int i = 0; i < NB; ++i, codes += codes_step) {
            d.codes[i] = u32x4{0, 0, 0, 0};
            if (16 * i + (lane >> 2) < rows_n && 16 * (lane & 3) < (left + 1) / 2)
                d.codes[i] = *reinterpret_cast<const u32x4*>(codes + code_at);
        }
        const uint8_t* x = x0 + int64_t(whole) * ROW;
        // of this lane's piece: a load of the 16 bytes that end with the row, if it has so many
        const int left_here = left * ES - 16 * (lane % PER), bytes = left_here < 16 ? left_here : 16;
        const bool is_long = a.k * ES >= 16;
#pragma unroll
        for (int q = 0; q < H::PIECES; ++q) {
            d.x[q] = u32x4{0, 0, 0, 0};
            if (STEP * q + lane / PER < rows_m && bytes > 0) {
                if (is_long) __builtin_memcpy(&d.x[q], x + q * x_step + x_at + bytes - 16, 16);
                else d.x[q] = load_short<ES>(x + q * x_step + x_at, bytes);
            }
        }
        if (is_long && bytes > 0) {
#pragma unroll
            for (int q = 0; q < H::PIECES; ++q) d.x[q] = to_front(d.x[q], bytes);
        }
        if constexpr (XT == X::F8_BLOCK) {
#pragma unroll
            for (int i = 0; i < MB; ++i) {
                d.xscale[i] = 0x7f7f7f7fu;
                if (16 * i + r >= rows_m) continue;
                const uint8_t* p = static_cast<const uint8_t*>(a.xscales) + (m0 + 16 * i + r) * a.ldxs + whole * 4;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j * kScaleBlock < left) d.xscale[i] = (d.xscale[i] & ~(255u << (8 * j))) | uint32_t(p[j]) << (8 * j);
            }
        }
    };

    // Into this wavefront's LDS.  The 16-byte slots of a row are permuted by the
    // row, so that the reads below (16 rows at a time) spread over all banks.
    auto& own = lds.of[wave];
    auto put_codes = [&](const H& d) {
#pragma unroll
        for (int i = 0; i < NB; ++i) own.codes[64 * i + (lane & ~3) + ((lane & 3) ^ (lane >> 4))] = d.codes[i];
    };
    auto mix = [](int row) { return SLOTS < 16 ? row >> 1 & 7 : MT <= 4 ? 4 * row : row & 15; };
    auto put_x = [&](const H& d) {
#pragma unroll
        for (int q = 0; q < H::PIECES; ++q) {
            const int row = STEP * q + lane / PER;
            if (H::BYTES >= 1024 || row < MT) own.x[row * SLOTS + (lane % PER ^ mix(row))] = MIXED ? mixed<EIGHT>(d.x[q]) : d.x[q];
        }
    };
    // Whether half precision holds the chunk's block-scaled x: scale bytes 112 to 127, for
    // e4m3 values, multiples of 2^-9, become multiples of its smallest step 2^-24.
    auto fits = [&](const H& d) {
        bool bad = false;
#pragma unroll
        for (int i = 0; i < MB; ++i) bad = bad || (16 * i + r < rows_m && (d.xscale[i] & 0xf0f0f0f0u) != 0x70707070u);
        return !__any(bad);
    };
    // Codes of product t for row lane % 16 of W: dword 4 t + lane / 16 of the row.
    auto get_codes = [&](int i, int t) {
        return reinterpret_cast<const uint32_t*>(&own.codes[64 * i + 4 * r + (t ^ (r >> 2))])[g];
    };
    // Columns 32 t + 8 g of row lane % 16 of x.
    auto get_x = [&](auto half, int i, int t, [[maybe_unused]] uint32_t scale) {
        constexpr bool HALF = decltype(half)::value;
        const int row = 16 * i + (MT < 16 ? r % MT : r), byte = (32 * t + 8 * g) * ES;
        const uint32_t* p = reinterpret_cast<const uint32_t*>(&own.x[row * SLOTS + (byte / 16 ^ mix(row))]);
        if constexpr (EIGHT) {
            const uint2 v = reinterpret_cast<const uint2*>(p)[g & 1];
            return from_e4m3<HALF>(v.x, v.y, XT != X::F8_BLOCK ? 1.0f : HALF ? power_of(scale >> (8 * t) & 255u) : block_power(scale >> (8 * t) & 255u));
        } else {
            return *reinterpret_cast<const Frag*>(p);
        }
    };

    f32x4 acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    // Multiplies the chunk that is in LDS; `group`: its first group, of those staged.
    auto products = [&](auto half, const uint32_t (&xscale)[MB], int group) {
        constexpr bool HALF = decltype(half)::value;
        float scale[NB][GROUPS];
        uint32_t zero[NB][GROUPS];
#pragma unroll
        for (int j = 0; j < NB; ++j) scales.get(16 * j + r, group, scale[j], zero[j]);
#pragma unroll
        for (int s = 0; s < GROUPS; ++s) {
            f32x4 part[MB][NB];
#pragma unroll
            for (int i = 0; i < MB; ++i)
#pragma unroll
                for (int j = 0; j < NB; ++j) part[i][j] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int q = 0; q < STEPS; ++q) {
                const int t = s * STEPS + q;
                Frag x[MB];
#pragma unroll
                for (int i = 0; i < MB; ++i) x[i] = get_x(half, i, t, xscale[i]);
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    const Frag w = unpack<HALF, F>(get_codes(j, t), Zero<HALF>(zero[j][s]));
#pragma unroll
                    for (int i = 0; i < MB; ++i) part[i][j] = product<HALF>(x[i], w, part[i][j]);
                }
            }
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                if constexpr (EITHER) scale[j][s] *= HALF ? 1.0f : kUnit<XT, F>;
#pragma unroll
                for (int i = 0; i < MB; ++i)
#pragma unroll
                    for (int e = 0; e < SUMS; ++e) acc[i][j][e] = fmadd(scale[j][s], part[i][j][e], acc[i][j][e]);
            }
        }
    };
    // The same for the chunk that is held, and loads chunk `next` if it is before `full`.
    auto multiply = [&](H& d, int group, int next, int full) {
        [[maybe_unused]] const bool half = EITHER && fits(d);
        wave_lds_sync();                                        // the last chunk has been read
        put_codes(d);
        put_x(d);
        uint32_t xscale[MB];
#pragma unroll
        for (int i = 0; i < MB; ++i) xscale[i] = XT == X::F8_BLOCK ? d.xscale[i] : 0;
        if (next < full) load(next, d);
        wave_lds_sync();
        if constexpr (EITHER) {
            if (half) return products(std::true_type{}, xscale, group);
        }
        products(std::bool_constant<in_half(XT)>{}, xscale, group);
    };

    constexpr int PHASE = kGroups / GROUPS;                     // chunks whose scales fit
    H held = {};
    for (int base = 0; base < chunks; base += PHASE) {
        const int end = base + PHASE < chunks ? base + PHASE : chunks;
        const int full = end < whole ? end : whole;             // of them, those that lie inside the row
        int c = base + wave;
        if (c < full) load(c, held);                            // on its way while the scales are staged
        const int g0 = base * GROUPS;
        if (base) __syncthreads();
        scales.stage(a, n0, g0, end * GROUPS < groups ? end * GROUPS - g0 : groups - g0);
        __syncthreads();
        for (; c < end; c += waves) {
            if (c >= whole) load_partial(held);
            multiply(held, (c - base) * GROUPS, c + waves, full);
        }
    }

    __syncthreads();                                            // the chunks' LDS is free
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int e = 0; e < SUMS; ++e) lds.sums[wave][(i * NB + j) * 4 + e][lane] = acc[i][j][e];
    __syncthreads();

    store_sums<F, GROUP, MB, NB>(a, XT, yt, m0, n0, rows_m, rows_n, waves, &lds.sums[0], EITHER ? 1.0f : kUnit<XT, F>,
                                XT == X::F8_ROW ? static_cast<const float*>(a.xscales) : nullptr);
}

template <X XT>
inline hipError_t weight_matvec_t(Type yt, Format f, int group, const MatvecArgs& a, hipStream_t s) {
    const int64_t chunks = (a.k + kChunk - 1) / kChunk;
    auto tile = [&](auto fmt, auto size, auto mt, auto nb, auto waves) {
        constexpr int MT = decltype(mt)::value, NB = decltype(nb)::value, WAVES = decltype(waves)::value;
        const dim3 block(uint32_t(64 * (chunks < WAVES ? chunks : WAVES)));
        const dim3 grid(uint32_t((a.n + 16 * NB - 1) / (16 * NB)), uint32_t((a.m + MT - 1) / MT));
        // One row, 32 rows of W: LDS that is not used keeps a compute unit at two workgroups.
        // A third one takes 1 x 28672 x 8192 in half precision and groups of 64 from 29.3 to
        // 32.2 us and 32768 rows of W from 32.9 to 35.3; 20480 of them gain (20.0 to 19.1).
        constexpr size_t unused = decltype(fmt)::value == Format::INTEGER && MT == 1 && NB == 2 ? 16384 : 0;
        return launch(weight_matvec_kernel<XT, decltype(fmt)::value, decltype(size)::value, MT, NB, WAVES>, grid, block, unused,
                      s, a, yt);
    };
    constexpr int FEW = is_eight(XT) ? 8 : 4;                   // rows that one load holds
    auto shape = [&](auto fmt, auto size) {
        // 32 rows of W to a workgroup where that leaves one for every compute unit, since x
        // and its fragments then serve twice (16 x 8192 x 8192 12.5 us, 13.8 with 16; 1 x
        // 28672 x 8192 30.0 and 32.5).  Where 16 rows leave one workgroup or none for a
        // compute unit, its wavefronts are twice as many (4 x 4096 x 14336 10.0 us, 11.7
        // with 8; at 4096 columns the call's overhead hides both).
        const bool wide = a.n >= 256 * 32;
        auto rows = [&](auto mt) {
            if (wide) return tile(fmt, size, mt, ic<2>{}, ic<8>{});
            if (a.n <= 256 * 16) return tile(fmt, size, mt, ic<1>{}, ic<16>{});
            return tile(fmt, size, mt, ic<1>{}, ic<8>{});
        };
        // The matrix cores take 16 rows of x in any case; loading, holding and joining
        // those that are there: 1 x 28672 x 8192 29.1 us (30.2 as 4 rows, 31.8 as 16), 4 x
        // 4096 x 14336 10.0 (12.2 as 16).
        return a.m == 1 ? rows(ic<1>{}) : a.m <= FEW ? rows(ic<FEW>{}) : rows(ic<16>{});
    };
    if (f == Format::FLOAT) return shape(std::integral_constant<Format, Format::FLOAT>{}, ic<32>{});
    using I = std::integral_constant<Format, Format::INTEGER>;
    return group == 32 ? shape(I{}, ic<32>{}) : group == 64 ? shape(I{}, ic<64>{}) : shape(I{}, ic<128>{});
}

}  // namespace weight_matvec_detail
}  // namespace bl
