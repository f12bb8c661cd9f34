// Device helpers shared by the 8-bit-integer layer operators (gfx950).
#pragma once

#include "integer.hpp"
#include "layer_impl.hpp"

namespace bl {
namespace layer {

// Eight elements from column c on of a row of n, in two parts: fetch() is one load of all
// lanes without a branch, so that many may be on their way; settle(), where they are used,
// puts them right in the lanes at the row's end.  Those load the row's last eight, which
// settle() moves to the front, with zeros after them (only zeros past the end); what they
// load of a neighbour's elements is dropped, so that the neighbour may have stored over it.
template <typename T>
__device__ __forceinline__ Raw8<T> fetch(const T* row, int c, int n) {
    if (n < 8) return load8(row + c, n - c);
    Raw8<T> r;
    __builtin_memcpy(&r, row + (c < n - 8 ? c : n - 8), sizeof(r));
    return r;
}
template <typename T>
__device__ __forceinline__ void settle(Raw8<T>& r, int c, int n) {
    const int by = c + 8 - n;                                   // elements to move by
    if (by <= 0 || n < 8) return;
    constexpr int WORDS = 2 * sizeof(T);
    auto words = [&](int by_words) {                            // a constant
#pragma unroll
        for (int i = 0; i < WORDS; ++i) r.word[i] = i + by_words < WORDS ? r.word[i + by_words] : 0;
    };
    if (by & 4) words(int(sizeof(T)));
    if (by & 2) words(int(sizeof(T)) / 2);
    if (by & 1) {
        if constexpr (sizeof(T) == 4) {
            words(1);
        } else {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) r.word[i] = __builtin_amdgcn_alignbit(i + 1 < WORDS ? r.word[i + 1] : 0, r.word[i], 16);
        }
    }
    if (by >= 8) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) r.word[i] = 0;
    }
}

constexpr float kCodeMax = 127.0f;

// The scale of a row from the bits of its largest magnitude: NaN where that is not finite.
__device__ __forceinline__ float code_scale(uint32_t top) {
    return top >= kInfBits ? __builtin_nanf("") : fmaxf(__builtin_bit_cast(float, top) / kCodeMax, kTiny);
}

// Codes of eight values under a normal positive scale s, rint(v / s) of the exact
// quotient, within -127..127; and codes as floats, for what they stand for.
//
// t = v (1 / s) is within a few ulp of the quotient, so rint(t) is wrong only next to
// a half.  There the remainder v - q s is exact in 32 bits (it is at most about s / 2
// and a multiple of half an ulp of s), and twice of it against s says on which side
// of the half the quotient is; on it, the even code is taken.  t is rounded by adding
// 3 2^22, which leaves the code in the lowest byte.
struct Codes {
    uint32_t word[2];
};
__device__ __forceinline__ Codes to_codes(const float (&v)[8], float s, float inverse, float (&q)[8]) {
    constexpr float kRound = 12582912.0f;
    float t[8], far = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        t[j] = fminf(fmaxf(v[j] * inverse, -kCodeMax), kCodeMax);
        q[j] = (t[j] + kRound) - kRound;
        far = fmaxf(far, fabsf(t[j] - q[j]));
    }
    if (far > 0.4999f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float d = 2 * fmadd(-q[j], s, v[j]);
            const bool odd = __builtin_bit_cast(uint32_t, q[j] + kRound) & 1;
            if (fabsf(d) > s || (fabsf(d) == s && odd)) q[j] += d > 0 ? 1.0f : -1.0f;
            q[j] = fminf(fmaxf(q[j], -kCodeMax), kCodeMax);
        }
    }
    uint32_t b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j] = __builtin_bit_cast(uint32_t, q[j] + kRound);
    auto four = [](uint32_t b0, uint32_t b1, uint32_t b2, uint32_t b3) {
        const uint32_t lo = __builtin_amdgcn_perm(b1, b0, 0x0c0c0400u), hi = __builtin_amdgcn_perm(b3, b2, 0x04000c0cu);
        return lo | hi;
    };
    return Codes{{four(b[0], b[1], b[2], b[3]), four(b[4], b[5], b[6], b[7])}};
}

// `count` of 8 codes; p is aligned to 8 bytes.
__device__ __forceinline__ void store_codes(int8_t* p, const Codes& c, int count) {
    if (count >= 8) {
        *reinterpret_cast<uint2*>(p) = uint2{c.word[0], c.word[1]};
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < count) p[i] = int8_t(c.word[i / 4] >> (8 * (i % 4)));
    }
}

// Stores past the caches, for what a launch writes once.  Whoever reads it next finds it in
// the last level either way: 1024 rows of 4096 in bf16 normed and their outputs
// multiplied take 16.2 us, with plain stores 19.2; 16384 rows 162 and 185.
template <typename T, int COUNT>
__device__ __forceinline__ void store_past(T* p, const T (&v)[COUNT]) {
    static_assert(sizeof(v) % 16 == 0);
    using Words = uint32_t __attribute__((ext_vector_type(4)));
    struct __attribute__((packed)) Place {
        Words w;
    };
    Words w[sizeof(v) / 16];
    __builtin_memcpy(w, v, sizeof(v));
#pragma unroll
    for (int i = 0; i < int(sizeof(v) / 16); ++i) __builtin_nontemporal_store(w[i], &(reinterpret_cast<Place*>(p) + i)->w);
}
template <typename T>
__device__ __forceinline__ void store8_past(T* p, const float (&f)[8], int count) {
    if (count < 8) return store8(p, f, count);
    T v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = T(f[i]);
    store_past(p, v);
}

}  // namespace layer
}  // namespace bl
