// What the norms share: a row's threads, its root, and the shape by its width.
#pragma once

#include "layer_impl.hpp"

namespace bl {
namespace rmsnorm_detail {

using namespace layer;

template <int TPR> struct Shape {
    static constexpr int threads = TPR < 256 ? 256 : TPR;     // of several rows, if a row has fewer
    static constexpr int rows = threads / TPR;
    static constexpr int waves = TPR < 64 ? 1 : TPR / 64;     // a row's
    // Which of the workgroup's rows a thread has, the same for a wavefront where it is:
    // a row's address is then scalar.
    static __device__ __forceinline__ int slot() {
        if constexpr (rows == 1) return 0;
        else if constexpr (TPR == 64) return __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
        else return threadIdx.x / TPR;
    }
};

// Squares leave the range of 32 bits where the row itself does not.  Outside
// this range of mean(h^2) + eps (inside it, what underflowed does not count) the
// sum is taken again of h times a power of two that brings the largest to about
// 1.  The branch is the same for all threads of a row.
__device__ __forceinline__ bool mean_in_range(float mean) { return mean > 0x1p-90f && mean < 0x1p90f; }
// That power of two, f, for a row whose largest magnitude has the bits `top`; 1 for a row that
// is not finite.  It brings the larger of that and sqrt(eps) to 1..2, so that eps f^2 stays
// below 4 whatever eps is, and the mean, then eps f^2 + mean((h f)^2), above 1 / n: squares
// that underflow beside such an eps do not count.
__device__ __forceinline__ float rescale(uint32_t top, float eps) {
    if (top >= kInfBits) return 1.0f;
    const uint32_t most = Max{}(top, __builtin_bit_cast(uint32_t, __builtin_amdgcn_sqrtf(eps)));
    const int e = 127 - int(most >> 23);           // -127..127, kept where f is normal; rows of zeros without eps: 100
    return __builtin_bit_cast(float, uint32_t((e < -126 ? -126 : e < 100 ? e : 100) + 127) << 23);
}

// 1 / sqrt(mean): the instruction's result (an ulp off) and a step of Newton's method
// with the products' own roundings, within half an ulp and a little; 0 and infinity,
// for which the step is not a number, stay.
__device__ __forceinline__ float inverse_root(float mean) {
    const float y = __builtin_amdgcn_rsqf(mean);
    const float t = mean * y, low = fmadd(mean, y, -t);
    const float better = fmadd(0.5f * y, fmadd(-low, y, fmadd(-t, y, 1.0f)), y);
    return better == better ? better : y;
}

// Calls f with the shape that holds a row of n columns: up to 1024 a wavefront or
// a part of it (no barrier), then 256 or 512 threads.  Lanes without columns hold
// registers and load nothing, hence the steps between.  bf16 with a residual, 16 M
// elements, in us:
//     128 columns   16 lanes 28.2, 64 lanes 66.3     256   32 lanes 27.4, 64: 38.4
//     1024          64 lanes 27.4, 256: 32.6         512   64 lanes 27.4, 256: 51.6
//     5120, 9001, 12288   3 vectors a thread 30.9, 35.5, 29.9, 4: 33.2, 43.3, 33.5
template <typename F>
inline hipError_t with_shape(int64_t n, F&& f) {
    const int64_t v = (n + 7) / 8;
    if (v <= 16) return f(ic<16>{}, ic<1>{});
    if (v <= 32) return f(ic<32>{}, ic<1>{});
    if (v <= 64) return f(ic<64>{}, ic<1>{});
    if (v <= 128) return f(ic<64>{}, ic<2>{});
    if (v <= 256) return f(ic<256>{}, ic<1>{});
    if (v <= 512) return f(ic<256>{}, ic<2>{});
    if (v <= 768) return f(ic<256>{}, ic<3>{});
    if (v <= 1024) return f(ic<256>{}, ic<4>{});
    if (v <= 1536) return f(ic<512>{}, ic<3>{});
    if (v <= 2048) return f(ic<512>{}, ic<4>{});
    return f(ic<512>{}, ic<8>{});
}

}  // namespace rmsnorm_detail
}  // namespace bl
