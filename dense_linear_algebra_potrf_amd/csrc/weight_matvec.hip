// Products of a few rows with 4-bit weights, y = x W^T.
//
// One wavefront per row of W: each lane takes 8 columns (a dword of codes) at
// a time, unpacks them to floats once and multiplies them with up to 8 rows of
// x; the lanes' sums are joined by a butterfly.
#include "layer_impl.hpp"

namespace bl {
namespace weight_matvec_detail {

using namespace layer;

constexpr int kRows = 8;

__device__ __forceinline__ float e4m3_value(uint32_t b) {
    return __builtin_amdgcn_cvt_f32_fp8(int(b), 0);
}

__device__ __forceinline__ float e2m1_value(uint32_t code) {
    const uint32_t c = code & 7;
    const float v = c < 2 ? 0.5f * float(c) : __builtin_bit_cast(float, (126 + (c >> 1)) << 23 | (c & 1) << 22);
    return code & 8 ? -v : v;
}

__device__ __forceinline__ float element(const MatvecArgs& a, Type xt, Scale xs, int64_t m, int64_t k) {
    if (xt == Type::BF16) return float(static_cast<const bf16*>(a.x)[m * a.ldx + k]);
    if (xt == Type::F16) return float(static_cast<const f16*>(a.x)[m * a.ldx + k]);
    const float v = e4m3_value(static_cast<const uint8_t*>(a.x)[m * a.ldx + k]);
    if (xs == Scale::ROW) return v;                     // the row's scale at the end
    return v * power_of(static_cast<const uint8_t*>(a.xscales)[m * a.ldxs + k / kScaleBlock]);
}

__global__ __launch_bounds__(256) void weight_matvec_kernel(MatvecArgs a, Type xt, Scale xs, Type yt, Format f,
                                                            int group) {
    const int lane = threadIdx.x & 63;
    const int64_t n = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (n >= a.n) return;
    const int64_t m0 = int64_t(blockIdx.y) * kRows;
    double sum[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) sum[i] = 0;
    for (int64_t k = lane * 8; k < a.k; k += 512) {
        const uint32_t codes = *reinterpret_cast<const uint32_t*>(a.codes + n * a.ldc + k / 2);
        const int64_t g = k / group;
        const float z = f == Format::FLOAT ? 0.0f : a.zeros ? float(a.zeros[n * a.ldz + g]) : 8.0f;
        const float scale = f == Format::FLOAT ? power_of(static_cast<const uint8_t*>(a.scales)[n * a.lds + g])
                                               : float(static_cast<const bf16*>(a.scales)[n * a.lds + g]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t u = codes >> (4 * j) & 15;
            // in 64 bits: a code times its scale, or x times a code, may leave the
            // range of 32 bits where the whole product does not
            const double w = double(f == Format::FLOAT ? e2m1_value(u) : float(u) - z) * double(scale);
            if (k + j < a.k) {
#pragma unroll
                for (int i = 0; i < kRows; ++i)
                    if (m0 + i < a.m) sum[i] = fmadd(w, double(element(a, xt, xs, m0 + i, k + j)), sum[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        double all = sum[i];
#pragma unroll
        for (int step = 1; step < 64; step *= 2) all += __shfl_xor(all, step);
        float v = float(all);
        if (lane != 0 || m0 + i >= a.m) continue;
        if (xs == Scale::ROW) v = float(all * double(static_cast<const float*>(a.xscales)[m0 + i]));
        const int64_t at = (m0 + i) * a.ldy + n;
        if (yt == Type::F32) static_cast<float*>(a.y)[at] = v;
        else if (yt == Type::F16) static_cast<f16*>(a.y)[at] = f16(v);
        else static_cast<bf16*>(a.y)[at] = bf16(v);
    }
}

}  // namespace weight_matvec_detail

hipError_t weight_matvec(Type xt, Scale xs, Type yt, Format f, int group, const MatvecArgs& a, hipStream_t s) {
    using namespace weight_matvec_detail;
    const dim3 grid(uint32_t((a.n + 3) / 4), uint32_t((a.m + kRows - 1) / kRows));
    return launch(weight_matvec_kernel, grid, dim3(256), 0, s, a, xt, xs, yt, f, group);
}

}  // namespace bl
