// Root-mean-square norm with the residual's addition and an output in 8 bits,
// and its gradient.
//
//     h = x + r,  s = 1 / sqrt(mean(h^2) + eps),  v = h s w,  q = e4m3(v / scale)
//
// A row is read once: it stays in the registers of the TPR threads that share
// it (VPT vectors of 8 elements each, vector i of thread t at column
// 8 (i TPR + t)) from the load through the sum of squares to the stores.  A
// block of 32 columns is then held by 4 neighbouring lanes, so its largest
// magnitude takes two quad permutes.
//
// HBM bounds it: 2 + 2 + 2 + 1 bytes an element in 16 bits with a residual.
// 8192 x 8192 bf16, residual, block scales: 97 us in calls back to back, 97 to 107
// (102 on average, 4.6 TB/s) in a profile; a large copy reaches 5.1.  A single row of
// 4096 takes 7.7 us a call, of which the kernel, 3.6, is less than the launch.  Loading a row ahead in a grid of 1280 workgroups
// took 102 us at that size (registers for half as many wavefronts), 3 to 7%
// less below 1024 columns: not done.
#pragma once

#include "norm_impl.hpp"

namespace bl {
namespace rmsnorm_detail {

using namespace layer;

template <typename T, int TPR, int VPT, bool BLOCK>
__global__ __launch_bounds__(Shape<TPR>::threads) void rmsnorm_quant_kernel(NormQuantArgs a) {
    using S = Shape<TPR>;
    __shared__ float sums[2][S::waves];
    __shared__ uint32_t tops[2][S::waves];
    const int t = threadIdx.x % TPR;
    const int n = int(a.n);
    const T* w = static_cast<const T*>(a.w);
    for (int64_t row = int64_t(blockIdx.x) * S::rows + threadIdx.x / TPR; row < a.rows;
         row += int64_t(gridDim.x) * S::rows) {
        const T* x = static_cast<const T*>(a.x) + row * a.ldx;
        float v[VPT][8];
        float sum = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 8 * (i * TPR + t), left = n - c;
            const Raw8<T> xr = load8(x + c, left);
            if (a.r) {
                const Raw8<T> rr = load8(static_cast<const T*>(a.r) + row * a.ldr + c, left);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = xr[j] + rr[j];
                if (a.h) store8(static_cast<T*>(a.h) + row * a.ldh + c, v[i], left);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = xr[j];
            }
            float square = 0;                                   // short chains: small errors
#pragma unroll
            for (int j = 0; j < 8; ++j) square = fmadd(v[i][j], v[i][j], square);
            sum += square;
        }
        sum = block_reduce<TPR>(sum, Add{}, sums[0]);
        float mean = sum / float(n) + a.eps;
        if (!mean_in_range(mean)) {
            uint32_t most = 0;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) most = Max{}(most, magnitude(v[i][j]));
            const float f = rescale(block_reduce<TPR>(most, Max{}, tops[0]), a.eps);
            sum = 0;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[i][j] *= f;
                    sum = fmadd(v[i][j], v[i][j], sum);
                }
            mean = block_reduce<TPR>(sum, Add{}, sums[1]) / float(n) + a.eps * f * f;
        }
        const float rs = inverse_root(mean);
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 8 * (i * TPR + t), left = n - c;
            const Raw8<T> wr = load8(w + c, left);
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // h rs w rounded once: an output next to a tie of its 8 bits should fall on
                // the definition's side
                const float u = v[i][j] * rs, low = fmadd(v[i][j], rs, -u), wj = wr[j];
                v[i][j] = fmadd(u, wj, low * wj);
                // elements past the row's end are not part of it (0 * inf is not 0)
                m = Max{}(m, j < left ? magnitude(v[i][j]) : 0u);
            }
            if constexpr (BLOCK) {
                const uint32_t b = e4m3_scale_byte(row_reduce<4>(m, Max{}));
                if ((t & 3) == 0 && left > 0)
                    static_cast<uint8_t*>(a.scales)[row * a.lds + c / kScaleBlock] = uint8_t(b);
                store_e4m3(a.q + row * a.ldq + c, v[i], power_of(b == 255 ? 255 : 254 - b), left);
            } else {
                top = Max{}(top, m);
            }
        }
        if constexpr (!BLOCK) {
            top = block_reduce<TPR>(top, Max{}, tops[1]);
            const float big = __builtin_bit_cast(float, top);
            const float scale = top >= kInfBits ? __builtin_nanf("") : fmaxf(big / kE4M3Max, kTiny);
            if (t == 0) static_cast<float*>(a.scales)[row] = scale;
            const float inverse = top >= kInfBits ? scale : fminf(kE4M3Max / big, 0x1p126f);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = 8 * (i * TPR + t);
                store_e4m3(a.q + row * a.ldq + c, v[i], inverse, n - c);
            }
        }
        if constexpr (S::waves > 1) __syncthreads();   // the next row's sums
    }
}

// The gradient, with g = dy w and the residual's own dh:
//     dx = s (g - h s^2 mean(g h)) + dh,   dw = sum over rows of dy h s.
// Each workgroup takes rows blockIdx, blockIdx + grid, ... and keeps its sum of
// dw in registers over them, joined over its rows in LDS (16384 x 1024 bf16: 30 us,
// 39 with a sum per row of the workgroup); the sums of the workgroups go to
// `partial` and are added in a fixed order by rmsnorm_dw_kernel: no atomics, so two
// runs agree bit for bit.
//
// HBM bounds it (four rows of 16 bits an element in and out with dh).  With
// only 512 workgroups to hide it, the latency of a row's load showed: 8192 x
// 4096 bf16 took 80 us a call, and 55.5 with the next row on its way while this one
// is reduced and stored (in a profile 50.9, 5.3 TB/s, and 5.0 for the sum of dw).  Where two rows and a sum do not fit the
// registers (more than 8 bytes a column and thread) it loads in order.
template <typename T, int TPR, int VPT>
__global__ __launch_bounds__(Shape<TPR>::threads) void rmsnorm_grad_kernel(NormGradArgs a, float* dw) {
    using S = Shape<TPR>;
    __shared__ float sums[3][S::waves];
    __shared__ uint32_t tops[S::waves];
    const int t = threadIdx.x % TPR;
    const int n = int(a.n);
    const int64_t first = int64_t(blockIdx.x) * S::rows + threadIdx.x / TPR;
    // w stays in registers where there is room for it, else it comes from the L2 for every row
    constexpr bool KEEP = VPT * sizeof(T) <= 8;
    const T* w = static_cast<const T*>(a.w);
    Raw8<T> kept[KEEP ? VPT : 1];
    float part[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = 8 * (i * TPR + t);
        if constexpr (KEEP) kept[i] = load8(w + c, n - c);
#pragma unroll
        for (int j = 0; j < 8; ++j) part[i][j] = 0;
    }
    const int64_t step = int64_t(gridDim.x) * S::rows;
    constexpr bool AHEAD = VPT * sizeof(T) <= 8;                // the next row is on its way, if there is room
    Raw8<T> hn[VPT], gn[VPT], en[VPT];
    auto load = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 8 * (i * TPR + t), left = n - c;
            hn[i] = load8(static_cast<const T*>(a.h) + row * a.ldh + c, left);
            gn[i] = load8(static_cast<const T*>(a.dy) + row * a.lddy + c, left);
            if (a.dh) en[i] = load8(static_cast<const T*>(a.dh) + row * a.lddh + c, left);
        }
    };
    if (AHEAD && first < a.rows) load(first);
    for (int64_t row = first; row < a.rows; row += step) {
        if (!AHEAD) load(row);
        Raw8<T> hr[VPT], gr[VPT], er[VPT];
        float square = 0, dot = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 8 * (i * TPR + t), left = n - c;
            float squares = 0, dots = 0;
            hr[i] = hn[i];
            gr[i] = gn[i];
            er[i] = en[i];
            const Raw8<T> wr = KEEP ? kept[KEEP ? i : 0] : load8(w + c, left);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float h = hr[i][j];
                squares = fmadd(h, h, squares);
                dots = fmadd(gr[i][j] * wr[j], h, dots);
            }
            square += squares;
            dot += dots;
        }
        if (AHEAD && row + step < a.rows) load(row + step);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            hr[i].keep_packed();
            gr[i].keep_packed();
        }
        square = block_reduce<TPR>(square, Add{}, sums[0]);
        dot = block_reduce<TPR>(dot, Add{}, sums[1]);
        float mean = square / float(n) + a.eps, f = 1;
        if (!mean_in_range(mean)) {
            uint32_t most = 0;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) most = Max{}(most, magnitude(hr[i][j]));
            f = rescale(block_reduce<TPR>(most, Max{}, tops), a.eps);
            square = dot = 0;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = 8 * (i * TPR + t);
                const Raw8<T> wr = KEEP ? kept[KEEP ? i : 0] : load8(w + c, n - c);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    square = fmadd(hr[i][j] * f, hr[i][j] * f, square);
                    dot = fmadd(gr[i][j] * wr[j], hr[i][j] * f, dot);
                }
            }
            if constexpr (S::waves > 1) __syncthreads();   // sums[1] is read by all before it is written again
            square = block_reduce<TPR>(square, Add{}, sums[2]);
            dot = block_reduce<TPR>(dot, Add{}, sums[1]);
            mean = square / float(n) + a.eps * f * f;
        }
        // with h f and rs = 1 / rms(h f): s = f rs, and h s = (h f) rs
        const float rs = inverse_root(mean), s = f * rs;
        const float back = rs * (dot / float(n));
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 8 * (i * TPR + t), left = n - c;
            const Raw8<T> wr = KEEP ? kept[KEEP ? i : 0] : load8(w + c, left);
            float d[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float h = hr[i][j], g = gr[i][j];
                const float unit = h * f * rs;
                d[j] = s * (g * wr[j] - unit * back);
                part[i][j] = fmadd(g, unit, part[i][j]);
            }
            if (a.dh) {
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] += er[i][j];
            }
            store8(static_cast<T*>(a.dx) + row * a.lddx + c, d, left);
        }
        if constexpr (S::waves > 1) __syncthreads();   // the next row's sums
    }
    if (!dw) return;
    float* out = dw + int64_t(blockIdx.x) * n;
    if constexpr (S::rows == 1) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 8 * (i * TPR + t);
            store8(out + c, part[i], n - c);
        }
    } else {
        __shared__ float join[S::rows][TPR * VPT * 8];
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) join[threadIdx.x / TPR][8 * (i * TPR + t) + j] = part[i][j];
        __syncthreads();
        for (int c = threadIdx.x; c < n; c += S::threads) {
            float sum = join[0][c];
#pragma unroll
            for (int i = 1; i < S::rows; ++i) sum += join[i][c];
            out[c] = sum;
        }
    }
}

// dw[c] = the sum of `count` rows of partial sums: 32 columns and 8 slices of
// the rows per workgroup, the slices joined in LDS.  Bound by latency: 512 rows
// of 4096 take 4 to 5 us with eight loads of a slice on their way at a time; one at
// a time cost 517 x 1537 f32 two of its 16 us.
static __global__ __launch_bounds__(256) void rmsnorm_dw_kernel(const float* partial, int64_t count, int n, float* dw) {
    __shared__ float slice[8][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + x;
    float sum = 0;
    if (c < n) {
        int64_t p = y;
        for (; p + 56 < count; p += 64) {                       // eight loads on their way at a time
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = partial[(p + 8 * i) * n + c];
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += v[i];
        }
        for (; p < count; p += 8) sum += partial[p * n + c];
    }
    slice[y][x] = sum;
    __syncthreads();
    if (y == 0 && c < n) {
#pragma unroll
        for (int i = 1; i < 8; ++i) sum += slice[i][x];
        dw[c] = sum;
    }
}

static __global__ __launch_bounds__(256) void rmsnorm_zero_kernel(float* dw, int n) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c < n) dw[c] = 0;
}

// ---------------------------------------------------------------- selection
// The gradient holds two rows and a sum, so it spreads them over more threads; for
// short rows as above (bf16 with dh, 16 M elements: 128 columns 29 us with 16 lanes,
// 130 with 64; 256 columns 29 with 32, 78 with 64).
// Three vectors in 16 bits: 34.8 us for 3276 x 5120 and 44.4 for 1365 x 12288
// (47.6 and 56.6 with the next power of two).  In 32 bits three vectors leave
// no room for the next row, which up to 8192 columns two vectors of 512 threads
// have: 56.0 us against 58.0 at 5120.
template <typename T, typename F>
inline hipError_t with_grad_shape(int64_t n, F&& f) {
    const int64_t v = (n + 7) / 8;
    if (v <= 16) return f(ic<16>{}, ic<1>{});
    if (v <= 32) return f(ic<32>{}, ic<1>{});
    if (v <= 64) return f(ic<64>{}, ic<1>{});
    if (v <= 128) return f(ic<64>{}, ic<2>{});
    if (v <= 256) return f(ic<256>{}, ic<1>{});
    if (v <= 512) return f(ic<256>{}, ic<2>{});
    if constexpr (sizeof(T) == 2)
        if (v <= 768) return f(ic<256>{}, ic<3>{});
    if (v <= 1024) return f(ic<512>{}, ic<2>{});
    if (v <= 1536) return f(ic<512>{}, ic<3>{});
    return f(ic<512>{}, ic<4>{});
}

constexpr int64_t kMostGroups = 1 << 20;    // workgroups of a launch; rows beyond it loop

template <typename T>
inline hipError_t rmsnorm_quant_t(Scale sc, const NormQuantArgs& a, hipStream_t s) {
    return with_shape(a.n, [&](auto tpr, auto vpt) {
        constexpr int TPR = decltype(tpr)::value, VPT = decltype(vpt)::value;
        using S = Shape<TPR>;
        const int64_t need = (a.rows + S::rows - 1) / S::rows;
        const dim3 grid(uint32_t(need < kMostGroups ? need : kMostGroups));
        return sc == Scale::BLOCK
                   ? launch(rmsnorm_quant_kernel<T, TPR, VPT, true>, grid, dim3(S::threads), 0, s, a)
                   : launch(rmsnorm_quant_kernel<T, TPR, VPT, false>, grid, dim3(S::threads), 0, s, a);
    });
}

// Workgroups of the gradient kernel: two a compute unit (8192 x 4096 bf16 52 us, 60
// with four), and not less than four rows for each of its groups of threads, whose
// sums of dw are then fewer (1024 x 4096 bf16 14.9 us, 17.1 with one).
template <int TPR>
inline int64_t grad_groups(int64_t rows) {
    const int64_t need = (rows + 4 * Shape<TPR>::rows - 1) / (4 * Shape<TPR>::rows);
    const int64_t most = 512;
    return need < most ? need : most;
}

// Partial sums of dw, one a workgroup.
template <typename T>
inline int64_t grad_partials(int64_t rows, int64_t n) {
    int64_t p = 0;
    with_grad_shape<T>(n, [&](auto tpr, auto) {
        p = grad_groups<decltype(tpr)::value>(rows);
        return hipSuccess;
    });
    return p;
}

template <typename T>
inline hipError_t rmsnorm_grad_t(const NormGradArgs& a, hipStream_t s) {
    if (a.rows == 0)
        return launch(rmsnorm_zero_kernel, dim3(uint32_t((a.n + 255) / 256)), dim3(256), 0, s, a.dw, int(a.n));
    const int64_t parts = grad_partials<T>(a.rows, a.n);
    float* out = !a.dw ? nullptr : parts > 1 ? a.partial : a.dw;
    const hipError_t e = with_grad_shape<T>(a.n, [&](auto tpr, auto vpt) {
        constexpr int TPR = decltype(tpr)::value, VPT = decltype(vpt)::value;
        return launch(rmsnorm_grad_kernel<T, TPR, VPT>, dim3(uint32_t(grad_groups<TPR>(a.rows))),
                      dim3(Shape<TPR>::threads), 0, s, a, out);
    });
    if (e != hipSuccess || parts == 1 || !a.dw) return e;
    return launch(rmsnorm_dw_kernel, dim3(uint32_t((a.n + 31) / 32)), dim3(256), 0, s,
                  static_cast<const float*>(a.partial), parts, int(a.n), a.dw);
}

}  // namespace rmsnorm_detail
}  // namespace bl
