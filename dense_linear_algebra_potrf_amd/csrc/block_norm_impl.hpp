// Norms after one block and before the next with the block's gate and the residual's
// scale in one pass, and their gradient.
//
//     u = post y / sqrt(mean(y^2) + eps),  h = c x + gate u,  v = w h / sqrt(mean(h^2) + eps)
//
// As in the norm to 8 bits, a row stays in the registers of the TPR threads that
// share it (VPT vectors of 8 elements each, vector i of thread t at column
// 8 (i TPR + t)) from its loads through both sums of squares to the stores.
//
// HBM bounds it: x, y, h and v (and a gate for each row), a pass each.
#pragma once

#include "integer_impl.hpp"
#include "norm_impl.hpp"

namespace bl {
namespace block_norm_detail {

using namespace layer;
using rmsnorm_detail::Shape;
using rmsnorm_detail::inverse_root;
using rmsnorm_detail::mean_in_range;
using rmsnorm_detail::rescale;

// Brings a row held as floats to unit root mean square: v becomes v f, and the result
// is what to multiply it by.  f is 1 unless its squares leave the range of 32 bits.
template <int TPR, int VPT>
__device__ __forceinline__ float unit_factor(float (&v)[VPT][8], int n, float eps, float* sums, float* again, uint32_t* tops) {
    float sum = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        float square = 0;                                       // short chains: small errors
#pragma unroll
        for (int j = 0; j < 8; ++j) square = fmadd(v[i][j], v[i][j], square);
        sum += square;
    }
    float mean = block_reduce<TPR>(sum, Add{}, sums) / float(n) + eps;
    if (!mean_in_range(mean)) {
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) most = Max{}(most, magnitude(v[i][j]));
        const float f = rescale(block_reduce<TPR>(most, Max{}, tops));
        sum = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] *= f;
                sum = fmadd(v[i][j], v[i][j], sum);
            }
        mean = block_reduce<TPR>(sum, Add{}, again) / float(n) + eps * f * f;
    }
    return inverse_root(mean);
}

template <typename T, int TPR, int VPT, bool POST, bool CODES>
__global__ __launch_bounds__(Shape<TPR>::threads) void block_norm_kernel(BlockNormArgs a) {
    using S = Shape<TPR>;
    __shared__ float sums[4][S::waves];
    __shared__ uint32_t tops[3][S::waves];
    const int t = threadIdx.x % TPR;
    const int n = int(a.n);
    const T* w = static_cast<const T*>(a.w);
    for (int64_t row = int64_t(blockIdx.x) * S::rows + S::slot(); row < a.rows;
         row += int64_t(gridDim.x) * S::rows) {
        const T* x = static_cast<const T*>(a.x) + row * a.ldx;
        const T* y = static_cast<const T*>(a.y) + row * a.ldy;
        const T* gate = static_cast<const T*>(a.gate) + (a.gate ? row / a.per * a.ldg : 0);
        float v[VPT][8];
        Raw8<T> held[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 8 * (i * TPR + t), left = n - c;
            const Raw8<T> yr = load8(y + c, left);
            held[i] = load8(x + c, left);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = yr[j];
        }
        [[maybe_unused]] float ts = 1;
        if constexpr (POST) ts = unit_factor<TPR>(v, n, a.eps, sums[0], sums[1], tops[0]);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 8 * (i * TPR + t), left = n - c;
            if constexpr (POST) {
                const Raw8<T> p = load8(static_cast<const T*>(a.post) + c, left);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * ts * p[j];
            }
            if (a.gate) {
                const Raw8<T> g = load8(gate + c, left);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = fmadd(v[i][j], g[j], a.c * held[i][j]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = fmadd(a.c, held[i][j], v[i][j]);
            }
            // elements past the row's end are not part of it (0 * inf is not 0)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = j < left ? v[i][j] : 0.0f;
            store8(static_cast<T*>(a.h) + row * a.ldh + c, v[i], left);
        }
        const float rs = unit_factor<TPR>(v, n, a.eps, sums[2], sums[3], tops[1]);
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 8 * (i * TPR + t), left = n - c;
            const Raw8<T> wr = load8(w + c, left);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] = v[i][j] * rs * wr[j];
                if constexpr (CODES) top = Max{}(top, j < left ? magnitude(v[i][j]) : 0u);
            }
            if constexpr (!CODES) store8(static_cast<T*>(a.v) + row * a.ldv + c, v[i], left);
        }
        if constexpr (CODES) {
            const float scale = code_scale(block_reduce<TPR>(top, Max{}, tops[2]));
            if (t == 0) a.scales[row] = scale;
            const float inverse = 1.0f / scale;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = 8 * (i * TPR + t);
                float q[8];
                Codes codes = to_codes(v[i], scale, inverse, q);
                if (!(inverse > 0)) codes = Codes{{0, 0}};      // a row that is not finite
                store_codes(static_cast<int8_t*>(a.v) + row * a.ldv + c, codes, n - c);
            }
        }
        if constexpr (S::waves > 1) __syncthreads();            // the next row's sums
    }
}

// ---------------------------------------------------------------- gradient
// With g = dv w, unit vectors h s and y t of the two norms, and the row's gate:
//     a = dh + s (g - (h s) mean(g h s)),   dx = c a,   b = a gate,
//     dy = t (b post - (y t) mean(b post y t)),
//     dw = sum dv (h s),  and S = sum a (y t) over the rows of one gate, from which
//     dgate = post S and dpost = sum over gates of gate S.
// Without post, y t is y itself, dy = b and dgate = S.
//
// Each group of TPR threads takes a run of consecutive rows and keeps its sums over
// them in registers: runs either lie within one gate's rows, whose sums S then go to
// the workspace, or hold whole gates, whose dgate is then written at each gate's end
// while gate S goes on in registers.  The workspace's sums are added in a fixed
// order by block_grad_sums_kernel: no atomics, so two runs agree bit for bit.
struct Runs {
    int64_t rows;        // of a run
    int64_t of_gate;     // runs of one gate; 0: a run holds whole gates (or there are none)
    int64_t count;
};

// Sums of three values over THREADS threads with one barrier.
template <int THREADS>
__device__ __forceinline__ void reduce3(float& a, float& b, float& c, float (*slot)[3]) {
    constexpr int LANES = THREADS < 64 ? THREADS : 64;
    a = wave_reduce<LANES>(a, Add{});
    b = wave_reduce<LANES>(b, Add{});
    c = wave_reduce<LANES>(c, Add{});
    if constexpr (THREADS > 64) {
        if ((threadIdx.x & 63) == 0) {
            slot[threadIdx.x >> 6][0] = a;
            slot[threadIdx.x >> 6][1] = b;
            slot[threadIdx.x >> 6][2] = c;
        }
        __syncthreads();
        a = slot[0][0], b = slot[0][1], c = slot[0][2];
#pragma unroll
        for (int i = 1; i < THREADS / 64; ++i) a += slot[i][0], b += slot[i][1], c += slot[i][2];
    }
}

// The next row is on its way while this one is reduced and stored, where the
// registers have room for two; else y and dh are loaded where they are used.
template <typename T, int VPT> constexpr bool kAhead = VPT * sizeof(T) <= 4;
// In the widest shape h and dv are loaded where they are used, too (from the cache).
template <int VPT> constexpr bool kHold = VPT <= 2;
// Then the loads of one vector also stay behind the work on the last.
template <bool AHEAD>
__device__ __forceinline__ void in_turn() {
    if constexpr (!AHEAD) {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    }
}

// The workspace: dw's sums, a row of n for each workgroup, then either S, a row for
// each run, or dpost's, a row for each workgroup.
template <typename T, int TPR, int VPT, bool POST>
__global__ __launch_bounds__(Shape<TPR>::threads) void block_grad_kernel(BlockGradArgs a, Runs runs, float* dw, float* second) {
    using S = Shape<TPR>;
    constexpr bool AHEAD = kAhead<T, VPT>, HOLD = kHold<VPT>;
    __shared__ float sums[2][S::waves][3], ysums[S::waves];
    __shared__ uint32_t tops[2][S::waves];
    const int t = threadIdx.x % TPR;
    const int n = int(a.n);
    const int64_t run = int64_t(blockIdx.x) * S::rows + S::slot();
    const T* const w = static_cast<const T*>(a.w);
    const T* const post = static_cast<const T*>(a.post);
    auto at = [&](const void* p, int64_t row, int64_t ld, int i) {
        const int c = 8 * (i * TPR + t);
        return load8(static_cast<const T*>(p) + row * ld + c, n - c);
    };
    auto put = [&](void* p, int64_t row, int64_t ld, int i, const float (&v)[8]) {
        const int c = 8 * (i * TPR + t);
        store8(static_cast<T*>(p) + row * ld + c, v, n - c);
    };
    // dpost's sum over whole gates is touched once a gate: it lies in LDS, a thread's
    // own slots, for the registers it would take
    __shared__ float psum[VPT][8][S::threads];
    __shared__ float glds[HOLD ? 1 : VPT][8][HOLD ? 1 : S::threads];    // S too, in the widest shape
    float wsum[VPT][8], gkept[HOLD ? VPT : 1][8];
    auto gsum = [&](int i, int j) -> float& {
        if constexpr (HOLD) return gkept[i][j];
        else return glds[i][j][threadIdx.x];
    };
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) psum[i][j][threadIdx.x] = wsum[i][j] = gsum(i, j) = 0;
    int64_t row = run * runs.rows, end = row + runs.rows;
    if (runs.of_gate) {
        const int64_t g = run / runs.of_gate;
        row = g * a.per + run % runs.of_gate * runs.rows;
        end = row + runs.rows < (g + 1) * a.per ? row + runs.rows : (g + 1) * a.per;
    }
    if (run >= runs.count) end = row;
    if (end > a.rows) end = a.rows;
    int64_t gate_row = a.gate && row < end ? row / a.per : 0;
    int64_t in_gate = a.gate && row < end ? row - gate_row * a.per : 0;
    Raw8<T> hn[AHEAD ? VPT : 1], vn[AHEAD ? VPT : 1], yn[AHEAD ? VPT : 1], en[AHEAD ? VPT : 1];
    auto load = [&](int64_t r) {
        if constexpr (AHEAD) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                hn[i] = at(a.h, r, a.ldh, i);
                vn[i] = at(a.dv, r, a.lddv, i);
                yn[i] = at(a.y, r, a.ldy, i);
                if (a.dh) en[i] = at(a.dh, r, a.lddh, i);
            }
        }
    };
    if (row < end) load(row);
    for (; row < end; ++row) {
        Raw8<T> hkept[HOLD ? VPT : 1], vkept[HOLD ? VPT : 1], ykept[AHEAD ? VPT : 1], ekept[AHEAD ? VPT : 1];
        float square = 0, dot = 0, ysquare = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            Raw8<T> hr, vr, yr;
            if constexpr (AHEAD) {
                hr = hn[i];
                vr = vn[i];
                yr = ykept[i] = yn[i];
                ekept[i] = en[i];
            } else {
                hr = at(a.h, row, a.ldh, i);
                vr = at(a.dv, row, a.lddv, i);
                if constexpr (POST) yr = at(a.y, row, a.ldy, i);
            }
            if constexpr (HOLD) {
                hkept[i] = hr;
                vkept[i] = vr;
            }
            const Raw8<T> wr = at(w, 0, 0, i);
            float squares = 0, dots = 0, ysquares = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                squares = fmadd(hr[j], hr[j], squares);
                dots = fmadd(vr[j] * wr[j], hr[j], dots);
                if constexpr (POST) ysquares = fmadd(yr[j], yr[j], ysquares);
            }
            square += squares;
            dot += dots;
            ysquare += ysquares;
            in_turn<AHEAD>();
        }
        if (AHEAD && row + 1 < end) load(row + 1);
        auto keep_packed = [&] {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if constexpr (HOLD) {
                    hkept[i].keep_packed();
                    vkept[i].keep_packed();
                }
                if constexpr (AHEAD) ykept[i].keep_packed();
            }
        };
        keep_packed();
        reduce3<TPR>(square, dot, ysquare, sums[0]);
        auto h_at = [&](int i) {
            if constexpr (HOLD) return hkept[i];
            else return at(a.h, row, a.ldh, i);
        };
        auto v_at = [&](int i) {
            if constexpr (HOLD) return vkept[i];
            else return at(a.dv, row, a.lddv, i);
        };
        auto y_at = [&](int i) {
            if constexpr (AHEAD) return ykept[i];
            else return at(a.y, row, a.ldy, i);
        };
        float mean = square / float(n) + a.eps, f = 1;
        if (!mean_in_range(mean)) {
            uint32_t most = 0;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const Raw8<T> hr = h_at(i);
#pragma unroll
                for (int j = 0; j < 8; ++j) most = Max{}(most, magnitude(hr[j]));
            }
            f = rescale(block_reduce<TPR>(most, Max{}, tops[0]));
            square = dot = 0;
            float none = 0;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const Raw8<T> wr = at(w, 0, 0, i), hr = h_at(i), vr = v_at(i);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    square = fmadd(hr[j] * f, hr[j] * f, square);
                    dot = fmadd(vr[j] * wr[j], hr[j] * f, dot);
                }
            }
            reduce3<TPR>(square, dot, none, sums[1]);
            mean = square / float(n) + a.eps * f * f;
        }
        const float rs = inverse_root(mean), s = f * rs, back = rs * (dot / float(n));
        float yf = 1, rt = 1;
        if constexpr (POST) {
            float ymean = ysquare / float(n) + a.eps;
            if (!mean_in_range(ymean)) {
                uint32_t most = 0;
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const Raw8<T> yr = y_at(i);
#pragma unroll
                    for (int j = 0; j < 8; ++j) most = Max{}(most, magnitude(yr[j]));
                }
                yf = rescale(block_reduce<TPR>(most, Max{}, tops[1]));
                ysquare = 0;
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const Raw8<T> yr = y_at(i);
#pragma unroll
                    for (int j = 0; j < 8; ++j) ysquare = fmadd(yr[j] * yf, yr[j] * yf, ysquare);
                }
                if constexpr (S::waves > 1) __syncthreads();    // sums[0] has been read
                float none = 0, nothing = 0;
                reduce3<TPR>(ysquare, none, nothing, sums[0]);
                ymean = ysquare / float(n) + a.eps * yf * yf;
            }
            rt = inverse_root(ymean);
        }
        keep_packed();
        const T* const gate = static_cast<const T*>(a.gate);
        float d[VPT][8];                                        // a
        [[maybe_unused]] float ydot = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const Raw8<T> wr = at(w, 0, 0, i), hr = h_at(i), vr = v_at(i), yr = y_at(i);
            Raw8<T> er;
            if constexpr (AHEAD) er = ekept[i];
            else if (a.dh) er = at(a.dh, row, a.lddh, i);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float unit = hr[j] * f * rs, g = vr[j];
                wsum[i][j] = fmadd(g, unit, wsum[i][j]);
                d[i][j] = s * (g * wr[j] - unit * back);
            }
            if (a.dh) {
#pragma unroll
                for (int j = 0; j < 8; ++j) d[i][j] += er[j];
            }
            float unit[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                unit[j] = POST ? yr[j] * yf * rt : yr[j];
                gsum(i, j) = fmadd(d[i][j], unit[j], gsum(i, j));
            }
            if constexpr (POST) {
                const Raw8<T> pr = at(post, 0, 0, i);
                float dots = 0;
                if (a.gate) {
                    const Raw8<T> gr = at(gate, gate_row, a.ldg, i);
#pragma unroll
                    for (int j = 0; j < 8; ++j) dots = fmadd(d[i][j] * gr[j] * pr[j], unit[j], dots);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) dots = fmadd(d[i][j] * pr[j], unit[j], dots);
                }
                ydot += dots;
            }
            in_turn<AHEAD>();
        }
        if constexpr (POST) ydot = block_reduce<TPR>(ydot, Add{}, ysums) / float(n);
        keep_packed();
        asm volatile("" : "+v"(rt));                            // y t is computed again: not kept from above
        const bool last = !runs.of_gate && a.gate && ++in_gate == a.per;    // of a gate, in a run of whole gates
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            Raw8<T> pr, gr;
            if constexpr (POST) pr = at(post, 0, 0, i);
            if (a.gate) gr = at(gate, gate_row, a.ldg, i);
            float dx[8], dy[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dx[j] = a.c * d[i][j];
                dy[j] = a.gate ? d[i][j] * gr[j] : d[i][j];
            }
            if constexpr (POST) {
                const Raw8<T> yr = y_at(i);
#pragma unroll
                for (int j = 0; j < 8; ++j) dy[j] = yf * rt * (dy[j] * pr[j] - yr[j] * yf * rt * ydot);
            }
            put(a.dx, row, a.lddx, i, dx);
            put(a.dy, row, a.lddy, i, dy);
            if (last) {
                float out[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    out[j] = POST ? gsum(i, j) * pr[j] : gsum(i, j);
                    psum[i][j][threadIdx.x] = fmadd(gr[j], gsum(i, j), psum[i][j][threadIdx.x]);
                    gsum(i, j) = 0;
                }
                const int c = 8 * (i * TPR + t);
                if (a.dgate && a.dgtype == Type::F32) store8(static_cast<float*>(a.dgate) + gate_row * a.lddg + c, out, n - c);
                else if (a.dgate) put(a.dgate, gate_row, a.lddg, i, out);
            }
            in_turn<AHEAD>();
        }
        if (last) {
            in_gate = 0;
            ++gate_row;
        }
        if constexpr (S::waves > 1) __syncthreads();            // the next row's sums
    }
    // a run's S, or the workgroup's sums of dw and dpost
    if (runs.of_gate && second && run < runs.count) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 8 * (i * TPR + t);
            float out[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) out[j] = gsum(i, j);
            store8(second + run * n + c, out, n - c);
        }
    }
    auto store_sum = [&](float* to, const float (&sum)[VPT][8]) {
        if constexpr (S::rows == 1) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = 8 * (i * TPR + t);
                store8(to + c, sum[i], n - c);
            }
        } else {
            __shared__ float join[S::rows][TPR * VPT * 8];
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) join[threadIdx.x / TPR][8 * (i * TPR + t) + j] = sum[i][j];
            __syncthreads();
            for (int c = threadIdx.x; c < n; c += S::threads) {
                float v = join[0][c];
#pragma unroll
                for (int i = 1; i < S::rows; ++i) v += join[i][c];
                to[c] = v;
            }
            __syncthreads();
        }
    };
    if (dw) store_sum(dw + int64_t(blockIdx.x) * n, wsum);
    if (!runs.of_gate && second) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) wsum[i][j] = a.gate ? psum[i][j][threadIdx.x] : gsum(i, j);
        store_sum(second + int64_t(blockIdx.x) * n, wsum);
    }
}

// What is added up from the workspace: blockIdx.y 0: dw, 1: dpost, 2 + g: dgate of
// gate g.  32 columns and 8 slices of the sums per workgroup, joined in LDS; eight
// loads of a slice are on their way at a time.
template <typename T>
__global__ __launch_bounds__(256) void block_grad_sums_kernel(BlockGradArgs a, Runs runs, const float* first, const float* second,
                                                              int64_t groups) {
    __shared__ float slice[8][33];
    const int n = int(a.n), x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + x;
    const int what = int(blockIdx.y);
    const float* from = what ? second : first;
    int64_t count = groups;
    if (what && runs.of_gate) {
        count = what == 1 ? runs.count : runs.of_gate;
        if (what > 1) from += (what - 2) * runs.of_gate * n;
    }
    const bool weighted = what == 1 && runs.of_gate;            // dpost = sum over gates of gate S
    const T* gate = static_cast<const T*>(a.gate);
    if (what == 0 ? !a.dw : what == 1 ? !a.dpost : !a.dgate) return;
    float sum = 0;
    if (c < n) {
        auto one = [&](int64_t p) {
            const float v = from[p * n + c];
            return weighted ? v * float(gate[p / runs.of_gate * a.ldg + c]) : v;
        };
        int64_t p = y;
        for (; p + 56 < count; p += 64) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = one(p + 8 * i);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += v[i];
        }
        for (; p < count; p += 8) sum += one(p);
    }
    slice[y][x] = sum;
    __syncthreads();
    if (y == 0 && c < n) {
#pragma unroll
        for (int i = 1; i < 8; ++i) sum += slice[i][x];
        if (what == 0) {
            a.dw[c] = sum;
        } else if (what == 1) {
            a.dpost[c] = sum;
        } else {
            if (a.post) sum *= float(static_cast<const T*>(a.post)[c]);
            const int64_t to = (what - 2) * a.lddg + c;
            if (a.dgtype == Type::F32) static_cast<float*>(a.dgate)[to] = sum;
            else static_cast<T*>(a.dgate)[to] = T(sum);
        }
    }
}

// No rows: what would be added up is zero.
template <typename T>
__global__ __launch_bounds__(256) void block_grad_zero_kernel(BlockGradArgs a) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= a.n) return;
    if (a.dw) a.dw[c] = 0;
    if (a.dpost) a.dpost[c] = 0;
    if (a.dgate)
        for (int64_t g = 0; g < a.gates; ++g) {
            if (a.dgtype == Type::F32) static_cast<float*>(a.dgate)[g * a.lddg + c] = 0;
            else static_cast<T*>(a.dgate)[g * a.lddg + c] = T(0.0f);
        }
}

constexpr int64_t kMostGroups = 1 << 20;    // workgroups of a launch; rows beyond it loop

template <typename T>
inline hipError_t block_norm_t(Scale sc, const BlockNormArgs& a, hipStream_t s) {
    return rmsnorm_detail::with_shape(a.n, [&](auto tpr, auto vpt) {
        constexpr int TPR = decltype(tpr)::value, VPT = decltype(vpt)::value;
        using S = Shape<TPR>;
        const int64_t need = (a.rows + S::rows - 1) / S::rows;
        const dim3 grid(uint32_t(need < kMostGroups ? need : kMostGroups)), block(S::threads);
        if (sc == Scale::ROW)
            return a.post ? launch(block_norm_kernel<T, TPR, VPT, true, true>, grid, block, 0, s, a)
                          : launch(block_norm_kernel<T, TPR, VPT, false, true>, grid, block, 0, s, a);
        return a.post ? launch(block_norm_kernel<T, TPR, VPT, true, false>, grid, block, 0, s, a)
                      : launch(block_norm_kernel<T, TPR, VPT, false, false>, grid, block, 0, s, a);
    });
}

// Runs of rows: two workgroups a compute unit, not less than four rows to a run.
// A gate with more rows is cut into equal runs, smaller ones are put together.
template <int TPR>
inline Runs make_runs(int64_t rows, int64_t per) {
    const int64_t slots = 512 * Shape<TPR>::rows;
    int64_t want = (rows + slots - 1) / slots;
    if (want < 4) want = 4;
    Runs r{want, 0, 0};
    if (per > want) {
        const int64_t parts = (per + want - 1) / want;
        r.rows = (per + parts - 1) / parts;
        r.of_gate = (per + r.rows - 1) / r.rows;
        r.count = rows / per * r.of_gate;
    } else {
        if (per > 0) r.rows = (want + per - 1) / per * per;
        r.count = (rows + r.rows - 1) / r.rows;
    }
    return r;
}

// Shapes of the gradient: as many threads as leave room for the next row, as above
// for short rows.
template <typename T, typename F>
inline hipError_t with_block_grad_shape(int64_t n, F&& f) {
    const int64_t v = (n + 7) / 8;
    if (v <= 16) return f(ic<16>{}, ic<1>{});
    if (v <= 32) return f(ic<32>{}, ic<1>{});
    if (v <= 64) return f(ic<64>{}, ic<1>{});
    if (v <= 128) return f(ic<64>{}, ic<2>{});
    if (v <= 256) return f(ic<256>{}, ic<1>{});
    if constexpr (sizeof(T) == 2) {
        if (v <= 512) return f(ic<256>{}, ic<2>{});
    } else {
        if (v <= 512) return f(ic<512>{}, ic<1>{});
    }
    if (v <= 1024) return f(ic<512>{}, ic<2>{});
    return f(ic<512>{}, ic<4>{});
}

template <typename T, typename F>
inline auto with_runs(int64_t rows, int64_t n, int64_t per, F&& f) {
    return with_block_grad_shape<T>(n, [&](auto tpr, auto vpt) {
        constexpr int TPR = decltype(tpr)::value;
        const Runs r = make_runs<TPR>(rows, per);
        return f(tpr, vpt, r, (r.count + Shape<TPR>::rows - 1) / Shape<TPR>::rows);
    });
}

template <typename T>
inline int64_t block_norm_grad_floats_t(int64_t rows, int64_t n, int64_t per) {
    int64_t floats = 0;
    with_runs<T>(rows, n, per, [&](auto, auto, const Runs& r, int64_t groups) {
        floats = (groups + (r.of_gate ? r.count : groups)) * n;
        return hipSuccess;
    });
    return floats;
}

template <typename T>
inline hipError_t block_norm_grad_t(const BlockGradArgs& a, hipStream_t s) {
    if (a.rows == 0)
        return launch(block_grad_zero_kernel<T>, dim3(uint32_t((a.n + 255) / 256)), dim3(256), 0, s, a);
    return with_runs<T>(a.rows, a.n, a.gate ? a.per : 0, [&](auto tpr, auto vpt, const Runs& r, int64_t groups) {
        constexpr int TPR = decltype(tpr)::value, VPT = decltype(vpt)::value;
        const dim3 grid{uint32_t(groups)}, block(Shape<TPR>::threads);
        float* const first = a.dw ? a.workspace : nullptr;
        float* const second = (r.of_gate ? a.dgate || a.dpost : a.dpost != nullptr) ? a.workspace + groups * a.n : nullptr;
        const hipError_t e = a.post ? launch(block_grad_kernel<T, TPR, VPT, true>, grid, block, 0, s, a, r, first, second)
                                    : launch(block_grad_kernel<T, TPR, VPT, false>, grid, block, 0, s, a, r, first, second);
        if (e != hipSuccess || (!first && !second)) return e;
        const int64_t gates = r.of_gate && a.dgate ? r.count / r.of_gate : 0;
        const dim3 sums(uint32_t((a.n + 31) / 32), uint32_t(gates ? 2 + gates : a.dpost ? 2 : 1));
        return launch(block_grad_sums_kernel<T>, sums, dim3(256), 0, s, a, r, static_cast<const float*>(a.workspace),
                      static_cast<const float*>(second), groups);
    });
}

}  // namespace block_norm_detail
}  // namespace bl
