// Norms after one block and before the next with the block's gate and the residual's
// scale in one pass, and their gradient.
//
//     u = post y / sqrt(mean(y^2) + eps),  h = c x + gate u,  v = w h / sqrt(mean(h^2) + eps)
//
// As in the norm to 8 bits, a row stays in the registers of the TPR threads that
// share it (VPT vectors of 8 elements each, vector i of thread t at column
// 8 (i TPR + t)) from its loads through both sums of squares to the stores.
//
// HBM bounds it: x, y, h and v (and a gate for each row), a pass each.  8192 rows of 8192
// in bf16 take 97 us (a copy of as many bytes 104), with codes 95 (91), of 4096 47 (52), in f32
// 110 (104).
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
        const float f = rescale(block_reduce<TPR>(most, Max{}, tops), eps);
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

// Rows of 16-bit types are stored past the caches: 8192 rows of 8192 take 97 us in place of
// 117, the gradient at 8192 rows of 4096 95 in place of 97.  In 32 bits a thread's eight
// columns take two stores, each of every other 16 bytes, and lose by it: 8192 rows
// of 4096 119 (110), the gradient 199 (168).
template <typename T>
__device__ __forceinline__ void store_row(T* p, const float (&f)[8], int count) {
    if constexpr (sizeof(T) == 2) store8_past(p, f, count);
    else store8(p, f, count);
}

// The weights and the gate are on their way before the sums that they wait for, where
// that costs few of the wavefronts a compute unit has room for: 8192 rows of 8192 in bf16 take
// 117 us where they took 121, to codes 101 (110), of 4096 in f32 110 (119), all stored through
// the caches.  In shapes
// where it costs more of them it loses: 65536 rows of 1024 114 (108), 2000 of 12000 with
// a gate each 61 (58).
template <int TPR, int VPT> constexpr bool kEarly = VPT == 1 || VPT == 4 || (VPT == 2 && TPR > 64);

template <typename T, int TPR, int VPT, bool POST, bool CODES>
__global__ __launch_bounds__(Shape<TPR>::threads) void block_norm_kernel(BlockNormArgs a) {
    using S = Shape<TPR>;
    __shared__ float sums[4][S::waves];
    __shared__ uint32_t tops[3][S::waves];
    const int t = threadIdx.x % TPR;
    const int n = int(a.n);
    constexpr bool EARLY = kEarly<TPR, VPT>;
    const T* w = static_cast<const T*>(a.w);
    // Where a row is shared by less than a wave, its end is in every wave's way: loads without
    // a branch took 124 us in place of 154 for 500000 rows of 100 in f16 (98 now).  In longer rows
    // the last threads alone take the branch, and 8192 rows of 8192 in bf16 took 121 us with it, 127
    // without.
    auto at = [&](const T* from, int c) {
        if constexpr (TPR >= 64) return load8(from + c, n - c);
        Raw8<T> r = fetch(from, c, n);
        settle(r, c, n);
        return r;
    };
    for (int64_t row = int64_t(blockIdx.x) * S::rows + S::slot(); row < a.rows;
         row += int64_t(gridDim.x) * S::rows) {
        const T* x = static_cast<const T*>(a.x) + row * a.ldx;
        const T* y = static_cast<const T*>(a.y) + row * a.ldy;
        const T* gate = static_cast<const T*>(a.gate) + (a.gate ? row / a.per * a.ldg : 0);
        float v[VPT][8];
        Raw8<T> held[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 8 * (i * TPR + t);
            const Raw8<T> yr = at(y, c);
            held[i] = at(x, c);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = yr[j];
        }
        [[maybe_unused]] float ts = 1;
        Raw8<T> pk[VPT], gk[VPT], wk[VPT];
        if constexpr (EARLY) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if constexpr (POST) pk[i] = at(static_cast<const T*>(a.post), 8 * (i * TPR + t));
                if (a.gate) gk[i] = at(gate, 8 * (i * TPR + t));
            }
        }
        if constexpr (POST) ts = unit_factor<TPR>(v, n, a.eps, sums[0], sums[1], tops[0]);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 8 * (i * TPR + t), left = n - c;
            if constexpr (POST) {
                const Raw8<T> p = EARLY ? pk[i] : at(static_cast<const T*>(a.post), c);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * ts * p[j];
            }
            if (a.gate) {
                const Raw8<T> g = EARLY ? gk[i] : at(gate, c);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = fmadd(v[i][j], g[j], a.c * held[i][j]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = fmadd(a.c, held[i][j], v[i][j]);
            }
            // elements past the row's end are not part of it (0 * inf is not 0)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = j < left ? v[i][j] : 0.0f;
            store_row(static_cast<T*>(a.h) + row * a.ldh + c, v[i], left);
        }
        if constexpr (EARLY) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) wk[i] = at(w, 8 * (i * TPR + t));
        }
        const float rs = unit_factor<TPR>(v, n, a.eps, sums[2], sums[3], tops[1]);
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = 8 * (i * TPR + t), left = n - c;
            const Raw8<T> wr = EARLY ? wk[i] : at(w, c);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] = v[i][j] * rs * wr[j];
                if constexpr (CODES) top = Max{}(top, j < left ? magnitude(v[i][j]) : 0u);
            }
            if constexpr (!CODES) store_row(static_cast<T*>(a.v) + row * a.ldv + c, v[i], left);
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
// With e = dv w, the unit rows u = h s and z = y t of the two norms, and the row's gate:
//     a = dh + s (e - u mean(e u)),   dx = c a,   b = a gate,
//     dy = t (b post - z mean(b post z)),
//     dw = sum dv u,  and S = sum a z over the rows of one gate, from which
//     dgate = post S and dpost = sum over gates of gate S.
// Without post, z is y itself, dy = b and dgate = S.
//
// With k = gate post y, the last mean comes apart into sums that need neither root nor
// the other mean, so that a row takes one reduction and one barrier:
//     sum(b post z) = t (sum(k dh) + s sum(k e) - s^2 mean(e u) sum(k h)).
// (Three reductions, one after the other, took 130 us where this took 97.)
//
// Each group of TPR threads takes a run of consecutive rows and keeps its sums over
// them in registers: runs either lie within one gate's rows, whose sums S then go to
// the workspace, or hold whole gates, whose dgate is then written at each gate's end
// while gate S goes on in LDS.  The workspace's sums are added in a fixed order by
// block_grad_sums_kernel: no atomics, so two runs agree bit for bit.
//
// HBM bounds it: dv, y, h and dh are read and dx and dy written once.  8192 rows of 4096 in bf16
// with eight gates take 95 us, 87 of them here and 8 in the sums (a copy of as many
// bytes 78), in f32 168 (157), 4096 of 8192 in bf16 89 (78).  517 rows of 1537 take
// 18 us, 11 here and 4 in the sums: the latency of two launches.
struct Runs {
    int64_t rows;        // of a run
    int64_t of_gate;     // runs of one gate, whole workgroups of them; 0: a run holds whole gates (or there are none)
    int64_t count;
};

// A row's sums: h^2, e h and, with post, y^2, k dh, k e and k h.
struct RowSums {
    float h2, eh, y2, kd, ke, kh;
};

// Their sums over THREADS threads, with one barrier.
template <int THREADS, bool POST>
__device__ __forceinline__ RowSums reduce(RowSums v, RowSums* slot) {
    constexpr int LANES = THREADS < 64 ? THREADS : 64;
    v.h2 = wave_reduce<LANES>(v.h2, Add{});
    v.eh = wave_reduce<LANES>(v.eh, Add{});
    if constexpr (POST) {
        v.y2 = wave_reduce<LANES>(v.y2, Add{});
        v.kd = wave_reduce<LANES>(v.kd, Add{});
        v.ke = wave_reduce<LANES>(v.ke, Add{});
        v.kh = wave_reduce<LANES>(v.kh, Add{});
    }
    if constexpr (THREADS > 64) {
        if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
        __syncthreads();
        v = slot[0];
#pragma unroll
        for (int i = 1; i < THREADS / 64; ++i) {
            const RowSums o = slot[i];
            v.h2 += o.h2, v.eh += o.eh;
            if constexpr (POST) v.y2 += o.y2, v.kd += o.kd, v.ke += o.ke, v.kh += o.kh;
        }
    }
    return v;
}

// What a shape's registers have room for: the weights over all rows and the next row
// while this one is reduced and stored; or only this row; or not even that (it then comes
// from the cache a second time, which rows beyond 8192 pay with 135 us where a copy takes 78).
template <typename T, int TPR, int VPT> constexpr bool kAhead = TPR <= 512 && VPT * sizeof(T) <= 4;
template <typename T, int TPR, int VPT> constexpr bool kHold = TPR <= 512 && VPT <= 2;

// The sums hold products of h and y with the gradients, which may be large or small
// themselves: h and y are scaled sooner than their squares alone would need.
__device__ __forceinline__ bool near_one(float mean) { return mean > 0x1p-48f && mean < 0x1p48f; }

// The workspace: dw's sums, a row of n for each workgroup, then as many of either S or
// dpost's.
template <typename T, int TPR, int VPT, bool POST>
__global__ __launch_bounds__(Shape<TPR>::threads) void block_grad_kernel(BlockGradArgs a, Runs runs, float* dw, float* second) {
    using S = Shape<TPR>;
    constexpr bool AHEAD = kAhead<T, TPR, VPT>, HOLD = kHold<T, TPR, VPT>;
    // by the row's parity, so that the next row's may be written while this one's are read
    __shared__ RowSums sums[2][S::waves], again[2][S::waves];
    __shared__ uint32_t tops[2][2][S::waves];
    const int t = threadIdx.x % TPR;
    const int n = int(a.n);
    const int64_t run = int64_t(blockIdx.x) * S::rows + S::slot();
    auto send_for = [&](const void* p, int64_t row, int64_t ld, int i) {
        int c = 8 * (i * TPR + t);
        asm volatile("" : "+v"(c));                             // no address is kept from one row to the next
        return fetch(static_cast<const T*>(p) + row * ld, c, n);
    };
    auto at = [&](const void* p, int64_t row, int64_t ld, int i) {
        Raw8<T> r = send_for(p, row, ld, i);
        settle(r, 8 * (i * TPR + t), n);
        return r;
    };
    auto put = [&](void* p, int64_t row, int64_t ld, int i, const float (&v)[8]) {
        const int c = 8 * (i * TPR + t);
        store_row(static_cast<T*>(p) + row * ld + c, v, n - c);
    };
    // dpost's sum over whole gates is touched once a gate: it lies in LDS, a thread's
    // own slots, for the registers it would take
    __shared__ float psum[VPT][8][S::threads];
    __shared__ float glds[HOLD ? 1 : VPT][8][HOLD ? 1 : S::threads];    // S too, in the widest shapes
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

    // where registers are short, a vector's loads stay behind the last one's work
    auto in_turn = [] {
        if constexpr (!HOLD) __builtin_amdgcn_sched_barrier(0);
    };
    // the next row on its way, and this one
    constexpr int NEXT = AHEAD ? VPT : 1, KEPT = HOLD ? VPT : 1;
    Raw8<T> hn[NEXT], vn[NEXT], yn[NEXT], dn[NEXT], hk[KEPT], vk[KEPT], yk[KEPT], dk[KEPT], wk[NEXT], pk[NEXT], gk[NEXT];
    auto load_next = [&](int64_t r) {
        if constexpr (AHEAD)
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                hn[i] = send_for(a.h, r, a.ldh, i);
                vn[i] = send_for(a.dv, r, a.lddv, i);
                yn[i] = send_for(a.y, r, a.ldy, i);
                if (a.dh) dn[i] = send_for(a.dh, r, a.lddh, i);
            }
    };
    if (AHEAD && row < end) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            wk[i] = at(a.w, 0, 0, i);
            if constexpr (POST) pk[i] = at(a.post, 0, 0, i);
            if (a.gate) gk[i] = at(a.gate, gate_row, a.ldg, i);
        }
        load_next(row);
    }
    auto w_at = [&](int i) {
        if constexpr (AHEAD) return wk[i];
        else return at(a.w, 0, 0, i);
    };
    auto p_at = [&](int i) {
        if constexpr (AHEAD) return pk[i];
        else return at(a.post, 0, 0, i);
    };
    auto g_at = [&](int i) {
        if constexpr (AHEAD) return gk[i];
        else return at(a.gate, gate_row, a.ldg, i);
    };
    for (int parity = 0; row < end; ++row, parity ^= 1) {
        auto h_at = [&](int i) {
            if constexpr (HOLD) return hk[i];
            else return at(a.h, row, a.ldh, i);
        };
        auto v_at = [&](int i) {
            if constexpr (HOLD) return vk[i];
            else return at(a.dv, row, a.lddv, i);
        };
        auto y_at = [&](int i) {
            if constexpr (HOLD) return yk[i];
            else return at(a.y, row, a.ldy, i);
        };
        auto d_at = [&](int i) {
            if constexpr (HOLD) return dk[i];
            else return at(a.dh, row, a.lddh, i);
        };
        // sums of h f and y yf in the place of h and y
        auto sum_up = [&](float f, float yf) {
            RowSums sum = {0, 0, 0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const Raw8<T> hr = h_at(i), vr = v_at(i), wr = w_at(i);
                RowSums part = {0, 0, 0, 0, 0, 0};              // short chains: small errors
                float e[8], h[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    e[j] = vr[j] * wr[j];
                    h[j] = hr[j] * f;
                    part.h2 = fmadd(h[j], h[j], part.h2);
                    part.eh = fmadd(e[j], h[j], part.eh);
                }
                in_turn();
                if constexpr (POST) {
                    const Raw8<T> yr = y_at(i), pr = p_at(i);
                    float k[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        k[j] = yr[j] * yf;
                        part.y2 = fmadd(k[j], k[j], part.y2);
                        k[j] *= pr[j];
                    }
                    in_turn();
                    if (a.gate) {
                        const Raw8<T> gr = g_at(i);
#pragma unroll
                        for (int j = 0; j < 8; ++j) k[j] *= gr[j];
                    }
                    in_turn();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        part.ke = fmadd(k[j], e[j], part.ke);
                        part.kh = fmadd(k[j], h[j], part.kh);
                    }
                    if (a.dh) {
                        const Raw8<T> dr = d_at(i);
#pragma unroll
                        for (int j = 0; j < 8; ++j) part.kd = fmadd(k[j], dr[j], part.kd);
                    }
                }
                sum.h2 += part.h2, sum.eh += part.eh;
                if constexpr (POST) sum.y2 += part.y2, sum.kd += part.kd, sum.ke += part.ke, sum.kh += part.kh;
                in_turn();
            }
            return sum;
        };
        if constexpr (HOLD) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if constexpr (AHEAD) {
                    hk[i] = hn[i], vk[i] = vn[i], yk[i] = yn[i], dk[i] = dn[i];
                } else {
                    hk[i] = send_for(a.h, row, a.ldh, i);
                    vk[i] = send_for(a.dv, row, a.lddv, i);
                    yk[i] = send_for(a.y, row, a.ldy, i);
                    if (a.dh) dk[i] = send_for(a.dh, row, a.lddh, i);
                }
            }
            if (AHEAD && row + 1 < end) load_next(row + 1);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = 8 * (i * TPR + t);
                settle(hk[i], c, n), settle(vk[i], c, n), settle(yk[i], c, n);
                if (a.dh) settle(dk[i], c, n);
            }
        }
        const bool last = !runs.of_gate && a.gate && ++in_gate == a.per;    // of a gate, in a run of whole gates
        RowSums sum = sum_up(1.0f, 1.0f);
        auto keep_packed = [&] {
            if constexpr (HOLD) {
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    hk[i].keep_packed(), vk[i].keep_packed(), yk[i].keep_packed(), dk[i].keep_packed();
                    if constexpr (AHEAD) wk[i].keep_packed(), pk[i].keep_packed(), gk[i].keep_packed();
                }
            }
        };
        keep_packed();
        sum = reduce<TPR, POST>(sum, sums[parity]);
        float f = 1, yf = 1, mean = sum.h2 / float(n) + a.eps, ymean = POST ? sum.y2 / float(n) + a.eps : 1.0f;
        if (!near_one(mean) || !near_one(ymean)) {
            uint32_t most = 0, ymost = 0;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const Raw8<T> hr = h_at(i);
#pragma unroll
                for (int j = 0; j < 8; ++j) most = Max{}(most, magnitude(hr[j]));
                if constexpr (POST) {
                    const Raw8<T> yr = y_at(i);
#pragma unroll
                    for (int j = 0; j < 8; ++j) ymost = Max{}(ymost, magnitude(yr[j]));
                }
                in_turn();
            }
            f = rescale(block_reduce<TPR>(most, Max{}, tops[parity][0]), a.eps);
            if constexpr (POST) yf = rescale(block_reduce<TPR>(ymost, Max{}, tops[parity][1]), a.eps);
            sum = reduce<TPR, POST>(sum_up(f, yf), again[parity]);
            mean = sum.h2 / float(n) + a.eps * f * f;
            if constexpr (POST) ymean = sum.y2 / float(n) + a.eps * yf * yf;
        }
        // with h f and rs = 1 / rms(h f): s = f rs, and h s = (h f) rs; likewise for y
        const float rs = inverse_root(mean), s = f * rs, back = rs * (sum.eh / float(n));
        [[maybe_unused]] float rt = 1, ts = 1, yback = 0;
        if constexpr (POST) {
            rt = inverse_root(ymean), ts = yf * rt;
            // kh with rs first: with back, which has the gradients' size, it would leave the range before ke does
            yback = rt * ((sum.kd + s * (sum.ke - back * (rs * sum.kh))) / float(n));
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const Raw8<T> hr = h_at(i), vr = v_at(i), wr = w_at(i);
            float d[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float unit = hr[j] * f * rs, v = vr[j];
                wsum[i][j] = fmadd(v, unit, wsum[i][j]);
                d[j] = s * (v * wr[j] - unit * back);
            }
            if (a.dh) {
                const Raw8<T> dr = d_at(i);
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] += dr[j];
            }
            float dx[8], z[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) dx[j] = a.c * d[j];
            const Raw8<T> yr = y_at(i);                         // before the stores: dx or dy may be y
            if constexpr (!HOLD) put(a.dx, row, a.lddx, i, dx);
            in_turn();
            Raw8<T> pr, gr;
            if constexpr (POST) pr = p_at(i);
            if (a.gate) gr = g_at(i);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                z[j] = POST ? yr[j] * yf * rt : yr[j];
                gsum(i, j) = fmadd(d[j], z[j], gsum(i, j));
            }
            if (a.gate) {
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] *= gr[j];
            }
            if constexpr (POST) {
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] = ts * (d[j] * pr[j] - z[j] * yback);
            }
            if constexpr (HOLD) put(a.dx, row, a.lddx, i, dx);
            put(a.dy, row, a.lddy, i, d);
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
            in_turn();
        }
        if (last) {
            in_gate = 0;
            ++gate_row;
            if (AHEAD && row + 1 < end) {
#pragma unroll
                for (int i = 0; i < VPT; ++i) gk[i] = at(a.gate, gate_row, a.ldg, i);
            }
        }
    }
    // the workgroup's sums of dw, and of S or dpost
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
    if (second) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) wsum[i][j] = a.gate && !runs.of_gate ? psum[i][j][threadIdx.x] : gsum(i, j);
        store_sum(second + int64_t(blockIdx.x) * n, wsum);
    }
}

// What is added up from the workspace: blockIdx.y 0: dw, 1: dpost, 2 + g: dgate of
// gate g, which has `of_gate` of the workgroups' sums (0: it is written already).  32
// columns and 32 slices of the sums per workgroup, joined in LDS, eight loads of a slice
// on their way at a time: it is bound by their latency.
template <typename T>
__global__ __launch_bounds__(1024) void block_grad_sums_kernel(BlockGradArgs a, const float* first, const float* second, int groups,
                                                               int of_gate) {
    constexpr int SLICES = 32;
    __shared__ float slice[SLICES][33];
    const int n = int(a.n), x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + x;
    const int what = int(blockIdx.y);
    if (what == 0 ? !a.dw : what == 1 ? !a.dpost : !a.dgate) return;
    const float* from = what ? second : first;
    int count = groups;
    if (what > 1) {
        count = of_gate;
        from += int64_t(what - 2) * of_gate * n;
    }
    const bool weighted = what == 1 && of_gate;                 // dpost = sum over gates of gate S
    const T* const gate = static_cast<const T*>(a.gate);
    float sum = 0;
    if (c < n) {
        auto add = [&](auto some) {                             // up to eight of them
            constexpr int MOST = decltype(some)::value;
            return [&, MOST](int p) {
                float v[MOST];
#pragma unroll
                for (int i = 0; i < MOST; ++i) v[i] = from[int64_t(p + SLICES * i) * n + c];
                if (weighted) {
#pragma unroll
                    for (int i = 0; i < MOST; ++i) v[i] *= float(gate[int64_t((p + SLICES * i) / of_gate) * a.ldg + c]);
                }
#pragma unroll
                for (int i = 0; i < MOST; ++i) sum += v[i];
            };
        };
        int p = y;
        for (; p + 7 * SLICES < count; p += 8 * SLICES) add(ic<8>{})(p);
        for (; p < count; p += SLICES) add(ic<1>{})(p);
    }
    slice[y][x] = sum;
    __syncthreads();
    if (y == 0 && c < n) {
#pragma unroll
        for (int i = 1; i < SLICES; ++i) sum += slice[i][x];
        if (what == 0) {
            a.dw[c] = sum;
        } else if (what == 1) {
            a.dpost[c] = sum;
        } else {
            if (a.post) sum *= float(static_cast<const T*>(a.post)[c]);
            const int64_t to = int64_t(what - 2) * a.lddg + c;
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

// Runs of rows: 512 workgroups for rows of up to 256 threads (the shapes of one vector a thread have
// registers for three a compute unit or more; what that would do for 513 to 768 rows, which are two
// to a run now, was not measured), 256 for wider ones, which have room for one.  A
// gate with more rows than a workgroup's groups of threads is cut into equal runs, whole
// workgroups of them, so that its S is joined there; smaller ones are put together.  Runs
// of one row, where there are few rows, cost the sums less than they save here: 64 rows
// of 4096 take 8 + 4 us, in runs of two 12 + 4.  Many short gates stay whole: cutting them
// saves about 2.7 us for each row less, adding them up costs about 1.5 for 512 workgroups of 32
// columns.  512 rows of 4096 with 256 gates take 21 us whole and 82 cut, with 64 gates 30 and
// 36, 4096 rows with 128 gates 99 and 81.
template <int TPR>
inline Runs make_runs(int64_t rows, int64_t n, int64_t per) {
    constexpr int64_t groups = Shape<TPR>::rows, slots = (TPR <= 256 ? 512 : 256) * groups;
    const int64_t want = (rows + slots - 1) / slots;
    Runs r{want, 0, 0};
    if (per > groups && (per - want) * 30000 > rows / per * n) {
        const int64_t parts = (per + want * groups - 1) / (want * groups) * groups;
        r.rows = (per + parts - 1) / parts;
        r.of_gate = ((per + r.rows - 1) / r.rows + groups - 1) / groups * groups;
        r.count = rows / per * r.of_gate;
    } else {
        if (per > 0) r.rows = (want + per - 1) / per * per;
        r.count = (rows + r.rows - 1) / r.rows;
    }
    return r;
}

// Shapes of the gradient: the fewest threads whose registers have room for the next row,
// so that two rows or more are under way on a compute unit.  In bf16, 8192 rows of 4096
// took 97 us in 256 threads and 106 in 512; 4096 rows of 8192 96 us in 512 and 151 in
// 1024, which have no room; 2048 rows of 16384, for which there is none, 153 us in 1024
// and 181 in 512 (before the stores past the caches).
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
    if constexpr (sizeof(T) == 2) return f(ic<1024>{}, ic<2>{});
    else return f(ic<512>{}, ic<4>{});
}

template <typename T, typename F>
inline auto with_runs(int64_t rows, int64_t n, int64_t per, F&& f) {
    return with_block_grad_shape<T>(n, [&](auto tpr, auto vpt) {
        constexpr int TPR = decltype(tpr)::value;
        const Runs r = make_runs<TPR>(rows, n, per);
        return f(tpr, vpt, r, (r.count + Shape<TPR>::rows - 1) / Shape<TPR>::rows);
    });
}

template <typename T>
inline int64_t block_norm_grad_floats_t(int64_t rows, int64_t n, int64_t per) {
    int64_t floats = 0;
    with_runs<T>(rows, n, per, [&](auto, auto, const Runs&, int64_t groups) {
        floats = 2 * groups * n;
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
        const int of_gate = int(r.of_gate / Shape<TPR>::rows);
        const int64_t gates = of_gate && a.dgate ? a.rows / a.per : 0;
        const dim3 sums(uint32_t((a.n + 31) / 32), uint32_t(gates ? 2 + gates : a.dpost ? 2 : 1));
        return launch(block_grad_sums_kernel<T>, sums, dim3(1024), 0, s, a, static_cast<const float*>(a.workspace),
                      static_cast<const float*>(second), int(groups), of_gate);
    });
}

}  // namespace block_norm_detail
}  // namespace bl
