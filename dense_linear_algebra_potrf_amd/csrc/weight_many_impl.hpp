// Products of more than 16 rows with 4-bit weights.
//
// As weight_matvec_impl.hpp, with up to 64 rows of x to a workgroup, so that the
// codes are read and unpacked once for them.  What bounds it then is x: every
// workgroup reads all of it, and in the layout of the matrix cores (16 bytes of
// each of 16 rows) a load makes 64 requests to the cache.  So x is laid out once
// before, in the caller's workspace, as the matrix cores take it: 1 KB for each
// 16 rows and 32 columns, 16 bytes to a lane, in 16-bit floats (8-bit values with
// their blocks' scale), the columns in the order in which integer codes come
// apart, rows and columns past the end zero.
#pragma once

#include "weight_matvec_impl.hpp"

namespace bl {
namespace weight_matvec_detail {

constexpr int kManyWaves = 8;

inline int64_t packed_bytes(int64_t m, int64_t k) {
    return (m + 15) / 16 * ((k + kChunk - 1) / kChunk) * 4096;
}

// One thread for 8 columns of a row.
template <X XT, bool MIXED>
__global__ __launch_bounds__(256) void pack_kernel(MatvecArgs a, u32x4* out) {
    const int64_t octets = (a.k + kChunk - 1) / kChunk * 16, rows = (a.m + 15) / 16 * 16;
    const int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (id >= rows * octets) return;
    const int64_t row = id / octets, k = (id - row * octets) * 8;
    const int left = row < a.m ? int(a.k - k < 8 ? a.k - k : 8) : 0;   // columns that there are
    u32x4 v = {0, 0, 0, 0};
    if constexpr (is_eight(XT)) {
        const uint8_t* p = static_cast<const uint8_t*>(a.x) + row * a.ldx + k;
        uint64_t e = 0;
        if (left >= 8) {
            __builtin_memcpy(&e, p, 8);
        } else {
#pragma unroll
            for (int j = 0; j < 7; ++j)
                if (j < left) e |= uint64_t(p[j]) << (8 * j);
        }
        float scale = 1;
        if (XT == X::F8_BLOCK && left > 0)
            scale = power_of(static_cast<const uint8_t*>(a.xscales)[row * a.ldxs + k / kScaleBlock]);
        const Frag f = from_e4m3<in_half(XT)>(uint32_t(e), uint32_t(e >> 32), scale);
        v = u32x4{f.word[0], f.word[1], f.word[2], f.word[3]};
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(a.x) + row * a.ldx + k;
        if (left >= 8) {
            __builtin_memcpy(&v, p, 16);
        } else {
#pragma unroll
            for (int j = 0; j < 7; ++j)
                if (j < left) v[j / 2] |= uint32_t(p[j]) << (16 * (j & 1));
        }
    }
    if constexpr (MIXED) v = mixed<false>(v);
    // (16 rows, 32 columns), then the lane: row, and which 8 of the columns
    out[((row / 16) * (octets / 4) + k / 32) * 64 + k % 32 / 8 * 16 + row % 16] = v;
}

template <bool HALF, Format F, int GROUP, int MT, int NB>
__global__ __launch_bounds__(64 * kManyWaves) void weight_many_kernel(MatvecArgs a, const u32x4* packed, X xt, Type yt) {
    constexpr bool OFFSET = F == Format::INTEGER;
    constexpr int MB = MT / 16, GROUPS = kChunk / GROUP, STEPS = GROUP / 32, TILE = 16 * NB;
    __shared__ uint32_t scales[kGroups][TILE];
    __shared__ union {
        u32x4 codes[kManyWaves][NB * 64];
        float sums[kManyWaves][MB * NB * 4][64];
    } lds;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6, r = lane & 15, g = lane >> 4;
    const int64_t n0 = int64_t(blockIdx.x) * TILE, m0 = int64_t(blockIdx.y) * MT;
    const int chunks = int((a.k + kChunk - 1) / kChunk), groups = int((a.k + GROUP - 1) / GROUP);
    const int rows_n = a.n - n0 < TILE ? int(a.n - n0) : TILE, rows_m = a.m - m0 < MT ? int(a.m - m0) : MT;

    // Codes: lane / 4 is the row, lane % 4 the 16 bytes of it.  Rows past the end
    // and bytes past a row's are not read: their results are not stored, and their
    // columns of x are zero.
    const uint32_t code_at = uint32_t(lane >> 2) * uint32_t(a.ldc) + 16 * (lane & 3);
    const uint8_t* const codes0 = a.codes + n0 * a.ldc;
    const int64_t codes_step = 16 * a.ldc;
    const int row_bytes = int((a.k + 1) / 2) - 16 * (lane & 3);
    auto load_codes = [&](int c, u32x4 (&d)[NB]) {
        const uint8_t* codes = codes0 + int64_t(c) * (kChunk / 2);
        const bool in = c * (kChunk / 2) < row_bytes;
#pragma unroll
        for (int i = 0; i < NB; ++i, codes += codes_step)
            if (in && 16 * i + (lane >> 2) < rows_n) d[i] = *reinterpret_cast<const u32x4*>(codes + code_at);
    };
    // x: tiles of 16 rows past the end are those of the last one
    const int last = int((a.m + 15) / 16 - 1 - m0 / 16);
    const u32x4* const x0 = packed + m0 / 16 * chunks * 256 + lane;
    auto load_x = [&](int c, int t, Frag (&x)[MB][4]) {
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            const u32x4 v = x0[(int64_t(i < last ? i : last) * chunks + c) * 256 + 64 * t];
            x[i][t] = Frag{{v[0], v[1], v[2], v[3]}};
        }
    };
    auto& own = lds.codes[wave];
    auto get_codes = [&](int i, int t) {
        return reinterpret_cast<const uint32_t*>(&own[64 * i + 4 * r + (t ^ (r >> 2))])[g];
    };

    f32x4 acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    constexpr int PHASE = kGroups / GROUPS;
    u32x4 held[NB] = {};
    Frag x[MB][4];
    for (int base = 0; base < chunks; base += PHASE) {
        const int end = base + PHASE < chunks ? base + PHASE : chunks;
        int c = base + wave;
        if (c < end) {                                          // on their way while the scales are staged
            load_codes(c, held);
#pragma unroll
            for (int t = 0; t < 4; ++t) load_x(c, t, x);
        }
        const int g0 = base * GROUPS;
        if (base) __syncthreads();
        stage_scales<F, GROUPS, TILE>(a, n0, g0, end * GROUPS < groups ? end * GROUPS - g0 : groups - g0, scales);
        __syncthreads();
        for (; c < end; c += waves) {
            const int next = c + waves < end ? c + waves : c, group = (c - base) * GROUPS;
            wave_lds_sync();                                    // the last chunk has been read
#pragma unroll
            for (int i = 0; i < NB; ++i) own[64 * i + (lane & ~3) + ((lane & 3) ^ (lane >> 4))] = held[i];
            load_codes(next, held);
            wave_lds_sync();
#pragma unroll
            for (int s = 0; s < GROUPS; ++s) {
                f32x4 part[MB][NB], ones[MB];
                float scale[NB], zero[NB];
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    const uint32_t v = scales[group + s][16 * j + r];
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
                    if constexpr (OFFSET) {
#pragma unroll
                        for (int i = 0; i < MB; ++i) ones[i] = product<HALF>(x[i][t], ones_of<HALF>(), ones[i]);
                    }
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        const Frag w = unpack<HALF, F, true>(get_codes(j, t));
#pragma unroll
                        for (int i = 0; i < MB; ++i) part[i][j] = product<HALF>(x[i][t], w, part[i][j]);
                    }
                    // x of the next chunk (of this one again, at the end), in the place of what has
                    // been multiplied; not earlier, or it would be held twice
                    __builtin_amdgcn_sched_barrier(0);
                    load_x(next, t, x);
                }
#pragma unroll
                for (int j = 0; j < NB; ++j)
#pragma unroll
                    for (int i = 0; i < MB; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float p = OFFSET ? fmadd(-zero[j], ones[i][e], part[i][j][e]) : part[i][j][e];
                            acc[i][j][e] = fmadd(scale[j], p, acc[i][j][e]);
                        }
            }
        }
    }

    __syncthreads();                                            // the codes' LDS is free
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) lds.sums[wave][(i * NB + j) * 4 + e][lane] = acc[i][j][e];
    __syncthreads();
    store_sums<F, GROUP, MB, NB>(a, xt, yt, m0, n0, rows_m, rows_n, waves, &lds.sums[0]);
}

template <bool HALF>
inline hipError_t weight_many_t(X xt, Type yt, Format f, int group, const MatvecArgs& a, const u32x4* packed, hipStream_t s) {
    const int64_t chunks = (a.k + kChunk - 1) / kChunk;
    const dim3 block(uint32_t(64 * (chunks < kManyWaves ? chunks : kManyWaves)));
    auto tile = [&](auto fmt, auto size, auto mt, auto nb) {
        constexpr int MT = decltype(mt)::value, NB = decltype(nb)::value;
        const dim3 grid(uint32_t((a.n + 16 * NB - 1) / (16 * NB)), uint32_t((a.m + MT - 1) / MT));
        return launch(weight_many_kernel<HALF, decltype(fmt)::value, decltype(size)::value, MT, NB>, grid, block, 0, s, a, packed,
                      xt, yt);
    };
    auto shape = [&](auto fmt, auto size) {
        const bool wide = a.n >= 256 * 32;                      // enough rows for every compute unit at 32 each
        if (a.m <= 32) return wide ? tile(fmt, size, ic<32>{}, ic<2>{}) : tile(fmt, size, ic<32>{}, ic<1>{});
        return wide ? tile(fmt, size, ic<64>{}, ic<2>{}) : tile(fmt, size, ic<64>{}, ic<1>{});
    };
    if (f == Format::FLOAT) return shape(std::integral_constant<Format, Format::FLOAT>{}, ic<32>{});
    using I = std::integral_constant<Format, Format::INTEGER>;
    return group == 32 ? shape(I{}, ic<32>{}) : group == 64 ? shape(I{}, ic<64>{}) : shape(I{}, ic<128>{});
}

template <X XT>
inline hipError_t pack_t(Format f, const MatvecArgs& a, u32x4* packed, hipStream_t s) {
    const int64_t threads = (a.m + 15) / 16 * 16 * ((a.k + kChunk - 1) / kChunk) * 16;
    const dim3 grid(uint32_t((threads + 255) / 256));
    return f == Format::INTEGER ? launch(pack_kernel<XT, true>, grid, dim3(256), 0, s, a, packed)
                                : launch(pack_kernel<XT, false>, grid, dim3(256), 0, s, a, packed);
}

}  // namespace weight_matvec_detail
}  // namespace bl
