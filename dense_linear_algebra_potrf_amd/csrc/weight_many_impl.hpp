// Products of more than 16 rows with 4-bit weights.
//
// As weight_matvec_impl.hpp, with up to 64 rows of x to a workgroup, so that the
// codes are read and unpacked once for them.  Every workgroup reads all of x, and
// in the layout of the matrix cores (16 bytes of each of 16 rows) a load makes 64
// requests to the cache.  So x is laid out once before, in the caller's workspace,
// as the matrix cores take it: 1 KB for each 16 rows and 32 columns, 16 bytes to a
// lane, the columns in the order in which integer codes come apart, rows and
// columns past the end zero.
//
// x keeps the type that a few rows are multiplied in (e4m3 values become 16-bit
// floats on that occasion), so every value of it goes into the product as it is.  In
// half precision for all kinds, with a power of two per row, the codes would come
// apart more cheaply, but what is far below the row's largest value would be lost, and
// it counts where that value has no weight.
//
// What bounds it is the work in the compute unit: for 64 x 8192 x 8192 bfloat16 in
// groups of 32 (23.3 us a call; in a profile 21.9 and 4.9 for the layout of x) the
// vector units are busy for 10.7 us (unpacking 4.1, scaling the sums 3.4, the rest
// mostly before and after the loop), the matrix cores for 3.4, and 1 MB of x goes from
// the L2 to each compute unit, 12 TB/s in all; the codes alone would take 7.  Groups of
// 128 take 21.4 us, 32 rows of x 18.0.  When it took 24.9, scaling the last group and
// unpacking the next one while a product runs gained nothing (24.8), nor did codes from
// the cache (24.3): the two wavefronts of a SIMD already overlap.
#pragma once

#include "weight_matvec_impl.hpp"

namespace bl {
namespace weight_matvec_detail {

// Eight bytes at p, of which `left` belong to the row; the others are zero.
__device__ __forceinline__ uint64_t load_octet(const uint8_t* p, int left) {
    uint64_t e = 0;
    if (left >= 8) {
        __builtin_memcpy(&e, p, 8);
    } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < left) e |= uint64_t(p[j]) << (8 * j);
    }
    return e;
}

// Lays out x.  A workgroup takes 16 rows and a chunk's 128 columns, a wavefront 32 of
// them, a lane 16 bytes of the result: 8 columns of row lane % 16.  2.0 to 4.9 us for
// 64 x 8192 in a launch of its own, which is latency: 2 MB in and out would take 0.4.
constexpr int kPackThreads = 256;

template <X XT, Format F>
__global__ __launch_bounds__(kPackThreads) void pack_kernel(MatvecArgs a, u32x4* out, float* row_scale, int chunks) {
    using T = std::conditional_t<XT == X::F16, f16, bf16>;
    const int tile = int(blockIdx.x) / chunks, chunk = int(blockIdx.x) % chunks, lane = threadIdx.x & 63;
    const int64_t row = tile * 16 + (lane & 15), k = int64_t(chunk) * kChunk + (threadIdx.x >> 6) * 32 + (lane >> 4) * 8;
    const int left = row >= a.m || a.k <= k ? 0 : a.k - k < 8 ? int(a.k - k) : 8;
    u32x4 v = {0, 0, 0, 0};
    if constexpr (is_eight(XT)) {
        if (left) {
            const uint64_t raw = load_octet(static_cast<const uint8_t*>(a.x) + row * a.ldx + k, left);
            const float block = XT == X::F8_BLOCK ? block_power(static_cast<const uint8_t*>(a.xscales)[row * a.ldxs + k / kScaleBlock]) : 1.0f;
            v = __builtin_bit_cast(u32x4, from_e4m3<in_half(XT)>(uint32_t(raw), uint32_t(raw >> 32), block));
        }
    } else {
        v = __builtin_bit_cast(u32x4, load8(static_cast<const T*>(a.x) + row * a.ldx + k, left));
    }
    out[int64_t(blockIdx.x) * kPackThreads + threadIdx.x] = F == Format::INTEGER ? mixed<false>(v) : v;
    if (chunk == 0 && threadIdx.x < 16 && row < a.m)
        row_scale[row] = kUnit<XT, F> * (XT == X::F8_ROW ? static_cast<const float*>(a.xscales)[row] : 1.0f);
}

// Joins the wavefronts' sums in their order (a lane's four of a tile of 16 x 16:
// rows 4 (lane / 16) .. + 3 of x, column lane % 16), times the scale of x's row, and
// stores y.  A wavefront takes a tile, with 16-byte reads; element by element, with
// the row's scale from memory, 64 x 28672 x 8192 in groups of 128 took 76.9 us
// instead of 72.9 (72.3 now), and 64 x 28672 x 512 20.0 instead of 15.4 (15.0 now).
template <Format F, int GROUP, int MB, int NB, int WAVES>
__device__ __forceinline__ void store_tiles(const MatvecArgs& a, X xt, Type yt, int64_t m0, int64_t n0, int rows_m, int rows_n,
                                            int waves, const f32x4 (*sums)[MB * NB][64], const float* row_scale) {
    const int lane = threadIdx.x & 63;
    for (int tile = threadIdx.x >> 6; tile < MB * NB; tile += waves) {
        const int ml = tile / NB * 16 + (lane >> 4) * 4, nl = tile % NB * 16 + (lane & 15);
        f32x4 v = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {                       // those of wavefronts that are not there are not added
            const f32x4 s = sums[w][tile][lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += w < waves ? s[e] : 0.0f;
        }
        bool odd = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = ml + e < rows_m && nl < rows_n ? v[e] * row_scale[ml + e] : 0;
            odd = odd || magnitude(v[e]) >= kInfBits;
        }
        if (__ballot(odd)) {
#pragma unroll 1
            for (int e = 0; e < 4; ++e) {
                float mine = e == 0 ? v[0] : e == 1 ? v[1] : e == 2 ? v[2] : v[3];
#pragma unroll 1
                for (uint64_t left = __ballot(magnitude(mine) >= kInfBits); left; left &= left - 1) {
                    const int at = __builtin_ctzll(left);
                    const double d = by_definition(a, xt, F, GROUP, m0 + tile / NB * 16 + (at >> 4) * 4 + e,
                                                   n0 + tile % NB * 16 + (at & 15));
                    if (lane == at) mine = float(d);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] = q == e ? mine : v[q];
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (ml + e >= rows_m || nl >= rows_n) continue;
            const int64_t to = (m0 + ml + e) * a.ldy + n0 + nl;
            if (yt == Type::F32) static_cast<float*>(a.y)[to] = v[e];
            else if (yt == Type::F16) static_cast<f16*>(a.y)[to] = f16(v[e]);
            else static_cast<bf16*>(a.y)[to] = bf16(v[e]);
        }
    }
}

template <bool HALF, Format F, int GROUP, int MT, int NB, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void weight_many_kernel(MatvecArgs a, const u32x4* packed, const float* row_scale,
                                                                     X xt, Type yt) {
    constexpr int MB = MT / 16, GROUPS = kChunk / GROUP, STEPS = GROUP / 32, TILE = 16 * NB;
    __shared__ Scales<F, GROUPS, TILE> scales;
    __shared__ union {
        u32x4 codes[WAVES][NB * 64];
        f32x4 sums[WAVES][MB * NB][64];
    } lds;
    __shared__ float factor[MT];                                // of x's rows

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

    if (threadIdx.x < rows_m) factor[threadIdx.x] = row_scale[m0 + threadIdx.x];
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
        scales.stage(a, n0, g0, end * GROUPS < groups ? end * GROUPS - g0 : groups - g0);
        __syncthreads();
        for (; c < end; c += waves) {
            const int next = c + waves < end ? c + waves : c, group = (c - base) * GROUPS;
            wave_lds_sync();                                    // the last chunk has been read
#pragma unroll
            for (int i = 0; i < NB; ++i) own[64 * i + (lane & ~3) + ((lane & 3) ^ (lane >> 4))] = held[i];
            load_codes(next, held);
            wave_lds_sync();
            float scale[NB][GROUPS];
            uint32_t zeros[NB][GROUPS];
#pragma unroll
            for (int j = 0; j < NB; ++j) scales.get(16 * j + r, group, scale[j], zeros[j]);
#pragma unroll
            for (int s = 0; s < GROUPS; ++s) {
                f32x4 part[MB][NB];
#pragma unroll
                for (int j = 0; j < NB; ++j)
#pragma unroll
                    for (int i = 0; i < MB; ++i) part[i][j] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int q = 0; q < STEPS; ++q) {
                    const int t = s * STEPS + q;
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        const Frag w = unpack<HALF, F>(get_codes(j, t), Zero<HALF>(zeros[j][s]));
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
                        for (int e = 0; e < 4; ++e) acc[i][j][e] = fmadd(scale[j][s], part[i][j][e], acc[i][j][e]);
            }
        }
    }

    __syncthreads();                                            // the codes' LDS is free
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) lds.sums[wave][i * NB + j][lane] = acc[i][j];
    __syncthreads();
    store_tiles<F, GROUP, MB, NB, WAVES>(a, xt, yt, m0, n0, rows_m, rows_n, waves, &lds.sums[0], factor);
}

// x's layout in the workspace: the tiles, then the rows' scales.
inline float* row_scales(const MatvecArgs& a, void* workspace) {
    return reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + packed_bytes(a.m, a.k));
}

template <Format F, int GROUP>
inline hipError_t weight_many_t(X xt, Type yt, const MatvecArgs& a, void* workspace, hipStream_t s) {
    const int64_t chunks = (a.k + kChunk - 1) / kChunk;
    auto tile = [&](auto mt, auto nb, auto waves) {
        constexpr int MT = decltype(mt)::value, NB = decltype(nb)::value, WAVES = decltype(waves)::value;
        const dim3 block(uint32_t(64 * (chunks < WAVES ? chunks : WAVES)));
        const dim3 grid(uint32_t((a.n + 16 * NB - 1) / (16 * NB)), uint32_t((a.m + MT - 1) / MT));
        auto go = [&](auto half) {
            return launch(weight_many_kernel<decltype(half)::value, F, GROUP, MT, NB, WAVES>, grid, block, 0, s, a,
                          static_cast<const u32x4*>(workspace), static_cast<const float*>(row_scales(a, workspace)), xt, yt);
        };
        return in_half(xt) ? go(std::true_type{}) : go(std::false_type{});
    };
    // 32 rows of W to a workgroup where that leaves one for every compute unit: x is read
    // half as often (64 x 8192 x 8192 in groups of 32 23.6 us, 33.4 with 16; 32 x 28672 x
    // 8192 52.7 and 68.0).  With 64 rows of x a compute unit has the registers and LDS of
    // one workgroup of 8 wavefronts, and waits while it starts and joins: two of 4 where
    // there are so many (64 x 28672 x 8192 72.3 us, 81.1 with 8; 64 x 16384 x 4096 20.8 and
    // 23.5; 64 x 28672 x 512 15.0 and 23.2).  32 rows of x leave room for several (32 x 16384
    // x 8192 in groups of 32 26.7 us, 32.3 with 4; 32 x 28672 x 8192 52.7 and 52.0).
    // 32 rows of x where there are no more (17 x 8192 x 8192 16.0 us, 19.8 as 64; 32 x 28672
    // x 8192 52.7 and 59.9).
    auto rows = [&](auto mt) {
        if constexpr (decltype(mt)::value == 64)
            if (a.n >= 512 * 32) return tile(mt, ic<2>{}, ic<4>{});
        if (a.n >= 256 * 32) return tile(mt, ic<2>{}, ic<8>{});
        return tile(mt, ic<1>{}, ic<8>{});
    };
    return a.m <= 32 ? rows(ic<32>{}) : rows(ic<64>{});
}

template <X XT>
inline hipError_t pack_t(Format f, const MatvecArgs& a, void* workspace, hipStream_t s) {
    const int64_t chunks = (a.k + kChunk - 1) / kChunk;
    const dim3 grid(uint32_t((a.m + 15) / 16 * chunks));
    u32x4* out = static_cast<u32x4*>(workspace);
    float* scales = row_scales(a, workspace);
    return f == Format::INTEGER ? launch(pack_kernel<XT, Format::INTEGER>, grid, dim3(kPackThreads), 0, s, a, out, scales, int(chunks))
                                : launch(pack_kernel<XT, Format::FLOAT>, grid, dim3(kPackThreads), 0, s, a, out, scales, int(chunks));
}

}  // namespace weight_matvec_detail
}  // namespace bl
