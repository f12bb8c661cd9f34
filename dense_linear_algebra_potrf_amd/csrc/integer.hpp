// Internal interface between the C-ABI layer (integer.cpp) and the kernels of the
// 8-bit-integer layer operators.  Arguments have been checked by the caller.
#pragma once

#include "layer.hpp"

namespace bl {

struct Int8QuantArgs {
    int64_t rows, n;
    const void* x; int64_t ldx;
    const float* given;                  // may be null
    int8_t* q; int64_t ldq;
    float* scales;                       // null where scales are given
    void* values; int64_t ldv;           // may be null
};
hipError_t int8_quant(Type t, const Int8QuantArgs& a, hipStream_t s);

struct Int8MatmulArgs {
    int64_t m, n, k;
    const int8_t* x; int64_t ldx;
    const float* xs;
    const int8_t* w; int64_t ldw;
    const float* ws;
    void* y; int64_t ldy;
};
// Largest sizes: sums of products up to 2^14 in 32 bits, and offsets within a tile
// of 256 rows in 32.
constexpr int64_t kIntMaxK = (int64_t(1) << 17) - 1, kIntMaxRows = int64_t(1) << 24, kIntMaxLd = int64_t(1) << 22;
hipError_t int8_matmul(Type yt, const Int8MatmulArgs& a, hipStream_t s);

// Widest rows: the norm and its gradient hold a row in registers.
constexpr int64_t kBlockNormMaxN = 32768, kBlockGradMaxN = 16384;

struct BlockNormArgs {
    int64_t rows, n;
    const void* y; int64_t ldy;
    const void* x; int64_t ldx;
    const void* w;
    const void* post;                    // may be null
    const void* gate; int64_t per, ldg;  // may be null; row i has gate row i / per
    float c, eps;
    void* h; int64_t ldh;
    void* v; int64_t ldv;
    float* scales;                       // with Scale::ROW
};
hipError_t block_norm(Type t, Scale sc, const BlockNormArgs& a, hipStream_t s);

struct BlockGradArgs {
    int64_t rows, n;
    const void* dv; int64_t lddv;
    const void* y; int64_t ldy;
    const void* h; int64_t ldh;
    const void* w;
    const void* post;                    // may be null
    const void* gate; int64_t per, ldg;  // may be null
    const void* dh; int64_t lddh;        // may be null
    float c, eps;
    void* dy; int64_t lddy;
    void* dx; int64_t lddx;
    Type dgtype;
    void* dgate; int64_t lddg;           // may be null
    float* dw;                           // may be null
    float* dpost;                        // may be null
    float* workspace;
    int64_t gates;                       // rows of the gate
};
// Floats of the workspace where everything is computed; per = 0: without a gate.
int64_t block_norm_grad_floats(Type t, int64_t rows, int64_t n, int64_t per);
hipError_t block_norm_grad(Type t, const BlockGradArgs& a, hipStream_t s);

}  // namespace bl
