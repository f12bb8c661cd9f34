// Internal interface between the C-ABI layer (layer.cpp) and the kernels of the
// low-bit layer operators.  Arguments have been checked by the caller.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace bl {

enum class Type : int { F32 = 0, F16 = 1, BF16 = 2, E4M3 = 3 };
enum class Scale : int { NONE = 0, ROW = 1, BLOCK = 2 };
enum class Format : int { INTEGER = 0, FLOAT = 1 };

// Widest rows: the norm and its gradient hold a row in registers.
constexpr int64_t kNormMaxN = 32768, kGradMaxN = 16384;
constexpr int kScaleBlock = 32;          // columns per scale of 8-bit values

struct NormQuantArgs {
    int64_t rows, n;
    const void* x; int64_t ldx;
    const void* r; int64_t ldr;          // may be null
    const void* w;
    float eps;
    void* h; int64_t ldh;                // may be null
    uint8_t* q; int64_t ldq;
    void* scales; int64_t lds;
};
hipError_t rmsnorm_quant(Type t, Scale sc, const NormQuantArgs& a, hipStream_t s);

struct NormGradArgs {
    int64_t rows, n;
    const void* dy; int64_t lddy;
    const void* h; int64_t ldh;
    const void* w;
    const void* dh; int64_t lddh;        // may be null
    float eps;
    void* dx; int64_t lddx;
    float* dw;                           // may be null
    float* partial;                      // rmsnorm_grad_partials(...) rows of n floats
};
// Partial sums of dw that the kernel writes; 1 means that it writes dw itself.
int64_t rmsnorm_grad_partials(Type t, int64_t rows, int64_t n);
hipError_t rmsnorm_grad(Type t, const NormGradArgs& a, hipStream_t s);

struct WeightQuantArgs {
    int64_t n, k;
    const void* W; int64_t ldw;
    uint8_t* codes; int64_t ldc;
    void* scales; int64_t lds;
    uint8_t* zeros; int64_t ldz;         // may be null
    void* values; int64_t ldv;           // may be null
    int64_t held;                        // bytes of a row that are written; 0: those with codes
};
hipError_t weight_quant(Type t, Format f, int group, const WeightQuantArgs& a, hipStream_t s);

struct MatvecArgs {
    int64_t m, n, k;
    const void* x; int64_t ldx;
    const void* xscales; int64_t ldxs;
    const uint8_t* codes; int64_t ldc;
    const void* scales; int64_t lds;
    const uint8_t* zeros; int64_t ldz;   // may be null
    void* y; int64_t ldy;
};
constexpr int64_t kFewRows = 16;         // above it x is laid out anew in the workspace first:
// 16-bit floats of whole tiles of 16 rows and 128 columns, then a scale for each row
inline int64_t packed_bytes(int64_t m, int64_t k) { return (m + 15) / 16 * ((k + 127) / 128) * 4096; }
inline int64_t weight_matvec_workspace(int64_t m, int64_t k) {
    return m <= kFewRows ? 0 : packed_bytes(m, k) + (m + 15) / 16 * 64;
}
hipError_t weight_matvec(Type xt, Scale xs, Type yt, Format f, int group, const MatvecArgs& a, void* workspace,
                         hipStream_t s);

}  // namespace bl
