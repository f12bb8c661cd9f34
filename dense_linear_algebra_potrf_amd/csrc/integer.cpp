// C-ABI entry points of the 8-bit-integer layer operators: argument validation.
// Declared in include/batchlas.h; everything here runs before anything is
// enqueued, and nothing is written on an error.
#include "../../include/batchlas.h"

#include <hip/hip_runtime.h>

#include <cmath>

#include "integer.hpp"
#include "layer_checks.hpp"
#include "status.hpp"

namespace {

using bl::Scale;
using bl::Type;
using bl::aligned;
using bl::check_norm_size;
using bl::check_norm_width;
using bl::fail;
using bl::guarded;
using bl::is_float;
using bl::kMost;
using bl::size_of;
using bl::spans;

batchlas_status do_int8_quant(int type, const bl::Int8QuantArgs& a, hipStream_t stream) {
    BL_REQUIRE(is_float(type), "type must be F32, F16 or BF16");
    batchlas_status st = check_norm_size(a.rows, a.n);
    if (st != BATCHLAS_OK) return st;
    BL_REQUIRE(a.ldx >= a.n, "ldx must be >= n");
    BL_REQUIRE(a.ldq >= a.n, "ldq must be >= n");
    BL_REQUIRE(a.ldq % 16 == 0, "ldq must be a multiple of 16");
    BL_REQUIRE(!a.values || a.ldv >= a.n, "ldv must be >= n");
    BL_REQUIRE(spans(a.rows, a.ldx) && spans(a.rows, a.ldq) && (!a.values || spans(a.rows, a.ldv)),
               "rows * leading dimension overflows");
    BL_REQUIRE(!a.given || !a.scales, "scales are either given or computed");
    if (a.rows > 0) {
        BL_POINTER(a.x, "x");
        BL_POINTER(a.q, "q");
        if (!a.given) BL_POINTER(a.scales, "scales");
    }
    BL_REQUIRE(aligned(a.q, 16), "q must be aligned to 16 bytes");
    BL_REQUIRE(aligned(a.x, size_of(type)) && aligned(a.values, size_of(type)) &&
                   aligned(a.given, 4) && aligned(a.scales, 4),
               "an array is not aligned to its element size");
    if (a.rows == 0) return BATCHLAS_OK;
    st = bl::check_device();
    if (st != BATCHLAS_OK) return st;
    return bl::hip_status(bl::int8_quant(static_cast<Type>(type), a, stream), "integer_quant launch");
}

batchlas_status do_int8_matmul(int ytype, const bl::Int8MatmulArgs& a, hipStream_t stream) {
    BL_REQUIRE(is_float(ytype), "ytype must be F32, F16 or BF16");
    BL_REQUIRE(a.m >= 0, "m must be >= 0");
    BL_REQUIRE(a.n >= 1, "n must be >= 1");
    BL_REQUIRE(a.k >= 1, "k must be >= 1");
    BL_REQUIRE(a.m < kMost && a.n < kMost && a.k < kMost, "m, n or k is out of range");
    BL_REQUIRE(a.ldx >= a.k, "ldx must be >= k");
    BL_REQUIRE(a.ldw >= a.k, "ldw must be >= k");
    BL_REQUIRE(a.ldx % 16 == 0 && a.ldw % 16 == 0, "ldx and ldw must be multiples of 16");
    BL_REQUIRE(a.ldy >= a.n, "ldy must be >= n");
    BL_REQUIRE(spans(a.m, a.ldx) && spans(a.n, a.ldw) && spans(a.m, a.ldy),
               "rows * leading dimension overflows");
    if (a.m > 0) {
        BL_POINTER(a.x, "x");
        BL_POINTER(a.xs, "xscales");
        BL_POINTER(a.w, "w");
        BL_POINTER(a.ws, "wscales");
        BL_POINTER(a.y, "y");
    }
    BL_REQUIRE(aligned(a.x, 16) && aligned(a.w, 16), "x and w must be aligned to 16 bytes");
    BL_REQUIRE(aligned(a.xs, 4) && aligned(a.ws, 4) && aligned(a.y, size_of(ytype)),
               "an array is not aligned to its element size");
    if (a.k > bl::kIntMaxK) return fail(BATCHLAS_NOT_SUPPORTED, "k is 2^17 or beyond");
    if (a.m > bl::kIntMaxRows || a.n > bl::kIntMaxRows)
        return fail(BATCHLAS_NOT_SUPPORTED, "m or n is beyond 2^24");
    // one launch's workgroups
    if (a.m * a.n > int64_t(1) << 36) return fail(BATCHLAS_NOT_SUPPORTED, "m * n is beyond 2^36");
    // offsets within a tile of rows are 32-bit
    if (a.ldx > bl::kIntMaxLd || a.ldw > bl::kIntMaxLd)
        return fail(BATCHLAS_NOT_SUPPORTED, "ldx or ldw is beyond 2^22");
    if (a.m == 0) return BATCHLAS_OK;
    const batchlas_status st = bl::check_device();
    if (st != BATCHLAS_OK) return st;
    return bl::hip_status(bl::int8_matmul(static_cast<Type>(ytype), a, stream),
                          "integer_matmul launch");
}

// Rows of a gate; `per` becomes the rows that share one.  An empty batch may have none.
batchlas_status check_gate(int64_t rows, int64_t gates, int64_t& per) {
    BL_REQUIRE(gates >= 1 || (gates == 0 && rows == 0), "gates must be >= 1");
    BL_REQUIRE(gates == 0 || rows % gates == 0, "gates must divide rows");
    per = gates ? rows / gates : 0;
    return BATCHLAS_OK;
}

batchlas_status check_factors(double c, double eps) {
    BL_REQUIRE(eps >= 0 && float(eps) <= 3.4028234e38f, "eps must be >= 0 and finite");
    BL_REQUIRE(std::isfinite(float(c)), "residual_scale must be finite");
    return BATCHLAS_OK;
}

batchlas_status do_block_norm(int type, int scale, bl::BlockNormArgs a, int64_t gates, double c,
                              double eps, hipStream_t stream) {
    BL_REQUIRE(is_float(type), "type must be F32, F16 or BF16");
    BL_REQUIRE(scale == BATCHLAS_SCALE_NONE || scale == BATCHLAS_SCALE_ROW,
               "scale must be NONE or ROW");
    const bool codes = scale == BATCHLAS_SCALE_ROW;
    batchlas_status st = check_norm_size(a.rows, a.n);
    if (st != BATCHLAS_OK) return st;
    if (a.gate && (st = check_gate(a.rows, gates, a.per)) != BATCHLAS_OK) return st;
    if ((st = check_factors(c, eps)) != BATCHLAS_OK) return st;
    BL_REQUIRE(a.ldy >= a.n, "ldy must be >= n");
    BL_REQUIRE(a.ldx >= a.n, "ldx must be >= n");
    BL_REQUIRE(!a.gate || a.ldg >= a.n, "ldg must be >= n");
    BL_REQUIRE(a.ldh >= a.n, "ldh must be >= n");
    BL_REQUIRE(a.ldv >= a.n, "ldv must be >= n");
    BL_REQUIRE(!codes || a.ldv % 16 == 0, "ldv must be a multiple of 16 for codes");
    BL_REQUIRE(spans(a.rows, a.ldy) && spans(a.rows, a.ldx) && spans(a.rows, a.ldh) &&
                   spans(a.rows, a.ldv) && (!a.gate || spans(gates, a.ldg)),
               "rows * leading dimension overflows");
    BL_REQUIRE(codes || !a.scales, "scales are for codes");
    if (a.rows > 0) {
        BL_POINTER(a.y, "y");
        BL_POINTER(a.x, "x");
        BL_POINTER(a.w, "w");
        BL_POINTER(a.h, "h");
        BL_POINTER(a.v, "v");
        if (codes) BL_POINTER(a.scales, "scales");
    }
    const int64_t es = size_of(type);
    BL_REQUIRE(!codes || aligned(a.v, 16), "codes must be aligned to 16 bytes");
    BL_REQUIRE(aligned(a.y, es) && aligned(a.x, es) && aligned(a.w, es) && aligned(a.post, es) &&
                   aligned(a.gate, es) && aligned(a.h, es) && (codes || aligned(a.v, es)) &&
                   aligned(a.scales, 4),
               "an array is not aligned to its element size");
    st = check_norm_width(a.n, bl::kBlockNormMaxN);
    if (st != BATCHLAS_OK || a.rows == 0) return st;
    BL_REQUIRE(a.h != a.v, "h and v must be different");
    st = bl::check_device();
    if (st != BATCHLAS_OK) return st;
    return bl::hip_status(bl::block_norm(static_cast<Type>(type), static_cast<Scale>(scale), a,
                                         stream),
                          "block_norm launch");
}

batchlas_status grad_bytes(int type, int64_t rows, int64_t n, int64_t gates, int64_t& bytes) {
    BL_REQUIRE(is_float(type), "type must be F32, F16 or BF16");
    batchlas_status st = check_norm_size(rows, n);
    if (st != BATCHLAS_OK) return st;
    int64_t per = 0;
    if (gates != 0 && (st = check_gate(rows, gates, per)) != BATCHLAS_OK) return st;
    st = check_norm_width(n, bl::kBlockGradMaxN);
    if (st != BATCHLAS_OK) return st;
    bytes = rows ? 4 * bl::block_norm_grad_floats(static_cast<Type>(type), rows, n, per) : 0;
    return BATCHLAS_OK;
}

batchlas_status do_block_norm_grad(int type, bl::BlockGradArgs a, int64_t gates, double c,
                                   double eps, int dgtype, int64_t bytes, hipStream_t stream) {
    BL_REQUIRE(is_float(type), "type must be F32, F16 or BF16");
    BL_REQUIRE(!a.dgate || dgtype == BATCHLAS_TYPE_F32 || dgtype == type,
               "dgtype must be F32 or the type");
    batchlas_status st = check_norm_size(a.rows, a.n);
    if (st != BATCHLAS_OK) return st;
    if (a.gate && (st = check_gate(a.rows, gates, a.per)) != BATCHLAS_OK) return st;
    a.gates = gates;
    if ((st = check_factors(c, eps)) != BATCHLAS_OK) return st;
    BL_REQUIRE(a.lddv >= a.n, "lddv must be >= n");
    BL_REQUIRE(a.ldy >= a.n, "ldy must be >= n");
    BL_REQUIRE(a.ldh >= a.n, "ldh must be >= n");
    BL_REQUIRE(!a.gate || a.ldg >= a.n, "ldg must be >= n");
    BL_REQUIRE(!a.dh || a.lddh >= a.n, "lddh must be >= n");
    BL_REQUIRE(a.lddy >= a.n, "lddy must be >= n");
    BL_REQUIRE(a.lddx >= a.n, "lddx must be >= n");
    BL_REQUIRE(!a.dgate || a.lddg >= a.n, "lddg must be >= n");
    BL_REQUIRE(spans(a.rows, a.lddv) && spans(a.rows, a.ldy) && spans(a.rows, a.ldh) &&
                   (!a.dh || spans(a.rows, a.lddh)) && spans(a.rows, a.lddy) &&
                   spans(a.rows, a.lddx) && (!a.gate || spans(gates, a.ldg)) &&
                   (!a.dgate || spans(gates, a.lddg)),
               "rows * leading dimension overflows");
    BL_REQUIRE(a.post || !a.dpost, "dpost needs post");
    BL_REQUIRE(a.gate || !a.dgate, "dgate needs a gate");
    if (a.rows > 0) {
        BL_POINTER(a.dv, "dv");
        BL_POINTER(a.y, "y");
        BL_POINTER(a.h, "h");
        BL_POINTER(a.w, "w");
        BL_POINTER(a.dy, "dy");
        BL_POINTER(a.dx, "dx");
    }
    const int64_t es = size_of(type);
    BL_REQUIRE(aligned(a.dv, es) && aligned(a.y, es) && aligned(a.h, es) && aligned(a.w, es) &&
                   aligned(a.post, es) && aligned(a.gate, es) && aligned(a.dh, es) &&
                   aligned(a.dy, es) && aligned(a.dx, es) &&
                   (!a.dgate || aligned(a.dgate, size_of(dgtype))) && aligned(a.dw, 4) &&
                   aligned(a.dpost, 4) && aligned(a.workspace, 4),
               "an array is not aligned to its element size");
    int64_t need = 0;
    st = grad_bytes(type, a.rows, a.n, a.gate ? gates : 0, need);
    if (st != BATCHLAS_OK) return st;
    if (!a.dw && !a.dpost && !a.dgate) need = 0;
    if (need) {
        BL_POINTER(a.workspace, "workspace");
        BL_REQUIRE(bytes >= need, "workspace_bytes is less than block_norm_grad_workspace gives");
    }
    BL_REQUIRE(a.rows == 0 || a.dy != a.dx, "dy and dx must be different");
    if (a.rows == 0 && !a.dw && !a.dpost && !a.dgate) return BATCHLAS_OK;
    st = bl::check_device();
    if (st != BATCHLAS_OK) return st;
    return bl::hip_status(bl::block_norm_grad(static_cast<Type>(type), a, stream),
                          "block_norm_grad launch");
}

}  // namespace

extern "C" {

batchlas_status batchlas_integer_quant(batchlas_type type, int64_t rows, int64_t n, const void* x,
                                       int64_t ldx, const float* given, int8_t* q, int64_t ldq,
                                       float* scales, void* values, int64_t ldv,
                                       batchlas_stream_t stream) {
    return guarded([&] {
        return do_int8_quant(type, {rows, n, x, ldx, given, q, ldq, scales, values, ldv},
                             reinterpret_cast<hipStream_t>(stream));
    });
}

batchlas_status batchlas_integer_matmul(batchlas_type ytype, int64_t m, int64_t n, int64_t k,
                                        const int8_t* x, int64_t ldx, const float* xscales,
                                        const int8_t* w, int64_t ldw, const float* wscales, void* y,
                                        int64_t ldy, batchlas_stream_t stream) {
    return guarded([&] {
        return do_int8_matmul(ytype, {m, n, k, x, ldx, xscales, w, ldw, wscales, y, ldy},
                              reinterpret_cast<hipStream_t>(stream));
    });
}

batchlas_status batchlas_block_norm(batchlas_type type, batchlas_scale scale, int64_t rows,
                                    int64_t n, const void* y, int64_t ldy, const void* x,
                                    int64_t ldx, const void* w, const void* post, const void* gate,
                                    int64_t gates, int64_t ldg, double residual_scale, double eps,
                                    void* h, int64_t ldh, void* v, int64_t ldv, float* scales,
                                    batchlas_stream_t stream) {
    return guarded([&] {
        return do_block_norm(type, scale,
                             {rows, n, y, ldy, x, ldx, w, post, gate, 0, ldg, float(residual_scale),
                              float(eps), h, ldh, v, ldv, scales},
                             gates, residual_scale, eps, reinterpret_cast<hipStream_t>(stream));
    });
}

batchlas_status batchlas_block_norm_grad(batchlas_type type, int64_t rows, int64_t n,
                                         const void* dv, int64_t lddv, const void* y, int64_t ldy,
                                         const void* h, int64_t ldh, const void* w,
                                         const void* post, const void* gate, int64_t gates,
                                         int64_t ldg, const void* dh, int64_t lddh,
                                         double residual_scale, double eps, void* dy, int64_t lddy,
                                         void* dx, int64_t lddx, batchlas_type dgtype, void* dgate,
                                         int64_t lddg, float* dw, float* dpost, void* workspace,
                                         int64_t workspace_bytes, batchlas_stream_t stream) {
    return guarded([&] {
        return do_block_norm_grad(
            type,
            {rows, n, dv, lddv, y, ldy, h, ldh, w, post, gate, 0, ldg, dh, lddh,
             float(residual_scale), float(eps), dy, lddy, dx, lddx, static_cast<Type>(dgtype), dgate,
             lddg, dw, dpost, static_cast<float*>(workspace), 0},
            gates, residual_scale, eps, dgtype, workspace_bytes,
            reinterpret_cast<hipStream_t>(stream));
    });
}

batchlas_status batchlas_block_norm_grad_workspace(batchlas_type type, int64_t rows, int64_t n,
                                                   int64_t gates, int64_t* bytes) {
    return guarded([&]() -> batchlas_status {
        BL_POINTER(bytes, "bytes");
        return grad_bytes(type, rows, n, gates, *bytes);
    });
}

}  // extern "C"
