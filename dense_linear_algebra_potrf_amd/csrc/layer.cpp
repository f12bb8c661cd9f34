// C-ABI entry points of the low-bit layer operators: argument validation.
// Declared in include/batchlas.h; everything here runs before anything is
// enqueued, and nothing is written on an error.
#include "../../include/batchlas.h"

#include <hip/hip_runtime.h>

#include <string>

#include "layer.hpp"
#include "status.hpp"

namespace {

using bl::Format;
using bl::Scale;
using bl::Type;
using bl::fail;
using bl::guarded;

batchlas_status invalid(const char* msg) { return fail(BATCHLAS_INVALID_VALUE, msg); }

int64_t size_of(int t) { return t == BATCHLAS_TYPE_F32 ? 4 : t == BATCHLAS_TYPE_E4M3 ? 1 : 2; }

bool is_float(int t) {
    return t == BATCHLAS_TYPE_F32 || t == BATCHLAS_TYPE_F16 || t == BATCHLAS_TYPE_BF16;
}

bool aligned(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// A row-major matrix whose last element's offset stays within 2^60 elements.
bool spans(int64_t rows, int64_t ld) {
    int64_t total = 0;
    return bl::mul_ok(rows, ld, total) && total < (int64_t(1) << 60);
}

#define BL_REQUIRE(cond, msg) \
    do {                      \
        if (!(cond)) return invalid(msg); \
    } while (0)
#define BL_POINTER(p, name) \
    do {                    \
        if (!(p)) return fail(BATCHLAS_NULL_POINTER, name " is NULL"); \
    } while (0)

constexpr int64_t kMost = int64_t(1) << 31;

batchlas_status check_norm_size(int64_t rows, int64_t n) {
    BL_REQUIRE(rows >= 0, "rows must be >= 0");
    BL_REQUIRE(n >= 1, "n must be >= 1");
    BL_REQUIRE(rows < kMost && n < kMost, "rows or n is out of range");
    return BATCHLAS_OK;
}

batchlas_status check_norm_width(int64_t n, int64_t most) {
    if (n > most)
        return fail(BATCHLAS_NOT_SUPPORTED,
                    "rows of at most " + std::to_string(most) + " columns are served");
    return BATCHLAS_OK;
}

batchlas_status check_format(int format, int64_t group) {
    BL_REQUIRE(format == BATCHLAS_FORMAT_INTEGER || format == BATCHLAS_FORMAT_FLOAT,
               "unknown format");
    if (format == BATCHLAS_FORMAT_INTEGER)
        BL_REQUIRE(group == 32 || group == 64 || group == 128, "group must be 32, 64 or 128");
    else
        BL_REQUIRE(group == 32, "group must be 32 for the float format");
    return BATCHLAS_OK;
}

batchlas_status check_codes(int64_t n, int64_t k, int64_t group, int64_t ldc, int64_t lds,
                            const void* zeros, int64_t ldz) {
    BL_REQUIRE(ldc >= (k + 1) / 2, "ldc must be >= (k + 1) / 2");
    BL_REQUIRE(ldc % 16 == 0, "ldc must be a multiple of 16");
    BL_REQUIRE(lds >= (k + group - 1) / group, "lds must be >= the groups of a row");
    BL_REQUIRE(!zeros || ldz >= (k + group - 1) / group, "ldz must be >= the groups of a row");
    BL_REQUIRE(spans(n, ldc) && spans(n, lds) && (!zeros || spans(n, ldz)),
               "rows * leading dimension overflows");
    return BATCHLAS_OK;
}

batchlas_status do_rmsnorm_quant(int type, int scale, const bl::NormQuantArgs& a,
                                 hipStream_t stream) {
    BL_REQUIRE(is_float(type), "type must be F32, F16 or BF16");
    BL_REQUIRE(scale == BATCHLAS_SCALE_ROW || scale == BATCHLAS_SCALE_BLOCK,
               "scale must be ROW or BLOCK");
    batchlas_status st = check_norm_size(a.rows, a.n);
    if (st != BATCHLAS_OK) return st;
    BL_REQUIRE(a.eps >= 0, "eps must be >= 0");
    BL_REQUIRE(a.ldx >= a.n, "ldx must be >= n");
    BL_REQUIRE(!a.r || a.ldr >= a.n, "ldr must be >= n");
    BL_REQUIRE(!a.h || a.ldh >= a.n, "ldh must be >= n");
    BL_REQUIRE(a.ldq >= a.n, "ldq must be >= n");
    const bool block = scale == BATCHLAS_SCALE_BLOCK;
    BL_REQUIRE(!block || a.lds >= (a.n + 31) / 32, "lds must be >= (n + 31) / 32");
    BL_REQUIRE(spans(a.rows, a.ldx) && (!a.r || spans(a.rows, a.ldr)) &&
                   (!a.h || spans(a.rows, a.ldh)) && spans(a.rows, a.ldq) &&
                   (!block || spans(a.rows, a.lds)),
               "rows * leading dimension overflows");
    BL_REQUIRE(a.r || !a.h, "h needs a residual r");
    if (a.rows > 0) {
        BL_POINTER(a.x, "x");
        BL_POINTER(a.w, "w");
        BL_POINTER(a.q, "q");
        BL_POINTER(a.scales, "scales");
    }
    const int64_t es = size_of(type);
    BL_REQUIRE(aligned(a.x, es) && aligned(a.r, es) && aligned(a.w, es) && aligned(a.h, es) &&
                   (block || aligned(a.scales, 4)),
               "an array is not aligned to its element size");
    st = check_norm_width(a.n, bl::kNormMaxN);
    if (st != BATCHLAS_OK || a.rows == 0) return st;
    st = bl::check_device();
    if (st != BATCHLAS_OK) return st;
    return bl::hip_status(bl::rmsnorm_quant(static_cast<Type>(type), static_cast<Scale>(scale), a,
                                            stream),
                          "rmsnorm_quant launch");
}

batchlas_status grad_bytes(int type, int64_t rows, int64_t n, int64_t& bytes) {
    BL_REQUIRE(is_float(type), "type must be F32, F16 or BF16");
    batchlas_status st = check_norm_size(rows, n);
    if (st != BATCHLAS_OK) return st;
    st = check_norm_width(n, bl::kGradMaxN);
    if (st != BATCHLAS_OK) return st;
    const int64_t p = rows ? bl::rmsnorm_grad_partials(static_cast<Type>(type), rows, n) : 0;
    bytes = p > 1 ? p * n * 4 : 0;
    return BATCHLAS_OK;
}

batchlas_status do_rmsnorm_grad(int type, const bl::NormGradArgs& a, int64_t bytes,
                                hipStream_t stream) {
    BL_REQUIRE(is_float(type), "type must be F32, F16 or BF16");
    batchlas_status st = check_norm_size(a.rows, a.n);
    if (st != BATCHLAS_OK) return st;
    BL_REQUIRE(a.eps >= 0, "eps must be >= 0");
    BL_REQUIRE(a.lddy >= a.n, "lddy must be >= n");
    BL_REQUIRE(a.ldh >= a.n, "ldh must be >= n");
    BL_REQUIRE(!a.dh || a.lddh >= a.n, "lddh must be >= n");
    BL_REQUIRE(a.lddx >= a.n, "lddx must be >= n");
    BL_REQUIRE(spans(a.rows, a.lddy) && spans(a.rows, a.ldh) && (!a.dh || spans(a.rows, a.lddh)) &&
                   spans(a.rows, a.lddx),
               "rows * leading dimension overflows");
    if (a.rows > 0) {
        BL_POINTER(a.dy, "dy");
        BL_POINTER(a.h, "h");
        BL_POINTER(a.w, "w");
        BL_POINTER(a.dx, "dx");
    }
    const int64_t es = size_of(type);
    BL_REQUIRE(aligned(a.dy, es) && aligned(a.h, es) && aligned(a.w, es) && aligned(a.dh, es) &&
                   aligned(a.dx, es) && aligned(a.dw, 4) && aligned(a.partial, 4),
               "an array is not aligned to its element size");
    int64_t need = 0;
    st = grad_bytes(type, a.rows, a.n, need);
    if (st != BATCHLAS_OK) return st;
    if (a.dw && need) {
        BL_POINTER(a.partial, "workspace");
        BL_REQUIRE(bytes >= need, "workspace_bytes is less than rmsnorm_grad_workspace gives");
    }
    if (a.rows == 0 && !a.dw) return BATCHLAS_OK;
    st = bl::check_device();
    if (st != BATCHLAS_OK) return st;
    return bl::hip_status(bl::rmsnorm_grad(static_cast<Type>(type), a, stream),
                          "rmsnorm_grad launch");
}

batchlas_status do_weight_quant(int type, int format, int64_t group, const bl::WeightQuantArgs& a,
                                hipStream_t stream) {
    BL_REQUIRE(is_float(type), "type must be F32, F16 or BF16");
    batchlas_status st = check_format(format, group);
    if (st != BATCHLAS_OK) return st;
    BL_REQUIRE(a.n >= 1, "n must be >= 1");
    BL_REQUIRE(a.k >= 1, "k must be >= 1");
    BL_REQUIRE(a.n < kMost && a.k <= kMost / 2, "n or k is out of range");
    BL_REQUIRE(a.ldw >= a.k, "ldw must be >= k");
    BL_REQUIRE(!a.values || a.ldv >= a.k, "ldv must be >= k");
    st = check_codes(a.n, a.k, group, a.ldc, a.lds, a.zeros, a.ldz);
    if (st != BATCHLAS_OK) return st;
    BL_REQUIRE(spans(a.n, a.ldw) && (!a.values || spans(a.n, a.ldv)),
               "rows * leading dimension overflows");
    BL_REQUIRE(!a.zeros || format == BATCHLAS_FORMAT_INTEGER, "the float format has no zeros");
    BL_POINTER(a.W, "W");
    BL_POINTER(a.codes, "codes");
    BL_POINTER(a.scales, "scales");
    const int64_t es = size_of(type);
    BL_REQUIRE(aligned(a.codes, 16), "codes must be aligned to 16 bytes");
    BL_REQUIRE(aligned(a.W, es) && aligned(a.values, es) &&
                   (format == BATCHLAS_FORMAT_FLOAT || aligned(a.scales, 2)),
               "an array is not aligned to its element size");
    st = bl::check_device();
    if (st != BATCHLAS_OK) return st;
    return bl::hip_status(bl::weight_quant(static_cast<Type>(type), static_cast<Format>(format),
                                           int(group), a, stream),
                          "weight_quant launch");
}

batchlas_status matvec_bytes(int64_t m, int64_t k, int64_t& bytes) {
    BL_REQUIRE(m >= 0, "m must be >= 0");
    BL_REQUIRE(k >= 1, "k must be >= 1");
    BL_REQUIRE(m < kMost && k <= kMost / 2, "m or k is out of range");
    if (m > (int64_t(1) << 21)) return fail(BATCHLAS_NOT_SUPPORTED, "m is beyond 2^21");
    const int64_t need = bl::weight_matvec_workspace(m, k);
    if (need > (int64_t(1) << 35)) return fail(BATCHLAS_NOT_SUPPORTED, "m * k is beyond 2^34");
    bytes = need;
    return BATCHLAS_OK;
}

batchlas_status do_weight_matvec(int xtype, int xscale, int ytype, int format, int64_t group,
                                 const bl::MatvecArgs& a, void* workspace, int64_t bytes,
                                 hipStream_t stream) {
    const bool eight = xtype == BATCHLAS_TYPE_E4M3;
    BL_REQUIRE(eight || xtype == BATCHLAS_TYPE_F16 || xtype == BATCHLAS_TYPE_BF16,
               "xtype must be F16, BF16 or E4M3");
    BL_REQUIRE(eight ? xscale == BATCHLAS_SCALE_ROW || xscale == BATCHLAS_SCALE_BLOCK
                     : xscale == BATCHLAS_SCALE_NONE,
               "xscale must be ROW or BLOCK for E4M3 and NONE otherwise");
    BL_REQUIRE(is_float(ytype), "ytype must be F32, F16 or BF16");
    batchlas_status st = check_format(format, group);
    if (st != BATCHLAS_OK) return st;
    BL_REQUIRE(a.m >= 0, "m must be >= 0");
    BL_REQUIRE(a.n >= 1, "n must be >= 1");
    BL_REQUIRE(a.k >= 1, "k must be >= 1");
    BL_REQUIRE(a.m < kMost && a.n < kMost && a.k <= kMost / 2, "m, n or k is out of range");
    BL_REQUIRE(a.ldx >= a.k, "ldx must be >= k");
    const bool block = xscale == BATCHLAS_SCALE_BLOCK;
    BL_REQUIRE(!block || a.ldxs >= (a.k + 31) / 32, "ldxs must be >= (k + 31) / 32");
    st = check_codes(a.n, a.k, group, a.ldc, a.lds, a.zeros, a.ldz);
    if (st != BATCHLAS_OK) return st;
    BL_REQUIRE(a.ldy >= a.n, "ldy must be >= n");
    BL_REQUIRE(spans(a.m, a.ldx) && (!block || spans(a.m, a.ldxs)) && spans(a.m, a.ldy),
               "rows * leading dimension overflows");
    BL_REQUIRE(!a.zeros || format == BATCHLAS_FORMAT_INTEGER, "the float format has no zeros");
    if (a.m > 0) {
        BL_POINTER(a.x, "x");
        if (eight) BL_POINTER(a.xscales, "xscales");
        BL_POINTER(a.codes, "codes");
        BL_POINTER(a.scales, "scales");
        BL_POINTER(a.y, "y");
    }
    BL_REQUIRE(aligned(a.codes, 16), "codes must be aligned to 16 bytes");
    BL_REQUIRE(aligned(workspace, 16), "workspace must be aligned to 16 bytes");
    BL_REQUIRE(aligned(a.x, size_of(xtype)) && aligned(a.y, size_of(ytype)) &&
                   (block || aligned(a.xscales, 4)) &&
                   (format == BATCHLAS_FORMAT_FLOAT || aligned(a.scales, 2)),
               "an array is not aligned to its element size");
    int64_t need = 0;
    st = matvec_bytes(a.m, a.k, need);
    if (st != BATCHLAS_OK) return st;
    if (a.n > (int64_t(1) << 24))
        return fail(BATCHLAS_NOT_SUPPORTED, "n is beyond 2^24");
    // offsets within a tile of rows are 32-bit
    if (a.ldx > (int64_t(1) << 27) || a.ldc > (int64_t(1) << 27))
        return fail(BATCHLAS_NOT_SUPPORTED, "ldx or ldc is beyond 2^27");
    if (a.m == 0) return BATCHLAS_OK;
    if (need) {
        BL_POINTER(workspace, "workspace");
        BL_REQUIRE(bytes >= need, "workspace_bytes is less than weight_matvec_workspace gives");
    }
    st = bl::check_device();
    if (st != BATCHLAS_OK) return st;
    return bl::hip_status(bl::weight_matvec(static_cast<Type>(xtype), static_cast<Scale>(xscale),
                                            static_cast<Type>(ytype), static_cast<Format>(format),
                                            int(group), a, workspace, stream),
                          "weight_matvec launch");
}

}  // namespace

extern "C" {

batchlas_status batchlas_rmsnorm_quant(batchlas_type type, batchlas_scale scale, int64_t rows,
                                       int64_t n, const void* x, int64_t ldx, const void* r,
                                       int64_t ldr, const void* w, double eps, void* h,
                                       int64_t ldh, uint8_t* q, int64_t ldq, void* scales,
                                       int64_t lds, batchlas_stream_t stream) {
    return guarded([&] {
        return do_rmsnorm_quant(type, scale,
                                {rows, n, x, ldx, r, ldr, w, float(eps), h, ldh, q, ldq, scales, lds},
                                reinterpret_cast<hipStream_t>(stream));
    });
}

batchlas_status batchlas_rmsnorm_grad(batchlas_type type, int64_t rows, int64_t n, const void* dy,
                                      int64_t lddy, const void* h, int64_t ldh, const void* w,
                                      const void* dh, int64_t lddh, double eps, void* dx,
                                      int64_t lddx, float* dw, void* workspace,
                                      int64_t workspace_bytes, batchlas_stream_t stream) {
    return guarded([&] {
        return do_rmsnorm_grad(type,
                               {rows, n, dy, lddy, h, ldh, w, dh, lddh, float(eps), dx, lddx, dw,
                                static_cast<float*>(workspace)},
                               workspace_bytes, reinterpret_cast<hipStream_t>(stream));
    });
}

batchlas_status batchlas_rmsnorm_grad_workspace(batchlas_type type, int64_t rows, int64_t n,
                                                int64_t* bytes) {
    return guarded([&]() -> batchlas_status {
        BL_POINTER(bytes, "bytes");
        return grad_bytes(type, rows, n, *bytes);
    });
}

batchlas_status batchlas_weight_quant(batchlas_type type, batchlas_format format, int64_t group,
                                      int64_t n, int64_t k, const void* W, int64_t ldw,
                                      uint8_t* codes, int64_t ldc, void* scales, int64_t lds,
                                      uint8_t* zeros, int64_t ldz, void* values, int64_t ldv,
                                      batchlas_stream_t stream) {
    return guarded([&] {
        return do_weight_quant(type, format, group,
                               {n, k, W, ldw, codes, ldc, scales, lds, zeros, ldz, values, ldv},
                               reinterpret_cast<hipStream_t>(stream));
    });
}

batchlas_status batchlas_weight_matvec(batchlas_type xtype, batchlas_scale xscale,
                                       batchlas_type ytype, batchlas_format format, int64_t group,
                                       int64_t m, int64_t n, int64_t k, const void* x,
                                       int64_t ldx, const void* xscales, int64_t ldxs,
                                       const uint8_t* codes, int64_t ldc, const void* scales,
                                       int64_t lds, const uint8_t* zeros, int64_t ldz, void* y,
                                       int64_t ldy, void* workspace, int64_t workspace_bytes,
                                       batchlas_stream_t stream) {
    return guarded([&] {
        return do_weight_matvec(xtype, xscale, ytype, format, group,
                                {m, n, k, x, ldx, xscales, ldxs, codes, ldc, scales, lds, zeros,
                                 ldz, y, ldy},
                                workspace, workspace_bytes, reinterpret_cast<hipStream_t>(stream));
    });
}

batchlas_status batchlas_weight_matvec_workspace(int64_t m, int64_t k, int64_t* bytes) {
    return guarded([&]() -> batchlas_status {
        BL_POINTER(bytes, "bytes");
        return matvec_bytes(m, k, *bytes);
    });
}

}  // extern "C"
