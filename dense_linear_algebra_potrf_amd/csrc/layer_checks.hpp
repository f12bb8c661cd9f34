// Argument checks shared by the C-ABI files of the layer operators (host only).
#pragma once

#include <cstdint>
#include <string>

#include "status.hpp"

namespace bl {

inline batchlas_status invalid(const char* msg) { return fail(BATCHLAS_INVALID_VALUE, msg); }

inline int64_t size_of(int t) { return t == BATCHLAS_TYPE_F32 ? 4 : t == BATCHLAS_TYPE_E4M3 ? 1 : 2; }

inline bool is_float(int t) {
    return t == BATCHLAS_TYPE_F32 || t == BATCHLAS_TYPE_F16 || t == BATCHLAS_TYPE_BF16;
}

inline bool aligned(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// A row-major matrix whose last element's offset stays within 2^60 elements.
inline bool spans(int64_t rows, int64_t ld) {
    int64_t total = 0;
    return mul_ok(rows, ld, total) && total < (int64_t(1) << 60);
}

#define BL_REQUIRE(cond, msg) \
    do {                      \
        if (!(cond)) return bl::invalid(msg); \
    } while (0)
#define BL_POINTER(p, name) \
    do {                    \
        if (!(p)) return bl::fail(BATCHLAS_NULL_POINTER, name " is NULL"); \
    } while (0)

constexpr int64_t kMost = int64_t(1) << 31;

inline batchlas_status check_norm_size(int64_t rows, int64_t n) {
    BL_REQUIRE(rows >= 0, "rows must be >= 0");
    BL_REQUIRE(n >= 1, "n must be >= 1");
    BL_REQUIRE(rows < kMost && n < kMost, "rows or n is out of range");
    return BATCHLAS_OK;
}

inline batchlas_status check_norm_width(int64_t n, int64_t most) {
    if (n > most)
        return fail(BATCHLAS_NOT_SUPPORTED,
                    "rows of at most " + std::to_string(most) + " columns are served");
    return BATCHLAS_OK;
}

}  // namespace bl
