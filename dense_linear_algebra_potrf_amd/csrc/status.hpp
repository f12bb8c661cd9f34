// Status, error text and device check shared by the C-ABI translation units
// (host only).
#pragma once

#include <hip/hip_runtime.h>

#include <exception>
#include <string>

#include "../../include/batchlas.h"

namespace bl {

// Records the message for batchlas_last_error (per host thread) and returns s.
batchlas_status fail(batchlas_status s, const std::string& msg);
const char* last_error();

// The library carries gfx950 code only; refuse other devices up front.
batchlas_status check_device();

batchlas_status hip_status(hipError_t e, const char* what);

// No C++ exception crosses the C interface.
template <typename F>
batchlas_status guarded(F&& f) {
    try {
        return f();
    } catch (const std::exception& e) {
        return fail(BATCHLAS_INTERNAL, std::string("internal error: ") + e.what());
    } catch (...) {
        return fail(BATCHLAS_INTERNAL, "internal error");
    }
}

inline bool mul_ok(int64_t a, int64_t b, int64_t& out) { return !__builtin_mul_overflow(a, b, &out); }

}  // namespace bl
