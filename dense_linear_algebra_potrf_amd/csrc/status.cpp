// Status, error text and device check of the C ABI (host only).
#include "status.hpp"

#include <atomic>
#include <cstring>

namespace bl {

namespace {
thread_local std::string g_last_error;
}

batchlas_status fail(batchlas_status s, const std::string& msg) {
    g_last_error = msg;
    return s;
}

const char* last_error() { return g_last_error.c_str(); }

batchlas_status check_device() {
    static std::atomic<int> state[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess)
        return fail(BATCHLAS_HIP_ERROR, "hipGetDevice failed");
    if (dev < 0 || dev >= 64) return fail(BATCHLAS_NOT_SUPPORTED, "device index out of range");
    int s = state[dev].load(std::memory_order_acquire);
    if (s == 0) {
        hipDeviceProp_t prop;
        if (hipGetDeviceProperties(&prop, dev) != hipSuccess)
            return fail(BATCHLAS_HIP_ERROR, "hipGetDeviceProperties failed");
        s = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
        state[dev].store(s, std::memory_order_release);
    }
    if (s != 1) return fail(BATCHLAS_NOT_SUPPORTED, "this library is built for gfx950 only");
    return BATCHLAS_OK;
}

batchlas_status hip_status(hipError_t e, const char* what) {
    if (e == hipSuccess) return BATCHLAS_OK;
    return fail(BATCHLAS_HIP_ERROR, std::string(what) + ": " + hipGetErrorString(e));
}

}  // namespace bl
