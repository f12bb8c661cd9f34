// RMS norm to 8 bits and its gradient for element type float (one translation
// unit per type).
#include "rmsnorm_impl.hpp"

namespace bl {

hipError_t rmsnorm_quant_f32(Scale sc, const NormQuantArgs& a, hipStream_t s) {
    return rmsnorm_detail::rmsnorm_quant_t<float>(sc, a, s);
}
hipError_t rmsnorm_grad_f32(const NormGradArgs& a, hipStream_t s) {
    return rmsnorm_detail::rmsnorm_grad_t<float>(a, s);
}
int64_t rmsnorm_grad_partials_f32(int64_t rows, int64_t n) {
    return rmsnorm_detail::grad_partials<float>(rows, n);
}

}  // namespace bl
