// RMS norm to 8 bits and its gradient for element type bf16 (one translation
// unit per type).
#include "rmsnorm_impl.hpp"

namespace bl {

hipError_t rmsnorm_quant_bf16(Scale sc, const NormQuantArgs& a, hipStream_t s) {
    return rmsnorm_detail::rmsnorm_quant_t<layer::bf16>(sc, a, s);
}
hipError_t rmsnorm_grad_bf16(const NormGradArgs& a, hipStream_t s) {
    return rmsnorm_detail::rmsnorm_grad_t<layer::bf16>(a, s);
}
int64_t rmsnorm_grad_partials_bf16(int64_t rows, int64_t n) {
    return rmsnorm_detail::grad_partials<layer::bf16>(rows, n);
}

}  // namespace bl
