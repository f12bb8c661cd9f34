// Norms around a block and their gradient for element type bf16 (one translation
// unit per type).
#include "block_norm_impl.hpp"

namespace bl {

hipError_t block_norm_bf16(Scale sc, const BlockNormArgs& a, hipStream_t s) {
    return block_norm_detail::block_norm_t<layer::bf16>(sc, a, s);
}
hipError_t block_norm_grad_bf16(const BlockGradArgs& a, hipStream_t s) {
    return block_norm_detail::block_norm_grad_t<layer::bf16>(a, s);
}
int64_t block_norm_grad_floats_bf16(int64_t rows, int64_t n, int64_t per) {
    return block_norm_detail::block_norm_grad_floats_t<layer::bf16>(rows, n, per);
}

}  // namespace bl
