// Norms around a block and their gradient for element type f32 (one translation
// unit per type).
#include "block_norm_impl.hpp"

namespace bl {

hipError_t block_norm_f32(Scale sc, const BlockNormArgs& a, hipStream_t s) {
    return block_norm_detail::block_norm_t<float>(sc, a, s);
}
hipError_t block_norm_grad_f32(const BlockGradArgs& a, hipStream_t s) {
    return block_norm_detail::block_norm_grad_t<float>(a, s);
}
int64_t block_norm_grad_floats_f32(int64_t rows, int64_t n, int64_t per) {
    return block_norm_detail::block_norm_grad_floats_t<float>(rows, n, per);
}

}  // namespace bl
