// Products with 4-bit weights for x of kind BF16 (one translation unit per kind).
#include "weight_matvec_impl.hpp"

namespace bl {

hipError_t weight_matvec_bf16(Type yt, Format f, int group, const MatvecArgs& a, hipStream_t s) {
    return weight_matvec_detail::weight_matvec_t<weight_matvec_detail::X::BF16>(yt, f, group, a, s);
}

}  // namespace bl
