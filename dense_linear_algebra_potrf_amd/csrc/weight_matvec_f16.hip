// Products with 4-bit weights for x of kind F16 (one translation unit per kind).
#include "weight_matvec_impl.hpp"

namespace bl {

hipError_t weight_matvec_f16(Type yt, Format f, int group, const MatvecArgs& a, hipStream_t s) {
    return weight_matvec_detail::weight_matvec_t<weight_matvec_detail::X::F16>(yt, f, group, a, s);
}

}  // namespace bl
