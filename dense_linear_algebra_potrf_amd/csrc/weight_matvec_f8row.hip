// Products with 4-bit weights for x of kind F8_ROW (one translation unit per kind).
#include "weight_matvec_impl.hpp"

namespace bl {

hipError_t weight_matvec_f8row(Type yt, Format f, int group, const MatvecArgs& a, hipStream_t s) {
    return weight_matvec_detail::weight_matvec_t<weight_matvec_detail::X::F8_ROW>(yt, f, group, a, s);
}

}  // namespace bl
