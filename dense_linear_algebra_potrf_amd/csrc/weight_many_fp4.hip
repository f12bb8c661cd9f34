// Products of many rows with 4-bit floats (one translation unit per form).
#include "weight_many_impl.hpp"

namespace bl {

hipError_t weight_many_fp4(Type xt, Scale xs, Type yt, const MatvecArgs& a, void* workspace, hipStream_t s) {
    return weight_matvec_detail::weight_many_t<Format::FLOAT, 32>(weight_matvec_detail::kind_of(xt, xs), yt, a, workspace, s);
}

}  // namespace bl
