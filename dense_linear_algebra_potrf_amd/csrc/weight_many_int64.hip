// Products of many rows with 4-bit integers in groups of 64 (one translation unit per form).
#include "weight_many_impl.hpp"

namespace bl {

hipError_t weight_many_int64(Type xt, Scale xs, Type yt, const MatvecArgs& a, void* workspace, hipStream_t s) {
    return weight_matvec_detail::weight_many_t<Format::INTEGER, 64>(weight_matvec_detail::kind_of(xt, xs), yt, a, workspace, s);
}

}  // namespace bl
