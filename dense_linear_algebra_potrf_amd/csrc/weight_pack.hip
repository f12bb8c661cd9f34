// Layout of x for products of many rows with 4-bit weights.
#include "weight_many_impl.hpp"

namespace bl {

hipError_t weight_pack(Type xt, Scale xs, Format f, const MatvecArgs& a, void* workspace, hipStream_t s) {
    using namespace weight_matvec_detail;
    switch (kind_of(xt, xs)) {
    case X::BF16: return pack_t<X::BF16>(f, a, workspace, s);
    case X::F16: return pack_t<X::F16>(f, a, workspace, s);
    case X::F8_BLOCK: return pack_t<X::F8_BLOCK>(f, a, workspace, s);
    case X::F8_ROW: return pack_t<X::F8_ROW>(f, a, workspace, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace bl
