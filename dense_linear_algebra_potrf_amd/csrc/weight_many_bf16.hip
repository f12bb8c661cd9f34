// Products of many rows with 4-bit weights where x is multiplied in bf16 (one
// translation unit per type).
#include "weight_many_impl.hpp"

namespace bl {

using weight_matvec_detail::X;

hipError_t weight_pack_bf16(Format f, const MatvecArgs& a, void* packed, hipStream_t s) {
    return weight_matvec_detail::pack_t<X::BF16>(f, a, static_cast<weight_matvec_detail::u32x4*>(packed), s);
}
hipError_t weight_pack_f8block(Format f, const MatvecArgs& a, void* packed, hipStream_t s) {
    return weight_matvec_detail::pack_t<X::F8_BLOCK>(f, a, static_cast<weight_matvec_detail::u32x4*>(packed), s);
}
hipError_t weight_many_bf16(bool eight, Type yt, Format f, int group, const MatvecArgs& a, const void* packed, hipStream_t s) {
    return weight_matvec_detail::weight_many_t<false>(eight ? X::F8_BLOCK : X::BF16, yt, f, group, a,
                                                      static_cast<const weight_matvec_detail::u32x4*>(packed), s);
}

}  // namespace bl
