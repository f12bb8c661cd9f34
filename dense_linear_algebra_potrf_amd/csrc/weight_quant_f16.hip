// Rounding of weights to 4 bits for element type f16 (one translation unit per
// type).
#include "weight_quant_impl.hpp"

namespace bl {

hipError_t weight_quant_f16(Format f, int group, const WeightQuantArgs& a, hipStream_t s) {
    return weight_quant_detail::weight_quant_t<layer::f16>(f, group, a, s);
}

}  // namespace bl
