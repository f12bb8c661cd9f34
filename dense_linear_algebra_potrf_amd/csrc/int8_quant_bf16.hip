// Rounding to 8-bit integers for element type bf16 (one translation unit per type).
#include "int8_quant_impl.hpp"

namespace bl {

hipError_t int8_quant_bf16(const Int8QuantArgs& a, hipStream_t s) { return int8_quant_detail::int8_quant_t<layer::bf16>(a, s); }

}  // namespace bl
