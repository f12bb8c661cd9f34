// Products of 8-bit integers with outputs of type bf16 (one translation unit per type).
#include "int8_matmul_impl.hpp"

namespace bl {

hipError_t int8_matmul_bf16(const Int8MatmulArgs& a, hipStream_t s) { return int8_matmul_detail::int8_matmul_t<layer::bf16>(a, s); }

}  // namespace bl
