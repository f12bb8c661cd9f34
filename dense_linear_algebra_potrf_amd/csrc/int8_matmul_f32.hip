// Products of 8-bit integers with outputs of type f32 (one translation unit per type).
#include "int8_matmul_impl.hpp"

namespace bl {

hipError_t int8_matmul_f32(const Int8MatmulArgs& a, hipStream_t s) { return int8_matmul_detail::int8_matmul_t<float>(a, s); }

}  // namespace bl
