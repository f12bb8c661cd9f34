// Dispatch of the 8-bit-integer layer operators by element type (host only).
#include "integer.hpp"

namespace bl {

#define BL_DECLARE_INTEGER(suf)                                                               \
    hipError_t int8_quant_##suf(const Int8QuantArgs& a, hipStream_t s);                       \
    hipError_t int8_matmul_##suf(const Int8MatmulArgs& a, hipStream_t s);                     \
    hipError_t block_norm_##suf(Scale sc, const BlockNormArgs& a, hipStream_t s);             \
    hipError_t block_norm_grad_##suf(const BlockGradArgs& a, hipStream_t s);                  \
    int64_t block_norm_grad_floats_##suf(int64_t rows, int64_t n, int64_t per);
BL_DECLARE_INTEGER(f32)
BL_DECLARE_INTEGER(f16)
BL_DECLARE_INTEGER(bf16)
#undef BL_DECLARE_INTEGER

#define BL_BY_TYPE(call)                    \
    switch (t) {                            \
    case Type::F32: return call(f32);       \
    case Type::F16: return call(f16);       \
    case Type::BF16: return call(bf16);     \
    case Type::E4M3: break;                 \
    }

hipError_t int8_quant(Type t, const Int8QuantArgs& a, hipStream_t s) {
#define BL_CALL(suf) int8_quant_##suf(a, s)
    BL_BY_TYPE(BL_CALL)
#undef BL_CALL
    return hipErrorInvalidValue;
}

hipError_t int8_matmul(Type t, const Int8MatmulArgs& a, hipStream_t s) {
#define BL_CALL(suf) int8_matmul_##suf(a, s)
    BL_BY_TYPE(BL_CALL)
#undef BL_CALL
    return hipErrorInvalidValue;
}

hipError_t block_norm(Type t, Scale sc, const BlockNormArgs& a, hipStream_t s) {
#define BL_CALL(suf) block_norm_##suf(sc, a, s)
    BL_BY_TYPE(BL_CALL)
#undef BL_CALL
    return hipErrorInvalidValue;
}

hipError_t block_norm_grad(Type t, const BlockGradArgs& a, hipStream_t s) {
#define BL_CALL(suf) block_norm_grad_##suf(a, s)
    BL_BY_TYPE(BL_CALL)
#undef BL_CALL
    return hipErrorInvalidValue;
}

int64_t block_norm_grad_floats(Type t, int64_t rows, int64_t n, int64_t per) {
#define BL_CALL(suf) block_norm_grad_floats_##suf(rows, n, per)
    BL_BY_TYPE(BL_CALL)
#undef BL_CALL
    return 0;
}

}  // namespace bl
