// Dispatch of the low-bit layer operators by element type (host only).
#include "layer.hpp"

namespace bl {

#define BL_DECLARE_LAYER(suf)                                                                 \
    hipError_t rmsnorm_quant_##suf(Scale sc, const NormQuantArgs& a, hipStream_t s);          \
    hipError_t rmsnorm_grad_##suf(const NormGradArgs& a, hipStream_t s);                      \
    int64_t rmsnorm_grad_partials_##suf(int64_t rows, int64_t n);                             \
    hipError_t weight_quant_##suf(Format f, int group, const WeightQuantArgs& a, hipStream_t s);
BL_DECLARE_LAYER(f32)
BL_DECLARE_LAYER(f16)
BL_DECLARE_LAYER(bf16)
#undef BL_DECLARE_LAYER

#define BL_BY_TYPE(call)                    \
    switch (t) {                            \
    case Type::F32: return call(f32);       \
    case Type::F16: return call(f16);       \
    case Type::BF16: return call(bf16);     \
    case Type::E4M3: break;                 \
    }

hipError_t rmsnorm_quant(Type t, Scale sc, const NormQuantArgs& a, hipStream_t s) {
#define BL_CALL(suf) rmsnorm_quant_##suf(sc, a, s)
    BL_BY_TYPE(BL_CALL)
#undef BL_CALL
    return hipErrorInvalidValue;
}

hipError_t rmsnorm_grad(Type t, const NormGradArgs& a, hipStream_t s) {
#define BL_CALL(suf) rmsnorm_grad_##suf(a, s)
    BL_BY_TYPE(BL_CALL)
#undef BL_CALL
    return hipErrorInvalidValue;
}

int64_t rmsnorm_grad_partials(Type t, int64_t rows, int64_t n) {
#define BL_CALL(suf) rmsnorm_grad_partials_##suf(rows, n)
    BL_BY_TYPE(BL_CALL)
#undef BL_CALL
    return 0;
}

hipError_t weight_quant(Type t, Format f, int group, const WeightQuantArgs& a, hipStream_t s) {
#define BL_CALL(suf) weight_quant_##suf(f, group, a, s)
    BL_BY_TYPE(BL_CALL)
#undef BL_CALL
    return hipErrorInvalidValue;
}

#define BL_DECLARE_MATVEC(suf) \
    hipError_t weight_matvec_##suf(Type yt, Format f, int group, const MatvecArgs& a, hipStream_t s);
BL_DECLARE_MATVEC(bf16)
BL_DECLARE_MATVEC(f16)
BL_DECLARE_MATVEC(f8block)
BL_DECLARE_MATVEC(f8row)
#undef BL_DECLARE_MATVEC

#define BL_DECLARE_MANY(suf)                                                                           \
    hipError_t weight_many_##suf(Type xt, Scale xs, Type yt, const MatvecArgs& a, void* workspace, hipStream_t s);
BL_DECLARE_MANY(int32)
BL_DECLARE_MANY(int64)
BL_DECLARE_MANY(int128)
BL_DECLARE_MANY(fp4)
#undef BL_DECLARE_MANY
hipError_t weight_pack(Type xt, Scale xs, Format f, const MatvecArgs& a, void* workspace, hipStream_t s);

hipError_t weight_matvec(Type xt, Scale xs, Type yt, Format f, int group, const MatvecArgs& a, void* workspace,
                         hipStream_t s) {
    if (a.m <= kFewRows) {
        if (xt == Type::BF16) return weight_matvec_bf16(yt, f, group, a, s);
        if (xt == Type::F16) return weight_matvec_f16(yt, f, group, a, s);
        return xs == Scale::BLOCK ? weight_matvec_f8block(yt, f, group, a, s) : weight_matvec_f8row(yt, f, group, a, s);
    }
    const hipError_t e = weight_pack(xt, xs, f, a, workspace, s);
    if (e != hipSuccess) return e;
    if (f == Format::FLOAT) return weight_many_fp4(xt, xs, yt, a, workspace, s);
    return group == 32   ? weight_many_int32(xt, xs, yt, a, workspace, s)
           : group == 64 ? weight_many_int64(xt, xs, yt, a, workspace, s)
                         : weight_many_int128(xt, xs, yt, a, workspace, s);
}

}  // namespace bl
