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

#define BL_DECLARE_PACK(suf) hipError_t weight_pack_##suf(Format f, const MatvecArgs& a, void* packed, hipStream_t s);
BL_DECLARE_PACK(bf16)
BL_DECLARE_PACK(f16)
BL_DECLARE_PACK(f8block)
BL_DECLARE_PACK(f8row)
#undef BL_DECLARE_PACK
#define BL_DECLARE_MANY(suf)                                                                          \
    hipError_t weight_many_##suf(bool eight, Type yt, Format f, int group, const MatvecArgs& a,       \
                                 const void* packed, hipStream_t s);
BL_DECLARE_MANY(bf16)
BL_DECLARE_MANY(f16)
#undef BL_DECLARE_MANY

int64_t weight_matvec_workspace(int64_t m, int64_t k) {
    // 16-bit floats of whole tiles of 16 rows and 128 columns
    return m <= kFewRows ? 0 : (m + 15) / 16 * ((k + 127) / 128) * 4096;
}

hipError_t weight_matvec(Type xt, Scale xs, Type yt, Format f, int group, const MatvecArgs& a, void* workspace,
                         hipStream_t s) {
    const bool block = xs == Scale::BLOCK;
    if (a.m <= kFewRows) {
        if (xt == Type::BF16) return weight_matvec_bf16(yt, f, group, a, s);
        if (xt == Type::F16) return weight_matvec_f16(yt, f, group, a, s);
        return block ? weight_matvec_f8block(yt, f, group, a, s) : weight_matvec_f8row(yt, f, group, a, s);
    }
    const hipError_t e = xt == Type::BF16  ? weight_pack_bf16(f, a, workspace, s)
                         : xt == Type::F16 ? weight_pack_f16(f, a, workspace, s)
                         : block           ? weight_pack_f8block(f, a, workspace, s)
                                           : weight_pack_f8row(f, a, workspace, s);
    if (e != hipSuccess) return e;
    const bool eight = xt == Type::E4M3;
    return xt == Type::BF16 || (eight && block) ? weight_many_bf16(eight, yt, f, group, a, workspace, s)
                                                : weight_many_f16(eight, yt, f, group, a, workspace, s);
}

}  // namespace bl
