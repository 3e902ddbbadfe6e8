// Checks that the C-ABI front ends of the layer operators share: sizes, strides,
// types and the overlap of buffers, on the host.
#pragma once

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "kda.h"
#include "layer_internal.h"

namespace kda {
namespace layer {

inline bool mul_ok(int64_t a, int64_t b, int64_t *r) { return !__builtin_mul_overflow(a, b, r); }
inline bool add_ok(int64_t a, int64_t b, int64_t *r) { return !__builtin_add_overflow(a, b, r); }

inline bool bf16_or_fp32(int32_t d) { return d == KDA_DTYPE_BF16 || d == KDA_DTYPE_FP32; }
inline int64_t bytes_of(int32_t d) { return d == KDA_DTYPE_BF16 ? 2 : 4; }
inline bool flag(int32_t v) { return v == 0 || v == 1; }
inline bool valid_eps(double e) { return std::isfinite(e) && e >= 0.0; }
// The kernels multiply in fp32: a scale has to be 0 or normal there.
inline bool fp32_scale(double s) { return s == 0.0 || std::isnormal(static_cast<float>(s)); }

// Byte range of a buffer.
struct Span {
    uintptr_t lo = 0, hi = 0;
    bool overlaps(const Span &o) const { return lo < o.hi && o.lo < hi; }
};
inline Span span(const void *p, int64_t bytes)
{
    Span s;
    if (p && bytes > 0) {
        s.lo = reinterpret_cast<uintptr_t>(p);
        s.hi = s.lo + static_cast<uintptr_t>(bytes);
    }
    return s;
}
inline bool any_overlap(const Span &out, std::initializer_list<Span> inputs)
{
    for (const Span &s : inputs)
        if (out.overlaps(s))
            return true;
    return false;
}

inline bool misaligned(const void *p, uintptr_t a) { return p != nullptr && reinterpret_cast<uintptr_t>(p) % a != 0; }

// Bytes from the first to past the last element of `outer` x `inner` rows of
// `width` adjacent elements with the given strides; false on a negative
// stride or overflow.
inline bool extent(int64_t outer, int64_t stride_o, int64_t inner, int64_t stride_i, int64_t width, int64_t elem,
            int64_t *bytes)
{
    int64_t a = 0, b = 0, n = 0;
    if (stride_o < 0 || stride_i < 0)
        return false;
    if (outer == 0 || inner == 0 || width == 0) {
        *bytes = 0;
        return true;
    }
    return mul_ok(outer - 1, stride_o, &a) && mul_ok(inner - 1, stride_i, &b) && add_ok(a, b, &n) &&
           add_ok(n, width, &n) && mul_ok(n, elem, bytes);
}

// The batch of sequences a call names: KDA_OK, or what is wrong with it.
inline kda_status check_seqs(const int64_t *cu, int64_t num_seqs, int64_t B, int64_t T, Seqs *s)
{
    if (B < 1 || T < 0 || T > INT32_MAX)
        return KDA_ERR_SIZE;
    if (cu && (B != 1 || num_seqs < 0))
        return KDA_ERR_VARLEN_BATCH;
    s->cu = cu;
    s->N = cu ? num_seqs : B;
    s->T = T;
    return s->N > INT32_MAX ? KDA_ERR_SIZE : KDA_OK;
}

inline kda_status check_states(const void *init, int32_t init_dtype, const void *fin, int32_t fin_dtype)
{
    if (init && !bf16_or_fp32(init_dtype))
        return init_dtype == KDA_DTYPE_NONE ? KDA_ERR_NULL_POINTER : KDA_ERR_STATE_DTYPE;
    if (fin && !bf16_or_fp32(fin_dtype))
        return fin_dtype == KDA_DTYPE_NONE ? KDA_ERR_NULL_POINTER : KDA_ERR_STATE_DTYPE;
    return init && fin && init_dtype != fin_dtype ? KDA_ERR_STATE_DTYPE : KDA_OK;
}

inline kda_status launched(hipError_t e)
{
    return e == hipSuccess ? KDA_OK : e == hipErrorInvalidConfiguration ? KDA_ERR_SIZE : KDA_ERR_LAUNCH;
}

}  // namespace layer
}  // namespace kda
