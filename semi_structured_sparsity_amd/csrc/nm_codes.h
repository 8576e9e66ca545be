// One-byte codes of quantised activations: the e4m3 code of a value and the quotient by a row's
// scale, correctly rounded.
#pragma once

#include "nm_internal.h"

namespace nm {

// OCP e4m3 code of v, |v| <= 448, finite: nearest code, ties to even.  With t the
// biased f32 exponent of |v| raised to that of 2^-6 (below it the codes are the
// subnormals m 2^-9), y = |v| 2^(3 - (t - 127)) is exact and lies in [8, 16) in a normal
// binade, [0, 8) in the subnormal one; rint(y) (ties to even) is the code's 3-bit
// mantissa plus 8, counted from the binade's first code (t - 121) * 8 - 8, and a value
// that rounds up to 16 carries into the next binade as the code arithmetic requires.
// -0 keeps its sign.
__device__ __forceinline__ uint32_t e4m3_code(float v) {
    const uint32_t bits = __builtin_bit_cast(uint32_t, v);
    const float a = __builtin_bit_cast(float, bits & 0x7fffffffu);
    const int t = max((int)((bits >> 23) & 0xffu), 121);
    const uint32_t r = (uint32_t)rintf(__builtin_ldexpf(a, 130 - t));
    return ((bits >> 24) & 0x80u) | ((uint32_t)(t - 121) * 8u + r);
}

// x / s rounded to nearest f32 for one row's scale s (finite, > 0) without a division per
// element: s and x are scaled by the same power of two so that s lies in [1, 2) (exact),
// r = RN(1 / s) is formed once, q0 = RN(x r) is within an ulp of x / s, the residual
// x - q0 s is exact in one fma, and RN(q0 + (x - q0 s) r) is RN(x / s) (Markstein's
// correction step).  The quotient carries x's sign (also for x = -0).  A quotient that
// the scaling pushes below the normal range is below 2^-125 and gives code 0 either way.
template <bool B>
struct BoolTag {
    static constexpr bool value = B;
};

struct RowDiv {
    int k;       // the scaling exponent
    float s1;    // s 2^k, in [1, 2)
    float r1;    // RN(1 / s1)
};
__device__ __forceinline__ RowDiv row_div(float s) {
    RowDiv d;
    d.k = 1 - __builtin_amdgcn_frexp_expf(s);
    d.s1 = __builtin_ldexpf(s, d.k);
    d.r1 = __fdiv_rn(1.0f, d.s1);
    return d;
}
__device__ __forceinline__ float row_quot(float x, const RowDiv& d) {
    const float xs = __builtin_ldexpf(x, d.k);
    const float q0 = xs * d.r1;
    const float rem = __builtin_fmaf(-q0, d.s1, xs);
    return __builtin_copysignf(__builtin_fmaf(rem, d.r1, q0), x);
}

}  // namespace nm
