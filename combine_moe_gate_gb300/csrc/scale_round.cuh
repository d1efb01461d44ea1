// A 16-byte chunk of a row times an fp32 gate, each product rounded once to the row's type.
#pragma once

#include "common.cuh"

namespace moe {

// g * d (fp32 times a bf16 value) correctly rounded to bf16, one rounding of
// the exact product, by round to odd: the product truncated to fp32 with its
// last bit set when it was inexact keeps 16 bits beyond bf16's precision, so
// rounding that to bf16 (nearest even) rounds the exact product once.  err is
// the exact remainder g*d - p (at most 8 significant bits).  Infinities and
// NaNs keep their bits.
__device__ __forceinline__ float mul_round_odd(float g, float d) {
    const float p = __fmul_rz(g, d);
    const float err = __fmaf_rn(g, d, -p);
    uint32_t u = __float_as_uint(p);
    if (err != 0.0f && (u & 0x7F800000u) != 0x7F800000u) u |= 1u;
    return __uint_as_float(u);
}

// Two of them, packed (lo in the low half).
__device__ __forceinline__ uint32_t mul_round_bf16x2(float g, float lo, float hi) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(mul_round_odd(g, lo), mul_round_odd(g, hi));
    return *reinterpret_cast<const uint32_t *>(&r);
}

template <typename T> struct ScaleRound;
template <> struct ScaleRound<float> {
    __device__ __forceinline__ static V16 apply(float g, const V16 &d) {
        V16 o;
#pragma unroll
        for (int i = 0; i < 4; i++) o.w[i] = __float_as_uint(__fmul_rn(g, __uint_as_float(d.w[i])));
        return o;
    }
};
template <> struct ScaleRound<__nv_bfloat16> {
    __device__ __forceinline__ static V16 apply(float g, const V16 &d) {
        V16 o;
#pragma unroll
        for (int i = 0; i < 4; i++) o.w[i] = mul_round_bf16x2(g, bf16lo(d.w[i]), bf16hi(d.w[i]));
        return o;
    }
};

}  // namespace moe
