// Correctly rounded reciprocals and quotients by fused corrections of an
// approximation (Markstein, "Computation of elementary functions on the IBM
// RISC System/6000 processor", 1990: with r = fma(-b, y, 1) exact, fma(r, y, y)
// rounds 1/b correctly; likewise a quotient from a faithful one).  They leave
// out the range checks of the general operations, so operands and results have
// to stay well inside the normal numbers.
#pragma once

#include "common.cuh"

namespace moe {

// 1 / x for 2^-120 <= x <= 2^126 (compared with __frcp_rn for each of these
// floats in tests/test_gpu_exact.py).
__device__ __forceinline__ float rcp_mid(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return __fmaf_rn(__fmaf_rn(-x, y, 1.0f), y, y);
}

// a / b with y = 1 / b rounded, for a = 0 or |a| >= 2^-100, and a quotient
// between 2^-120 and 2^120 (sampled against __fdiv_rn there, to both ends).
__device__ __forceinline__ float div_mid(float a, float b, float y) {
    float q = __fmul_rn(a, y);
    q = __fmaf_rn(__fmaf_rn(-q, b, a), y, q);
    return __fmaf_rn(__fmaf_rn(-q, b, a), y, q);
}

}  // namespace moe
