// Launchers of the 8-bit integer rows' kernels (int8.cu; the tensor-core product is ffn_int8.cuh).
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {

// Four 8-bit integers -> fp16 pairs: 1024 + (b + 128) is the fp16 number 0x6400 | (b ^ 0x80).
__device__ __forceinline__ void i8_widen(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t l = __byte_perm(u, 0x64646464u, 0x4140), h = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 off = __half2half2(__ushort_as_half(0x6480));   // 1152
    const __half2 a = __hsub2(*reinterpret_cast<const __half2 *>(&l), off);
    const __half2 b = __hsub2(*reinterpret_cast<const __half2 *>(&h), off);
    lo = *reinterpret_cast<const uint32_t *>(&a);
    hi = *reinterpret_cast<const uint32_t *>(&b);
}

// The two scales' product is formed first where it is a normal number (or a factor is 0, infinite or a NaN, which
// it shows as well); elsewhere it would lose its bits, or be an infinity that a sum of 0 makes a NaN, so there all
// factors meet in 64 bits, where the scales' product is exact.
__device__ __forceinline__ bool i8_scales_ok(float a, float b) {   // a, b: magnitudes
    const float p = a * b;
    return (p >= 1.17549435e-38f && p <= 3.40282347e38f) || !(a > 0.0f && a < INFINITY) || !(b > 0.0f && b < INFINITY);
}
__device__ __forceinline__ float i8_scaled_far(double sum, float a, float b, float bias) {
    return (float)fma(sum, (double)a * (double)b, (double)bias);
}

enum I8Act { I8_BIAS = 0, I8_RELU = 1, I8_GELU = 2, I8_SWIGLU = 3 };   // what becomes of a sum

moe_status i8_gemm_launch(const void *x16, const float *x_scale, const SortedRows &so, const void *w,
                          const float *w_scale, const void *w3, const float *w3_scale, const void *bias, int epi,
                          bool f32, int e, int K, int n_out, void *out, int32_t *st, cudaStream_t stream);

}  // namespace moe
