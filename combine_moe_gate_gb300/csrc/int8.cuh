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

// A channel's scale, as s * up with |s| in 2^-126 .. 2^96 (up is 1 but for scales of no model): a sum, in magnitude 0
// or 1 to 2^31, times s is 0 or a normal number, and that times the row's scale loses bits or overflows only where
// the result does.  (Row scale times channel scale first would lose bits below 2^-126 and be an infinity above
// 2^128, which a sum of 0 makes a NaN.)
struct I8Scale { float s, up; };
__device__ __forceinline__ I8Scale i8_scale(float w) {
    const float a = fabsf(w);
    if (a > 7.9228163e28f && a < INFINITY) return {w * 5.421010862427522e-20f, 1.8446744073709552e19f};   // 2^-64, 2^64
    if (a < 1.17549435e-38f) return {w * 1.8446744073709552e19f, 5.421010862427522e-20f};
    return {w, 1.0f};
}
__device__ __forceinline__ float i8_scaled(float sum, float row, const I8Scale &w, float bias) {
    return __fmaf_rn(__fmul_rn(__fmul_rn(sum, w.s), row), w.up, bias);
}

enum I8Act { I8_BIAS = 0, I8_RELU = 1, I8_GELU = 2, I8_SWIGLU = 3 };   // what becomes of a sum

moe_status i8_gemm_launch(const void *x16, const float *x_scale, const SortedRows &so, const void *w,
                          const float *w_scale, const void *w3, const float *w3_scale, const void *bias, int epi,
                          bool f32, int e, int K, int n_out, void *out, int32_t *st, cudaStream_t stream);

}  // namespace moe
