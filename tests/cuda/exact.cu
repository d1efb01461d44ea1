// csrc/exact.cuh against CUDA's own operations, and CUDA's expf for the tests'
// fp32 restatements.
#include "exact.cuh"

namespace {

__device__ __forceinline__ uint32_t mix(uint32_t x) {
    x ^= x >> 16; x *= 0x7feb352du; x ^= x >> 15; x *= 0x846ca68bu; return x ^ (x >> 16);
}

// rcp_mid of the first n mantissas at one exponent (one float per thread).
__global__ void rcp_kernel(uint32_t exponent, uint32_t n, unsigned long long *bad) {
    const uint32_t m = blockIdx.x * blockDim.x + threadIdx.x;
    if (m >= n) return;
    const float x = __uint_as_float(exponent << 23 | m);
    if (__float_as_uint(moe::rcp_mid(x)) != __float_as_uint(__frcp_rn(x))) atomicAdd(bad, 1ull);
}

// A mantissa: any, or one of those near a power of two.
__device__ __forceinline__ uint32_t mantissa(uint32_t h) {
    const uint32_t m = mix(h) & 0x7fffffu;
    return (h & 3u) == 0 ? m & 0xffu : (h & 3u) == 1 ? 0x7fffffu - (m & 0xffu) : m;
}

// div_mid of `per` pairs a thread, exponents uniform in [a0, a1] and [b0, b1].
__global__ void div_kernel(uint32_t seed, int per, int a0, int a1, int b0, int b1, unsigned long long *bad) {
    const uint32_t t = blockIdx.x * blockDim.x + threadIdx.x;
    for (int i = 0; i < per; i++) {
        const uint32_t h = mix(t + mix(seed * 4096u + i)), u = mix(h + 1u), v = mix(h + 2u);
        const float a = (h & 63u) == 63u ? 0.0f
                                         : __uint_as_float((uint32_t)(127 + a0 + (int)(u % (uint32_t)(a1 - a0 + 1))) << 23 | mantissa(v));
        const float b = __uint_as_float((uint32_t)(127 + b0 + (int)(mix(u) % (uint32_t)(b1 - b0 + 1))) << 23 | mantissa(mix(v)));
        if (__float_as_uint(moe::div_mid(a, b, __frcp_rn(b))) != __float_as_uint(__fdiv_rn(a, b))) atomicAdd(bad, 1ull);
    }
}

__global__ void exp_kernel(const float *x, float *y, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) y[i] = expf(x[i]);
}

}  // namespace

extern "C" {

int exact_rcp(uint32_t exponent, uint32_t n, unsigned long long *bad) {
    rcp_kernel<<<(n + 1023) / 1024, 1024>>>(exponent, n, bad);
    return (int)cudaGetLastError();
}

int exact_div(uint32_t seed, int blocks, int per, int a0, int a1, int b0, int b1, unsigned long long *bad) {
    div_kernel<<<blocks, 256>>>(seed, per, a0, a1, b0, b1, bad);
    return (int)cudaGetLastError();
}

int exact_exp(const float *x, float *y, int64_t n) {
    exp_kernel<<<(unsigned)((n + 255) / 256), 256>>>(x, y, n);
    return (int)cudaGetLastError();
}

}
