// Microscaled 4-bit blocks: the arithmetic and the storage order that the
// quantiser, the products' epilogues and the expander share.
//
// A block of B values (MX: 32, NV: 16) is stored as e2m1 codes and one scale
// byte; value = code * scale.  The order of the scale bytes (tiles of 128 rows
// x 4 blocks, 512 bytes) is the one tcgen05.cp .32x128b reads: 32 rows of 16
// bytes, row r of the tile at 16-byte row r % 32, 4-byte column r / 32.
#pragma once

#include <cuda_fp16.h>

#include "exact.cuh"

namespace moe {

template <int FMT> struct Fp4;
template <> struct Fp4<MOE_FP4_MX> {
    static constexpr int BLK = 32;
    static constexpr uint32_t NAN_SCALE = 0xFFu;
};
template <> struct Fp4<MOE_FP4_NV> {
    static constexpr int BLK = 16;
    static constexpr uint32_t NAN_SCALE = 0x7Fu;
};

__host__ __device__ inline int fp4_blk(moe_fp4 fmt) { return fmt == MOE_FP4_MX ? 32 : 16; }
// 512-byte scale tiles along one row of `cols` values, and bytes per batch.
__host__ __device__ inline int64_t fp4_scale_tiles(int blk, int cols) { return (cols / blk + 3) / 4; }
__host__ __device__ inline int64_t fp4_scale_bytes(int blk, int64_t rows, int cols) {
    return (rows + 127) / 128 * fp4_scale_tiles(blk, cols) * 512;
}
// Byte of (row, block) within a batch's scales (ntiles = fp4_scale_tiles()).
__device__ __forceinline__ int64_t fp4_scale_at(int64_t row, int b, int64_t ntiles) {
    return ((row >> 7) * ntiles + (b >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (b & 3);
}

// Nearest e4m3 code of v >= 0 (ties to even, at most 448).
__device__ __forceinline__ uint32_t e4m3_of(float v) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
    return r & 0xFFu;
}
// The value of an e4m3 code (exact in fp16).
__device__ __forceinline__ float e4m3_value(uint32_t code) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)code));
    return __half2float(__ushort_as_half((unsigned short)(h & 0xFFFFu)));
}
// 2^(code - 127); code 0 is the subnormal 2^-127.
__device__ __forceinline__ float e8m0_value(uint32_t code) {
    return code == 0xFFu ? NAN : __uint_as_float(code ? code << 23 : 1u << 22);
}

// A batch's factor g (NV) with what its blocks' scales divide by.
struct Fp4Factor {
    float g, g6, y6;   // g, 6 g, and 1 / (6 g) rounded (0: not in the middle of the range)
};
__device__ __forceinline__ Fp4Factor fp4_factor(float g) {
    Fp4Factor f;
    f.g = g;
    f.g6 = __fmul_rn(g, 6.0f);
    f.y6 = f.g6 >= 0x1p-40f && f.g6 <= 0x1p40f ? __frcp_rn(f.g6) : 0.0f;
    return f;
}

// Scale byte of a block with largest magnitude amax, and what its values are
// multiplied by (1 / scale; 0 where that is not finite).
template <int FMT>
__device__ __forceinline__ uint32_t fp4_scale(float amax, const Fp4Factor &f, float &inv) {
    if (FMT == MOE_FP4_NV && f.y6 != 0.0f && amax <= 0x1p60f && (amax >= 0x1p-60f || amax == 0.0f)) {
        const uint32_t s8 = e4m3_of(div_mid(amax, f.g6, f.y6));
        const float y = rcp_mid(__fmul_rn(e4m3_value(s8), f.g));
        inv = s8 ? y : 0.0f;
        return s8;
    }
    if (!(amax < INFINITY)) {   // an infinity or a NaN
        inv = 0.0f;
        return Fp4<FMT>::NAN_SCALE;
    }
    if (FMT == MOE_FP4_MX) {
        const int ex = (int)(__float_as_uint(amax) >> 23);   // biased exponent
        const int sc = amax == 0.0f ? 127 : max(ex - 2, 0);
        inv = __uint_as_float((uint32_t)(254 - sc) << 23);
        return (uint32_t)sc;
    }
    const uint32_t s8 = e4m3_of(__fdiv_rn(amax, f.g6));
    const float y = __frcp_rn(__fmul_rn(e4m3_value(s8), f.g));
    inv = y > 0.0f && y < INFINITY ? y : 0.0f;   // a scale of 0, or below 2^-128: zeros
    return s8;
}

// Eight codes, value i in bits 4i .. 4i + 3 (nearest-even, saturating).
__device__ __forceinline__ uint32_t e2m1x8(const float *v) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// The larger magnitude of the two, with some sign; a NaN stays one.
__device__ __forceinline__ float amax_nan(float m, float v) {
    float r;
    asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(v));
    return r;
}

}  // namespace moe
