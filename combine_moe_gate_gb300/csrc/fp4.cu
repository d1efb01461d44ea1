// Quantiser and expander of microscaled 4-bit rows (MX: e8m0 scales over 32
// values; NV: e4m3 scales over 16 with one fp32 factor per batch).
#include <cuda_fp16.h>

#include "fp4.cuh"

namespace moe {
namespace {

constexpr int Q_THREADS = 256;

// 32 bytes at a time (one sector a lane: a warp's access is 1 KB in a row).
__device__ __forceinline__ void ld32(const void *p, uint32_t (&w)[8]) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
}
__device__ __forceinline__ void st32(void *p, const float (&f)[8]) {
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(f[0]), "f"(f[1]), "f"(f[2]),
                 "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                 : "memory");
}

// 16 consecutive values (rows start on 64-byte boundaries: cols % 32 == 0).
__device__ __forceinline__ void ld_values(const float *p, float (&f)[16]) {
    uint32_t w[8];
#pragma unroll
    for (int h = 0; h < 2; h++) {
        ld32(p + 8 * h, w);
#pragma unroll
        for (int i = 0; i < 8; i++) f[8 * h + i] = __uint_as_float(w[i]);
    }
}
__device__ __forceinline__ void ld_values(const __nv_bfloat16 *p, float (&f)[16]) {
    uint32_t w[8];
    ld32(p, w);
#pragma unroll
    for (int i = 0; i < 8; i++) { f[2 * i] = bf16lo(w[i]); f[2 * i + 1] = bf16hi(w[i]); }
}

// Kept rows of batch b.
__device__ __forceinline__ int64_t live_rows(const int32_t *counts, const int32_t *c_dev, int64_t b, int64_t rpb) {
    return counts ? min((int64_t)max(counts[b], 0), min((int64_t)*c_dev, rpb)) : rpb;
}

// One lane per 16 values (an MX block is a pair of lanes); T lanes share a row,
// 32 / T rows a warp.  A row takes a whole number of scale tiles' worth of
// steps (4 blocks each): the lanes past its last block write the zeros of its
// last tile.  Four neighbouring lanes gather the bytes that one row has in a
// tile into one 4-byte store.  Bound by HBM: 2.56 bytes a value.
template <typename T_, int FMT, int T>
__global__ void __launch_bounds__(Q_THREADS)
quantize_fp4_kernel(const T_ *__restrict__ src, int64_t batches, int64_t rpb, int cols, int64_t ntiles,
                    const float *__restrict__ global, const int32_t *__restrict__ counts,
                    const int32_t *__restrict__ c_dev, uint8_t *__restrict__ q,
                    uint8_t *__restrict__ scale, int32_t *status) {
    pdl_enter();
    if (status_bad(status)) return;
    constexpr int TPB = Fp4<FMT>::BLK / 16;   // lanes per block
    constexpr int RPC = Q_THREADS / T;        // rows per CTA and pass
    const int steps = (int)ntiles * 4 * TPB, nch = cols / 16;
    const int64_t batch_bytes = (rpb + 127) / 128 * ntiles * 512;
    const int lane = threadIdx.x & 31, sub = lane % T;
    for (int64_t b = blockIdx.y; b < batches; b += gridDim.y) {
        const int64_t rows = live_rows(counts, c_dev, b, rpb);
        const float g = FMT == MOE_FP4_NV && global ? global[b] : 1.0f;
        const float g6 = __fmul_rn(g, 6.0f);
        const int row_in = (int)threadIdx.x / T;
        // the warp's first row decides how often the warp goes round
        for (int64_t r = (int64_t)blockIdx.x * RPC + row_in; r - lane / T < rows; r += (int64_t)gridDim.x * RPC) {
            const bool live = r < rows;
            const int64_t at = (b * rpb + r) * cols;
            uint8_t *srow = scale + b * batch_bytes;
#pragma unroll 2
            for (int ch = sub; ch < steps; ch += T) {
                const bool on = live && ch < nch;
                float f[16] = {};
                float amax = 0.0f, inv;
                if (on) ld_values(src + at + ch * 16, f);
#pragma unroll
                for (int i = 0; i < 16; i++) amax = amax_nan(amax, f[i]);
                if (TPB == 2) amax = amax_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                uint32_t sc = fp4_scale<FMT>(amax, g, g6, inv);
#pragma unroll
                for (int i = 0; i < 16; i++) f[i] = __fmul_rn(f[i], inv);
                if (on) *reinterpret_cast<uint2 *>(q + (at + ch * 16) / 2) = make_uint2(e2m1x8(f), e2m1x8(f + 8));
                else sc = 0;   // past the row's last block
                uint32_t word = sc;
#pragma unroll
                for (int i = 1; i < 4; i++) word |= __shfl_down_sync(0xffffffffu, sc, i * TPB) << (8 * i);
                if (live && lane % (4 * TPB) == 0)
                    *reinterpret_cast<uint32_t *>(srow + fp4_scale_at(r, ch / TPB, ntiles)) = word;
            }
        }
    }
}

// Eight codes to their values (exact).
__device__ __forceinline__ void e2m1_values(uint32_t w, float (&f)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
    }
}

// One lane per 8 values, T lanes a row.  Bound by the bytes written.
template <typename T_, int FMT, int T>
__global__ void __launch_bounds__(Q_THREADS)
dequantize_fp4_kernel(const uint8_t *__restrict__ q, const uint8_t *__restrict__ scale, int64_t batches,
                      int64_t rpb, int cols, int64_t ntiles, const float *__restrict__ global,
                      const int32_t *__restrict__ counts, const int32_t *__restrict__ c_dev,
                      T_ *__restrict__ dst, int32_t *status) {
    pdl_enter();
    if (status_bad(status)) return;
    constexpr int RPC = Q_THREADS / T;
    const int nch = cols / 8, sub = (int)threadIdx.x % T;
    const int64_t batch_bytes = (rpb + 127) / 128 * ntiles * 512;
    for (int64_t b = blockIdx.y; b < batches; b += gridDim.y) {
        const int64_t rows = live_rows(counts, c_dev, b, rpb);
        const float g = FMT == MOE_FP4_NV && global ? global[b] : 1.0f;
        for (int64_t r = (int64_t)blockIdx.x * RPC + threadIdx.x / T; r < rows; r += (int64_t)gridDim.x * RPC) {
            const int64_t at = (b * rpb + r) * cols;
            const uint8_t *srow = scale + b * batch_bytes;
#pragma unroll 4
            for (int ch = sub; ch < nch; ch += T) {
                const uint32_t w = __ldg(reinterpret_cast<const uint32_t *>(q + at / 2) + ch);
                const uint32_t code = __ldg(srow + fp4_scale_at(r, ch * 8 / Fp4<FMT>::BLK, ntiles));
                const float s = FMT == MOE_FP4_MX ? e8m0_value(code) : __fmul_rn(e4m3_value(code), g);
                float f[8];
                e2m1_values(w, f);
#pragma unroll
                for (int i = 0; i < 8; i++) f[i] = __fmul_rn(f[i], s);
                if constexpr (sizeof(T_) == 4) st32(dst + at + ch * 8, f);
                else st_v16(dst + at + ch * 8, Elt<__nv_bfloat16>::pack(f));
            }
        }
    }
}

int sms() {
    static int cached[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
    if (!cached[dev]) {
        int v = 0;
        cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
        cached[dev] = v > 0 ? v : 148;
    }
    return cached[dev];
}

// Batches along y; rows along x, at most about one resident wave of CTAs.
dim3 grid_for(int64_t batches, int64_t rpb, int rows_per_cta) {
    const int64_t y = batches < 65535 ? batches : 65535;
    const int64_t want = (rpb + rows_per_cta - 1) / rows_per_cta;
    const int64_t cap = ((int64_t)sms() * 8 + y - 1) / y;
    return dim3((unsigned)(want < cap ? want : cap), (unsigned)y);
}

template <typename T_, int FMT, int T>
moe_status quantize_t(const void *src, int64_t batches, int64_t rpb, int cols, const float *global,
                      const int32_t *counts, const int32_t *c_dev, void *q, void *scale,
                      int32_t *st, cudaStream_t stream) {
    return launch_pdl(quantize_fp4_kernel<T_, FMT, T>, grid_for(batches, rpb, Q_THREADS / T), dim3(Q_THREADS), 0,
                      stream, (const T_ *)src, batches, rpb, cols, fp4_scale_tiles(Fp4<FMT>::BLK, cols), global,
                      counts, c_dev, (uint8_t *)q, (uint8_t *)scale, st);
}

template <typename T_, int FMT, int T>
moe_status dequantize_t(const void *q, const void *scale, int64_t batches, int64_t rpb, int cols,
                        const float *global, const int32_t *counts, const int32_t *c_dev, void *dst,
                        int32_t *st, cudaStream_t stream) {
    return launch_pdl(dequantize_fp4_kernel<T_, FMT, T>, grid_for(batches, rpb, Q_THREADS / T), dim3(Q_THREADS), 0,
                      stream, (const uint8_t *)q, (const uint8_t *)scale, batches, rpb, cols,
                      fp4_scale_tiles(Fp4<FMT>::BLK, cols), global, counts, c_dev, (T_ *)dst, st);
}

// Lanes a row: a whole warp from 512 values on, a quarter of one below (rows
// of a few blocks would leave most of a warp without work).
constexpr int Q_WIDE = 512;

}  // namespace

#define MOE_FP4_PICK(F)                                                                                   \
    (dt == MOE_F32 ? (fmt == MOE_FP4_MX ? (wide ? F<float, MOE_FP4_MX, 32> : F<float, MOE_FP4_MX, 8>)     \
                                        : (wide ? F<float, MOE_FP4_NV, 32> : F<float, MOE_FP4_NV, 8>))    \
                   : (fmt == MOE_FP4_MX ? (wide ? F<bf, MOE_FP4_MX, 32> : F<bf, MOE_FP4_MX, 8>)           \
                                        : (wide ? F<bf, MOE_FP4_NV, 32> : F<bf, MOE_FP4_NV, 8>)))

moe_status quantize_fp4_launch(const void *src, moe_dtype dt, int64_t batches, int64_t rpb, int cols,
                               moe_fp4 fmt, const float *global, const int32_t *counts,
                               const int32_t *c_dev, void *q, void *scale, int32_t *st,
                               cudaStream_t stream) {
    using bf = __nv_bfloat16;
    const bool wide = cols >= Q_WIDE;
    return MOE_FP4_PICK(quantize_t)(src, batches, rpb, cols, global, counts, c_dev, q, scale, st, stream);
}

moe_status dequantize_fp4_launch(const void *q, const void *scale, int64_t batches, int64_t rpb,
                                 int cols, moe_fp4 fmt, const float *global, const int32_t *counts,
                                 const int32_t *c_dev, void *dst, moe_dtype dt, int32_t *st,
                                 cudaStream_t stream) {
    using bf = __nv_bfloat16;
    const bool wide = cols >= Q_WIDE;
    return MOE_FP4_PICK(dequantize_t)(q, scale, batches, rpb, cols, global, counts, c_dev, dst, st, stream);
}
#undef MOE_FP4_PICK

}  // namespace moe
