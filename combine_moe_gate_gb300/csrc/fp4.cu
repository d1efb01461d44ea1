// Quantiser and expander of microscaled 4-bit rows (MX: e8m0 scales over 32
// values; NV: e4m3 scales over 16 with one fp32 factor per batch).
#include "fp4.cuh"

namespace moe {
namespace {

constexpr int Q_THREADS = 256;

template <typename T> struct Ld16;   // 16 consecutive values
template <> struct Ld16<float> {
    __device__ __forceinline__ static void get(const float *p, float *f) {
#pragma unroll
        for (int i = 0; i < 4; i++) Elt<float>::unpack(ld_v16(p + 4 * i), f + 4 * i);
    }
    __device__ __forceinline__ static void put(float *p, const float *f) {
#pragma unroll
        for (int i = 0; i < 4; i++) st_v16(p + 4 * i, Elt<float>::pack(f + 4 * i));
    }
};
template <> struct Ld16<__nv_bfloat16> {
    __device__ __forceinline__ static void get(const __nv_bfloat16 *p, float *f) {
        Elt<__nv_bfloat16>::unpack(ld_v16(p), f);
        Elt<__nv_bfloat16>::unpack(ld_v16(p + 8), f + 8);
    }
    __device__ __forceinline__ static void put(__nv_bfloat16 *p, const float *f) {
        st_v16(p, Elt<__nv_bfloat16>::pack(f));
        st_v16(p + 8, Elt<__nv_bfloat16>::pack(f + 8));
    }
};

// One thread per 16 values (an MX block is a pair of lanes).  A row takes a
// whole number of scale tiles' worth of threads (4 blocks each); the threads
// past its last block write the zeros of the last tile.  Four neighbouring
// lanes gather the bytes of one row of a tile into one 4-byte store.
template <typename T, int FMT>
__global__ void __launch_bounds__(Q_THREADS)
quantize_fp4_kernel(const T *__restrict__ src, int64_t batches, int64_t rpb, int cols, int64_t ntiles,
                    const float *__restrict__ global, const int32_t *__restrict__ counts,
                    const int32_t *__restrict__ c_dev, uint8_t *__restrict__ q,
                    uint8_t *__restrict__ scale, int32_t *status) {
    pdl_enter();
    if (status_bad(status)) return;
    constexpr int TPB = Fp4<FMT>::BLK / 16;   // threads per block
    const int per_row = (int)ntiles * 4 * TPB, nch = cols / 16;
    const int64_t total = batches * rpb * per_row;
    const int64_t batch_bytes = (rpb + 127) / 128 * ntiles * 512;
    const int64_t c_eff = counts ? min((int64_t)*c_dev, rpb) : rpb;
    const int lane = threadIdx.x & 31;
    for (int64_t base = (int64_t)blockIdx.x * Q_THREADS; base < total; base += (int64_t)gridDim.x * Q_THREADS) {
        const int64_t at = base + threadIdx.x;
        const int64_t row = at / per_row;
        const int ch = (int)(at - row * per_row);
        const int64_t b = row / rpb, r = row - b * rpb;
        const bool live = at < total && (!counts || r < min((int64_t)max(counts[b], 0), c_eff));
        float f[16] = {};
        float amax = 0.0f;
        if (live && ch < nch) {
            Ld16<T>::get(src + row * cols + ch * 16, f);
#pragma unroll
            for (int i = 0; i < 16; i++) amax = amax_nan(amax, f[i]);
        }
        if (TPB == 2) amax = amax_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        const float g = FMT == MOE_FP4_NV && global && live ? global[b] : 1.0f;
        float inv;
        uint32_t sc = fp4_scale<FMT>(amax, g, __fmul_rn(g, 6.0f), inv);
        if (live && ch < nch) {
            uint32_t w[2];
#pragma unroll
            for (int i = 0; i < 16; i++) f[i] = __fmul_rn(f[i], inv);
            w[0] = e2m1x8(f);
            w[1] = e2m1x8(f + 8);
            *reinterpret_cast<uint2 *>(q + (row * cols + ch * 16) / 2) = make_uint2(w[0], w[1]);
        } else {
            sc = 0;   // a block past the row's last
        }
        uint32_t word = sc;
#pragma unroll
        for (int i = 1; i < 4; i++) word |= __shfl_down_sync(0xffffffffu, sc, i * TPB) << (8 * i);
        if (live && lane % (4 * TPB) == 0)
            *reinterpret_cast<uint32_t *>(scale + b * batch_bytes + fp4_scale_at(r, ch / TPB, ntiles)) = word;
    }
}

template <typename T, int FMT>
__global__ void __launch_bounds__(Q_THREADS)
dequantize_fp4_kernel(const uint8_t *__restrict__ q, const uint8_t *__restrict__ scale, int64_t batches,
                      int64_t rpb, int cols, int64_t ntiles, const float *__restrict__ global,
                      const int32_t *__restrict__ counts, const int32_t *__restrict__ c_dev,
                      T *__restrict__ dst, int32_t *status) {
    pdl_enter();
    if (status_bad(status)) return;
    const int nch = cols / 16;
    const int64_t total = batches * rpb * nch;
    const int64_t batch_bytes = (rpb + 127) / 128 * ntiles * 512;
    const int64_t c_eff = counts ? min((int64_t)*c_dev, rpb) : rpb;
    for (int64_t at = (int64_t)blockIdx.x * Q_THREADS + threadIdx.x; at < total;
         at += (int64_t)gridDim.x * Q_THREADS) {
        const int64_t row = at / nch;
        const int ch = (int)(at - row * nch);
        const int64_t b = row / rpb, r = row - b * rpb;
        if (counts && r >= min((int64_t)max(counts[b], 0), c_eff)) continue;
        const uint32_t code = scale[b * batch_bytes + fp4_scale_at(r, ch * 16 / Fp4<FMT>::BLK, ntiles)];
        float s;
        if (FMT == MOE_FP4_MX) s = e8m0_value(code);
        else s = __fmul_rn(e4m3_value(code), global ? global[b] : 1.0f);
        const uint2 w = *reinterpret_cast<const uint2 *>(q + (row * cols + ch * 16) / 2);
        float f[16];
#pragma unroll
        for (int i = 0; i < 8; i++) {
            f[i] = __fmul_rn(e2m1_value(w.x >> (4 * i)), s);
            f[8 + i] = __fmul_rn(e2m1_value(w.y >> (4 * i)), s);
        }
        Ld16<T>::put(dst + row * cols + ch * 16, f);
    }
}

// One resident wave at most: the kernels stride.
int grid_for(int64_t threads) {
    int dev = 0, sms = 152;
    if (cudaGetDevice(&dev) == cudaSuccess)
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t want = (threads + Q_THREADS - 1) / Q_THREADS, cap = (int64_t)sms * 8;
    return (int)(want < cap ? want : cap);
}

template <typename T, int FMT>
moe_status quantize_t(const void *src, int64_t batches, int64_t rpb, int cols, const float *global,
                      const int32_t *counts, const int32_t *c_dev, void *q, void *scale,
                      int32_t *st, cudaStream_t stream) {
    const int64_t nt = fp4_scale_tiles(Fp4<FMT>::BLK, cols);
    return launch_pdl(quantize_fp4_kernel<T, FMT>,
                      dim3(grid_for(batches * rpb * nt * 4 * (Fp4<FMT>::BLK / 16))), dim3(Q_THREADS), 0,
                      stream, (const T *)src, batches, rpb, cols, nt, global, counts, c_dev,
                      (uint8_t *)q, (uint8_t *)scale, st);
}

template <typename T, int FMT>
moe_status dequantize_t(const void *q, const void *scale, int64_t batches, int64_t rpb, int cols,
                        const float *global, const int32_t *counts, const int32_t *c_dev, void *dst,
                        int32_t *st, cudaStream_t stream) {
    return launch_pdl(dequantize_fp4_kernel<T, FMT>, dim3(grid_for(batches * rpb * (cols / 16))),
                      dim3(Q_THREADS), 0, stream, (const uint8_t *)q, (const uint8_t *)scale, batches,
                      rpb, cols, fp4_scale_tiles(Fp4<FMT>::BLK, cols), global, counts, c_dev, (T *)dst,
                      st);
}

}  // namespace

moe_status quantize_fp4_launch(const void *src, moe_dtype sdt, int64_t batches, int64_t rpb, int cols,
                               moe_fp4 fmt, const float *global, const int32_t *counts,
                               const int32_t *c_dev, void *q, void *scale, int32_t *st,
                               cudaStream_t stream) {
    using bf = __nv_bfloat16;
    auto f = sdt == MOE_F32 ? (fmt == MOE_FP4_MX ? quantize_t<float, MOE_FP4_MX> : quantize_t<float, MOE_FP4_NV>)
                            : (fmt == MOE_FP4_MX ? quantize_t<bf, MOE_FP4_MX> : quantize_t<bf, MOE_FP4_NV>);
    return f(src, batches, rpb, cols, global, counts, c_dev, q, scale, st, stream);
}

moe_status dequantize_fp4_launch(const void *q, const void *scale, int64_t batches, int64_t rpb,
                                 int cols, moe_fp4 fmt, const float *global, const int32_t *counts,
                                 const int32_t *c_dev, void *dst, moe_dtype ddt, int32_t *st,
                                 cudaStream_t stream) {
    using bf = __nv_bfloat16;
    auto f = ddt == MOE_F32 ? (fmt == MOE_FP4_MX ? dequantize_t<float, MOE_FP4_MX> : dequantize_t<float, MOE_FP4_NV>)
                            : (fmt == MOE_FP4_MX ? dequantize_t<bf, MOE_FP4_MX> : dequantize_t<bf, MOE_FP4_NV>);
    return f(q, scale, batches, rpb, cols, global, counts, c_dev, dst, st, stream);
}

}  // namespace moe
