// Quantiser and expander of microscaled 4-bit rows (MX: e8m0 scales over 32
// values; NV: e4m3 scales over 16 with one fp32 factor per batch).
#include "fp4.cuh"

namespace moe {
namespace {

constexpr int Q_THREADS = 256;

// 32 bytes at a time (one sector a lane: a warp's access is 1 KB in a row).
// `wide`: p lies on a 32-byte boundary (callers' buffers have to on 16 only).
__device__ __forceinline__ void ld32(const void *p, uint32_t (&w)[8], bool wide) {
    if (!wide) {
        const V16 a = ld_stream(p), b = ld_stream(reinterpret_cast<const char *>(p) + 16);
#pragma unroll
        for (int i = 0; i < 4; i++) { w[i] = a.w[i]; w[4 + i] = b.w[i]; }
        return;
    }
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
}
__device__ __forceinline__ void st32(void *p, const float (&f)[8], bool wide) {
    if (!wide) {
        st_v16(p, Elt<float>::pack(f));
        st_v16(reinterpret_cast<char *>(p) + 16, Elt<float>::pack(f + 4));
        return;
    }
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(f[0]), "f"(f[1]), "f"(f[2]),
                 "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                 : "memory");
}

// 16 consecutive values as loaded (rows start on 64-byte boundaries: cols % 32
// == 0), their largest magnitude (a NaN counts as one above infinity: as bits,
// magnitudes order like integers) and the values.
template <typename T> struct Raw;
template <> struct Raw<float> {
    uint32_t w[2][8];
    __device__ __forceinline__ void load(const float *p, bool wide) {
        ld32(p, w[0], wide);
        ld32(p + 8, w[1], wide);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 8; i++) w[0][i] = w[1][i] = 0u;
    }
    __device__ __forceinline__ float amax() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) m = max(m, max(w[0][i] & 0x7FFFFFFFu, w[1][i] & 0x7FFFFFFFu));
        return __uint_as_float(m);
    }
    __device__ __forceinline__ float2 pair(int i) const {
        return make_float2(__uint_as_float(w[i / 4][2 * (i % 4)]), __uint_as_float(w[i / 4][2 * (i % 4) + 1]));
    }
};
template <> struct Raw<__nv_bfloat16> {
    uint32_t w[8];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, bool wide) { ld32(p, w, wide); }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 8; i++) w[i] = 0u;
    }
    __device__ __forceinline__ float amax() const {
        uint32_t m = 0;   // two at a time, as 16-bit integers
#pragma unroll
        for (int i = 0; i < 8; i++) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
        return __uint_as_float(max(m << 16, m & 0xFFFF0000u));
    }
    __device__ __forceinline__ float2 pair(int i) const { return make_float2(bf16lo(w[i]), bf16hi(w[i])); }
};

// Kept rows of batch b.
__device__ __forceinline__ int64_t live_rows(const int32_t *counts, const int32_t *c_dev, int64_t b, int64_t rpb) {
    return counts ? min((int64_t)max(counts[b], 0), min((int64_t)*c_dev, rpb)) : rpb;
}

// One lane per 16 values (an MX block is a pair of lanes); T lanes share a row,
// 32 / T rows a warp; a CTA takes its rows' steps of one segment (blockIdx.z).
// A row takes a whole number of scale tiles' worth of steps (4 blocks each):
// the lanes past its last block write the zeros of its last tile.  Four
// neighbouring lanes gather the bytes that one row has in a tile into one
// 4-byte store.  Bound by HBM (2.56 bytes a value) and, close behind, by
// instructions: U steps are loaded before the first is used.  12592 rows of
// 4096 bf16: 25.5 us, 5.2 TB/s (one or two steps at a time: 28 to 34 us).
template <typename T_, int FMT, int T>
__global__ void __launch_bounds__(Q_THREADS)
quantize_fp4_kernel(const T_ *__restrict__ src, int64_t batches, int64_t rpb, int cols, int64_t ntiles, int seg,
                    int wide,
                    const float *__restrict__ global, const int32_t *__restrict__ counts,
                    const int32_t *__restrict__ c_dev, uint8_t *__restrict__ q,
                    uint8_t *__restrict__ scale, int32_t *status) {
    pdl_enter();
    if (status_bad(status)) return;
    constexpr int TPB = Fp4<FMT>::BLK / 16;   // lanes per block
    constexpr int RPC = Q_THREADS / T;        // rows per CTA and pass
    constexpr int U = sizeof(T_) == 2 ? 4 : 2;
    const int steps = (int)ntiles * 4 * TPB, nch = cols / 16;
    const int first = (int)blockIdx.z * seg, last = min(first + seg, steps);   // seg: a multiple of T
    const int64_t batch_bytes = (rpb + 127) / 128 * ntiles * 512;
    const int lane = threadIdx.x & 31, sub = lane % T;
    for (int64_t b = blockIdx.y; b < batches; b += gridDim.y) {
        const int64_t rows = live_rows(counts, c_dev, b, rpb);
        const Fp4Factor g = fp4_factor(FMT == MOE_FP4_NV && global ? global[b] : 1.0f);
        const int row_in = (int)threadIdx.x / T;
        // the warp's first row decides how often the warp goes round
        for (int64_t r = (int64_t)blockIdx.x * RPC + row_in; r - lane / T < rows; r += (int64_t)gridDim.x * RPC) {
            const bool live = r < rows;
            const T_ *srow = src + (b * rpb + r) * cols;
            uint8_t *qrow = q + (b * rpb + r) * cols / 2;
            uint8_t *scrow = scale + b * batch_bytes + fp4_scale_at(r, 0, ntiles);
            for (int c0 = first + sub; c0 - sub < last; c0 += U * T) {
                Raw<T_> v[U];
#pragma unroll
                for (int u = 0; u < U; u++) {
                    v[u].zero();
                    if (live && c0 + u * T < min(last, nch)) v[u].load(srow + (c0 + u * T) * 16, wide);
                }
#pragma unroll
                for (int u = 0; u < U; u++) {
                    const int ch = c0 + u * T;
                    if (ch - sub >= last) break;   // the same in the lanes of a row's step
                    float amax = v[u].amax(), inv;
                    if (TPB == 2)
                        amax = __uint_as_float(max(__float_as_uint(amax),
                                                   __shfl_xor_sync(0xffffffffu, __float_as_uint(amax), 1)));
                    uint32_t sc = fp4_scale<FMT>(amax, g, inv);
                    float f[16];
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        const float2 p = __fmul2_rn(v[u].pair(i), make_float2(inv, inv));
                        f[2 * i] = p.x;
                        f[2 * i + 1] = p.y;
                    }
                    const bool on = live && ch < nch;
                    if (on) *reinterpret_cast<uint2 *>(qrow + ch * 8) = make_uint2(e2m1x8(f), e2m1x8(f + 8));
                    else sc = 0;   // past the row's last block
                    uint32_t word = sc;
#pragma unroll
                    for (int i = 1; i < 4; i++) word |= __shfl_down_sync(0xffffffffu, sc, i * TPB) << (8 * i);
                    if (live && ch < last && lane % (4 * TPB) == 0)
                        *reinterpret_cast<uint32_t *>(scrow + (int64_t)(ch / (4 * TPB)) * 512) = word;
                }
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

// One lane per 16 values, T lanes a row.  Bound by the bytes written: the same
// rows to fp32, 40.6 us, 5.8 TB/s.
template <typename T_, int FMT, int T>
__global__ void __launch_bounds__(Q_THREADS)
dequantize_fp4_kernel(const uint8_t *__restrict__ q, const uint8_t *__restrict__ scale, int64_t batches,
                      int64_t rpb, int cols, int64_t ntiles, int seg, int wide,
                      const float *__restrict__ global,
                      const int32_t *__restrict__ counts, const int32_t *__restrict__ c_dev,
                      T_ *__restrict__ dst, int32_t *status) {
    pdl_enter();
    if (status_bad(status)) return;
    constexpr int RPC = Q_THREADS / T, U = 4;
    const int first = (int)blockIdx.z * seg, last = min(first + seg, cols / 16), sub = (int)threadIdx.x % T;
    const int64_t batch_bytes = (rpb + 127) / 128 * ntiles * 512;
    for (int64_t b = blockIdx.y; b < batches; b += gridDim.y) {
        const int64_t rows = live_rows(counts, c_dev, b, rpb);
        const float g = FMT == MOE_FP4_NV && global ? global[b] : 1.0f;
        for (int64_t r = (int64_t)blockIdx.x * RPC + threadIdx.x / T; r < rows; r += (int64_t)gridDim.x * RPC) {
            const uint2 *qrow = reinterpret_cast<const uint2 *>(q + (b * rpb + r) * cols / 2);
            T_ *drow = dst + (b * rpb + r) * cols;
            const uint8_t *scrow = scale + b * batch_bytes + fp4_scale_at(r, 0, ntiles);
            for (int c0 = first + sub; c0 < last; c0 += U * T) {
                uint2 w[U];
                uint32_t code[U];
#pragma unroll
                for (int u = 0; u < U; u++) {
                    const int ch = min(c0 + u * T, last - 1), blk = ch * 16 / Fp4<FMT>::BLK;
                    w[u] = __ldg(qrow + ch);
                    code[u] = __ldg(scrow + (int64_t)(blk >> 2) * 512 + (blk & 3));
                }
#pragma unroll
                for (int u = 0; u < U; u++) {
                    const int ch = c0 + u * T;
                    if (ch >= last) break;
                    const float s = FMT == MOE_FP4_MX ? e8m0_value(code[u]) : __fmul_rn(e4m3_value(code[u]), g);
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        float f[8];
                        e2m1_values(h ? w[u].y : w[u].x, f);
#pragma unroll
                        for (int i = 0; i < 8; i++) f[i] = __fmul_rn(f[i], s);
                        if constexpr (sizeof(T_) == 4) st32(drow + ch * 16 + 8 * h, f, wide);
                        else st_v16(drow + ch * 16 + 8 * h, Elt<__nv_bfloat16>::pack(f));
                    }
                }
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

// Rows along x, batches along y, and where those are too few for the device,
// segments of a row along z: `per` steps of 16 values each, a multiple of T.
// CTAs per multiprocessor: 8 for the quantiser (16: 10% slower on 16384 x 2048),
// 16 for the expander (8: 7% slower on 8 x 2048 x 4096).
dim3 grid_for(int64_t batches, int64_t rpb, int T, int steps, int ctas_per_sm, int &per) {
    const int64_t y = batches < 65535 ? batches : 65535, want = (int64_t)sms() * ctas_per_sm;
    const int64_t rows = (rpb * T + Q_THREADS - 1) / Q_THREADS, cap = (want + y - 1) / y;
    const int64_t x = rows < cap ? rows : cap;
    const int rounds = (steps + T - 1) / T;   // of a row's lanes
    const int64_t z = want / (x * y) < rounds ? want / (x * y) : rounds;
    per = (int)((rounds + (z > 1 ? z : 1) - 1) / (z > 1 ? z : 1)) * T;
    return dim3((unsigned)x, (unsigned)y, (unsigned)((steps + per - 1) / per));
}

template <typename T_, int FMT, int T>
moe_status quantize_t(const void *src, int64_t batches, int64_t rpb, int cols, const float *global,
                      const int32_t *counts, const int32_t *c_dev, void *q, void *scale,
                      int32_t *st, cudaStream_t stream) {
    const int64_t nt = fp4_scale_tiles(Fp4<FMT>::BLK, cols);
    int per;
    const dim3 grid = grid_for(batches, rpb, T, (int)nt * (Fp4<FMT>::BLK / 4), 8, per);
    return launch_pdl(quantize_fp4_kernel<T_, FMT, T>, grid, dim3(Q_THREADS), 0, stream, (const T_ *)src, batches,
                      rpb, cols, nt, per, ((uintptr_t)src & 31) == 0, global, counts, c_dev, (uint8_t *)q, (uint8_t *)scale, st);
}

template <typename T_, int FMT, int T>
moe_status dequantize_t(const void *q, const void *scale, int64_t batches, int64_t rpb, int cols,
                        const float *global, const int32_t *counts, const int32_t *c_dev, void *dst,
                        int32_t *st, cudaStream_t stream) {
    int per;
    const dim3 grid = grid_for(batches, rpb, T, cols / 16, 16, per);
    return launch_pdl(dequantize_fp4_kernel<T_, FMT, T>, grid, dim3(Q_THREADS), 0, stream, (const uint8_t *)q,
                      (const uint8_t *)scale, batches, rpb, cols, fp4_scale_tiles(Fp4<FMT>::BLK, cols), per,
                      ((uintptr_t)dst & 31) == 0, global,
                      counts, c_dev, (T_ *)dst, st);
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
