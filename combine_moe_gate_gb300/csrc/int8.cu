// 8-bit integer rows: the quantiser, and the order of the launches.
//
//   scale = amax / 127, code = rn(x * (127 / amax))   per row, in fp32
#include "int8.cuh"

namespace moe {
namespace {

int sm_count() {
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

// ------------------------------------------------------------- the quantiser
// W warps share a row, each lane holds QC 16-byte chunks of it in registers (every load before any
// use: the row is read once); a longer row is read twice.  The maximum is taken of the magnitudes' bits as
// integers, where an infinity and a NaN are larger than every number.  Bound by HBM (16384 rows of 8192 to
// fp16 codes: 82 us, 6.5 TB/s; tokens into their 16384 rows of 4096: 32 us).
//   FAN: the row of token t goes to its routes' rows rows[r, t] (one read, up to k writes)
//   else row t to row t, of the first *end rows (null: all)
// OUT: int8_t, or __half for the codes as fp16 numbers, which the tensor-core product reads.
constexpr int QN_NT = 256, QN_NW = QN_NT / 32, QC = 8;
constexpr uint32_t TINY_BITS = (127u - 100u) << 23;   // 2^-100

struct QuantArgs {
    const void *src;         // [s, cols]
    const int32_t *rows;     // [k, s] (FAN)
    const int32_t *end;
    void *q;                 // [n, cols]
    float *scale;            // [n]
    int64_t s, n;
    int cols, k;
    int32_t *status;
};

// The codes of one chunk (8 bf16 or 4 fp32 values).
template <int V, typename OUT>
struct Codes {
    uint32_t w[V * sizeof(OUT) / 4];
    __device__ __forceinline__ void make(const float *f, float inv) {
        uint32_t c[V];   // rounded by adding 1.5 * 2^23: the code is the sum's low byte
#pragma unroll
        for (int i = 0; i < V; i++) c[i] = __float_as_uint(__fadd_rn(__fmul_rn(f[i], inv), 12582912.0f));
#pragma unroll
        for (int i = 0; i < V / 4; i++) {
            const uint32_t p = __byte_perm(__byte_perm(c[4 * i], c[4 * i + 1], 0x0040),
                                           __byte_perm(c[4 * i + 2], c[4 * i + 3], 0x0040), 0x5410);
            if constexpr (sizeof(OUT) == 1) w[i] = p;
            else i8_widen(p, w[2 * i], w[2 * i + 1]);
        }
    }
    __device__ __forceinline__ void store(OUT *p) const {
        if constexpr (sizeof(w) == 16) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (sizeof(w) == 8) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t *>(p) = w[0];
    }
};

template <typename T, typename OUT, int W, bool FAN>
__global__ void __launch_bounds__(QN_NT)
quantize_int8_kernel(const QuantArgs g) {
    constexpr int V = Elt<T>::VEC, RPC = QN_NW / W;
    __shared__ uint32_t part[QN_NW];
    pdl_enter();
    if (status_bad(g.status)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % W;
    const int nch = g.cols / V;
    const bool whole = nch <= W * 32 * QC;   // the row fits the registers
    const int64_t last = FAN || !g.end ? g.s : min((int64_t)max(*g.end, 0), g.s);
    for (int64_t t0 = (int64_t)blockIdx.x * RPC; t0 < last; t0 += (int64_t)gridDim.x * RPC) {
        const int64_t t = t0 + warp / W;
        const bool mine = t < last;
        const T *xr = static_cast<const T *>(g.src) + (mine ? t : 0) * g.cols;
        int row = -1;   // lane r: route r's row
        if (FAN && mine && lane < g.k) {
            row = g.rows[(int64_t)lane * g.s + t];
            if (row < -1 || row >= g.n) {
                set_status(g.status, MOE_ERR_INVALID_ARG);
                row = -1;
            }
        }
        V16 v[QC];
        uint32_t top = 0;
        auto see = [&](const V16 &c) {
            float f[V];
            Elt<T>::unpack(c, f);
#pragma unroll
            for (int i = 0; i < V; i++) top = max(top, __float_as_uint(f[i]) & 0x7FFFFFFFu);
        };
        if (mine) {
            if (whole) {
#pragma unroll
                for (int i = 0; i < QC; i++) {
                    const int c = (i * W + sub) * 32 + lane;
                    if (c < nch) v[i] = ld_stream(xr + (int64_t)c * V);
                }
#pragma unroll
                for (int i = 0; i < QC; i++)
                    if ((i * W + sub) * 32 + lane < nch) see(v[i]);
            } else {
                for (int c = sub * 32 + lane; c < nch; c += W * 32) see(ld_v16(xr + (int64_t)c * V));
            }
        }
        top = __reduce_max_sync(0xffffffffu, top);
        if (W > 1) {
            if (lane == 0) part[warp] = top;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < W; w++) top = max(top, part[warp - sub + w]);
            __syncthreads();
        }
        if (!mine) continue;
        const bool live = top >= TINY_BITS, number = top < 0x7F800000u;
        const float amax = __uint_as_float(top);
        const float scale = !number ? __uint_as_float(0x7FC00000u) : live ? __fdiv_rn(amax, 127.0f) : 1.0f;
        const float inv = live && number ? __fdiv_rn(127.0f, amax) : 0.0f;
        const unsigned to = FAN ? __ballot_sync(0xffffffffu, row >= 0) : 1u;
        if (sub == 0) {
            if (FAN) { if (row >= 0) g.scale[row] = scale; }
            else if (lane == 0) g.scale[t] = scale;
        }
        // chunk c of the row, by the whole warp (lanes past the row's end bring nothing)
        auto put = [&](const V16 &x, int c) {
            float f[V];
            Elt<T>::unpack(x, f);
            Codes<V, OUT> o;
#pragma unroll
            for (int i = 0; i < V; i++) f[i] = number ? f[i] : 0.0f;
            o.make(f, inv);
            OUT *q = static_cast<OUT *>(g.q) + (int64_t)c * V;
            if (FAN) {
                for (unsigned km = to; km; km &= km - 1) {
                    const int64_t r = __shfl_sync(0xffffffffu, row, __ffs(km) - 1);
                    if (c < nch) o.store(q + r * g.cols);
                }
            } else if (c < nch) {
                o.store(q + t * g.cols);
            }
        };
        if (whole) {
#pragma unroll
            for (int i = 0; i < QC; i++)
                if ((i * W + sub) * 32 < nch) put(v[i], (i * W + sub) * 32 + lane);
        } else {
            for (int c0 = sub * 32; c0 < nch; c0 += W * 32) {
                V16 x{};
                if (c0 + lane < nch) x = ld_v16(xr + (int64_t)(c0 + lane) * V);
                put(x, c0 + lane);
            }
        }
    }
}

template <typename T, typename OUT, bool FAN>
moe_status quantize_typed(const QuantArgs &g, cudaStream_t stream) {
    const int nch = g.cols / Elt<T>::VEC, sms = sm_count();
    // the fewest warps that hold a row, and more while the rows alone leave warps idle
    int w = 1;
    while (w < QN_NW && nch > w * 32 * QC) w *= 2;
    while (w < QN_NW && nch > w * 32 && g.s * w < (int64_t)sms * 16) w *= 2;
    const int64_t ctas = (g.s * w + QN_NW - 1) / QN_NW, cap = (int64_t)sms * 4;
    const dim3 grid((unsigned)(ctas < cap ? ctas : cap)), blk(QN_NT);
    switch (w) {
        case 1: return launch_pdl(quantize_int8_kernel<T, OUT, 1, FAN>, grid, blk, 0, stream, g);
        case 2: return launch_pdl(quantize_int8_kernel<T, OUT, 2, FAN>, grid, blk, 0, stream, g);
        case 4: return launch_pdl(quantize_int8_kernel<T, OUT, 4, FAN>, grid, blk, 0, stream, g);
        default: return launch_pdl(quantize_int8_kernel<T, OUT, 8, FAN>, grid, blk, 0, stream, g);
    }
}

// Codes as fp16 numbers: dst[i] = src[i] over the first *end rows of `chunks` x 8 codes.  A thread takes 8
// codes at a time, so that its warp writes 512 bytes in a row (16384 rows of 4096: 30 us, 6.7 TB/s).
constexpr int WN_U = 8;   // loads under way a thread

__global__ void __launch_bounds__(256)
widen_rows_kernel(const uint2 *__restrict__ src, uint4 *__restrict__ dst, const int32_t *end, int64_t n, int chunks,
                  int32_t *status) {
    pdl_enter();
    if (status_bad(status)) return;
    const int64_t total = (end ? min((int64_t)max(*end, 0), n) : n) * chunks;
    for (int64_t i0 = (int64_t)blockIdx.x * 256 * WN_U + threadIdx.x; i0 < total; i0 += (int64_t)gridDim.x * 256 * WN_U) {
        uint2 v[WN_U];
#pragma unroll
        for (int u = 0; u < WN_U; u++)
            if (i0 + 256 * u < total) v[u] = __ldg(src + i0 + 256 * u);
#pragma unroll
        for (int u = 0; u < WN_U; u++) {
            if (i0 + 256 * u >= total) continue;
            uint4 o;
            i8_widen(v[u].x, o.x, o.y);
            i8_widen(v[u].y, o.z, o.w);
            dst[i0 + 256 * u] = o;
        }
    }
}

// ---------------------------------------------------------- products of few rows
// A warp forms CPW = 2 output channels (SwiGLU: one of W1 and the same of
// W3) with every row of the channel's expert, R at a time; its lanes walk along K in 16-byte pieces
// with dp4a, so the sums are exact integers.  Bound by the weights' bytes: FU pieces of both channels are
// in flight a lane.  CTA (x, y): channels, and the expert whose first row is row y (others leave).
// (mma.sync on 8-bit integers, 8 rows at a time, was slower here already at one row: 18 us against 13 for the FFN of
// a row of 64 experts, 1024 x 704.)
constexpr int FU = 4, CPW = 2;

struct FewArgs {
    const int8_t *x, *w, *w3;
    const float *x_scale, *w_scale, *w3_scale;
    const __nv_bfloat16 *bias;
    void *out;
    SortedRows so;
    int e, K, n_out;
    int32_t *status;
};

__device__ __forceinline__ int dot16(const uint4 &a, const uint4 &b, int acc) {
    acc = __dp4a((int)a.x, (int)b.x, acc);
    acc = __dp4a((int)a.y, (int)b.y, acc);
    acc = __dp4a((int)a.z, (int)b.z, acc);
    return __dp4a((int)a.w, (int)b.w, acc);
}

template <int ACT, int R, typename OUT>
__global__ void __launch_bounds__(256)
int8_few_kernel(const FewArgs g) {
    pdl_enter();
    if (status_bad(g.status)) return;
    constexpr bool SWI = ACT == I8_SWIGLU;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, y = blockIdx.y;
    int j = 0;
    int64_t lo = 0, count = g.so.n;
    if (g.so.offsets) {
        bool bad = false;
        for (int b = lane; b < g.e; b += 32) {   // experts that end at or before row y
            const int o = g.so.offsets[b], p = g.so.offsets[b + 1];
            j += p <= y;
            bad |= o < 0 || p < o || p > g.so.n || (b == 0 && o != 0);
        }
        if (bad) set_status(g.status, MOE_ERR_INVALID_ARG);
        j = __reduce_add_sync(0xffffffffu, j);
        if (__any_sync(0xffffffffu, bad) || j >= g.e) return;
        sorted_span(g.so, j, lo, count);
        if (lo != y) return;
    } else if (y != 0) {
        return;
    }
    const int ch = (blockIdx.x * 8 + warp) * (SWI ? 1 : CPW);
    if (ch >= g.n_out) return;
    const int pieces = g.K / 16;
    const uint4 *wp[CPW];
#pragma unroll
    for (int c = 0; c < CPW; c++) {
        const int8_t *base = SWI && c == 1 ? g.w3 : g.w;
        wp[c] = reinterpret_cast<const uint4 *>(base + ((int64_t)j * g.n_out + ch + (SWI ? 0 : c)) * g.K);
    }
    const uint4 *xp = reinterpret_cast<const uint4 *>(g.x);
    for (int64_t r0 = lo; r0 < lo + count; r0 += R) {
        int acc[CPW][R] = {};
        for (int p0 = lane; p0 < pieces; p0 += 32 * FU) {
            uint4 wv[FU][CPW];
#pragma unroll
            for (int u = 0; u < FU; u++)
#pragma unroll
                for (int c = 0; c < CPW; c++) {
                    const V16 q = ld_stream_if(wp[c] + p0 + 32 * u, p0 + 32 * u < pieces);
                    wv[u][c] = make_uint4(q.w[0], q.w[1], q.w[2], q.w[3]);
                }
#pragma unroll
            for (int u = 0; u < FU; u++) {
                if (p0 + 32 * u >= pieces) continue;
#pragma unroll
                for (int r = 0; r < R; r++) {
                    if (r0 + r >= lo + count) continue;
                    const uint4 xv = __ldg(xp + (r0 + r) * pieces + p0 + 32 * u);
#pragma unroll
                    for (int c = 0; c < CPW; c++) acc[c][r] = dot16(wv[u][c], xv, acc[c][r]);
                }
            }
        }
        // lane r * CH + c finishes row r's channel c (SwiGLU: lane r, of both sums), all of them at once
        constexpr int CH = SWI ? 1 : CPW;
        int sum[CPW] = {};
#pragma unroll
        for (int r = 0; r < R; r++)
#pragma unroll
            for (int c = 0; c < CPW; c++) {
                const int s = __reduce_add_sync(0xffffffffu, acc[c][r]);
                if (lane == r * CH + (SWI ? 0 : c)) sum[SWI ? c : 0] = s;
            }
        const int64_t row = r0 + lane / CH;
        if (lane >= R * CH || row >= lo + count) continue;
        const int64_t at = (int64_t)j * g.n_out + ch + lane % CH, to = row * g.n_out + ch + lane % CH;   // n_out is even
        const float sx = g.x_scale[row];
        if constexpr (SWI) {
            const float a = i8_scaled(__int2float_rn(sum[0]), sx, i8_scale(g.w_scale[at]), 0.0f);
            const float b = i8_scaled(__int2float_rn(sum[1]), sx, i8_scale(g.w3_scale[at]), 0.0f);
            static_cast<__nv_bfloat16 *>(g.out)[to] = __float2bfloat16_rn(a / (1.0f + expf(-a)) * b);
        } else {
            float v = i8_scaled(__int2float_rn(sum[0]), sx, i8_scale(g.w_scale[at]),
                                g.bias ? __bfloat162float(g.bias[at]) : 0.0f);
            if (ACT == I8_RELU) v = v < 0.0f ? 0.0f : v;
            if (ACT == I8_GELU) {   // Phi(v) from below where v is negative: no cancellation in the tail
                const float t = 0.5f * erfcf(fabsf(v) * 0.70710678118654752f);
                v *= v < 0.0f ? t : 1.0f - t;
            }
            if constexpr (sizeof(OUT) == 2) static_cast<__nv_bfloat16 *>(g.out)[to] = __float2bfloat16_rn(v);
            else static_cast<float *>(g.out)[to] = v;
        }
    }
}

template <int ACT, typename OUT>
moe_status few_launch(const FewArgs &g, cudaStream_t stream) {
    const int per = 8 * (ACT == I8_SWIGLU ? 1 : CPW);
    const dim3 grid((unsigned)((g.n_out + per - 1) / per), (unsigned)(g.so.offsets ? g.so.n : 1));
    // rows in one pass over an expert's weights: up to 4 experts get two rows in all, and of many experts few
    // have more than two
    if (g.so.n == 1) return launch_pdl(int8_few_kernel<ACT, 1, OUT>, grid, dim3(256), 0, stream, g);
    return launch_pdl(int8_few_kernel<ACT, 2, OUT>, grid, dim3(256), 0, stream, g);
}

moe_status few(int act, bool f32, const FewArgs &g, cudaStream_t stream) {
    switch (act) {
        case I8_RELU: return few_launch<I8_RELU, __nv_bfloat16>(g, stream);
        case I8_GELU: return few_launch<I8_GELU, __nv_bfloat16>(g, stream);
        case I8_SWIGLU: return few_launch<I8_SWIGLU, __nv_bfloat16>(g, stream);
        default: return f32 ? few_launch<I8_BIAS, float>(g, stream) : few_launch<I8_BIAS, __nv_bfloat16>(g, stream);
    }
}

// Whether n rows in all go by dot products.  Each row costs them time, the tiles hardly any, so that the rows an
// expert has decide, of which the host knows only the average (FFN, cold, dot products | tiles, us): 1 expert
// 4096 x 8192, 2 rows 34 | 52, 4 rows 53 | 52; 8 experts of that size, 4 rows 56 | 56, 8 rows 83 | 74; 64 experts
// 1024 x 704, 32 rows 32 | 39, 64 rows 48 | 48; 256 experts 2048 x 512, 64 rows 70 | 75.  That is spread routing.
// With all rows on one expert, whose weights are then read once for every two rows, this is the slower side (SwiGLU;
// 64 experts 1024 x 704, 16 rows 38, 32 rows 62 | 28; 256 experts 2048 x 512, 32 rows 83, 64 rows 150 | 34).
bool few_rows8(int64_t n, int e) { return n <= (e <= 4 ? 2 : e < 128 ? e / 2 : 64); }

constexpr int64_t up256(int64_t b) { return (b + 255) & ~(int64_t)255; }

const int32_t *rows_end(const SortedRows &so, int e) { return so.offsets ? so.offsets + e : nullptr; }

moe_status widen(const void *q, void *dst, const SortedRows &so, int e, int cols, int32_t *st, cudaStream_t stream) {
    const int64_t per = 256 * WN_U, want = (so.n * (cols / 8) + per - 1) / per, cap = (int64_t)sm_count() * 8;
    return launch_pdl(widen_rows_kernel, dim3((unsigned)(want < cap ? want : cap)), dim3(256), 0, stream,
                      (const uint2 *)q, (uint4 *)dst, rows_end(so, e), so.n, cols / 8, st);
}

}  // namespace

moe_status quantize_rows_int8_launch(const void *src, moe_dtype sdt, const int32_t *rows, int64_t s, int cols, int k,
                                     int64_t n, void *q, float *scale, int32_t *st, cudaStream_t stream) {
    const QuantArgs g{src, rows, nullptr, q, scale, s, n, cols, k, st};
    if (rows)
        return sdt == MOE_BF16 ? quantize_typed<__nv_bfloat16, int8_t, true>(g, stream)
                               : quantize_typed<float, int8_t, true>(g, stream);
    return sdt == MOE_BF16 ? quantize_typed<__nv_bfloat16, int8_t, false>(g, stream)
                           : quantize_typed<float, int8_t, false>(g, stream);
}

// The rows as fp16 numbers, for the tensor-core form.
size_t product_int8_workspace_bytes(int e, int64_t n, int k) {
    return (size_t)(few_rows8(n, e) ? 256 : up256(n * k * 2));
}

moe_status product_int8_launch(const void *a_q, const float *a_scale, const SortedRows &so, const void *b_q,
                               const float *b_scale, const void *bias, int e, int k, int n_out, void *ws, void *out,
                               bool f32, int32_t *st, cudaStream_t stream) {
    if (few_rows8(so.n, e)) {
        const FewArgs g{(const int8_t *)a_q, (const int8_t *)b_q, nullptr, a_scale, b_scale, nullptr,
                        (const __nv_bfloat16 *)bias, out, so, e, k, n_out, st};
        return few(I8_BIAS, f32, g, stream);
    }
    const moe_status r = widen(a_q, ws, so, e, k, st, stream);
    if (r != MOE_OK) return r;
    return i8_gemm_launch(ws, a_scale, so, b_q, b_scale, nullptr, nullptr, bias, I8_BIAS, f32, e, k, n_out, out, st,
                          stream);
}

// Workspace of the FFN: the hidden (bf16), its scales, its codes (int8 or fp16), the rows as fp16.
struct FfnInt8Layout {
    int64_t hid, scale, code, x16, total;
};

FfnInt8Layout ffn_int8_layout(int e, int64_t n, int m, int h) {
    FfnInt8Layout L{};
    L.scale = up256(n * h * 2);
    L.code = L.scale + up256(n * 4);
    L.x16 = L.code + up256(n * h * (few_rows8(n, e) ? 1 : 2));
    L.total = L.x16 + (few_rows8(n, e) ? 0 : up256(n * m * 2));
    return L;
}

size_t ffn_int8_workspace_bytes(int e, int64_t n, int m, int h) { return (size_t)ffn_int8_layout(e, n, m, h).total; }

moe_status ffn_int8_launch(const void *x_q, const float *x_scale, const SortedRows &so, const void *w1_q,
                           const float *w1_scale, const void *b1, const void *w3_q, const float *w3_scale,
                           const void *w2_q, const float *w2_scale, const void *b2, moe_act act, int e, int m, int h,
                           void *ws, void *out, int32_t *st, cudaStream_t stream) {
    const FfnInt8Layout L = ffn_int8_layout(e, so.n, m, h);
    char *w = (char *)ws;
    const int a = act == MOE_ACT_RELU ? I8_RELU : act == MOE_ACT_GELU ? I8_GELU : I8_SWIGLU;
    float *hs = (float *)(w + L.scale);
    const QuantArgs hq{w + L.hid, nullptr, rows_end(so, e), w + L.code, hs, so.n, so.n, h, 0, st};
    moe_status r;
    if (few_rows8(so.n, e)) {
        const FewArgs g1{(const int8_t *)x_q, (const int8_t *)w1_q, (const int8_t *)w3_q, x_scale, w1_scale, w3_scale,
                         (const __nv_bfloat16 *)b1, w + L.hid, so, e, m, h, st};
        if ((r = few(a, false, g1, stream)) != MOE_OK) return r;
        if ((r = quantize_typed<__nv_bfloat16, int8_t, false>(hq, stream)) != MOE_OK) return r;
        const FewArgs g2{(const int8_t *)(w + L.code), (const int8_t *)w2_q, nullptr, hs, w2_scale, nullptr,
                         (const __nv_bfloat16 *)b2, out, so, e, h, m, st};
        return few(I8_BIAS, false, g2, stream);
    }
    if ((r = widen(x_q, w + L.x16, so, e, m, st, stream)) != MOE_OK) return r;
    r = i8_gemm_launch(w + L.x16, x_scale, so, w1_q, w1_scale, w3_q, w3_scale, b1, a, false, e, m, h, w + L.hid, st,
                       stream);
    if (r != MOE_OK) return r;
    if ((r = quantize_typed<__nv_bfloat16, __half, false>(hq, stream)) != MOE_OK) return r;
    return i8_gemm_launch(w + L.code, hs, so, w2_q, w2_scale, nullptr, nullptr, b2, I8_BIAS, false, e, h, m, out, st,
                          stream);
}

}  // namespace moe
