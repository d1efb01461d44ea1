// The expert FFN on few sorted rows (bf16), which the grouped tiles of 256 rows would be mostly empty for.
//
//   hid = act(x W1^T + b1), or silu(x W1^T) * (x W3^T); out = hid W2^T + b2
//
// Bound by the weights' bytes, so the weights are read once for up to 32 rows of one expert (of many: once for every
// 8 rows) and little else is asked of the multiprocessor.  A CTA owns 16 output channels (SwiGLU: of W1 and of W3); its warps share K, 256 bytes
// of a channel's row at a time, and add up in shared memory in order.  The arithmetic is mma.sync
// (16 channels x 8 rows): tcgen05 would want 128 channels, and too few CTAs would then hold the loads.
// A sum may take its terms in any order, so the MMAs' K slots are filled as the loads come: lane 4 g + t
// reads 16 bytes of channels g and g + 8 and of row g at the same place, and two MMAs take them.
// CTA (x, y): channels, and the expert whose first row is row y (the others leave).
// Measured: 5 tokens x 4 of 64 SwiGLU experts, 1024 x 704 (18 experts' weights, 78 MB): 19 us in calls, 4 TB/s; one
// row of an expert of 4096 x 8192 (134 MB): 33 us, 4 TB/s: the two launches' ramps.
#include "common.cuh"

namespace moe {
namespace {

using bf = __nv_bfloat16;
constexpr int FU = 4;       // 64-byte blocks of K under way
enum { FEW_OUT = 3 };       // beside the activations (moe_act): the second product

struct FewArgs {
    const bf *x, *w, *w3, *bias;
    bf *out, *pre;          // pre: null, or the pre-activation (SwiGLU: a, then b)
    SortedRows so;
    int e, K, n_out;
    int32_t *status;
};

__device__ __forceinline__ void mma_row(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// NB: blocks of 8 rows in one pass over the weights.  FW: warps a CTA.
template <int ACT, int NB, int FW>
__global__ void __launch_bounds__(FW * 32, ACT == MOE_ACT_SWIGLU || NB > 1 ? 16 / FW : 32 / FW)
ffn_few_kernel(const FewArgs g) {
    pdl_enter();
    if (status_bad(g.status)) return;
    constexpr bool SWI = ACT == MOE_ACT_SWIGLU;
    constexpr int M = SWI ? 2 : 1;
    __shared__ float part[FW][M][16][NB * 8 + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, y = blockIdx.y;
    int j = 0;
    bool bad = false;
    for (int b = lane; b < g.e; b += 32) {   // experts that end at or before row y
        const int o = g.so.offsets[b], p = g.so.offsets[b + 1];
        j += p <= y;
        bad |= o < 0 || p < o || p > g.so.n || (b == 0 && o != 0);
    }
    if (bad) set_status(g.status, MOE_ERR_INVALID_ARG);
    j = __reduce_add_sync(0xffffffffu, j);
    if (__any_sync(0xffffffffu, bad) || j >= g.e) return;   // the same in every warp of the CTA
    int64_t lo, count;
    sorted_span(g.so, j, lo, count);
    if (lo != y) return;
    const int gr = lane >> 2, t = lane & 3, ch0 = blockIdx.x * 16;
    const int pieces = g.K / 8, groups = (pieces + 4 * FU - 1) / (4 * FU);
    const bool upper = ch0 + 8 < g.n_out;   // n_out is a multiple of 8: whole halves
    const V16 *wp[M][2];
#pragma unroll
    for (int q = 0; q < M; q++)
#pragma unroll
        for (int hf = 0; hf < 2; hf++)
            wp[q][hf] = reinterpret_cast<const V16 *>(q ? g.w3 : g.w) +
                        ((int64_t)j * g.n_out + ch0 + gr + (hf && upper ? 8 : 0)) * pieces + t;
    const V16 *xp = reinterpret_cast<const V16 *>(g.x) + t;
    for (int64_t r0 = lo; r0 < lo + count; r0 += 8 * NB) {
        float acc[M][NB][4] = {};
        for (int gi = warp; gi < groups; gi += FW) {
            const int p0 = gi * 4 * FU;
            V16 wv[FU][M][2];
#pragma unroll
            for (int u = 0; u < FU; u++)
#pragma unroll
                for (int q = 0; q < M; q++)
#pragma unroll
                    for (int hf = 0; hf < 2; hf++)
                        wv[u][q][hf] = ld_stream_if(wp[q][hf] + p0 + 4 * u, p0 + 4 * u + t < pieces && (!hf || upper));
#pragma unroll
            for (int u = 0; u < FU; u++)
#pragma unroll
                for (int b = 0; b < NB; b++) {
                    const int64_t row = r0 + 8 * b + gr;
                    const V16 xv = ld_v16_if(xp + row * pieces + p0 + 4 * u, p0 + 4 * u + t < pieces && row < lo + count);
#pragma unroll
                    for (int q = 0; q < M; q++) {
                        const V16 &a = wv[u][q][0], &c = wv[u][q][1];
                        const uint32_t f0[4] = {a.w[0], c.w[0], a.w[1], c.w[1]}, f1[4] = {a.w[2], c.w[2], a.w[3], c.w[3]};
                        mma_row(acc[q][b], f0, xv.w[0], xv.w[1]);
                        mma_row(acc[q][b], f1, xv.w[2], xv.w[3]);
                    }
                }
        }
#pragma unroll
        for (int q = 0; q < M; q++)
#pragma unroll
            for (int b = 0; b < NB; b++)
#pragma unroll
                for (int i = 0; i < 4; i++) part[warp][q][gr + (i >> 1) * 8][8 * b + 2 * t + (i & 1)] = acc[q][b][i];
        __syncthreads();
        const int c = threadIdx.x & 15, ch = ch0 + c;
        for (int rr = threadIdx.x >> 4; rr < 8 * NB; rr += FW * 2) {
            const int64_t row = r0 + rr;
            if (row >= lo + count || ch >= g.n_out) continue;
            float sum[M];
#pragma unroll
            for (int q = 0; q < M; q++) {
                sum[q] = part[0][q][c][rr];
#pragma unroll
                for (int w = 1; w < FW; w++) sum[q] += part[w][q][c][rr];
            }
            float v = sum[0];
            if (!SWI && g.bias) v += __bfloat162float(g.bias[(int64_t)j * g.n_out + ch]);
            if (ACT != FEW_OUT && g.pre) {
                bf *pre = g.pre + row * M * g.n_out + ch;
                pre[0] = __float2bfloat16_rn(v);
                if (SWI) pre[g.n_out] = __float2bfloat16_rn(sum[M - 1]);
            }
            if (ACT == MOE_ACT_RELU) v = relu_nan(v);
            if (ACT == MOE_ACT_GELU)   // Phi(v) from below where v is negative: no cancellation in the tail
                v = v < 0.0f ? v * 0.5f * erfcf(-v * 0.70710678118654752f)
                             : v * (1.0f - 0.5f * erfcf(v * 0.70710678118654752f));
            if (SWI) v = v / (1.0f + expf(-v)) * sum[M - 1];
            g.out[row * g.n_out + ch] = __float2bfloat16_rn(v);
        }
        __syncthreads();   // part is written again in the next pass
    }
}

template <int ACT, int NB>
moe_status few_launch(const FewArgs &g, cudaStream_t stream) {
    const unsigned ctas = (unsigned)((g.n_out + 15) / 16);
    const dim3 grid(ctas, (unsigned)g.so.n);
    // 16 warps where the channels of the experts at work (at most one a row) give few CTAs to a multiprocessor
    if constexpr (NB == 1)
        if ((int64_t)ctas * (g.so.n < g.e ? g.so.n : g.e) <= 304)
            return launch_pdl(ffn_few_kernel<ACT, NB, 16>, grid, dim3(512), 0, stream, g);
    return launch_pdl(ffn_few_kernel<ACT, NB, 8>, grid, dim3(256), 0, stream, g);
}

template <int ACT>
moe_status few_typed(const FewArgs &g, cudaStream_t stream) {
    // rows in one pass: all of them with one expert; of many experts few have more than 8
    if (g.e > 1 || g.so.n <= 8) return few_launch<ACT, 1>(g, stream);
    return g.so.n <= 16 ? few_launch<ACT, 2>(g, stream) : few_launch<ACT, 4>(g, stream);
}

}  // namespace

// Whether n rows in all go this way: more rows an expert, of which the host knows only the average, cost more here
// and nothing there (FFN, cold, here | tiles, us): 1 expert 4096 x 8192, 1 row 34 | 110, 16 rows 56 | 109, 32
// rows 91 | 108, 64 rows 173 | 110; 8 experts of that size, 16 rows 174 | 204, 32 rows 189 | 204, 48 rows 243 | 204;
// 64 experts 1024 x 704, 64 rows 45 | 67, 128 rows 65 | 72; 256 experts 2048 x 512, 128 rows 128 | 155.  That is
// spread routing.  With all rows on one expert, whose weights are then read once for every eight rows, many rows are
// slower here (SwiGLU; 64 experts 1024 x 704, 32 rows 21, 64 rows 35, 128 rows 58 | 38; 256 experts 2048 x 512, 32 rows
// 31, 64 rows 52, 128 rows 95 | 42).
bool few_rows(int64_t n, int e) { return n <= (e <= 16 ? 32 : e < 64 ? 2 * e : 128); }

moe_status ffn_few_launch(const void *x, const SortedRows &so, const void *w1, const void *b1, const void *w3,
                          const void *w2, const void *b2, moe_act act, int e, int m, int h, void *hid, void *pre,
                          void *out, int32_t *st, cudaStream_t stream) {
    const FewArgs g1{(const bf *)x, (const bf *)w1, (const bf *)w3, (const bf *)b1, (bf *)hid, (bf *)pre, so, e, m, h, st};
    const moe_status r = act == MOE_ACT_RELU   ? few_typed<MOE_ACT_RELU>(g1, stream)
                         : act == MOE_ACT_GELU ? few_typed<MOE_ACT_GELU>(g1, stream)
                                               : few_typed<MOE_ACT_SWIGLU>(g1, stream);
    if (r != MOE_OK) return r;
    const FewArgs g2{(const bf *)hid, (const bf *)w2, nullptr, (const bf *)b2, (bf *)out, nullptr, so, e, h, m, st};
    return few_typed<FEW_OUT>(g2, stream);
}

}  // namespace moe
