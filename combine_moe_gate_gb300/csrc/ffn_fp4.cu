// Grouped products of microscaled 4-bit operands and the expert FFN made of
// them.  Simple form: one CTA per 32 x 64 output tile, operands expanded to
// fp32 in shared memory, fp32 fused multiply-adds.
#include "fp4.cuh"

namespace moe {
namespace {

constexpr int BM = 32, BN = 64, BK = 32, NT = 256;

struct Operand {
    const uint8_t *q;
    const uint8_t *scale;
    const float *global;
};

template <int FMT>
__device__ __forceinline__ float value_at(const uint8_t *q, const uint8_t *sc, int64_t row, int k, int K,
                                          int64_t ntiles) {
    const uint32_t by = q[(row * K + k) / 2];
    const uint32_t code = k & 1 ? by >> 4 : by & 15u;
    const uint32_t s = sc[fp4_scale_at(row, k / Fp4<FMT>::BLK, ntiles)];
    return e2m1_value(code) * (FMT == MOE_FP4_MX ? e8m0_value(s) : e4m3_value(s));
}

__device__ __forceinline__ float act_of(float v, int act) {
    if (act == MOE_ACT_RELU) return fmaxf(v, 0.0f);
    return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
}

// act < 0: bf16 out = product + bias; else the activation (SwiGLU with b3),
// quantised to out_q / out_scale with the factors out_global.
template <int FMT>
__global__ void __launch_bounds__(NT)
fp4_product_kernel(Operand a, Operand b, Operand b3, const __nv_bfloat16 *__restrict__ bias,
                   const int32_t *__restrict__ counts, const int32_t *__restrict__ c_dev, int64_t c_max,
                   int K, int N, int act, __nv_bfloat16 *__restrict__ out, uint8_t *__restrict__ out_q,
                   uint8_t *__restrict__ out_scale, const float *__restrict__ out_global, int32_t *status) {
    pdl_enter();
    if (status_bad(status)) return;
    constexpr int BLK = Fp4<FMT>::BLK;
    __shared__ float As[BK][BM + 1], Bs[BK][BN + 1], B3s[BK][BN + 1], Hs[BM][BN + 1];
    const int j = blockIdx.z;
    const int rows = (int)min((int64_t)max(counts[j], 0), min((int64_t)*c_dev, c_max));
    const int r0 = blockIdx.y * BM, n0 = blockIdx.x * BN;
    if (r0 >= rows) return;
    const int64_t nt = fp4_scale_tiles(BLK, K);
    const uint8_t *aq = a.q + j * c_max * (K / 2), *asc = a.scale + j * fp4_scale_bytes(BLK, c_max, K);
    const uint8_t *bq = b.q + (int64_t)j * N * (K / 2), *bsc = b.scale + j * fp4_scale_bytes(BLK, N, K);
    const uint8_t *cq = b3.q + (int64_t)j * N * (K / 2), *csc = b3.scale + j * fp4_scale_bytes(BLK, N, K);
    const int tid = threadIdx.x, tn = tid % 16, tm = tid / 16;
    float acc[2][4] = {}, acc3[2][4] = {};
    for (int k0 = 0; k0 < K; k0 += BK) {
        for (int i = tid; i < BM * BK; i += NT) {
            const int r = i / BK, kk = i % BK;
            As[kk][r] = r0 + r < rows ? value_at<FMT>(aq, asc, r0 + r, k0 + kk, K, nt) : 0.0f;
        }
        for (int i = tid; i < BN * BK; i += NT) {
            const int n = i / BK, kk = i % BK;
            Bs[kk][n] = n0 + n < N ? value_at<FMT>(bq, bsc, n0 + n, k0 + kk, K, nt) : 0.0f;
            if (act == MOE_ACT_SWIGLU) B3s[kk][n] = n0 + n < N ? value_at<FMT>(cq, csc, n0 + n, k0 + kk, K, nt) : 0.0f;
        }
        __syncthreads();
        for (int kk = 0; kk < BK; kk++)
            for (int r = 0; r < 2; r++)
                for (int c = 0; c < 4; c++) {
                    acc[r][c] = fmaf(As[kk][tm * 2 + r], Bs[kk][tn * 4 + c], acc[r][c]);
                    if (act == MOE_ACT_SWIGLU)
                        acc3[r][c] = fmaf(As[kk][tm * 2 + r], B3s[kk][tn * 4 + c], acc3[r][c]);
                }
        __syncthreads();
    }
    const float ga = a.global ? a.global[j] : 1.0f;
    const float s1 = ga * (b.global ? b.global[j] : 1.0f), s3 = ga * (b3.global ? b3.global[j] : 1.0f);
    for (int r = 0; r < 2; r++)
        for (int c = 0; c < 4; c++) {
            const int row = tm * 2 + r, n = n0 + tn * 4 + c;
            float v = acc[r][c] * s1;
            if (bias && n < N) v += __bfloat162float(bias[(int64_t)j * N + n]);
            if (act == MOE_ACT_SWIGLU) v = v / (1.0f + expf(-v)) * (acc3[r][c] * s3);
            else if (act >= 0) v = act_of(v, act);
            if (act < 0) {
                if (r0 + row < rows && n < N) out[(j * c_max + r0 + row) * N + n] = __float2bfloat16_rn(v);
            } else {
                Hs[row][tn * 4 + c] = n < N ? v : 0.0f;
            }
        }
    if (act < 0) return;
    __syncthreads();
    const float g = FMT == MOE_FP4_NV && out_global ? out_global[j] : 1.0f;
    const int64_t hnt = fp4_scale_tiles(BLK, N);
    uint8_t *osc = out_scale + j * fp4_scale_bytes(BLK, c_max, N);
    for (int i = tid; i < BM * (BN / BLK); i += NT) {
        const int row = i / (BN / BLK), blk = i % (BN / BLK), n = n0 + blk * BLK;
        if (r0 + row >= rows) continue;
        float f[BLK], amax = 0.0f, inv;
        for (int x = 0; x < BLK; x++) { f[x] = Hs[row][blk * BLK + x]; amax = amax_nan(amax, f[x]); }
        const uint32_t sc = fp4_scale<FMT>(amax, g, __fmul_rn(g, 6.0f), inv);
        if (n / BLK < hnt * 4) osc[fp4_scale_at(r0 + row, n / BLK, hnt)] = (uint8_t)(n < N ? sc : 0u);
        if (n >= N) continue;
        for (int x = 0; x < BLK; x++) f[x] *= inv;
        for (int x = 0; x < BLK; x += 8)
            *reinterpret_cast<uint32_t *>(out_q + ((j * c_max + r0 + row) * N + n + x) / 2) = e2m1x8(f + x);
    }
    // the last scale tile's blocks past the row, where it reaches past this CTA's columns
    if (n0 + BN >= N)
        for (int i = tid; i < BM * 4; i += NT) {
            const int row = i / 4;
            const int64_t blk = (n0 + BN) / BLK + i % 4;
            if (r0 + row < rows && blk < hnt * 4) osc[fp4_scale_at(r0 + row, (int)blk, hnt)] = 0;
        }
}

moe_status product(moe_fp4 fmt, const Operand &a, const Operand &b, const Operand &b3, const void *bias,
                   const int32_t *counts, const int32_t *c_dev, int e, int64_t c_max, int K, int N, int act,
                   void *out, void *out_q, void *out_scale, const float *out_global, int32_t *st,
                   cudaStream_t stream) {
    auto kern = fmt == MOE_FP4_MX ? fp4_product_kernel<MOE_FP4_MX> : fp4_product_kernel<MOE_FP4_NV>;
    return launch_pdl(kern, dim3((N + BN - 1) / BN, (unsigned)((c_max + BM - 1) / BM), e), dim3(NT), 0, stream,
                      a, b, b3, (const __nv_bfloat16 *)bias, counts, c_dev, c_max, K, N, act,
                      (__nv_bfloat16 *)out, (uint8_t *)out_q, (uint8_t *)out_scale, out_global, st);
}

}  // namespace

moe_status product_fp4_launch(const void *a_q, const void *a_scale, const float *a_global,
                              const int32_t *counts, const int32_t *c_dev, const void *b_q,
                              const void *b_scale, const float *b_global, const void *bias,
                              moe_fp4 fmt, int e, int64_t c_max, int k, int n, void *out,
                              int32_t *st, cudaStream_t stream) {
    const Operand a{(const uint8_t *)a_q, (const uint8_t *)a_scale, a_global};
    const Operand b{(const uint8_t *)b_q, (const uint8_t *)b_scale, b_global};
    return product(fmt, a, b, b, bias, counts, c_dev, e, c_max, k, n, -1, out, nullptr, nullptr, nullptr,
                   st, stream);
}

moe_status ffn_fp4_launch(const void *buf_q, const void *buf_scale, const float *buf_global,
                          const float *hid_global, const int32_t *counts, const int32_t *c_dev,
                          const void *w1_q, const void *w1_scale, const float *w1_global,
                          const void *b1, const void *w3_q, const void *w3_scale,
                          const float *w3_global, const void *w2_q, const void *w2_scale,
                          const float *w2_global, const void *b2, moe_fp4 fmt, moe_act act, int e,
                          int64_t c_max, int m, int h, void *hid_q, void *hid_scale, void *out,
                          int32_t *st, cudaStream_t stream) {
    const Operand x{(const uint8_t *)buf_q, (const uint8_t *)buf_scale, buf_global};
    const Operand w1{(const uint8_t *)w1_q, (const uint8_t *)w1_scale, w1_global};
    const Operand w3{(const uint8_t *)w3_q, (const uint8_t *)w3_scale, w3_global};
    const Operand w2{(const uint8_t *)w2_q, (const uint8_t *)w2_scale, w2_global};
    const Operand hid{(const uint8_t *)hid_q, (const uint8_t *)hid_scale, hid_global};
    moe_status r = product(fmt, x, w1, act == MOE_ACT_SWIGLU ? w3 : w1, b1, counts, c_dev, e, c_max, m, h,
                           (int)act, nullptr, hid_q, hid_scale, hid_global, st, stream);
    if (r != MOE_OK) return r;
    return product(fmt, hid, w2, w2, b2, counts, c_dev, e, c_max, h, m, -1, out, nullptr, nullptr, nullptr,
                   st, stream);
}

}  // namespace moe
