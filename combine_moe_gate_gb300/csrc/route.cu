// Routing from router logits: scores, balance bias, group-limited top-k, and
// the gradient of the gates with respect to the logits.
//
// Per token, with l the e logits:
//   score_j  = 1 / (1 + exp(-l_j))                      (sigmoid), or
//              exp(l_j - max l) / sum_i exp(l_i - max l) (softmax);
//   choice_j = score_j + bias_j; -inf for a masked expert (l_j = -inf) or NaN;
//   group value = sum of the group's best group_top live choices (-inf: none);
//   idx = the k best experts of the topk_groups best groups by (choice
//   descending, index ascending); gates = score[idx] (/ their sum) * scale.
// The bias steers the choice only, so it has no gradient and the gates stay
// the scores' own.  Scores use the correctly rounded division and one fixed
// summation order (adjacent pairs over the width padded to a power of two),
// so idx is reproducible bit for bit.
#include "common.cuh"

namespace moe {
namespace {

constexpr int RT_WARPS = 8;

template <typename T> __device__ __forceinline__ float ld_logit(const T *p);
template <> __device__ __forceinline__ float ld_logit<float>(const float *p) { return __ldg(p); }
template <> __device__ __forceinline__ float ld_logit<__nv_bfloat16>(const __nv_bfloat16 *p) {
    return __bfloat162float(*p);
}

// Order-preserving map of a float to an unsigned key (-0 as +0); never 0.
__device__ __forceinline__ uint32_t order_key(float f) {
    const uint32_t b = __float_as_uint(__fadd_rn(f, 0.0f));
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The sigmoid; the additions and the division are single IEEE operations.
__device__ __forceinline__ float sigmoid_rn(float l) { return __frcp_rn(__fadd_rn(1.0f, expf(-l))); }

// Scores of one token over a warp: lane holds experts lane * V .. + V - 1.
// Padding enters as exp = 0.
template <int V, bool SOFTMAX>
__device__ __forceinline__ void scores(const float (&l)[V], int e, int lane, float (&sc)[V]) {
    if (!SOFTMAX) {
#pragma unroll
        for (int i = 0; i < V; i++) sc[i] = sigmoid_rn(l[i]);
        return;
    }
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; i++) top = fmaxf(top, l[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (top == -INFINITY) {   // nothing left (scores 0), or nothing but NaN and -inf
        bool nan = false;
#pragma unroll
        for (int i = 0; i < V; i++) nan |= l[i] != l[i];
        const float v = __any_sync(0xffffffffu, nan) ? NAN : 0.0f;
#pragma unroll
        for (int i = 0; i < V; i++) sc[i] = v;
        return;
    }
    float t[V];
#pragma unroll
    for (int i = 0; i < V; i++) {
        sc[i] = lane * V + i < e ? expf(__fsub_rn(l[i], top)) : 0.0f;
        t[i] = sc[i];
    }
#pragma unroll
    for (int n = V; n > 1; n >>= 1)
#pragma unroll
        for (int i = 0; i < n / 2; i++) t[i] = __fadd_rn(t[2 * i], t[2 * i + 1]);
    float sum = t[0];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, o));
#pragma unroll
    for (int i = 0; i < V; i++) sc[i] = __fdiv_rn(sc[i], sum);
}

// One warp per token, V = 2^p / 32 experts per lane in index order.
template <typename T, int V, bool SOFTMAX>
__global__ void __launch_bounds__(RT_WARPS * 32)
route_topk_kernel(const T *__restrict__ logits, const float *__restrict__ bias, int64_t s, int e,
                  int k, int groups, int topk_groups, int group_top, float scale, int normalize,
                  int32_t *__restrict__ idx, float *__restrict__ gates, int32_t *status) {
    __shared__ float s_choice[RT_WARPS][V * 32];
    pdl_enter();
    if (status_bad(status)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gs = e / groups;
    for (int64_t t = (int64_t)blockIdx.x * RT_WARPS + warp; t < s; t += (int64_t)gridDim.x * RT_WARPS) {
        float l[V], sc[V];
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int j = lane * V + i;
            l[i] = j < e ? ld_logit(logits + t * e + j) : -INFINITY;
        }
        scores<V, SOFTMAX>(l, e, lane, sc);
        float ch[V];
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int j = lane * V + i;
            ch[i] = bias && j < e ? __fadd_rn(sc[i], bias[j]) : sc[i];
            if (l[i] == -INFINITY || ch[i] != ch[i]) ch[i] = -INFINITY;
        }
        uint32_t kept = 0xffffffffu;
        if (groups > 1) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < V; i++) s_choice[warp][lane * V + i] = ch[i];
            __syncwarp();
            uint32_t gk = 0;   // no group on this lane: below every group
            if (lane < groups) {
                float a = -INFINITY, b = -INFINITY;   // the two best of this lane's group
                for (int i = 0; i < gs; i++) {
                    const float v = s_choice[warp][lane * gs + i];
                    b = fmaxf(b, fminf(a, v));
                    a = fmaxf(a, v);
                }
                gk = order_key(group_top == 2 && b > -INFINITY ? __fadd_rn(a, b) : a);
            }
            int ahead = 0;
            for (int g = 0; g < groups; g++) {
                const uint32_t o = __shfl_sync(0xffffffffu, gk, g);
                ahead += o > gk || (o == gk && g < lane);
            }
            kept = __ballot_sync(0xffffffffu, lane < groups && ahead < topk_groups);
        }
        uint32_t key[V];
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int j = lane * V + i;
            key[i] = j < e && (groups == 1 || (kept >> (j / gs) & 1)) ? order_key(ch[i]) : 0u;
        }
        float g_mine = 0.0f, sum = 0.0f;
        int j_mine = 0;
        for (int r = 0; r < k; r++) {
            uint32_t best = 0;
#pragma unroll
            for (int i = 0; i < V; i++) best = max(best, key[i]);
            const uint32_t top = __reduce_max_sync(0xffffffffu, best);
            const int src = __ffs(__ballot_sync(0xffffffffu, best == top)) - 1;
            int j = 0;
            float g = 0.0f;
            bool taken = false;
#pragma unroll
            for (int i = 0; i < V; i++)
                if (lane == src && !taken && key[i] == top) {
                    taken = true;
                    key[i] = 0u;
                    j = lane * V + i;
                    g = sc[i];
                }
            j = __shfl_sync(0xffffffffu, j, src);
            g = __shfl_sync(0xffffffffu, g, src);
            sum = __fadd_rn(sum, g);
            if (lane == r) { j_mine = j; g_mine = g; }
        }
        if (lane < k) {
            if (normalize) g_mine = sum == 0.0f ? 0.0f : __fdiv_rn(g_mine, sum);
            idx[(int64_t)lane * s + t] = j_mine;
            gates[(int64_t)lane * s + t] = g_mine * scale;
        }
    }
}

// d_logits of one token per warp.  With g the selected scores, G = g / sum g
// (normalised) and A = sum_r dg_r G_r:
//   softmax, normalised: scale G (dg - A) at the selection, 0 elsewhere;
//   softmax, raw:        scale (p dg [selected] - p sum_r dg_r p_r) everywhere;
//   sigmoid, normalised: scale G (dg - A)(1 - g) at the selection;
//   sigmoid, raw:        scale dg g (1 - g) at the selection.
template <typename T, typename D, int V, bool SOFTMAX>
__global__ void __launch_bounds__(RT_WARPS * 32)
route_bwd_kernel(const T *__restrict__ logits, const int32_t *__restrict__ idx,
                 const float *__restrict__ d_gates, int64_t s, int e, int k, float scale,
                 int normalize, D *__restrict__ d_logits, int32_t *status) {
    __shared__ float s_d[RT_WARPS][V * 32];
    pdl_enter();
    if (status_bad(status)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t t = (int64_t)blockIdx.x * RT_WARPS + warp; t < s; t += (int64_t)gridDim.x * RT_WARPS) {
        float l[V], sc[V];
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int j = lane * V + i;
            l[i] = j < e ? ld_logit(logits + t * e + j) : -INFINITY;
        }
        scores<V, SOFTMAX>(l, e, lane, sc);
        int j = lane < k ? idx[(int64_t)lane * s + t] : 0;
        if (__any_sync(0xffffffffu, j < 0 || j >= e)) {
            if (lane == 0) set_status(status, MOE_ERR_INVALID_ARG);
            return;
        }
        const float dg = lane < k ? d_gates[(int64_t)lane * s + t] : 0.0f;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < V; i++) s_d[warp][lane * V + i] = sc[i];
        __syncwarp();
        const float g = lane < k ? s_d[warp][j] : 0.0f;
        float total = g, dot = dg * g;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            total += __shfl_xor_sync(0xffffffffu, total, o);
            dot += __shfl_xor_sync(0xffffffffu, dot, o);
        }
        float d;
        if (normalize) d = total == 0.0f ? 0.0f : scale * (g / total) * (dg - dot / total);
        else d = scale * dg * g;
        if (!SOFTMAX) d *= 1.0f - g;
        const float back = SOFTMAX && !normalize ? scale * dot : 0.0f;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < V; i++) s_d[warp][lane * V + i] = -sc[i] * back;
        __syncwarp();
        if (lane < k) s_d[warp][j] += d;
        __syncwarp();
        for (int i = lane; i < e; i += 32) d_logits[t * e + i] = (D)s_d[warp][i];
        __syncwarp();
    }
}

int grid_for(int64_t s) {
    static int cached[64] = {0};
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64) {
        if (!cached[dev]) cudaDeviceGetAttribute(&cached[dev], cudaDevAttrMultiProcessorCount, dev);
        if (cached[dev] > 0) sms = cached[dev];
    }
    const int64_t want = (s + RT_WARPS - 1) / RT_WARPS, cap = (int64_t)sms * 8;
    return (int)(want < cap ? want : cap);
}

template <typename T, int V>
moe_status topk_v(const void *logits, const float *bias, int64_t s, int e, int k, bool softmax,
                  int groups, int topk_groups, int group_top, float scale, int normalize,
                  int32_t *idx, float *gates, int32_t *st, cudaStream_t stream) {
    auto kern = softmax ? route_topk_kernel<T, V, true> : route_topk_kernel<T, V, false>;
    return launch_pdl(kern, dim3(grid_for(s)), dim3(RT_WARPS * 32), 0, stream, (const T *)logits,
                      bias, s, e, k, groups, topk_groups, group_top, scale, normalize, idx, gates, st);
}

template <typename T, typename D, int V>
moe_status bwd_v(const void *logits, const int32_t *idx, const float *d_gates, int64_t s, int e,
                 int k, bool softmax, float scale, int normalize, void *d_logits, int32_t *st,
                 cudaStream_t stream) {
    auto kern = softmax ? route_bwd_kernel<T, D, V, true> : route_bwd_kernel<T, D, V, false>;
    return launch_pdl(kern, dim3(grid_for(s)), dim3(RT_WARPS * 32), 0, stream, (const T *)logits,
                      idx, d_gates, s, e, k, scale, normalize, (D *)d_logits, st);
}

}  // namespace

// Experts per lane: e padded to a power of two of at least 32.
#define MOE_BY_V(CALL)                 \
    if (e <= 32) return CALL(1);       \
    if (e <= 64) return CALL(2);       \
    if (e <= 128) return CALL(4);      \
    if (e <= 256) return CALL(8);      \
    if (e <= 512) return CALL(16);     \
    return CALL(32)

moe_status route_topk_launch(const void *logits, moe_dtype ldt, const float *bias, int64_t s, int e,
                             int k, moe_score score, int groups, int topk_groups, int group_top,
                             float scale, unsigned flags, int32_t *idx, float *gates, int32_t *st,
                             cudaStream_t stream) {
    const bool sm = score == MOE_SCORE_SOFTMAX;
    const int nrm = (flags & MOE_FLAG_NORMALIZE_GATES) != 0;
#define MOE_F(V) topk_v<float, V>(logits, bias, s, e, k, sm, groups, topk_groups, group_top, scale, nrm, idx, gates, st, stream)
#define MOE_B(V) topk_v<__nv_bfloat16, V>(logits, bias, s, e, k, sm, groups, topk_groups, group_top, scale, nrm, idx, gates, st, stream)
    if (ldt == MOE_F32) { MOE_BY_V(MOE_F); }
    MOE_BY_V(MOE_B);
#undef MOE_F
#undef MOE_B
}

moe_status route_bwd_launch(const void *logits, moe_dtype ldt, const int32_t *idx,
                            const float *d_gates, int64_t s, int e, int k, moe_score score,
                            float scale, unsigned flags, void *d_logits, moe_dtype ddt, int32_t *st,
                            cudaStream_t stream) {
    const bool sm = score == MOE_SCORE_SOFTMAX;
    const int nrm = (flags & MOE_FLAG_NORMALIZE_GATES) != 0;
    using bf = __nv_bfloat16;
#define MOE_FF(V) bwd_v<float, float, V>(logits, idx, d_gates, s, e, k, sm, scale, nrm, d_logits, st, stream)
#define MOE_FB(V) bwd_v<float, bf, V>(logits, idx, d_gates, s, e, k, sm, scale, nrm, d_logits, st, stream)
#define MOE_BF(V) bwd_v<bf, float, V>(logits, idx, d_gates, s, e, k, sm, scale, nrm, d_logits, st, stream)
#define MOE_BB(V) bwd_v<bf, bf, V>(logits, idx, d_gates, s, e, k, sm, scale, nrm, d_logits, st, stream)
    if (ldt == MOE_F32 && ddt == MOE_F32) { MOE_BY_V(MOE_FF); }
    if (ldt == MOE_F32) { MOE_BY_V(MOE_FB); }
    if (ddt == MOE_F32) { MOE_BY_V(MOE_BF); }
    MOE_BY_V(MOE_BB);
#undef MOE_FF
#undef MOE_FB
#undef MOE_BF
#undef MOE_BB
}
#undef MOE_BY_V

}  // namespace moe
