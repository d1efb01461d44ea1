// Routing from router logits: scores, balance bias, group-limited top-k, and
// the gradient of the gates with respect to the logits.
//
// Per token, with l the e logits:
//   score_j  = 1 / (1 + exp(-l_j))                      (sigmoid), or
//              exp(l_j - max l) / sum_i exp(l_i - max l) (softmax);
//   choice_j = score_j + bias_j; -inf for a masked expert (l_j = -inf) or NaN;
//   group value = sum of the group's best group_top (1|2) live choices (-inf: none);
//   idx = the k best experts of the topk_groups best groups by (choice
//   descending, index ascending); gates = score[idx] (/ their sum) * scale.
// The bias steers the choice only, so it has no gradient and the gates stay
// the scores' own.  Scores use the correctly rounded division and one fixed
// summation order (adjacent pairs over the width padded to a power of two),
// so idx is reproducible bit for bit.
//
// Forward and backward read or write each logit once; at the sizes of a layer
// the forward is bound by its instructions (a sigmoid's exp and division are
// about 20 per expert), so its layout is chosen to spend few of them: L lanes
// share a token and hold V = width / L consecutive experts each, with V = 8
// where the width allows, so that 32 / L tokens run in one warp.  Measured: 16384
// x 256 sigmoid, 8 groups, top 8: 14.9 us (17.9 MB; 73% of the issue slots);
// 65536 x 64 softmax, top 2: 12.2 us; one token: 2.9 us.  The gradient of 16384
// x 256: 6.2 us, renormalised softmax 7.8.
#include "exact.cuh"

namespace moe {
namespace {

constexpr int RT_THREADS = 256;
constexpr int RT_WARPS = RT_THREADS / 32;

template <typename T> __device__ __forceinline__ float ld_logit(const T *p);
template <> __device__ __forceinline__ float ld_logit<float>(const float *p) { return __ldg(p); }
template <> __device__ __forceinline__ float ld_logit<__nv_bfloat16>(const __nv_bfloat16 *p) {
    return __bfloat162float(*p);
}

// V logits of a token from expert j0 on; `pad` past the last expert.  vec: rows
// are whole 16-byte chunks (e * sizeof(T) % 16 == 0), so a chunk is either
// inside a row or past it.
template <typename T, int V>
__device__ __forceinline__ void ld_logits(const T *row, int j0, int e, bool vec, float pad, float (&l)[V]) {
    constexpr int N = Elt<T>::VEC;
    if (V % N == 0 && vec) {
#pragma unroll
        for (int c = 0; c < V / N; c++) {
            if (j0 + c * N < e) {
                float f[N];
                Elt<T>::unpack(ld_stream(row + j0 + c * N), f);
#pragma unroll
                for (int i = 0; i < N; i++) l[c * N + i] = f[i];
            } else {
#pragma unroll
                for (int i = 0; i < N; i++) l[c * N + i] = pad;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; i++) l[i] = j0 + i < e ? ld_logit(row + j0 + i) : pad;
    }
}

// Order-preserving map of a float to an unsigned key; never 0.  (A choice is a
// score, at least +0, or its sum with a bias, and a group's value a sum of
// choices: none of them is -0.)
__device__ __forceinline__ uint32_t order_key(float f) {
    const uint32_t b = __float_as_uint(f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// The sigmoid; the addition and the division are single IEEE operations.
__device__ __forceinline__ float sigmoid_rn(float l) { return __frcp_rn(__fadd_rn(1.0f, expf(-l))); }

// Scores of a token over its L lanes, V consecutive experts a lane.  Padding:
// logits of 0 (sigmoid; its scores are not looked at) or -inf (softmax; it adds
// nothing).  Returns whether the choices are numbers where the logits are: not
// for a softmax with a NaN or +inf in it.
template <int V, int L, bool SOFTMAX>
__device__ __forceinline__ bool scores(const float (&l)[V], float (&sc)[V]) {
    if (!SOFTMAX) {
        float x[V];
        bool general = false;   // logits below -87: a subnormal score, or 0
#pragma unroll
        for (int i = 0; i < V; i++) {
            x[i] = __fadd_rn(1.0f, expf(-l[i]));
            general |= x[i] > 0x1p126f;
            sc[i] = rcp_mid(x[i]);
        }
        if (general)
#pragma unroll
            for (int i = 0; i < V; i++) sc[i] = __frcp_rn(x[i]);
        return true;
    }
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; i++) top = fmaxf(top, l[i]);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    // nothing left: exp(-inf - 0) = 0 everywhere (a NaN among the -inf still shows)
    const float base = top == -INFINITY ? 0.0f : top;
    float t[V];
    uint32_t least = 0xffffffffu;   // of the exponentials' bits - 1 (0 comes out largest)
#pragma unroll
    for (int i = 0; i < V; i++) {
        sc[i] = expf(__fsub_rn(l[i], base));
        least = min(least, __float_as_uint(sc[i]) - 1u);
        t[i] = sc[i];
    }
#pragma unroll
    for (int n = V; n > 1; n >>= 1)
#pragma unroll
        for (int i = 0; i < n / 2; i++) t[i] = __fadd_rn(t[2 * i], t[2 * i + 1]);
    float sum = t[0];
#pragma unroll
    for (int o = 1; o < L; o <<= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, o));
    if (sum == 0.0f) return true;   // every score is 0 already
    const float y = rcp_mid(sum);
    if (least < __float_as_uint(0x1p-100f) - 1u) {   // tiny exponentials: the general division
#pragma unroll
        for (int i = 0; i < V; i++) sc[i] = __fdiv_rn(sc[i], sum);
    } else {
#pragma unroll
        for (int i = 0; i < V; i++) sc[i] = div_mid(sc[i], sum, y);
    }
    return sum == sum;
}

// Largest of u over a token's L lanes.
template <int L>
__device__ __forceinline__ uint32_t max_over(uint32_t u) {
    if constexpr (L == 32) {
        return __reduce_max_sync(0xffffffffu, u);
    } else {
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) u = max(u, __shfl_xor_sync(0xffffffffu, u, o));
        return u;
    }
}

// The lowest of a token's lanes where p holds (0 if nowhere), as its place.
template <int L>
__device__ __forceinline__ int first_lane(bool p, int lane) {
    uint32_t b = __ballot_sync(0xffffffffu, p);
    if constexpr (L < 32) b = (b >> (lane & ~(L - 1))) & ((1u << L) - 1);
    return max(__ffs(b) - 1, 0);
}

// Merge the two best (a >= b) of another lane into this lane's.
__device__ __forceinline__ void merge_top2(float &a, float &b, float oa, float ob) {
    b = fmaxf(fminf(a, oa), fmaxf(b, ob));
    a = fmaxf(a, oa);
}

// Groups whose lanes are a power of two: whether this lane's group stays.  Its
// two best choices come by shuffles, then every lane meets the other groups' keys.
template <int V, int L>
__device__ __forceinline__ bool my_group_stays(const float (&ch)[V], int sub, int groups, int gl, int topk_groups,
                                               int group_top) {
    float a = -INFINITY, b = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; i++) {
        b = fmaxf(b, fminf(a, ch[i]));
        a = fmaxf(a, ch[i]);
    }
    for (int o = 1; o < gl; o <<= 1)
        merge_top2(a, b, __shfl_xor_sync(0xffffffffu, a, o), __shfl_xor_sync(0xffffffffu, b, o));
    const uint32_t gk = order_key(group_top == 2 && b > -INFINITY ? __fadd_rn(a, b) : a);
    int ahead = 0;
#pragma unroll 4
    for (int l = 0; l < groups * gl; l += gl) {
        const uint32_t o = __shfl_sync(0xffffffffu, gk, l, L);
        ahead += o > gk || (o == gk && l + gl <= sub);
    }
    return ahead < topk_groups;
}

// Other groups: which of a token's stay, as a bit mask, from its choices in
// shared memory; the groups' keys meet in `keys` (32 per token).
template <int V, int L>
__device__ __forceinline__ uint32_t kept_groups(const float (&ch)[V], float *choices, uint32_t *keys, int sub,
                                                int groups, int gs, int topk_groups, int group_top) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < V; i++) choices[sub * V + i] = ch[i];
    __syncwarp();
    for (int g = sub; g < groups; g += L) {
        float a = -INFINITY, b = -INFINITY;
        for (int i = 0; i < gs; i++) {
            const float v = choices[g * gs + i];
            b = fmaxf(b, fminf(a, v));
            a = fmaxf(a, v);
        }
        keys[g] = order_key(group_top == 2 && b > -INFINITY ? __fadd_rn(a, b) : a);
    }
    __syncwarp();
    uint32_t kept = 0;
    for (int g = sub; g < groups; g += L) {
        const uint32_t mine = keys[g];
        int ahead = 0;
        for (int o = 0; o < groups; o++) {
            const uint32_t other = keys[o];
            ahead += other > mine || (other == mine && o < g);
        }
        if (ahead < topk_groups) kept |= 1u << g;
    }
    if constexpr (L == 32) {
        return __reduce_or_sync(0xffffffffu, kept);
    } else {
#pragma unroll
        for (int o = 1; o < L; o <<= 1) kept |= __shfl_xor_sync(0xffffffffu, kept, o);
        return kept;
    }
}

template <int N> struct alignas(4 * N) Vec { float f[N]; };

// L lanes per token.
template <typename T, int V, int L, bool SOFTMAX>
__global__ void __launch_bounds__(RT_THREADS)
route_topk_kernel(const T *__restrict__ logits, const float *__restrict__ bias, int64_t s, int e,
                  int k, int groups, int topk_groups, int group_top, float scale, int normalize, int vec,
                  int32_t *__restrict__ idx, float *__restrict__ gates, int32_t *status) {
    constexpr int TPW = 32 / L;   // tokens per warp
    __shared__ __align__(16) float s_val[RT_WARPS][V * 32];   // choices, then scores
    constexpr int CAND = V <= 8 ? V * L : 32;    // room for every expert, where it is small
    __shared__ uint2 s_cand[L == 32 ? RT_WARPS : 1][CAND];   // candidates
    __shared__ int32_t s_sel[RT_WARPS][TPW * 32];   // the selection, by route
    pdl_enter();
    const bool stop = status_bad(status);   // asked for now, needed before the first store
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & (L - 1), tw = lane / L;
    constexpr int VS = V < 4 ? V : 4;
    const int gs = e / groups, gl = gs / V;   // experts and (where whole) lanes per group
    const bool by_lane = gs % V == 0 && (gl & (gl - 1)) == 0;
    const bool whole = e == V * L;                    // every lane holds V experts
    const int mine = min(max(e - sub * V, 0), V);     // experts on this lane
    float *val = s_val[warp] + tw * (V * L);
    int32_t *sel = s_sel[warp] + tw * 32;
    float bs[V];
#pragma unroll
    for (int i = 0; i < V; i++) {
        bs[i] = bias && sub * V + i < e ? bias[sub * V + i] : 0.0f;
        if (bs[i] != bs[i]) bs[i] = -INFINITY;   // a NaN choice ranks like a masked expert
    }
    const int64_t step = (int64_t)gridDim.x * RT_WARPS * TPW;
    for (int64_t t0 = ((int64_t)blockIdx.x * RT_WARPS + warp) * TPW; t0 < s; t0 += step) {
        const int64_t t = min(t0 + tw, s - 1);   // lanes past the end repeat the last token
        float l[V], sc[V], ch[V];
        ld_logits<T, V>(logits + t * e, sub * V, e, vec, SOFTMAX ? -INFINITY : 0.0f, l);
        const bool numbers = scores<V, L, SOFTMAX>(l, sc);
#pragma unroll
        for (int i = 0; i < V; i++) {
            const float c = __fadd_rn(sc[i], bs[i]);   // without a bias: + 0
            ch[i] = l[i] > -INFINITY && (!SOFTMAX || numbers) ? c : -INFINITY;   // (a NaN is not > -inf)
        }
        if (!whole) {
#pragma unroll
            for (int i = 0; i < V; i++) ch[i] = i < mine ? ch[i] : -INFINITY;
        }
        // keys: 0 below everything (not an expert, or of a group that does not stay)
        uint32_t key[V];
        if (groups == 1 || by_lane) {
            const bool in = groups == 1 || my_group_stays<V, L>(ch, sub, groups, gl, topk_groups, group_top);
#pragma unroll
            for (int i = 0; i < V; i++) key[i] = in ? order_key(ch[i]) : 0u;
            if (!whole) {
#pragma unroll
                for (int i = 0; i < V; i++) key[i] = i < mine ? key[i] : 0u;
            }
        } else {
            const uint32_t kept = kept_groups<V, L>(ch, val, reinterpret_cast<uint32_t *>(sel), sub, groups, gs,
                                                    topk_groups, group_top);
#pragma unroll
            for (int i = 0; i < V; i++)
                key[i] = i < mine && (kept >> ((sub * V + i) / gs) & 1) ? order_key(ch[i]) : 0u;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < V; i += VS)   // scores by expert
            *reinterpret_cast<Vec<VS> *>(val + sub * V + i) = *reinterpret_cast<const Vec<VS> *>(sc + i);
        bool done = false;
        if (L == 32) {
            // A token's k best are no less than the k-th largest of its lanes'
            // maxima; the few that are not go to a list, and their places in it
            // are counted.  More than 32 of them (equal choices): below.
            uint32_t best = 0;
#pragma unroll
            for (int i = 0; i < V; i++) best = max(best, key[i]);
            uint32_t m = best, low = 0;
#pragma unroll 4
            for (int r = 0; r < k; r++) {   // (equal maxima leave together: the bound is lower then, never higher)
                low = __reduce_max_sync(0xffffffffu, m);
                m = m == low ? 0u : m;
            }
            low = max(low, 1u);
            int n = 0;
#pragma unroll
            for (int i = 0; i < V; i++) {
                const uint32_t b = __ballot_sync(0xffffffffu, key[i] >= low);
                const int at = n + __popc(b & ((1u << lane) - 1));
                if (key[i] >= low && (CAND == V * L || at < 32)) s_cand[warp][at] = make_uint2(key[i], sub * V + i);
                n += __popc(b);
            }
            __syncwarp();
            if (n <= 32) {
                const uint2 c = s_cand[warp][lane];
                int rank = 0;
#pragma unroll 4
                for (int q = 0; q < n; q++) {
                    const uint2 o = s_cand[warp][q];
                    rank += o.x > c.x || (o.x == c.x && o.y < c.y);
                }
                if (lane < n && rank < k) sel[rank] = (int32_t)c.y;
                done = true;
            }
        }
        if (!done) {
            for (int r = 0; r < k; r++) {
                uint32_t best = 0;
#pragma unroll
                for (int i = 0; i < V; i++) best = max(best, key[i]);
                const uint32_t top = max_over<L>(best);
                const bool mine = first_lane<L>(best == top, lane) == sub;
                int pos = 0;
#pragma unroll
                for (int i = V - 1; i >= 0; i--) pos = key[i] == top ? i : pos;
                if (mine) sel[r] = sub * V + pos;
                if (r + 1 == k) break;
#pragma unroll
                for (int i = 0; i < V; i++) key[i] = mine && i == pos ? 0u : key[i];
            }
        }
        __syncwarp();
        // lane (place) r: route r, and with fewer lanes than routes r + L, ...
        int j = sub < k ? sel[sub] : 0;
        float g = sub < k ? val[j] : 0.0f, sum = 0.0f;
        if (normalize) {
            if (k <= L) {
#pragma unroll 4
                for (int r = 0; r < k; r++) sum = __fadd_rn(sum, __shfl_sync(0xffffffffu, g, r, L));
            } else {
                for (int r = 0; r < k; r++) sum = __fadd_rn(sum, val[sel[r]]);
            }
        }
        if (__any_sync(0xffffffffu, stop)) return;
        if (t0 + tw < s)
            for (int r = sub; r < k; r += L) {
                if (r != sub) {
                    j = sel[r];
                    g = val[j];
                }
                if (normalize) g = sum == 0.0f ? 0.0f : __fdiv_rn(g, sum);
                idx[(int64_t)r * s + t] = j;
                gates[(int64_t)r * s + t] = g * scale;
            }
        __syncwarp();
    }
}

// ---------------------------------------------------------------- backward
// A CTA takes `tb` consecutive tokens (a multiple of 8): their rows of
// d_logits are formed in shared memory and leave as one contiguous run of
// 16-byte stores, whatever e is.
constexpr int BWD_FLOATS = 8192;   // 8 tokens of 1024 experts
constexpr int BWD_LANES = 8;       // lanes per token for its routes

// Tokens per CTA (16384 x 256: 7.3 us with 16, 8.4 with 32, 9.1 with 8).
__host__ __device__ inline int bwd_tokens(int e) { return e <= 64 ? 32 : e <= 256 ? 16 : 8; }

template <typename D>
__device__ __forceinline__ void store_rows(const float *rows, int64_t n, D *out) {
    constexpr int N = Elt<D>::VEC;
    for (int64_t i = threadIdx.x; i < n / N; i += RT_THREADS) st_v16(out + i * N, Elt<D>::pack(rows + i * N));
    for (int64_t i = n / N * N + threadIdx.x; i < n; i += RT_THREADS) out[i] = (D)rows[i];
}

// A logit's bits as loaded, issued here (a plain load may sink to its use), and
// its value.
__device__ __forceinline__ uint32_t ld_early(const float *p) {
    uint32_t r;
    asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(r) : "l"(p));
    return r;
}
__device__ __forceinline__ uint32_t ld_early(const __nv_bfloat16 *p) {
    uint16_t r;
    asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(r) : "l"(p));
    return r;
}
template <typename T> __device__ __forceinline__ float of_bits(uint32_t w) {
    return __uint_as_float(sizeof(T) == 2 ? w << 16 : w);
}

// The larger of two; a NaN stays one.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Of a 16-byte chunk's values.
template <typename T>
__device__ __forceinline__ float max_of(const V16 &v) {
    constexpr int N = Elt<T>::VEC;
    float f[N];
    Elt<T>::unpack(v, f);
#pragma unroll
    for (int n = N / 2; n > 0; n >>= 1)
#pragma unroll
        for (int i = 0; i < n; i++) f[i] = max_nan(f[i], f[i + n]);
    return f[0];
}

// A row's softmax sum in the forward's order (adjacent pairs over the padded
// width: a pair is added as soon as its second half is complete), by one thread.
template <typename T>
__device__ __noinline__ float softmax_sum(const T *row, int e, float top) {
    float part[11], v = 0.0f;   // part[n]: the open run of 2^n exponentials
    for (int i = 0; i < e; i++) {
        v = expf(__fsub_rn(ld_logit(row + i), top));
        int n = 0;
        for (; i >> n & 1; n++) v = __fadd_rn(part[n], v);
        part[n] = v;
    }
    bool any = false;
    for (int n = 0; n < 11; n++) {
        if (!(e >> n & 1)) continue;
        v = any ? __fadd_rn(part[n], v) : part[n];
        any = true;
    }
    return v;
}

// Gradients that live on the selection: with g the selected scores, G = g / sum
// g and A = sum_r dg_r G_r,
//   softmax, normalised: scale G (dg - A);
//   sigmoid, normalised: scale G (dg - A) (1 - g);
//   sigmoid, raw:        scale dg g (1 - g).
// A softmax's G is formed from the selected logits alone, exp(l - their largest),
// which is closer than the quotient of two scores.  What the forward's gates do
// besides comes from the row's largest logit: they are NaN where that is a NaN or
// +inf, and the constant 0 where all chosen scores round to 0 (from about 97 below
// it on; settled by the forward's own operations).
// Bound by the e values written; sigmoid reads k logits a token, softmax all:
// 16384 x 256 fp32, k = 8: 6.2 us sigmoid, 7.8 softmax (6.4 if the row is not
// looked at); 65536 x 64 bf16, k = 2: 11.3 (8.6 sigmoid).  CTAs a multiprocessor:
// softmax four, 64 registers (five: 8.0, three: 8.5); sigmoid five, 48 registers
// (four: 6.6).
template <typename T, typename D, bool SOFTMAX>
__global__ void __launch_bounds__(RT_THREADS, SOFTMAX ? 4 : 5)
route_bwd_sel_kernel(const T *__restrict__ logits, const int32_t *__restrict__ idx,
                     const float *__restrict__ d_gates, int64_t s, int e, int k, float scale,
                     int normalize, D *__restrict__ d_logits, int32_t *status) {
    __shared__ __align__(16) float rows[BWD_FLOATS];
    __shared__ float row_top[SOFTMAX ? RT_THREADS / BWD_LANES : 1];   // largest logit by token
    pdl_enter();
    const bool stop = status_bad(status);
    const int tb = bwd_tokens(e), sub = threadIdx.x % BWD_LANES, tok = threadIdx.x / BWD_LANES;
    for (int64_t t0 = (int64_t)blockIdx.x * tb; t0 < s; t0 += (int64_t)gridDim.x * tb) {
        const int nt = (int)min((int64_t)tb, s - t0);
        const int64_t t = t0 + tok;
        const bool on = tok < nt;
        // this lane's routes sub, sub + 8, ... of its token (q * 8 < k is the same
        // in all threads: up to eight routes skip the other three)
        int j[4];
        float x[4], dg[4], g[4];
        bool bad = false;
        float top = -INFINITY;
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const int r = sub + q * BWD_LANES;
            const bool have = on && r < k;
            j[q] = have ? idx[(int64_t)r * s + t] : -1;
            dg[q] = have ? d_gates[(int64_t)r * s + t] : 0.0f;
        }
        // softmax: RT_THREADS / tb lanes (8, 16 or 32) look for a row's largest logit;
        // the first loads are on their way together with the selection's
        constexpr int N = Elt<T>::VEC, AHEAD = 4;
        const int lg = e <= 64 ? 3 : e <= 256 ? 4 : 5, lanes = 1 << lg;   // bwd_tokens(e) * lanes = RT_THREADS
        const int rl = threadIdx.x & (lanes - 1), rtok = threadIdx.x >> lg;
        const T *row = logits + (t0 + min(rtok, nt - 1)) * e;
        const bool chunks = e % N == 0;
        V16 ahead[SOFTMAX ? AHEAD : 1];
        if (SOFTMAX && chunks) {
#pragma unroll
            for (int i = 0; i < AHEAD; i++) {
                const int c = (rl + i * lanes) * N;
                if (c < e) ahead[i] = ld_stream(row + c);
            }
        } else if (SOFTMAX) {   // single values
#pragma unroll
            for (int i = 0; i < 2 * AHEAD; i++) {
                const int c = rl + i * lanes;
                ahead[i / 4].w[i % 4] = sizeof(T) == 2 ? 0xFF80u : 0xFF800000u;   // -inf
                if (c < e) ahead[i / 4].w[i % 4] = ld_early(row + c);
            }
        }
        float4 *z = reinterpret_cast<float4 *>(rows);   // zeros while those loads are on their way
        for (int i = threadIdx.x; i < (nt * e + 3) / 4; i += RT_THREADS) z[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int q = 0; q < 4; q++) {
            if (q * BWD_LANES >= k) break;
            if (on && sub + q * BWD_LANES < k && (j[q] < 0 || j[q] >= e)) { bad = true; j[q] = -1; }
            x[q] = j[q] >= 0 ? ld_logit(logits + t * e + j[q]) : -INFINITY;
            top = fmaxf(top, x[q]);
        }
        if (bad) set_status(status, MOE_ERR_INVALID_ARG);
        float total = 0.0f;
        if (SOFTMAX) {
            float m = -INFINITY;
            if (chunks) {
#pragma unroll
                for (int i = 0; i < AHEAD; i++)
                    if ((rl + i * lanes) * N < e) m = max_nan(m, max_of<T>(ahead[i]));
#pragma unroll 1
                for (int c = (rl + AHEAD * lanes) * N; c < e; c += lanes * N) m = max_nan(m, max_of<T>(ld_stream(row + c)));
            } else {
#pragma unroll
                for (int i = 0; i < 2 * AHEAD; i++) m = max_nan(m, of_bits<T>(ahead[i / 4].w[i % 4]));
#pragma unroll 4
                for (int c = rl + 2 * AHEAD * lanes; c < e; c += lanes) m = max_nan(m, ld_logit(row + c));
            }
            for (int o = lanes / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (rl == 0) row_top[rtok] = m;
#pragma unroll
            for (int o = BWD_LANES / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        }
#pragma unroll
        for (int q = 0; q < 4; q++) {
            if (q * BWD_LANES >= k) break;
            if (j[q] < 0 || (SOFTMAX && top == -INFINITY)) g[q] = 0.0f;
            else g[q] = SOFTMAX ? expf(x[q] - top) : sigmoid_rn(x[q]);
            total += g[q];
        }
        // A from the quotients G themselves: of a single route (G = 1) it is dg, and
        // the gradient 0 without a rounding error
        float G[4], A = 0.0f;
        if (normalize) {
#pragma unroll
            for (int o = BWD_LANES / 2; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
#pragma unroll
            for (int q = 0; q < 4; q++) {
                if (q * BWD_LANES >= k) break;
                G[q] = total == 0.0f ? 0.0f : g[q] / total;
                A += dg[q] * G[q];
            }
#pragma unroll
            for (int o = BWD_LANES / 2; o > 0; o >>= 1) A += __shfl_xor_sync(0xffffffffu, A, o);
        }
        // the rows are zero; another CTA's error may have come up meanwhile, so the
        // threads leave together
        if (__syncthreads_or(stop)) return;
        float f = scale;   // NaN or 0: as the gates are
        if (SOFTMAX && on) {
            const float rt = row_top[tok];
            if (!(rt < INFINITY)) f = NAN;
            else if (top - rt < -96.0f && __fdiv_rn(expf(__fsub_rn(top, rt)), softmax_sum(logits + t * e, e, rt)) == 0.0f)
                f = 0.0f;
        }
#pragma unroll
        for (int q = 0; q < 4; q++) {
            if (q * BWD_LANES >= k) break;
            if (j[q] < 0) continue;
            float d;
            if (normalize) d = f * G[q] * (dg[q] - A);
            else d = scale * dg[q] * g[q];
            if (!SOFTMAX) d *= 1.0f - g[q];
            rows[tok * e + j[q]] = d;
        }
        __syncthreads();
        store_rows(rows, (int64_t)nt * e, d_logits + t0 * e);
        __syncthreads();   // rows is rewritten
    }
}

// Raw softmax gates: d_j = scale p_j (dg_j [selected] - sum_r dg_r p_r) for every
// expert.  L lanes a token as in the forward.
template <typename T, typename D, int V, int L>
__global__ void __launch_bounds__(RT_THREADS)
route_bwd_all_kernel(const T *__restrict__ logits, const int32_t *__restrict__ idx,
                     const float *__restrict__ d_gates, int64_t s, int e, int k, float scale, int vec,
                     D *__restrict__ d_logits, int32_t *status) {
    constexpr int TPC = RT_THREADS / L;   // tokens per CTA and pass
    constexpr int ROUTES = 32 / L;        // routes per lane, at most
    __shared__ __align__(16) float rows[TPC * V * L];
    pdl_enter();
    const bool stop = status_bad(status);
    const int sub = threadIdx.x & (L - 1), tok = threadIdx.x / L;
    for (int64_t t0 = (int64_t)blockIdx.x * TPC; t0 < s; t0 += (int64_t)gridDim.x * TPC) {
        const int nt = (int)min((int64_t)TPC, s - t0);
        const int64_t t = t0 + min(tok, nt - 1);
        float l[V], p[V];
        ld_logits<T, V>(logits + t * e, sub * V, e, vec, -INFINITY, l);
        scores<V, L, true>(l, p);
        float *row = rows + tok * e;
        const bool on = tok < nt;   // lanes past the end repeat the last token's scores, and write nothing
        if (on)
#pragma unroll
            for (int i = 0; i < V; i++)
                if (sub * V + i < e) row[sub * V + i] = p[i];
        __syncwarp();
        float dot = 0.0f, pj[ROUTES], dg[ROUTES];
        int j[ROUTES];
#pragma unroll
        for (int q = 0; q < ROUTES; q++) {
            const int r = sub + q * L;
            j[q] = on && r < k ? idx[(int64_t)r * s + t] : -1;
            if (on && r < k && (j[q] < 0 || j[q] >= e)) {
                set_status(status, MOE_ERR_INVALID_ARG);
                j[q] = -1;
            }
            dg[q] = j[q] >= 0 ? d_gates[(int64_t)r * s + t] : 0.0f;
            pj[q] = j[q] >= 0 ? row[j[q]] : 0.0f;
            dot += dg[q] * pj[q];
        }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        __syncwarp();
        if (on)
#pragma unroll
            for (int i = 0; i < V; i++)
                if (sub * V + i < e) row[sub * V + i] = -scale * p[i] * dot;
        __syncwarp();
#pragma unroll
        for (int q = 0; q < ROUTES; q++)
            if (j[q] >= 0) row[j[q]] = scale * pj[q] * (dg[q] - dot);
        if (__syncthreads_or(stop)) return;
        store_rows(rows, (int64_t)nt * e, d_logits + t0 * e);
        __syncthreads();
    }
}

// CTAs for `units` CTA-sized pieces of work: at most `per_sm` a multiprocessor
// (the kernels stride).
int grid_for(int64_t units, int per_sm) {
    static int cached[64] = {0};
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64) {
        if (!cached[dev]) cudaDeviceGetAttribute(&cached[dev], cudaDevAttrMultiProcessorCount, dev);
        if (cached[dev] > 0) sms = cached[dev];
    }
    const int64_t cap = (int64_t)sms * per_sm;
    return (int)(units < cap ? units : cap);
}

template <typename T, int V, int L>
moe_status topk_v(const void *logits, const float *bias, int64_t s, int e, int k, bool softmax,
                  int groups, int topk_groups, int group_top, float scale, int normalize,
                  int32_t *idx, float *gates, int32_t *st, cudaStream_t stream) {
    auto kern = softmax ? route_topk_kernel<T, V, L, true> : route_topk_kernel<T, V, L, false>;
    constexpr int TPC = RT_THREADS / L;
    // about twice what is resident (512 experts: 16.3 us with 4, 20.9 with 8)
    constexpr int PER_SM = V <= 8 ? 8 : V == 16 ? 4 : 2;
    return launch_pdl(kern, dim3(grid_for((s + TPC - 1) / TPC, PER_SM)), dim3(RT_THREADS), 0, stream,
                      (const T *)logits, bias, s, e, k, groups, topk_groups, group_top, scale, normalize,
                      e % Elt<T>::VEC == 0 ? 1 : 0, idx, gates, st);
}

template <typename T, typename D, int V, int L>
moe_status bwd_all_v(const void *logits, const int32_t *idx, const float *d_gates, int64_t s, int e, int k,
                     float scale, void *d_logits, int32_t *st, cudaStream_t stream) {
    constexpr int TPC = RT_THREADS / L;
    return launch_pdl(route_bwd_all_kernel<T, D, V, L>, dim3(grid_for((s + TPC - 1) / TPC, 8)), dim3(RT_THREADS), 0,
                      stream, (const T *)logits, idx, d_gates, s, e, k, scale, e % Elt<T>::VEC == 0 ? 1 : 0,
                      (D *)d_logits, st);
}

template <typename T, typename D>
moe_status bwd_sel(const void *logits, const int32_t *idx, const float *d_gates, int64_t s, int e, int k,
                   bool softmax, float scale, int normalize, void *d_logits, int32_t *st, cudaStream_t stream) {
    auto kern = softmax ? route_bwd_sel_kernel<T, D, true> : route_bwd_sel_kernel<T, D, false>;
    const int tb = bwd_tokens(e);
    return launch_pdl(kern, dim3(grid_for((s + tb - 1) / tb, 8)), dim3(RT_THREADS), 0, stream, (const T *)logits, idx,
                      d_gates, s, e, k, scale, normalize, (D *)d_logits, st);
}

}  // namespace

// Experts and lanes per token: e padded to a power of two, eight experts a
// lane between 32 and 256.
#define MOE_BY_E(CALL)                 \
    if (e <= 8) return CALL(2, 4);     \
    if (e <= 16) return CALL(4, 4);    \
    if (e <= 32) return CALL(8, 4);    \
    if (e <= 64) return CALL(8, 8);    \
    if (e <= 128) return CALL(8, 16);  \
    if (e <= 256) return CALL(8, 32);  \
    if (e <= 512) return CALL(16, 32); \
    return CALL(32, 32)

moe_status route_topk_launch(const void *logits, moe_dtype ldt, const float *bias, int64_t s, int e,
                             int k, moe_score score, int groups, int topk_groups, int group_top,
                             float scale, unsigned flags, int32_t *idx, float *gates, int32_t *st,
                             cudaStream_t stream) {
    const bool sm = score == MOE_SCORE_SOFTMAX;
    const int nrm = (flags & MOE_FLAG_NORMALIZE_GATES) != 0;
    using bf = __nv_bfloat16;
#define MOE_F(V, L) topk_v<float, V, L>(logits, bias, s, e, k, sm, groups, topk_groups, group_top, scale, nrm, idx, gates, st, stream)
#define MOE_B(V, L) topk_v<bf, V, L>(logits, bias, s, e, k, sm, groups, topk_groups, group_top, scale, nrm, idx, gates, st, stream)
    if (ldt == MOE_F32) { MOE_BY_E(MOE_F); }
    MOE_BY_E(MOE_B);
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
    if (!sm || nrm) {
        auto f = ldt == MOE_F32 ? (ddt == MOE_F32 ? bwd_sel<float, float> : bwd_sel<float, bf>)
                                : (ddt == MOE_F32 ? bwd_sel<bf, float> : bwd_sel<bf, bf>);
        return f(logits, idx, d_gates, s, e, k, sm, scale, nrm, d_logits, st, stream);
    }
#define MOE_FF(V, L) bwd_all_v<float, float, V, L>(logits, idx, d_gates, s, e, k, scale, d_logits, st, stream)
#define MOE_FB(V, L) bwd_all_v<float, bf, V, L>(logits, idx, d_gates, s, e, k, scale, d_logits, st, stream)
#define MOE_BF(V, L) bwd_all_v<bf, float, V, L>(logits, idx, d_gates, s, e, k, scale, d_logits, st, stream)
#define MOE_BB(V, L) bwd_all_v<bf, bf, V, L>(logits, idx, d_gates, s, e, k, scale, d_logits, st, stream)
    if (ldt == MOE_F32 && ddt == MOE_F32) { MOE_BY_E(MOE_FF); }
    if (ldt == MOE_F32) { MOE_BY_E(MOE_FB); }
    if (ddt == MOE_F32) { MOE_BY_E(MOE_BF); }
    MOE_BY_E(MOE_BB);
#undef MOE_FF
#undef MOE_FB
#undef MOE_BF
#undef MOE_BB
}
#undef MOE_BY_E

}  // namespace moe
