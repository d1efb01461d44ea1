// Rows sorted by expert, without a capacity: the order of the routes, the tokens' rows on their
// way in and back, and the gradients of both.
//
// The routes of expert j take the rows offsets[j] .. offsets[j + 1] - 1 of one [n, m] buffer, in
// route-priority order (the flat [k, s] table's own order), so the order is a stable counting sort
// of the table by expert.  A route whose expert is -1 has no row.
#include "common.cuh"
#include "scale_round.cuh"

namespace moe {
namespace {

// ------------------------------------------------------------------- the sort
// Buckets 0 .. e-1 are the experts, bucket e the routes without one (source[] says -1 behind the
// last row, so they are ranked like the others).
constexpr int SS_NT = 1024, SS_NW = SS_NT / 32, SS_MAXE = 256, SS_MAXN = 2048;   // one launch
constexpr int ST_NT = 256, ST_NW = ST_NT / 32, ST_BLK = 256;                      // two launches
constexpr int ST_HELD = 8;                                                        // rounds kept in registers
constexpr int SORT_MAXB = 1025;                                                   // buckets

__device__ __forceinline__ int bucket_of(int v, int e, int32_t *status) {
    if ((unsigned)v < (unsigned)e) return v;
    if (v != -1) set_status(status, MOE_ERR_INVALID_ARG);
    return e;
}

// cnt[b] += 1 for every lane's bucket b (b < 0: none), one atomic a distinct bucket of the warp: a
// popular expert would serialise one a lane.
__device__ __forceinline__ void count_warp(int32_t *cnt, int b, unsigned lt) {
    const unsigned peers = __match_any_sync(0xffffffffu, b);
    if (b >= 0 && (peers & lt) == 0) atomicAdd(cnt + b, __popc(peers));
}

// start[b] = sum of tot[0 .. b-1] over nb <= 5 * NT buckets, by the whole CTA; start[nb] too.
template <int NT>
__device__ __forceinline__ void exclusive_scan(const int32_t *tot, int32_t *start, int nb, int32_t *part) {
    constexpr int PER = (SORT_MAXB + NT - 1) / NT;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int32_t v[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; i++) {
        const int b = tid * PER + i;
        v[i] = sum;
        sum += b < nb ? tot[b] : 0;
    }
    int32_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) part[warp] = inc;
    __syncthreads();
    int32_t ahead = inc - sum;
    for (int w = 0; w < warp; w++) ahead += part[w];
#pragma unroll
    for (int i = 0; i < PER; i++) {
        const int b = tid * PER + i;
        if (b <= nb) start[b] = ahead + v[i];
    }
    __syncthreads();
}

// A route's row, and its route back.  A position is inside the table whenever every count was made; warps that
// found dev_status set (by another CTA or stream) while the others went on have made none of theirs.
__device__ __forceinline__ void put_route(int64_t j, int b, int32_t pos, int64_t n, int e, int32_t *__restrict__ rows,
                                          int32_t *__restrict__ source) {
    rows[j] = b < e ? pos : -1;
    if (source && pos >= 0 && pos < n) source[pos] = b < e ? (int32_t)j : -1;
}

// The positions of `rounds` x 32 consecutive routes from `at` on, the warp's next free position of
// each bucket in next[].
__device__ __forceinline__ void place_segment(const int32_t *__restrict__ idx, int64_t at, int rounds, int64_t n,
                                              int e, int32_t *next, int32_t *__restrict__ rows,
                                              int32_t *__restrict__ source, int32_t *status, unsigned lt) {
    const int lane = threadIdx.x & 31;
    for (int r = 0; r < rounds; r++) {
        const int64_t j = at + r * 32 + lane;
        const int b = j < n ? bucket_of(__ldg(idx + j), e, status) : -1;
        const unsigned peers = __match_any_sync(0xffffffffu, b);
        const int32_t first = b >= 0 ? next[b] : 0;
        __syncwarp();
        if (b >= 0 && (peers & lt) == 0) next[b] = first + __popc(peers);
        __syncwarp();
        if (b >= 0) put_route(j, b, first + __popc(peers & lt), n, e, rows, source);
    }
}

// Up to 2048 routes of up to 256 experts: one launch, a CTA of 32 warps for 1024 routes.  Every
// CTA counts all routes and those before its own, so none waits for another.  (16384 routes this way: 29 us;
// a match of a warp's buckets costs about 50 clocks of the multiprocessor.)
__global__ void __launch_bounds__(SS_NT)
sort_small_kernel(const int32_t *__restrict__ idx, int n, int e, int32_t *__restrict__ rows,
                  int32_t *__restrict__ offsets, int32_t *__restrict__ source, int32_t *status) {
    pdl_enter();
    if (status_bad(status)) return;
    extern __shared__ int32_t sm[];
    __shared__ int32_t part[SS_NW];
    const int nb = e + 1, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int32_t *tot = sm, *before = sm + nb, *start = before + nb, *cnt = start + nb + 1;   // cnt [32][nb]
    const unsigned lt = (1u << lane) - 1u;
    for (int q = tid; q < 2 * nb; q += SS_NT) sm[q] = 0;
    for (int q = tid; q < SS_NW * nb; q += SS_NT) cnt[q] = 0;
    __syncthreads();
    const int own = blockIdx.x * SS_NT;
    for (int q0 = 0; q0 < n; q0 += SS_NT) {
        const int q = q0 + tid;
        const int b = q < n ? bucket_of(__ldg(idx + q), e, status) : -1;
        count_warp(tot, b, lt);
        if (q0 < own) count_warp(before, b, lt);   // own is a multiple of the step
        else if (q0 == own) count_warp(cnt + warp * nb, b, lt);
    }
    __syncthreads();
    exclusive_scan<SS_NT>(tot, start, nb, part);
    for (int b = tid; b < nb; b += SS_NT) {   // counts of the warps -> their first positions
        int32_t run = start[b] + before[b];
        for (int w = 0; w < SS_NW; w++) {
            const int32_t c = cnt[w * nb + b];
            cnt[w * nb + b] = run;
            run += c;
        }
    }
    if (blockIdx.x == 0)
        for (int b = tid; b < nb; b += SS_NT) offsets[b] = start[b];
    __syncthreads();
    place_segment(idx, own + warp * 32, 1, n, e, cnt + warp * nb, rows, source, status, lt);
}

// Larger tables (131072 routes of 64 experts: 8.8 us, 16384: 7.5 us, two launches of latency: index loads, counts,
// placing): CTA b counts its chunk of `rounds` x 256 routes into hist[bucket][b] ...
__global__ void __launch_bounds__(ST_NT)
sort_hist_kernel(const int32_t *__restrict__ idx, int64_t n, int e, int rounds, int32_t *__restrict__ hist,
                 int32_t *status) {
    pdl_enter();
    if (status_bad(status)) return;
    __shared__ int32_t cnt[SORT_MAXB];
    const int nb = e + 1, lane = threadIdx.x & 31;
    const unsigned lt = (1u << lane) - 1u;
    for (int q = threadIdx.x; q < nb; q += ST_NT) cnt[q] = 0;
    __syncthreads();
    const int64_t base = (int64_t)blockIdx.x * rounds * ST_NT;
    for (int r0 = 0; r0 < rounds; r0 += ST_HELD) {
        // all loads in flight before the first is looked at; a place past the table's end is known by its
        // position alone (an entry may hold any value)
        int v[ST_HELD];
        auto in_table = [&](int r) { return r0 + r < rounds && base + (r0 + r) * ST_NT + threadIdx.x < n; };
#pragma unroll
        for (int r = 0; r < ST_HELD; r++) v[r] = in_table(r) ? __ldg(idx + base + (r0 + r) * ST_NT + threadIdx.x) : -1;
#pragma unroll
        for (int r = 0; r < ST_HELD; r++)
            if (r0 + r < rounds) count_warp(cnt, in_table(r) ? bucket_of(v[r], e, status) : -1, lt);
    }
    __syncthreads();
    for (int q = threadIdx.x; q < nb; q += ST_NT) hist[(int64_t)q * gridDim.x + blockIdx.x] = cnt[q];
}

// ... and places them: a warp adds up a bucket's counts, those of the chunks before (all of the at
// most 256 chunks are read by every CTA: a third launch to sum them once costs more), and takes
// `rounds` x 32 consecutive routes.  HELD: at most ST_HELD rounds, kept in registers with their ranks in the
// warp; otherwise the routes are counted first and read again to be placed.
template <bool HELD>
__global__ void __launch_bounds__(ST_NT)
sort_place_kernel(const int32_t *__restrict__ idx, int64_t n, int e, int rounds, const int32_t *__restrict__ hist,
                  int32_t *__restrict__ rows, int32_t *__restrict__ offsets, int32_t *__restrict__ source,
                  int32_t *status) {
    pdl_enter();
    if (status_bad(status)) return;
    extern __shared__ int32_t sm[];
    __shared__ int32_t part[ST_NW];
    const int nb = e + 1, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nblk = gridDim.x;
    int32_t *start = sm, *before = start + nb + 1, *tot = before + nb, *cnt = tot + nb;   // cnt [8][nb]
    const unsigned lt = (1u << lane) - 1u;
    const int64_t at = ((int64_t)blockIdx.x * ST_NW + warp) * rounds * 32;
    int bucket[ST_HELD], rank[ST_HELD];
    auto in_table = [&](int r) { return r < rounds && at + r * 32 + lane < n; };
    if (HELD) {
#pragma unroll
        for (int r = 0; r < ST_HELD; r++) bucket[r] = in_table(r) ? __ldg(idx + at + r * 32 + lane) : -1;
    }
    for (int q = tid; q < ST_NW * nb; q += ST_NT) cnt[q] = 0;
    // four buckets a turn: up to 32 loads under way before the first is added
    for (int b0 = warp; b0 < nb; b0 += 4 * ST_NW) {
        int32_t c[4][ST_BLK / 32], all[4], pre[4];
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int q = 0; q < ST_BLK / 32; q++) {
                const int b = b0 + i * ST_NW, k = 32 * q + lane;
                c[i][q] = b < nb && k < nblk ? hist[(int64_t)b * nblk + k] : 0;
            }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            all[i] = pre[i] = 0;
#pragma unroll
            for (int q = 0; q < ST_BLK / 32; q++) {
                all[i] += c[i][q];
                pre[i] += 32 * q + lane < (int)blockIdx.x ? c[i][q] : 0;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int b = b0 + i * ST_NW;
            all[i] = __reduce_add_sync(0xffffffffu, all[i]);
            pre[i] = __reduce_add_sync(0xffffffffu, pre[i]);
            if (lane == 0 && b < nb) { tot[b] = all[i]; before[b] = pre[i]; }
        }
    }
    __syncthreads();
    int32_t *mine = cnt + warp * nb;
    if (HELD) {
#pragma unroll
        for (int r = 0; r < ST_HELD; r++)
            bucket[r] = in_table(r) ? bucket_of(bucket[r], e, status) : -1;
#pragma unroll
        for (int r = 0; r < ST_HELD; r++) {
            if (r >= rounds) break;
            const int b = bucket[r];
            const unsigned peers = __match_any_sync(0xffffffffu, b);
            const int32_t first = b >= 0 ? mine[b] : 0;
            __syncwarp();
            if (b >= 0 && (peers & lt) == 0) mine[b] = first + __popc(peers);
            __syncwarp();
            rank[r] = first + __popc(peers & lt);
        }
    } else {
        for (int r = 0; r < rounds; r++) {
            const int64_t j = at + r * 32 + lane;
            count_warp(mine, j < n ? bucket_of(__ldg(idx + j), e, status) : -1, lt);
        }
    }
    exclusive_scan<ST_NT>(tot, start, nb, part);
    for (int b = tid; b < nb; b += ST_NT) {
        int32_t run = start[b] + before[b];
        for (int w = 0; w < ST_NW; w++) {
            const int32_t c = cnt[w * nb + b];
            cnt[w * nb + b] = run;
            run += c;
        }
    }
    if (blockIdx.x == 0)
        for (int b = tid; b < nb; b += ST_NT) offsets[b] = start[b];
    __syncthreads();
    if (HELD) {
#pragma unroll
        for (int r = 0; r < ST_HELD; r++) {
            if (r >= rounds) break;
            const int b = bucket[r];
            const int64_t j = at + r * 32 + lane;
            if (b >= 0) put_route(j, b, mine[b] + rank[r], n, e, rows, source);
        }
    } else {
        place_segment(idx, at, rounds, n, e, mine, rows, source, status, lt);
    }
}

// ------------------------------------------------------------ rows in and back
// One kernel for the four movements.  Per token t with row a[t] and routes r to the rows b[rows[r, t]]:
//   IN    b_r = g_r a                            (no gates: a copy)
//   BACK  a = sum_r g_r b_r                      (no gates: g = 1)
//   DOTS  d_r = <a, b_r>, alone or with one of them (the gates' gradient: the way back's is
//         IN | DOTS with a = dy and the incoming rows b, the way in's is BACK | DOTS)
// Bound by HBM: each row is read once and written once (65536 x 2 rows of 8 KB in 254 us, 6.3 TB/s; back with
// gates, 8191 x 8 rows of 4 KB, 54 us, 5.6 TB/s).  W warps share a token (a whole number of
// tokens a CTA), KG routes' rows are in flight together for U chunks of 32 x 16 bytes.  Sums over
// routes run in ascending order in fp32 with fused multiply-add; a dot product is summed by each lane in
// ascending chunks, over the lanes by halving, over the W warps in order: no atomics, W set by the shape.
enum { IN = 1, BACK = 2, DOTS = 4, GATES = 8 };
constexpr int MV_NT = 256, MV_NW = MV_NT / 32;

struct MoveArgs {
    const void *a, *b;      // rows read: tokens [s, m], routes [n, m]
    void *a_out, *b_out;    // rows written: tokens (BACK), routes (IN)
    const int32_t *rows;    // [k, s]
    const float *gates;     // [k, s] (GATES)
    float *dots;            // [k, s] (DOTS)
    int64_t s, n;
    int m, k, wpt;          // wpt: warps per token
    int32_t *status;
};

// Sums of v[0 .. KG) over the 32 lanes: lane l ends with the sum of value l % KG (KG a power of two).
template <int KG>
__device__ __forceinline__ float reduce_many(float (&v)[KG], int lane) {
#pragma unroll
    for (int w = KG / 2, o = KG / 2; w > 0; w >>= 1, o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < w; i++) {
            const float send = up ? v[i] : v[i + w], keep = up ? v[i + w] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
#pragma unroll
    for (int o = KG; o < 32; o <<= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    return v[0];
}

// CTAs a multiprocessor: what the loads in flight and the sums leave room for (six forms spill 8 to 52 bytes a thread, the
// most at one route a token with dot products).
template <int MODE, int KG, int U>
constexpr int mv_ctas() {
    return KG * U >= 8 ? 2 : MODE & DOTS ? 3 : 4;
}

// KT: routes whose dot products are summed in one pass over the row (DOTS; a multiple of KG).
template <typename T, int MODE, int KT, int KG, int U>
__global__ void __launch_bounds__(MV_NT, (mv_ctas<MODE, KG, U>()))
move_rows_kernel(const MoveArgs g) {
    pdl_enter();
    if (status_bad(g.status)) return;
    constexpr bool in = MODE & IN, back = MODE & BACK, dots = MODE & DOTS, gated = MODE & GATES;
    constexpr bool read_a = in || dots, read_b = back || dots;
    constexpr int VEC = Elt<T>::VEC;
    __shared__ float part[MV_NW][KT];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tpc = MV_NW / g.wpt;                   // tokens a CTA holds at a time
    const int sub = warp % g.wpt;                    // this warp's share of its token
    const int nch = g.m / VEC, k = g.k;
    const int64_t step = (int64_t)gridDim.x * tpc;
    int64_t t = (int64_t)blockIdx.x * tpc + warp / g.wpt;
    // lane r holds route r; the next token's entries travel while this token's rows move
    auto fetch = [&](int64_t q, int &row, float &w) {
        row = -1;
        w = 0.0f;
        if (lane < k && q < g.s) {
            row = g.rows[(int64_t)lane * g.s + q];
            if (gated) w = g.gates[(int64_t)lane * g.s + q];
        }
    };
    int row_n;
    float w_n;
    fetch(t, row_n, w_n);
    // every warp of the CTA makes the same number of turns (the dot products meet at a barrier)
    for (int64_t t0 = (int64_t)blockIdx.x * tpc; t0 < g.s; t0 += step, t += step) {
        int row = row_n;
        const float wt = w_n;
        fetch(t + step, row_n, w_n);
        if (row < -1 || row >= g.n) {
            set_status(g.status, MOE_ERR_INVALID_ARG);
            row = -1;
        }
        const unsigned live = __ballot_sync(0xffffffffu, row >= 0);
        const bool mine = t < g.s;
        const V16 *ap = reinterpret_cast<const V16 *>(static_cast<const T *>(g.a) + (mine ? t : 0) * g.m);
        V16 *ao = reinterpret_cast<V16 *>(static_cast<T *>(g.a_out) + (mine ? t : 0) * g.m);
        const V16 *bp = static_cast<const V16 *>(g.b);
        V16 *bo = static_cast<V16 *>(g.b_out);
        // this lane's 16-byte piece of route r's row
        auto piece = [&](int r, int c) {
            return (int64_t)__shfl_sync(0xffffffffu, row, r & 31) * nch + c;
        };
        for (int rg = 0; rg < (dots ? k : 1); rg += KT) {
            float dot[KT];
#pragma unroll
            for (int i = 0; i < KT; i++) dot[i] = 0.0f;
            if (mine) {
                for (int c0 = sub * 32 * U; c0 < nch; c0 += g.wpt * 32 * U) {
                    const int c = c0 + lane;
                    V16 av[U];
                    if (read_a) {
#pragma unroll
                        for (int u = 0; u < U; u++)
                            if (c + 32 * u < nch) av[u] = k > KT ? ld_v16(ap + c + 32 * u) : ld_stream(ap + c + 32 * u);
                    }
                    float acc[U][VEC];
                    if (back) {
#pragma unroll
                        for (int u = 0; u < U; u++)
#pragma unroll
                            for (int i = 0; i < VEC; i++) acc[u][i] = 0.0f;
                    }
                    // KG routes from r0 on; their dot products are dot[d0 ..]
                    auto group = [&](int r0, float *dt) {
                        V16 bv[KG][U];
                        if (read_b) {
#pragma unroll
                            for (int i = 0; i < KG; i++) {
                                const int64_t o = piece(r0 + i, c);
                                if (r0 + i < k && ((live >> (r0 + i)) & 1u)) {
#pragma unroll
                                    for (int u = 0; u < U; u++)
                                        if (c + 32 * u < nch) bv[i][u] = ld_stream(bp + o + 32 * u);
                                }
                            }
                        }
#pragma unroll
                        for (int i = 0; i < KG; i++) {
                            int64_t o = 0;
                            if (in) o = piece(r0 + i, c);
                            const float w = gated ? __shfl_sync(0xffffffffu, wt, (r0 + i) & 31) : 1.0f;
                            if (r0 + i < k && ((live >> (r0 + i)) & 1u)) {
#pragma unroll
                                for (int u = 0; u < U; u++) {
                                    if (c + 32 * u >= nch) continue;
                                    if (in) st_v16(bo + o + 32 * u, gated ? ScaleRound<T>::apply(w, av[u]) : av[u]);
                                    if (!read_b) continue;
                                    float f[VEC];
                                    Elt<T>::unpack(bv[i][u], f);
                                    if (back) {
#pragma unroll
                                        for (int q = 0; q < VEC; q++)
                                            acc[u][q] = gated ? __fmaf_rn(w, f[q], acc[u][q]) : acc[u][q] + f[q];
                                    }
                                    if (dots) {
                                        float x[VEC];
                                        Elt<T>::unpack(av[u], x);
#pragma unroll
                                        for (int q = 0; q < VEC; q++) dt[i] = __fmaf_rn(x[q], f[q], dt[i]);
                                    }
                                }
                            }
                        }
                    };
                    if constexpr (dots) {
#pragma unroll
                        for (int d0 = 0; d0 < KT; d0 += KG) group(rg + d0, dot + d0);
                    } else {
                        for (int r0 = 0; r0 < k; r0 += KG) group(r0, dot);
                    }
                    if (back) {
#pragma unroll
                        for (int u = 0; u < U; u++)
                            if (c + 32 * u < nch) st_v16_cs(ao + c + 32 * u, Elt<T>::pack(acc[u]));
                    }
                }
            }
            if (dots) {   // lane i < KT: route rg + i
                float sum = reduce_many<KT>(dot, lane);
                if (g.wpt > 1) {
                    if (lane < KT) part[warp][lane] = sum;
                    __syncthreads();
                    if (sub == 0 && lane < KT) {
                        sum = part[warp][lane];
                        for (int w = 1; w < g.wpt; w++) sum += part[warp + w][lane];
                    }
                    __syncthreads();
                }
                if (mine && sub == 0 && lane < KT && rg + lane < k)
                    g.dots[(int64_t)(rg + lane) * g.s + t] = (live >> (rg + lane)) & 1u ? sum : 0.0f;
            }
        }
    }
}

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

template <typename T, int MODE, int KT, int KG, int U>
moe_status move_launch(MoveArgs g, cudaStream_t stream) {
    // as many warps a token as there are turns of 32 U chunks for, while the tokens alone leave warps idle
    const int sms = sm_count(), turns = (g.m / Elt<T>::VEC + 32 * U - 1) / (32 * U);
    g.wpt = 1;
    while (g.wpt < MV_NW && g.wpt < turns && g.s * g.wpt < (int64_t)sms * 24) g.wpt *= 2;
    const int64_t ctas = (g.s * g.wpt + MV_NW - 1) / MV_NW;
    const int64_t cap = (int64_t)sms * mv_ctas<MODE, KG, U>();   // resident at once
    return launch_pdl(move_rows_kernel<T, MODE, KT, KG, U>, dim3((unsigned)(ctas < cap ? ctas : cap)), dim3(MV_NT), 0,
                      stream, g);
}

// Eight or more 16-byte loads a lane under way, of at least two neighbouring chunks of a row: with one (512
// bytes a row and turn) the way back of 8191 x 8 rows of 4 KB took 111 us, with two 54; the way in's gradient
// with dot products 112 and 57.
template <typename T, int MODE>
moe_status move_typed(const MoveArgs &g, cudaStream_t stream) {
    if constexpr (!(MODE & (BACK | DOTS))) {
        return move_launch<T, MODE, 1, 1, 4>(g, stream);
    } else {
        if (g.k == 1) return move_launch<T, MODE, 1, 1, 4>(g, stream);
        if (g.k == 2) return move_launch<T, MODE, 2, 2, 4>(g, stream);
        if (g.k <= 4 || !(MODE & DOTS)) return move_launch<T, MODE, 4, 4, 2>(g, stream);
        return move_launch<T, MODE, 8, 8, 2>(g, stream);
    }
}

template <int MODE>
moe_status move(moe_dtype dt, const MoveArgs &g, cudaStream_t stream) {
    return dt == MOE_BF16 ? move_typed<__nv_bfloat16, MODE>(g, stream) : move_typed<float, MODE>(g, stream);
}

int sort_rounds(int64_t n) {   // rounds of 256 routes a CTA: at least 4, at most 256 CTAs
    const int64_t r = (n + (int64_t)ST_NT * ST_BLK - 1) / ((int64_t)ST_NT * ST_BLK);
    return (int)(r < 4 ? 4 : r);
}

}  // namespace

size_t sort_workspace_bytes(int64_t s, int e, int k) {
    const int64_t n = s * k, per = (int64_t)ST_NT * sort_rounds(n);
    return ((size_t)((n + per - 1) / per) * (size_t)(e + 1) * 4 + 255) & ~(size_t)255;
}

moe_status sort_routes_launch(const int32_t *idx, int64_t s, int e, int k, int32_t *rows, int32_t *offsets,
                              int32_t *source, void *ws, int32_t *st, cudaStream_t stream) {
    const int64_t n = s * k;
    const int nb = e + 1;
    if (n <= SS_MAXN && e <= SS_MAXE)
        return launch_pdl(sort_small_kernel, dim3((unsigned)((n + SS_NT - 1) / SS_NT)), dim3(SS_NT),
                          (size_t)(3 * nb + 1 + SS_NW * nb) * 4, stream, idx, (int)n, e, rows, offsets, source, st);
    const int rounds = sort_rounds(n);
    const unsigned nblk = (unsigned)((n + (int64_t)ST_NT * rounds - 1) / ((int64_t)ST_NT * rounds));
    moe_status r = launch_pdl(sort_hist_kernel, dim3(nblk), dim3(ST_NT), 0, stream, idx, n, e, rounds, (int32_t *)ws,
                              st);
    if (r != MOE_OK) return r;
    return launch_pdl(rounds <= ST_HELD ? sort_place_kernel<true> : sort_place_kernel<false>, dim3(nblk), dim3(ST_NT),
                      (size_t)(3 * nb + 1 + ST_NW * nb) * 4, stream, idx, n, e, rounds, (const int32_t *)ws, rows,
                      offsets, source, st);
}

moe_status encode_sorted_launch(const void *x, moe_dtype dt, const int32_t *rows, const float *gates, int64_t s, int m,
                                int k, int64_t n, void *out, int32_t *st, cudaStream_t stream) {
    const MoveArgs g{x, nullptr, nullptr, out, rows, gates, nullptr, s, n, m, k, 1, st};
    return gates ? move<IN | GATES>(dt, g, stream) : move<IN>(dt, g, stream);
}

moe_status decode_sorted_launch(const void *xs, moe_dtype dt, const int32_t *rows, const float *gates, int64_t s,
                                int m, int k, int64_t n, void *y, int32_t *st, cudaStream_t stream) {
    const MoveArgs g{nullptr, xs, y, nullptr, rows, gates, nullptr, s, n, m, k, 1, st};
    return gates ? move<BACK | GATES>(dt, g, stream) : move<BACK>(dt, g, stream);
}

moe_status decode_sorted_bwd_launch(const void *dy, const void *xs, moe_dtype dt, const int32_t *rows,
                                    const float *gates, int64_t s, int m, int k, int64_t n, void *d_xs,
                                    float *d_gates, int32_t *st, cudaStream_t stream) {
    const MoveArgs g{dy, xs, nullptr, d_xs, rows, gates, d_gates, s, n, m, k, 1, st};
    return move<IN | DOTS | GATES>(dt, g, stream);
}

moe_status encode_sorted_bwd_launch(const void *d_out, const void *x, moe_dtype dt, const int32_t *rows,
                                    const float *gates, int64_t s, int m, int k, int64_t n, void *d_x,
                                    float *d_gates, int32_t *st, cudaStream_t stream) {
    const MoveArgs g{x, d_out, d_x, nullptr, rows, gates, d_gates, s, n, m, k, 1, st};
    if (!gates) return move<BACK>(dt, g, stream);
    if (!d_gates) return move<BACK | GATES>(dt, g, stream);
    if (k <= 8) return move<BACK | DOTS | GATES>(dt, g, stream);   // all routes of a token in one group
    const moe_status r = move<BACK | GATES>(dt, g, stream);
    if (r != MOE_OK) return r;
    return dt == MOE_BF16 ? move_launch<__nv_bfloat16, DOTS, 8, 8, 2>(g, stream)
                          : move_launch<float, DOTS, 8, 8, 2>(g, stream);
}

}  // namespace moe
