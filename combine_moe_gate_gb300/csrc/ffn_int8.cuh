// Grouped products of 8-bit integer rows and weights on the tensor cores.  Included by ffn_tc.cu,
// whose barrier, copy and TMEM helpers it shares (and, of the 4-bit products, the GELU).
//
//   out[i, :] = act(s_x[i] s_w[j] (X[i] W[j]^T) + bias[j])   for the rows i of every expert j
//
// sm_103a has no integer tcgen05 (kind::i8), and its mma.sync integers run at a small part of the
// 16-bit rate.  Every 8-bit integer is an fp16 number, and a product of two is exact in fp32, so the
// products run as kind::f16 on fp16 operands with fp32 sums: exact while a partial sum is below
// 2^24 (always for K <= 1024), otherwise with fp32's rounding.  The weights stay 8-bit in memory and
// in shared memory and become fp16 on the way from there to TMEM, where the MMA reads them as its A
// operand; the rows (few bytes beside the weights, or reused by many weight tiles) are widened once
// before.  So a stage costs shared memory 8 KB of weights in and out and 12 KB of rows in and out per
// 64 of K and SM, 320 clocks at 128 bytes a clock, against 384 clocks of MMA.
//
// One persistent kernel on CTA pairs, tiles of 256 output channels (M: 128 a CTA) by up to 192 rows
// (N, a multiple of 32 that the expert's rows are cut into evenly), 512 threads a CTA:
//   warp 0       weights: 128 x 128 bytes a stage
//   warps 2, 3   rows: this CTA's half of the tile's rows, each one half of the stage's K, in boxes of
//                32 rows x 64 fp16
//   warps 4-11   widen: two groups of four warps take the stages in turn; a lane reads its channel's
//                128 bytes and writes 64 TMEM columns
//   warp 1       allocates TMEM; in the even CTA issues the pair's MMAs (A from TMEM, K = 16 each)
//   warps 12-15  epilogue: TMEM holds channels by rows, so a lane has one channel's scale and bias;
//                the block is turned in shared memory and stored as rows
// TMEM (512 columns), by the largest N of the launch's tiles: the way from a stage's MMAs over the widening
// warps to the MMAs that read what they wrote takes about 2000 clocks (two barriers across the pair), so
// three or four stages of A (64 columns each) have to be under way:
//   N <= 64    accumulators at 0 and 64,   4 stages from 128
//   N <= 128   accumulators at 0 and 128,  4 stages from 256
//   N <= 192   accumulators at 0 and 128,  3 stages from 320: they share columns 128 .. 191, so the next
//              tile's MMAs wait until the epilogue has read those
//
// Measured (GB300).  8 experts, 16384 rows, 4096 <-> 8192: 582 us (GELU) and 546 us, 1.89 and 2.01 PFLOP/s, the
// tensor pipe active 83% and 88% of the time: bound by it.  Decoding over 256 SwiGLU experts, 7168 x 2048: 480 and
// 225 us, the weights at 5.8 and 6.1 TB/s: bound by HBM.  16 experts, 2000 tokens x 2, 2048 -> 1048: 27 us, two
// tiles for most pairs: set-up 3 us, two main loops of 5 us, the last epilogue 2.5 us.
// (tests/test_int8_ring_host.py runs the barriers and roles under schedules that hold one of them back.)
#pragma once

#include "int8.cuh"

namespace moe {
namespace {

constexpr int I8_NT = 192;                       // rows per tile at most
constexpr int I8_BK = 128;                       // K per stage
constexpr int I8_W_BYTES = UM * I8_BK;           // weights of a stage, one CTA
constexpr int I8_BOX = 32;                       // rows of one row copy
constexpr int I8_BOX_BYTES = I8_BOX * 128;       // 64 fp16 each
constexpr int I8_XH_BYTES = I8_NT / 2 * 128;     // rows of half a stage, one CTA
constexpr int I8_X_BYTES = 2 * I8_XH_BYTES;
constexpr int I8_WST = 6, I8_XST = 4;            // stages of weights, of rows
static_assert(I8_WST % 2 == 0 && (I8_XST & (I8_XST - 1)) == 0, "the widening groups take the stages in turn");
constexpr int I8_CVT0 = 4, I8_EPI0 = 12;         // first warp of the two roles
constexpr int I8_THREADS = 512;
constexpr int I8_STG_BYTES = 32 * 32 * 4;        // output staging per epilogue warp

struct I8Layout {
    uint32_t acc1, slot0;        // first column of the second accumulator, of the stages of A
    int slots;                   // at most I8_XST
    bool shared;                 // the accumulators share columns [128, 192)
};

__device__ __forceinline__ I8Layout i8_layout(int max_n) {
    if (max_n <= 64) return I8Layout{64, 128, 4, false};
    if (max_n <= 128) return I8Layout{128, 256, 4, false};
    return I8Layout{128, 320, 3, true};
}

// Step i of the pair (a stage of K) uses the weights' barriers i % WST, the rows' i % XST and the TMEM
// slot i % slots.  A wait for a parity is sound while its barrier is neither two phases ahead of the
// waiter (the next phase needs the waiter) nor one behind (the waiter has seen the phase before, or what
// follows from it):
//   wfull (copies): waited for by the 4 widening warps of the CTA that take step i (they took step i - WST
//     as well), each of which then arrives at wempty; wempty (4): waited for by the weights' producer, who
//     issues the next copies.
//   full (even CTA: 4 widening warps of each CTA, and its two rows' producers with the bytes of both CTAs):
//     waited for by the MMA issuer.  (A tile has N / 2 rows for each CTA, N at least 32: all always copy.)
//     A widening warp arrives for step i after the MMAs of step i - slots, so that of i - XST is complete.
//   empty (per CTA, a commit after the step's MMAs): waited for by the rows' producers before step
//     i + XST, whose MMAs are its next phase and need their bytes; and by the widening warps of step
//     i + slots before they write the slot: as XST is even, a barrier is always met by the same group, at
//     each of its phases, and the next phase comes after or with the MMAs of step i + slots.
//   dfull (a commit, per CTA): waited for by its 4 epilogue warps, each of which then arrives at dempty
//     (even CTA, 8), waited for by the MMA issuer, who commits the next dfull: two of each, by the tile's
//     number.  drain: one phase.
// All roles of both CTAs go through the same tiles.
struct I8Ctl {
    uint64_t wfull[I8_WST], wempty[I8_WST];
    uint64_t full[I8_XST], empty[I8_XST];
    uint64_t dfull[2], dempty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int32_t abort;
    int32_t total_tiles;
    int32_t max_n;               // largest N of any tile
    int32_t tile_start[MAX_E + 1];
    int32_t first[MAX_E + 1];    // the offsets, inside the buffer and ascending
};

constexpr size_t I8_SMEM = 1024 + (size_t)I8_WST * I8_W_BYTES + (size_t)I8_XST * I8_X_BYTES + 4 * I8_STG_BYTES + sizeof(I8Ctl);
static_assert(I8_SMEM + 4 * I8_NT * 4 + 64 <= 227 * 1024, "shared memory");   // with what is not dynamic

struct I8Args {
    SortedRows so;               // offsets null: one expert has all n rows
    int32_t *status;
    const float *x_scale;        // [n]
    const float *w_scale;        // [e, n_out]
    const float *w3_scale;       // SwiGLU
    const __nv_bfloat16 *bias;   // [e, n_out] or nullptr
    void *out;                   // [n, n_out]
    int e;
    int K;
    int n_out;
    int32_t stall;               // tests: the producers issue no copies
};

struct I8Tile {
    int j, ct, row0, rows, n;    // expert, channel tile, first row, live rows, N
};

// Rows of a tile: even cuts, a multiple of 32.  (As rows > 192 (tiles - 1), none of the tiles is empty.  The sum
// is unsigned: rows of more than 2^31 - 2^31 / 193 and their tiles pass 2^31.)
__device__ __forceinline__ int i8_cut(int rows, int tiles) {
    return (int)((((uint32_t)rows + (uint32_t)tiles - 1u) / (uint32_t)tiles + 31u) & ~31u);
}

// Tile t; an expert's row tiles vary fastest, so neighbouring CTAs read the same weights.
__device__ __forceinline__ I8Tile i8_tile(const I8Ctl *ctl, int e, int t) {
    int lo = 0, hi = e;   // largest j with tile_start[j] <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (ctl->tile_start[mid] <= t) lo = mid; else hi = mid;
    }
    I8Tile T;
    T.j = lo;
    const int first = ctl->first[lo], rows = ctl->first[lo + 1] - first;
    const int tiles = (rows + I8_NT - 1) / I8_NT, local = t - ctl->tile_start[lo];
    const int per = i8_cut(rows, tiles);
    T.ct = local / tiles;
    const int rt = local - T.ct * tiles;
    T.row0 = first + rt * per;
    T.rows = min(per, rows - rt * per);
    T.n = (T.rows + 31) & ~31;
    return T;
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// 2-SM MMA with A (fp16, two a column, lane = row) in both CTAs' TMEM, by the lane with `one`.
__device__ __forceinline__ void umma_pair_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate,
                                             uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(one)
        : "memory");
}

__device__ __forceinline__ void umma_commit_pair_one(uint64_t *bar, uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
            su32(bar)),
        "h"((uint16_t)3u), "r"(one)
        : "memory");
}

// Whether the phase with `parity` is complete, without waiting.
template <bool CL>
__device__ __forceinline__ bool mbar_test(uint64_t *b, uint32_t parity) {
    uint32_t ok;
    if (CL)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(su32(b)), "r"(parity)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(su32(b)), "r"(parity)
            : "memory");
    return ok != 0;
}

// mbar_wait for the waits on the way of every 64 of K: the clock is read only after some tries.
template <bool CL>
__device__ __forceinline__ bool i8_wait(uint64_t *b, uint32_t parity, int32_t *abort_flag, int32_t *status) {
#pragma unroll 1
    for (int i = 0; i < 64; i++)
        if (mbar_try<CL>(b, parity)) return true;
    return mbar_wait<CL>(b, parity, abort_flag, status);
}

// GELU with a relative error, as the 4-bit products': a row that lies in the tail is scaled by it.  (There an
// infinity becomes a NaN; both make the row's scale one.)
__device__ __forceinline__ float2 i8_gelu2(float2 a) {
    const float2 g = f4_gelu2(a);
    return make_float2(a.x == INFINITY ? a.x : g.x, a.y == INFINITY ? a.y : g.y);
}

__device__ __forceinline__ float i8_relu(float v) { return v < 0.0f ? 0.0f : v; }   // a NaN stays one

template <int EPI, typename OUT>
__global__ void __launch_bounds__(I8_THREADS, 1)
i8_group_gemm(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmW3,
              const __grid_constant__ CUtensorMap tmX, const I8Args args) {
    constexpr bool SWI = EPI == I8_SWIGLU;
    constexpr int CH = SWI ? 64 : UM;             // output channels per CTA and tile
    __shared__ int32_t s_bad;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sW = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *sX = sW + I8_WST * I8_W_BYTES;
    uint8_t *stg_all = sX + I8_XST * I8_X_BYTES;
    I8Ctl *ctl = (I8Ctl *)(stg_all + 4 * I8_STG_BYTES);
    __shared__ __align__(16) float s_scale[4][I8_NT];   // per epilogue warp: the tile's row scales
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int tile0 = blockIdx.x / 2, tile_step = gridDim.x / 2;
    const int nct = (args.n_out + 2 * CH - 1) / (2 * CH);
    const int nk = (args.K + I8_BK - 1) / I8_BK;

    // barriers and TMEM before the wait for the kernel before, what the offsets say after it
    if (warp == 0 && lane == 0) {
        ctl->abort = 0;
        for (int s = 0; s < I8_WST; s++) {
            mbar_init(&ctl->wfull[s], 1);
            mbar_init(&ctl->wempty[s], 4);
        }
        for (int s = 0; s < I8_XST; s++) {
            mbar_init(&ctl->full[s], 10);
            mbar_init(&ctl->empty[s], 1);
        }
        for (int s = 0; s < 2; s++) {
            mbar_init(&ctl->dfull[s], 1);
            mbar_init(&ctl->dempty[s], 8);
        }
        mbar_init(&ctl->drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    } else if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&ctl->tmem_base)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    __syncwarp();
    pdl_enter();
    // one thread an expert, so that the loads travel together; the status by a warp that has none of the first 32
    if (threadIdx.x == I8_THREADS - 1) s_bad = status_bad(args.status) ? 1 : 0;
    bool bad = false;
    for (int j = threadIdx.x; j <= args.e; j += I8_THREADS) {
        int o = j ? (int)args.so.n : 0;
        if (args.so.offsets) {
            const int before = args.so.offsets[max(j - 1, 0)];
            o = args.so.offsets[j];
            bad |= o < 0 || o > args.so.n || before > o || (j == 0 && o != 0);
        }
        ctl->first[j] = o;
    }
    bad = __syncthreads_or(bad);
    if (warp == 0) {
        if (bad && lane == 0) set_status(args.status, MOE_ERR_INVALID_ARG);   // and no tiles
        int run = 0, max_n = 0;
        for (int base = 0; base < args.e; base += 32) {
            const int j = base + lane;
            const int rows = j < args.e && !bad ? ctl->first[j + 1] - ctl->first[j] : 0;
            const int cuts = (rows + I8_NT - 1) / I8_NT, own = cuts * nct;
            if (rows) max_n = max(max_n, i8_cut(rows, cuts));
            int v = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            if (j < args.e) ctl->tile_start[j] = run + v - own;
            run += __shfl_sync(0xffffffffu, v, 31);
        }
        max_n = __reduce_max_sync(0xffffffffu, max_n);
        if (lane == 0) {
            ctl->max_n = max_n;
            ctl->tile_start[args.e] = run;
            ctl->total_tiles = run;
        }
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    int total = ctl->total_tiles;
    {
        int any_bad = 0;   // the same decision in both CTAs
        for (uint32_t r = 0; r < 2; r++) {
            int b;
            asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(b) : "r"(map_to_rank(su32(&s_bad), r)));
            any_bad |= b;
        }
        if (any_bad) total = 0;
    }
    int32_t *abort_flag = &ctl->abort;
    const I8Layout L = i8_layout(ctl->max_n);

    if (warp == 0) {
        if (elect_one()) {
            int s = 0;
            uint32_t ph = 1;
            bool ok = true, ready = false;   // ready: the next stage was seen free
            for (int t = tile0; t < total && !args.stall && ok; t += tile_step) {
                const I8Tile T = i8_tile(ctl, args.e, t);
                const int ch = T.j * args.n_out + T.ct * 2 * CH + (int)rank * CH;
                for (int kb = 0; kb < nk; kb++) {
                    ok = ready || i8_wait<false>(&ctl->wempty[s], ph, abort_flag, args.status);
                    if (!ok) break;
                    const int sn = s + 1 == I8_WST ? 0 : s + 1;
                    ready = mbar_test<false>(&ctl->wempty[sn], sn ? ph : ph ^ 1u);
                    mbar_expect_tx(&ctl->wfull[s], I8_W_BYTES);
                    tma_load_2d(sW + s * I8_W_BYTES, &tmW, kb * I8_BK, ch, &ctl->wfull[s]);
                    if (SWI)
                        tma_load_2d(sW + s * I8_W_BYTES + I8_W_BYTES / 2, &tmW3, kb * I8_BK, ch, &ctl->wfull[s]);
                    s = sn;
                    if (s == 0) ph ^= 1u;
                }
            }
        }
    } else if (warp == 2 || warp == 3) {
        // (elected lanes issue copies faster than a branch on the lane number, as they do MMAs: six copies
        // took 730 clocks of a stage's 768)
        if (elect_one()) {
            const int hf = warp - 2;
            const uint32_t fb0 = map_to_rank(su32(&ctl->full[0]), 0);
            uint8_t *sh = sX + hf * I8_XH_BYTES;
            int s = 0;
            uint32_t ph = 1;
            bool ok = true, ready = false;
            for (int t = tile0; t < total && !args.stall && ok; t += tile_step) {
                const I8Tile T = i8_tile(ctl, args.e, t);
                const int half = T.n / 2, boxes = (half + I8_BOX - 1) / I8_BOX;
                const int r0 = T.row0 + (int)rank * half;
                for (int kb = 0; kb < nk; kb++) {
                    ok = ready || i8_wait<true>(&ctl->empty[s], ph, abort_flag, args.status);
                    if (!ok) break;
                    const int sn = (s + 1) & (I8_XST - 1);
                    ready = mbar_test<true>(&ctl->empty[sn], sn ? ph : ph ^ 1u);
                    if (rank == 0) mbar_expect_tx(&ctl->full[s], 2 * boxes * I8_BOX_BYTES);
                    for (int b = 0; b < boxes; b++)
                        tma_load_2d_pair(sh + s * I8_X_BYTES + b * I8_BOX_BYTES, &tmX, kb * I8_BK + hf * 64,
                                         r0 + b * I8_BOX, fb0 + 8 * s);
                    s = sn;
                    if (s == 0) ph ^= 1u;
                }
            }
        }
    } else if (warp == 1) {
        // The whole warp goes along and one lane's instructions count: in a branch of one lane the
        // descriptors would be moved to uniform registers for every MMA (about 95 clocks each).
        if (rank == 0) {
            const uint32_t one = elect_one();
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint64_t x0 = sdesc<128>(__shfl_sync(0xffffffffu, su32(sX), 0));
            const uint32_t slot0 = __shfl_sync(0xffffffffu, L.slot0, 0), acc1 = __shfl_sync(0xffffffffu, L.acc1, 0);
            const int slots = __shfl_sync(0xffffffffu, L.slots, 0);
            int s = 0, slot = 0, i = 0;      // i: the pair's tiles so far
            uint32_t ph = 0;
            bool ok = true, ready = false;   // ready: the next step's full was seen
            for (int t = tile0; t < total && ok; t += tile_step, i++) {
                const int n = __shfl_sync(0xffffffffu, i8_tile(ctl, args.e, t).n, 0);
                const uint32_t idesc = (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)((2 * UM) >> 4) << 24);
                // the accumulator's last tile is read, or (shared) the columns that the one before holds too
                const int last = L.shared ? i - 1 : i - 2;
                if (last >= 0) ok = i8_wait<true>(&ctl->dempty[last & 1], (last >> 1) & 1, abort_flag, args.status);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                const uint32_t d = tm + (i & 1 ? acc1 : 0);
                for (int kb = 0; kb < nk; kb++) {
                    ok = ready || i8_wait<true>(&ctl->full[s], ph, abort_flag, args.status);
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                    tc_fence_after();
                    const uint64_t b0 = x0 + (uint64_t)(s * (I8_X_BYTES >> 4));
                    const uint32_t a0 = tm + slot0 + (uint32_t)(slot * 64);
                    // a look at the next step's barrier travels while this step's MMAs are issued
                    const int sn = (s + 1) & (I8_XST - 1);
                    ready = mbar_test<true>(&ctl->full[sn], sn ? ph : ph ^ 1u);
#pragma unroll
                    for (int kk = 0; kk < 8; kk++)
                        umma_pair_ts(d, a0 + kk * 8, b0 + (((kk >> 2) * I8_XH_BYTES + (kk & 3) * 32) >> 4), idesc,
                                     (kb | kk) != 0, one);
                    umma_commit_pair_one(&ctl->empty[s], one);
                    if (++slot == slots) slot = 0;
                    s = sn;
                    if (s == 0) ph ^= 1u;
                }
                if (!ok) break;
                umma_commit_pair_one(&ctl->dfull[i & 1], one);
            }
            umma_commit_pair_one(&ctl->drain, one);
        }
        unsigned long long t0 = gtimer();
        while (!mbar_try<true>(&ctl->drain, 0) && gtimer() - t0 < WAIT_NS) {
        }
    } else if (warp >= I8_CVT0 && warp < I8_EPI0) {
        // ------------------------------------------------------------- widen
        const int g = (warp - I8_CVT0) >> 2, quarter = warp & 3;
        const int row = SWI ? (lane < 16 ? quarter * 16 + lane : 48 + quarter * 16 + lane) : quarter * 32 + lane;
        const uint32_t ta = tmem + L.slot0 + ((uint32_t)(quarter * 32) << 16);
        const int tiles = total > tile0 ? (total - tile0 + tile_step - 1) / tile_step : 0;
        const uint32_t steps = (uint32_t)tiles * (uint32_t)nk;
        int s = g, slot = g;
        uint32_t ph = 0;
        bool ready = false;                                   // the next step's weights were seen
        const uint32_t slots = (uint32_t)L.slots;
        for (uint32_t step = g; step < steps; step += 2) {
            bool ok = ready || i8_wait<false>(&ctl->wfull[s], ph, abort_flag, args.status);
            if (!__all_sync(0xffffffffu, ok)) break;
            const uint8_t *src = sW + s * I8_W_BYTES + row * 128;
            const int sn = s + 2 >= I8_WST ? s + 2 - I8_WST : s + 2;
#pragma unroll
            for (int hf = 0; hf < 2; hf++) {
                uint32_t r[32];
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(src + (((hf * 4 + c) ^ (row & 7)) << 4));
                    i8_widen(v.x, r[8 * c], r[8 * c + 1]);
                    i8_widen(v.y, r[8 * c + 2], r[8 * c + 3]);
                    i8_widen(v.z, r[8 * c + 4], r[8 * c + 5]);
                    i8_widen(v.w, r[8 * c + 6], r[8 * c + 7]);
                }
                if (hf == 0 && step >= slots) {
                    const uint32_t last = step - slots;   // of the slot
                    ok = i8_wait<true>(&ctl->empty[last & (I8_XST - 1)], last / I8_XST & 1u, abort_flag, args.status);
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                    tc_fence_after();
                }
                if (hf == 1) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl->wempty[s]);
                    ready = mbar_test<false>(&ctl->wfull[sn], sn > s ? ph : ph ^ 1u);
                }
                tmem_st32(ta + (uint32_t)(slot * 64 + hf * 32), r);
            }
            if (!ok) break;
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_to_rank(su32(&ctl->full[step & (I8_XST - 1)]), 0));
            slot += 2;
            if (slot >= L.slots) slot -= L.slots;
            if (sn < s) ph ^= 1u;
            s = sn;
        }
    } else if (warp >= I8_EPI0) {
        // ---------------------------------------------------------- epilogue
        const int quarter = warp & 3;
        uint8_t *stg = stg_all + quarter * I8_STG_BYTES;
        float *ssc = s_scale[quarter];
        int i = 0;
        for (int t = tile0; t < total; t += tile_step, i++) {
            const I8Tile T = i8_tile(ctl, args.e, t);
            // this warp's first output channel, and this lane's
            const int ch0 = T.ct * 2 * CH + (int)rank * CH + quarter * (CH / 4);
            const int ch = ch0 + (SWI ? lane & 15 : lane);
            float sb = 0.0f, bias = 0.0f;
            if (ch < args.n_out) {
                const int64_t at = (int64_t)T.j * args.n_out + ch;
                sb = SWI && lane >= 16 ? args.w3_scale[at] : args.w_scale[at];
                if (!SWI && args.bias) bias = __bfloat162float(args.bias[at]);
            }
            const I8Scale w = i8_scale(sb);
            const float2 ws = make_float2(w.s, w.s), wu = make_float2(w.up, w.up), bias2 = make_float2(bias, bias);
            for (int r = lane; r < T.n; r += 32) ssc[r] = r < T.rows ? args.x_scale[(int64_t)T.row0 + r] : 0.0f;
            __syncwarp();
            const bool ok = i8_wait<true>(&ctl->dfull[i & 1], (i >> 1) & 1, abort_flag, args.status);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const uint32_t tb = tmem + ((uint32_t)(quarter * 32) << 16) + (i & 1 ? L.acc1 : 0);
            // shared accumulators: the blocks that the next tile's accumulator holds too come first (of an
            // even tile columns 128 .., of an odd one 0 .. 63), then the issuer may go on
            const int blocks = T.n / 32, begin = L.shared && !(i & 1) && blocks > 4 ? 4 : 0;
            const int both = !L.shared ? 0 : i & 1 ? min(2, blocks) : blocks - begin < blocks ? blocks - begin : 0;
            auto next_tile = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(map_to_rank(su32(&ctl->dempty[i & 1]), 0));
            };
            if (L.shared && both == 0) next_tile();
            for (int q = 0; q < blocks; q++) {
                const int at = begin + q, c0 = 32 * (at < blocks ? at : at - blocks);
                uint32_t r[32];
                tmem_ld32(tb + (uint32_t)c0, r);
                const int left = T.rows - c0;          // live rows of this block (32 or fewer)
                tmem_wait_ld(r);
                if (q + 1 == both) next_tile();
                float v[32];
                // as i8_scaled, two rows at a time
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    const float2 sum = make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1]));
                    const float2 sa = *reinterpret_cast<const float2 *>(ssc + c0 + i);
                    const float2 o = __ffma2_rn(__fmul2_rn(__fmul2_rn(sum, ws), sa), wu, bias2);
                    v[i] = o.x;
                    v[i + 1] = o.y;
                }
                if constexpr (SWI) {
                    // lane l < 16 holds a, lane l + 16 b of a channel: the first takes rows 0-15, the
                    // second rows 16-31
                    __nv_bfloat16 *sp = reinterpret_cast<__nv_bfloat16 *>(stg);
                    const bool up = lane >= 16;
                    bool mid = true;
#pragma unroll
                    for (int i = 0; i < 16; i++) {
                        const float other = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + 16], 16);
                        const float ga = up ? other : v[i], gb = up ? v[i + 16] : other;
                        v[i] = ga;
                        v[i + 16] = gb;
                        mid &= i + (lane & 16) >= left || silu_mid_ok(ga);
                    }
                    if (__all_sync(0xffffffffu, mid)) {
#pragma unroll
                        for (int i = 0; i < 16; i++)
                            sp[(i + (lane & 16)) * 16 + (lane & 15)] = __float2bfloat16_rn(silu_mid(v[i]) * v[i + 16]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; i++)
                            sp[(i + (lane & 16)) * 16 + (lane & 15)] = __float2bfloat16_rn(silu(v[i]) * v[i + 16]);
                    }
                    __syncwarp();
#pragma unroll
                    for (int q = lane; q < 64; q += 32) {
                        const int row = q >> 1, part = (q & 1) * 8;
                        if (row < left && ch0 + part < args.n_out)
                            *reinterpret_cast<uint4 *>((__nv_bfloat16 *)args.out +
                                                       ((int64_t)T.row0 + c0 + row) * args.n_out + ch0 + part) =
                                *reinterpret_cast<const uint4 *>(sp + row * 16 + part);
                    }
                } else {
                    OUT *sp = reinterpret_cast<OUT *>(stg);
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        float2 a = make_float2(v[i], v[i + 1]);
                        if (EPI == I8_GELU) a = i8_gelu2(a);
                        if (EPI == I8_RELU) a = make_float2(i8_relu(a.x), i8_relu(a.y));
                        if constexpr (sizeof(OUT) == 2) {
                            sp[i * 32 + lane] = __float2bfloat16_rn(a.x);
                            sp[(i + 1) * 32 + lane] = __float2bfloat16_rn(a.y);
                        } else {
                            sp[i * 32 + lane] = a.x;
                            sp[(i + 1) * 32 + lane] = a.y;
                        }
                    }
                    __syncwarp();
                    constexpr int PER = 16 / sizeof(OUT), PARTS = 32 / PER;   // values and pieces of a row
#pragma unroll
                    for (int q = lane; q < 32 * PARTS; q += 32) {
                        const int row = q / PARTS, part = (q % PARTS) * PER;
                        if (row < left && ch0 + part < args.n_out)
                            *reinterpret_cast<uint4 *>((OUT *)args.out + ((int64_t)T.row0 + c0 + row) * args.n_out +
                                                       ch0 + part) =
                                *reinterpret_cast<const uint4 *>(sp + row * 32 + part);
                    }
                }
                __syncwarp();   // staging is rewritten for the next block, the scales for the next tile
            }
            if (!L.shared) next_tile();
        }
    }

    __syncwarp();   // the elected lanes are back
    tc_fence_before();
    if (*(volatile int32_t *)abort_flag) {   // copies may still be landing: they take microseconds
        unsigned long long t0 = gtimer();
        while (gtimer() - t0 < 1000000ull) {
        }
    }
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
    }
}

template <int EPI, typename OUT>
moe_status launch_i8(const void *x16, const void *w, const void *w3, I8Args args, cudaStream_t stream) {
    args.stall = take_gemm_stall() ? 1 : 0;
    constexpr bool SWI = EPI == I8_SWIGLU;
    constexpr int CH = SWI ? 64 : UM;
    CUtensorMap mW, mW3, mX;
    if (!make_map_u8(&mW, w, (uint64_t)args.e * args.n_out, (uint64_t)args.K, CH) ||
        !make_map_u8(&mW3, SWI ? w3 : w, (uint64_t)args.e * args.n_out, (uint64_t)args.K, CH) ||
        !make_map(&mX, x16, (uint64_t)args.so.n, (uint64_t)args.K, I8_BOX, 64))   // fp16: 16-bit elements
        return MOE_ERR_CUDA;
    auto kern = i8_group_gemm<EPI, OUT>;
    static int units[64] = {0};   // resident clusters per device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
    int nunits = dev >= 0 && dev < 64 ? units[dev] : 0;
    if (!nunits) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)I8_SMEM) != cudaSuccess)
            return MOE_ERR_CUDA;
        nunits = max_clusters(kern, I8_SMEM, 2, I8_THREADS);
        if (dev >= 0 && dev < 64) units[dev] = nunits;
    }
    const int64_t nct = (args.n_out + 2 * CH - 1) / (2 * CH);
    const int64_t upper = (args.so.n / I8_NT + (args.so.n < args.e ? args.so.n : args.e)) * nct;
    const int64_t grid = upper < nunits ? upper : nunits;
    return launch_cluster_pdl(kern, dim3((unsigned)(2 * grid)), dim3(I8_THREADS), I8_SMEM, 2, stream, mW, mW3, mX,
                              args);
}

}  // namespace

// out [n, n_out] (bf16, or fp32 when f32: the plain product only) from the rows' codes as fp16 numbers.
moe_status i8_gemm_launch(const void *x16, const float *x_scale, const SortedRows &so, const void *w,
                          const float *w_scale, const void *w3, const float *w3_scale, const void *bias, int epi,
                          bool f32, int e, int K, int n_out, void *out, int32_t *st, cudaStream_t stream) {
    I8Args g{so, st, x_scale, w_scale, w3_scale, (const __nv_bfloat16 *)bias, out, e, K, n_out, 0};
    switch (epi) {
        case I8_RELU: return launch_i8<I8_RELU, __nv_bfloat16>(x16, w, w3, g, stream);
        case I8_GELU: return launch_i8<I8_GELU, __nv_bfloat16>(x16, w, w3, g, stream);
        case I8_SWIGLU: return launch_i8<I8_SWIGLU, __nv_bfloat16>(x16, w, w3, g, stream);
        default:
            return f32 ? launch_i8<I8_BIAS, float>(x16, w, w3, g, stream)
                       : launch_i8<I8_BIAS, __nv_bfloat16>(x16, w, w3, g, stream);
    }
}

}  // namespace moe
