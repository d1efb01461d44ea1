// Grouped products of microscaled 4-bit operands on the tensor cores, and the
// expert FFN made of them.  Included by ffn_tc.cu, whose barrier, copy, TMEM
// and store helpers it shares.
//
//   out[j] = g_a[j] g_b[j] (A[j] B[j]^T) + bias[j]            (bf16), or
//   hid[j] = quantise(act(...))   (e2m1 codes and block scales, for fc2)
//
// over the first min(counts[j], c) rows of every expert j.  The block scales
// enter the tensor core with the operands (kind::mxf4 with one e8m0 byte per
// 32 values, kind::mxf4nvf4 with one e4m3 byte per 16), so the accumulator is
// the sum of the values the codes stand for, in fp32.
//
// One persistent kernel on CTA pairs, 256 x 256 tiles (M = 256 over the pair),
// the roles of tc_group_gemm: four producer warps, one MMA issuer, eight
// epilogue warps.  A stage is 256 values of K: 128-byte swizzled rows of 128 A
// and 128 B rows per CTA, and the 512-byte scale tiles of those A rows and of
// all 256 B rows (each CTA's half of the product needs every column's scale).
// tcgen05.cp copies a stage's scale tiles into TMEM ahead of its four K = 64
// MMAs; the two run in the order of issue, so a stage's copies wait for the
// MMAs that still read the columns they overwrite.
//
// TMEM: two 256-column accumulators do not fit beside the scales, so they
// overlap in 64 columns: [0, 256) and [192, 448).  Each epilogue warp first
// loads its part of the overlap (one chunk of 32 columns) and then lets the next
// tile's MMAs begin; the rest of the epilogue runs under that main loop.  (An
// overlap of 128 columns held twice the registers and spilled: 8 GELU experts
// of 2048 rows, m 4096, h 8192: 331 us, 306 like this.  Twelve epilogue warps on
// top of the wide overlap took 318 us, but under a profiler one of its bounded
// waits ran out now and then: it had the lap that F4_FULL_ARRIVALS closes, which
// may or may not have been the cause, and it is not used.)
//
// What bounds it: a stage fills 38 KB of shared memory per SM (NV; MX 35) and
// its MMAs read 32, against 128 bytes a clock; 8192^3 runs at 6.5 to 7.3 PFLOP/s
// (MX 7.1 to 7.6, by the power cap), 4096 x 4096 x 8192 (7 tiles a pair) at 5.8 to 6.1.  With few rows an
// expert it is the weights' bytes: 6.3 TB/s at K = 7168, 5.9 at K = 2048.
#pragma once

#include "fp4.cuh"

namespace moe {
namespace {

enum Fp4Epi { FP4_BIAS = 0, FP4_RELU = 1, FP4_GELU = 2, FP4_SWIGLU = 3 };

constexpr int F4_BK = 256;                     // values of K per stage (128 bytes a row)
constexpr int F4_BOX_BYTES = 64 * 128;         // one operand copy: 64 rows
constexpr int F4_OP_BYTES = 2 * F4_BOX_BYTES;  // one operand per CTA and stage
constexpr uint32_t F4_SF_COL = 448;            // first TMEM column of the scales
constexpr uint32_t F4_ACC_STEP = 192;          // first column of the odd tiles' accumulator

template <int FMT>
struct F4Tiling {
    static constexpr int KT = F4_BK / (4 * Fp4<FMT>::BLK);   // scale tiles along a stage's K
    static constexpr int SF_BYTES = KT * 512;                // of 128 rows
    static constexpr int STAGE_BYTES = 2 * F4_OP_BYTES + 3 * SF_BYTES;
    static constexpr int STAGES = 215 * 1024 / STAGE_BYTES;  // 5 (NV), 6 (MX)
    static constexpr uint32_t SF_COLS = 12 * KT;             // TMEM columns of a stage's scales
    static constexpr uint32_t SETS = (TMEM_COLS - F4_SF_COL) / SF_COLS;   // stages whose scales TMEM holds
    static_assert(SETS >= 1, "TMEM");
};

template <int FMT>
constexpr size_t f4_smem_bytes() {
    using TL = F4Tiling<FMT>;
    return 1024 + (size_t)TL::STAGES * TL::STAGE_BYTES + sizeof(Ctl<TL::STAGES>);
}

struct F4Args {
    const int32_t *counts;
    const int32_t *c_dev;
    int32_t *status;
    const float *a_global;      // [e] or nullptr: 1
    const float *b_global;
    const float *b3_global;     // SwiGLU
    const __nv_bfloat16 *bias;  // [e, n_out] or nullptr
    __nv_bfloat16 *out;         // FP4_BIAS: [e, c_max, n_out]
    uint8_t *out_q;             // else: codes [e, c_max, n_out / 2],
    uint8_t *out_scale;         // scale tiles, and
    const float *out_global;    // factors [e] or nullptr
    int64_t c_max;
    int e;
    int K;
    int n_out;
    int32_t wide;               // rows of out are whole 32-byte sectors
    int32_t stall;              // tests: the producers issue no copies
    int32_t lag;                // tests: the second CTA's A producers fall behind
};

// Arrivals per phase of a stage's full barrier: the four producers of the first
// CTA (with the bytes of both CTAs) and the two A producers of the second.
//
// A wait for a parity is sound while its barrier cannot get two phases ahead of
// the waiter; the next phase of every barrier needs each of its waiters:
//   empty (per CTA, a commit of the MMAs): waited for by the CTA's producers, and
//     the MMAs need the stage's full phase, for which every producer arrives or
//     brings bytes.  The second CTA's A producers may have nothing to copy, where
//     a tile's rows all lie in the first CTA: they arrive all the same.  (Without
//     that the ring could go round twice while one of them looked away, and its
//     wait ran out.)
//   full (first CTA): waited for by the MMA issuer, which frees the stage.
//   tfull (per CTA, a commit): waited for by the epilogue warps; the next tile's
//     MMAs begin when all 16 of both CTAs have arrived at tempty, each after its
//     wait.  tempty: waited for by the MMA issuer, which commits the next tfull.
//   drain: one phase.
// All roles go through the same tiles: both CTAs form the list from the same
// counts, and agree on the status word before the first.
constexpr int F4_FULL_ARRIVALS = 6;

// Instruction descriptor of the block-scaled 4-bit kinds: A and B e2m1 (1 at
// bits 7 and 10), both K-major, N >> 3 at bit 17, scale type at bit 23 (1:
// e8m0), M >> 7 at bit 27; which two of a column's four scale bytes a K = 64
// step uses (0 or 2; four of them: 0) at bits 4 (B) and 29 (A).
template <int FMT>
__device__ __forceinline__ uint32_t f4_idesc(uint32_t sf_id) {
    return (1u << 7) | (1u << 10) | ((uint32_t)(BN >> 3) << 17) | (FMT == MOE_FP4_MX ? 1u << 23 : 0u) |
           ((uint32_t)((2 * UM) >> 7) << 27) | (sf_id << 4) | (sf_id << 29);
}

template <int FMT>
__device__ __forceinline__ void umma_pair_f4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                             uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    if (FMT == MOE_FP4_MX)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
}

// One 512-byte scale tile from each CTA's shared memory into four columns of
// its own TMEM, the 32 lanes repeated in all four lane quarters.
__device__ __forceinline__ void cp_scales_pair(uint32_t tmem, uint32_t saddr) {
    // no swizzle: 8-row groups of 16-byte rows, 128 bytes apart
    const uint64_t desc = (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

__device__ __forceinline__ void tma_load_3d_pair(void *dst, const CUtensorMap *map, int x, int y, int z,
                                                 uint32_t bar_cluster) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(su32(dst)),
        "l"((uint64_t)map), "r"(x), "r"(y), "r"(z), "r"(bar_cluster)
        : "memory");
}

// One lane of a converged warp.  The compiler knows that a single thread runs
// what this guards and issues its tcgen05 instructions back to back: a row of
// tcgen05.cp takes 17 cycles each, against 59 behind a comparison of the lane
// number (4096 x 4096 x 8192, NV: 93 us with the comparison, 48 us with this).
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// mbar_wait by a whole warp: the same answer in every lane (what follows is
// warp-wide).
__device__ __forceinline__ bool warp_wait(uint64_t *b, uint32_t parity, int32_t *abort_flag, int32_t *status) {
    return __all_sync(0xffffffffu, mbar_wait<true>(b, parity, abort_flag, status));
}

// silu(a) = a / (1 + e^-a), about 2 units in the last place: e^-a as 2^t with
// the rounding error of t = -a log2(e) put back, one approximate reciprocal.
// (With the general exp and division the epilogue of a tile with few rows took
// longer than its main loop: 16 decoded tokens over 256 experts, 505 us; 402.)
__device__ __forceinline__ float f4_silu(float a) {
    const float t = a * -1.4426950408889634f;
    const float r = __fmaf_rn(a, -1.4426950408889634f, -t);
    float e, q;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    e = e < INFINITY ? __fmaf_rn(e, r * 0.6931471805599453f, e) : e;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(1.0f + e));
    return a * q;
}

// ReLU; a NaN stays one.
__device__ __forceinline__ float f4_relu(float a) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(0.0f));
    return r;
}

// GELU, exact erf form, two values at a time: a Phi(a) = max(a, 0) - |a| Phi(-|a|)
// on both sides of zero.  log2 Phi(-x) is a polynomial, fitted (weighted least
// squares, weights raised where the error is largest) to its values on [0, 8], so
// that the error is relative: a block of hidden values that all lie in the tail is
// scaled by the tail.  Relative error of Phi(-x): 1.5e-6 up to x = 4, 7e-6 up to 6,
// 1.3e-4 up to 8, a tenth at 10; of GELU 2e-7 absolute, 17 instructions a pair.
// (The leading coefficient is negative: far out the power is 0.)
__device__ __forceinline__ float2 f4_gelu2(float2 a) {
    const float2 x = make_float2(fabsf(a.x), fabsf(a.y));
    constexpr float C[11] = {-9.999992940e-01f, -1.151132071e+00f, -4.590410182e-01f, -5.288755060e-02f,
                               7.504534765e-03f, -3.964193125e-04f, -1.097939049e-04f, 3.183589297e-05f,
                               -3.947251672e-06f, 2.523481067e-07f, -6.728881193e-09f};
    float2 p = make_float2(C[10], C[10]);
#pragma unroll
    for (int i = 9; i >= 0; i--) p = __ffma2_rn(x, p, make_float2(C[i], C[i]));
    float2 q;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(q.x) : "f"(p.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(q.y) : "f"(p.y));
    return __ffma2_rn(make_float2(-x.x, -x.y), q, make_float2(fmaxf(a.x, 0.0f), fmaxf(a.y, 0.0f)));
}

// Accumulators of rows that are not kept may be anything: zeros in their place
// keep the arithmetic off its slow paths.
__device__ __forceinline__ void f4_zero_unless(bool valid, uint32_t (&r)[32]) {
#pragma unroll
    for (int i = 0; i < 32; i++) r[i] = valid ? r[i] : 0u;
}

// One lane's 32 output columns from gcol on, straight to its row: through
// shared memory and TMA (a box of 32 rows) the copy in and out took as much of
// shared memory's bandwidth as a fifth of a main loop's MMAs.  `wide`: rows are
// whole 32-byte sectors.
__device__ __forceinline__ void f4_store32(__nv_bfloat16 *row, const float (&v)[32], int gcol, int n_out, int wide) {
#pragma unroll
    for (int q = 0; q < 2; q++) {
        const int c = gcol + 16 * q;
        uint32_t p[8];
#pragma unroll
        for (int i = 0; i < 8; i++) p[i] = pack_bf16(v[16 * q + 2 * i], v[16 * q + 2 * i + 1]);
        if (wide) {
            if (c < n_out)
                asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(row + c), "r"(p[0]), "r"(p[1]),
                             "r"(p[2]), "r"(p[3]), "r"(p[4]), "r"(p[5]), "r"(p[6]), "r"(p[7])
                             : "memory");
        } else {
#pragma unroll
            for (int h = 0; h < 2; h++) {
                V16 w;
                w.w[0] = p[4 * h]; w.w[1] = p[4 * h + 1]; w.w[2] = p[4 * h + 2]; w.w[3] = p[4 * h + 3];
                if (c + 8 * h < n_out) st_v16(row + c + 8 * h, w);
            }
        }
    }
}

// One lane's 32 hidden values to codes and the bytes of their block scales (0
// unless `live`).
template <int FMT>
__device__ __forceinline__ void f4_quantise32(float (&v)[32], const Fp4Factor &g, bool live, uint32_t (&codes)[4],
                                              uint32_t &word) {
    constexpr int BLK = Fp4<FMT>::BLK;
#pragma unroll
    for (int b = 0; b < 32 / BLK; b++) {
        float m[4] = {0.0f, 0.0f, 0.0f, 0.0f}, inv;
#pragma unroll
        for (int i = 0; i < BLK; i++) m[i & 3] = amax_nan(m[i & 3], v[b * BLK + i]);
        const float amax = amax_nan(amax_nan(m[0], m[1]), amax_nan(m[2], m[3]));
        const uint32_t sc = fp4_scale<FMT>(fabsf(amax), g, inv);
        if (live) word |= sc << (8 * b);
#pragma unroll
        for (int i = 0; i < BLK; i += 2) {
            const float2 p = __fmul2_rn(make_float2(v[b * BLK + i], v[b * BLK + i + 1]), make_float2(inv, inv));
            v[b * BLK + i] = p.x;
            v[b * BLK + i + 1] = p.y;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; i++) codes[i] = e2m1x8(v + 8 * i);
}

template <int FMT, int EPI>
__global__ void __launch_bounds__(NUM_THREADS, 1)
fp4_group_gemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
               const __grid_constant__ CUtensorMap tmB3, const __grid_constant__ CUtensorMap tmSA,
               const __grid_constant__ CUtensorMap tmSB, const __grid_constant__ CUtensorMap tmSB3,
               const F4Args args) {
    using TL = F4Tiling<FMT>;
    constexpr bool SWIGLU = EPI == FP4_SWIGLU;
    constexpr int NOUT_TILE = SWIGLU ? BN / 2 : BN;
    constexpr int BLK = Fp4<FMT>::BLK, KT = TL::KT, STAGES = TL::STAGES;
    __shared__ int32_t s_bad;
    __shared__ int32_t kept_rows[MAX_E];
    __shared__ __align__(16) uint2 epi_bias[EPI_WARPS][32];   // 128 bf16 per epilogue warp
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *sA = smem, *sB = smem + STAGES * F4_OP_BYTES, *sSF = sB + STAGES * F4_OP_BYTES;
    Ctl<STAGES> *ctl = (Ctl<STAGES> *)(smem + STAGES * TL::STAGE_BYTES);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e = args.e;
    const uint32_t prank = cluster_rank();
    const int tile0 = (int)(blockIdx.x / 2), tile_step = (int)(gridDim.x / 2);
    const int ntn = (args.n_out + NOUT_TILE - 1) / NOUT_TILE;
    const int nk = (args.K + F4_BK - 1) / F4_BK;

    // what needs no result of the previous kernel: barriers, TMEM, descriptors
    if (warp == 0) {
        if (lane == 0) {
            ctl->abort = 0;
            for (int s = 0; s < STAGES; s++) { mbar_init(&ctl->full[s], F4_FULL_ARRIVALS); mbar_init(&ctl->empty[s], 1); }
            mbar_init(&ctl->tfull[0], 1);
            mbar_init(&ctl->tempty[0], 2 * EPI_WARPS);
            mbar_init(&ctl->drain, 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
    } else if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         su32(&ctl->tmem_base)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else if (warp == 2 && lane < 4) {
        const CUtensorMap *m = lane == 0 ? &tmA : lane == 1 ? &tmB : lane == 2 ? &tmSA : &tmSB;
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)m) : "memory");
    }
    pdl_enter();
    if (threadIdx.x == 0) s_bad = status_bad(args.status) ? 1 : 0;
    {
        const int c_eff = (int)min((int64_t)*args.c_dev, args.c_max);
        for (int j = threadIdx.x; j < e; j += NUM_THREADS) kept_rows[j] = max(0, min(args.counts[j], c_eff));
    }
    __syncthreads();
    if (warp == 0) {   // first tile of every expert: each lane sums a run of them
        const int per = (e + 31) / 32, j0 = min(lane * per, e), j1 = min(j0 + per, e);
        int own = 0;
        for (int j = j0; j < j1; j++) own += (kept_rows[j] + 2 * UM - 1) / (2 * UM) * ntn;
        int v = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        int at = v - own;
        for (int j = j0; j < j1; j++) {
            ctl->tile_start[j] = at;
            at += (kept_rows[j] + 2 * UM - 1) / (2 * UM) * ntn;
        }
        if (lane == 31) {
            ctl->tile_start[e] = v;
            ctl->total_tiles = v;
        }
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    int total = ctl->total_tiles;
    {
        int bad0, bad1;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(bad0) : "r"(map_to_rank(su32(&s_bad), 0)));
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(bad1) : "r"(map_to_rank(su32(&s_bad), 1)));
        if (bad0 | bad1) total = 0;   // the same decision in both CTAs
    }
    int32_t *abort_flag = &ctl->abort;

    if (warp == 0 || warp >= PROD_WARP0) {
        // Producers 0 and 2: the two row halves of this CTA's A rows; 1 and 3:
        // those of its B rows (SwiGLU: the first CTA's are W1's, the second's
        // W3's).  0 also brings the A scales, 1 and 3 the scales of the first
        // and second 128 columns of the tile.  A rows come in boxes of 32, and
        // only those that hold kept rows (the others' accumulators are never
        // stored).
        const int prod = warp == 0 ? 0 : warp - PROD_WARP0 + 1;
        const bool is_a = (prod & 1) == 0;
        const int hh = prod >> 1;
        const CUtensorMap *op = is_a ? &tmA : SWIGLU && prank ? &tmB3 : &tmB;
        const CUtensorMap *sf = is_a ? &tmSA : SWIGLU && hh ? &tmSB3 : &tmSB;
        const int a_tiles = (int)((args.c_max + 127) / 128), b_tiles = (args.n_out + 127) / 128;
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        if (elect_one()) {
            for (int t = tile0; t < total && !args.stall; t += tile_step) {
                const Tile T = decode_tile(ctl->tile_start, e, t, 2 * UM, kept_rows, 0, nk, F4_BK);
                // this CTA's boxes of A, and the bytes of both CTAs' copies
                const int left = T.rows - T.mt * 2 * UM - hh * 64;
                const int n0 = min(max((left + 31) / 32, 0), 2), n1 = min(max((left - UM + 31) / 32, 0), 2);
                const int boxes = prank ? n1 : n0;
                const bool sf_here = !is_a || (hh == 0 && boxes > 0);
                const uint32_t bytes = is_a ? (uint32_t)(n0 + n1) * (F4_BOX_BYTES / 2) +
                                                  (hh == 0 ? (uint32_t)((n0 > 0) + (n1 > 0)) * TL::SF_BYTES : 0u)
                                            : 2u * (F4_BOX_BYTES + TL::SF_BYTES);
                int row, sf_row;
                if (is_a) {
                    row = (int)(T.j * args.c_max + (int64_t)T.mt * 2 * UM) + (int)prank * UM + hh * 64;
                    sf_row = T.j * a_tiles + T.mt * 2 + (int)prank;
                } else {
                    row = T.j * args.n_out + T.nt * NOUT_TILE + (SWIGLU ? 0 : (int)prank * UM) + hh * 64;
                    sf_row = T.j * b_tiles + (SWIGLU ? T.nt : T.nt * 2 + hh);
                }
                uint8_t *dst = (is_a ? sA : sB) + hh * F4_BOX_BYTES;
                uint8_t *sf_dst = sSF + (is_a ? 0 : (1 + hh) * TL::SF_BYTES);
                for (int kb = 0; kb < nk; kb++) {
                    if (args.lag && is_a && prank) __nanosleep(20000);
                    if (!mbar_wait<true>(&ctl->empty[stage], phase ^ 1u, abort_flag, args.status)) goto producer_done;
                    const uint32_t fb = map_to_rank(su32(&ctl->full[stage]), 0);
                    if (prank == 0) mbar_expect_tx(&ctl->full[stage], bytes);
                    else if (is_a) mbar_arrive_cluster(fb);
                    uint8_t *to = dst + stage * F4_OP_BYTES;
                    if (!is_a || boxes > 0) tma_load_2d_pair(to, op, kb * (F4_BK / 2), row, fb);
                    if (is_a && boxes > 1) tma_load_2d_pair(to + F4_BOX_BYTES / 2, op, kb * (F4_BK / 2), row + 32, fb);
                    if (sf_here) tma_load_3d_pair(sf_dst + stage * 3 * TL::SF_BYTES, sf, 0, kb * KT, sf_row, fb);
                    issued++;
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
        producer_done:
            // bounded wait for this thread's copies in flight (the second CTA's are
            // covered by the MMAs that consume them, or by the delay after an abort)
            if (prank == 0) {
                for (int i = max(0, issued - STAGES); i < issued; i++) {
                    unsigned long long t0 = gtimer();
                    while (!mbar_try<true>(&ctl->full[i % STAGES], (uint32_t)((i / STAGES) & 1)) &&
                           gtimer() - t0 < WAIT_NS) {
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == 1 && elect_one()) {
        if (prank == 0) {
            int stage = 0;
            uint32_t phase = 0, sf_set = 0;
            int done = 0;   // tiles begun by this pair
            for (int t = tile0; t < total; t += tile_step, done++) {
                // the previous tile's epilogue has the columns that this tile shares with it
                if (done && !mbar_wait<true>(&ctl->tempty[0], (uint32_t)((done - 1) & 1), abort_flag, args.status))
                    break;
                tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(done & 1) * F4_ACC_STEP;
                bool ok = true;
                for (int kb = 0; kb < nk; kb++) {
                    if (!mbar_wait<true>(&ctl->full[stage], phase, abort_flag, args.status)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t a0 = su32(sA + stage * F4_OP_BYTES), b0 = su32(sB + stage * F4_OP_BYTES);
                    const uint32_t s0 = su32(sSF + stage * 3 * TL::SF_BYTES);
                    const uint32_t sfa = tmem + F4_SF_COL + sf_set * TL::SF_COLS, sfb = sfa + 4 * KT;
                    const int steps = min(F4_BK / 64, (args.K - kb * F4_BK + 63) / 64);
#pragma unroll
                    for (int x = 0; x < KT; x++) {
                        cp_scales_pair(sfa + 4 * x, s0 + x * 512);
                        cp_scales_pair(sfb + 8 * x, s0 + TL::SF_BYTES + x * 512);
                        cp_scales_pair(sfb + 8 * x + 4, s0 + 2 * TL::SF_BYTES + x * 512);
                    }
#pragma unroll
                    for (int kk = 0; kk < F4_BK / 64; kk++) {
                        if (kk < steps) {
                            const int x = FMT == MOE_FP4_MX ? kk / 2 : kk;   // its scale tile
                            umma_pair_f4<FMT>(d, sdesc<128>(a0 + kk * 32), sdesc<128>(b0 + kk * 32),
                                              f4_idesc<FMT>(FMT == MOE_FP4_MX ? (kk & 1) * 2 : 0), sfa + 4 * x,
                                              sfb + 8 * x, (kb | kk) != 0);
                        }
                    }
                    umma_commit_pair(&ctl->empty[stage], 3);
                    if (++sf_set == TL::SETS) sf_set = 0;
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
                if (!ok) break;
                umma_commit_pair(&ctl->tfull[0], 3);
            }
            umma_commit_pair(&ctl->drain, 3);
        }
        unsigned long long t0 = gtimer();
        while (!mbar_try<true>(&ctl->drain, 0) && gtimer() - t0 < WAIT_NS) {
        }
    } else if (warp >= 2 && warp < PROD_WARP0) {
        // Epilogue: warp (sub, half) has rows sub * 32 .. of this CTA and every other
        // chunk of 32 columns: half, half + 2, ...  The next tile overwrites the last
        // two chunks of an even tile and the first two of an odd one: each warp
        // begins with its own of them and then lets that tile's MMAs go ahead.
        const int ew = warp - 2, sub = warp & 3, half = ew >> 2;
        uint2 *bsl = epi_bias[ew];
        int done = 0;
        for (int t = tile0; t < total; t += tile_step, done++) {
            const Tile T = decode_tile(ctl->tile_start, e, t, 2 * UM, kept_rows, 0, nk, F4_BK);
            const int row = T.mt * 2 * UM + (int)prank * UM + sub * 32 + lane;
            const bool any = row - lane < T.rows;   // of the warp's rows
            const bool valid = row < T.rows, all_kept = row - lane + 31 < T.rows;
            const int64_t grow = (int64_t)T.j * args.c_max + row;
            const float ga = args.a_global ? args.a_global[T.j] : 1.0f;
            const float s1 = ga * (args.b_global ? args.b_global[T.j] : 1.0f);
            const float s3 = SWIGLU ? ga * (args.b3_global ? args.b3_global[T.j] : 1.0f) : 0.0f;
            const Fp4Factor og = fp4_factor(EPI != FP4_BIAS && args.out_global ? args.out_global[T.j] : 1.0f);
            if (!SWIGLU && args.bias) {
                // this warp's bias, four chunks of 32: chunk i at bsl + 8 i
                const int g = T.nt * NOUT_TILE + ((lane >> 3) * 2 + half) * 32 + (lane & 7) * 4;
                bsl[lane] = g < args.n_out ? *reinterpret_cast<const uint2 *>(args.bias + (int64_t)T.j * args.n_out + g)
                                           : make_uint2(0u, 0u);
            }
            __syncwarp();
            if (!warp_wait(&ctl->tfull[0], (uint32_t)(done & 1), abort_flag, args.status)) break;
            tc_fence_after();
            const uint32_t tb = tmem + ((uint32_t)(sub * 32) << 16) + (uint32_t)(done & 1) * F4_ACC_STEP;
            const int first = done & 1 ? half : 6 + half;   // the chunk to load first
            uint32_t r[32];
            if (any) {
                tmem_ld32(tb + 32 * first, r);
                tmem_wait_ld(r);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_to_rank(su32(&ctl->tempty[0]), 0));
            if (!any) continue;
            // 32 hidden values (columns gcol ..) of this lane's row to their place
            auto put_hidden = [&](float (&v)[32], int gcol) {
                const int64_t ont = fp4_scale_tiles(BLK, args.n_out);   // scale tiles of a row
                uint32_t codes[4], word = 0;
                const bool live = gcol < args.n_out;
                f4_quantise32<FMT>(v, og, live, codes, word);
                if (valid && live) {
                    V16 w;
                    w.w[0] = codes[0]; w.w[1] = codes[1]; w.w[2] = codes[2]; w.w[3] = codes[3];
                    st_v16(args.out_q + (grow * args.n_out + gcol) / 2, w);
                }
                if (valid && gcol < ont * 4 * BLK) {   // the last tile's blocks past the row: zeros
                    uint8_t *p = args.out_scale + T.j * fp4_scale_bytes(BLK, args.c_max, args.n_out) +
                                 fp4_scale_at(row, gcol / BLK, ont);
                    if (FMT == MOE_FP4_NV) *reinterpret_cast<uint16_t *>(p) = (uint16_t)word;
                    else *p = (uint8_t)word;
                }
            };
            if constexpr (SWIGLU) {
                // output chunk c pairs chunk c (a) with chunk c + 4 (b)
#pragma unroll 1
                for (int i = 0; i < 2; i++) {
                    const int c = (i == 0 ? first : first ^ 2) & 3;
                    uint32_t o[32];
                    if (i) {
                        tmem_ld32(tb + 32 * c, r);
                        tmem_ld32(tb + 32 * (c + 4), o);
                    } else {
                        tmem_ld32(tb + 32 * (first ^ 4), o);
                    }
                    tmem_wait_ld(o);
                    tmem_tie(r);
                    if (!all_kept) {
                        f4_zero_unless(valid, o);
                        f4_zero_unless(valid, r);
                    }
                    const bool r_is_b = i == 0 && first >= 4;   // what was loaded first
                    float v[32];
#pragma unroll
                    for (int x = 0; x < 32; x++) {
                        const float p = __uint_as_float(r[x]), q = __uint_as_float(o[x]);
                        v[x] = f4_silu((r_is_b ? q : p) * s1) * ((r_is_b ? p : q) * s3);
                    }
                    put_hidden(v, T.nt * NOUT_TILE + 32 * c);
                }
            } else {
#pragma unroll 1
                for (int i = 0; i < 4; i++) {
                    const int c = (first + 2 * i) & 7;
                    if (i) {
                        tmem_ld32(tb + 32 * c, r);
                        tmem_wait_ld(r);
                    }
                    if (EPI != FP4_BIAS && !all_kept) f4_zero_unless(valid, r);
                    const int gcol = T.nt * NOUT_TILE + 32 * c;
                    const uint4 *bp = reinterpret_cast<const uint4 *>(bsl + 8 * (c >> 1));
                    float v[32];
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        uint32_t bw[4] = {0u, 0u, 0u, 0u};   // eight columns' bias
                        if (args.bias) {
                            const uint4 u = bp[q];
                            bw[0] = u.x; bw[1] = u.y; bw[2] = u.z; bw[3] = u.w;
                        }
#pragma unroll
                        for (int y = 0; y < 4; y++) {
                            const int x = 8 * q + 2 * y;
                            float2 a = __ffma2_rn(make_float2(__uint_as_float(r[x]), __uint_as_float(r[x + 1])),
                                                  make_float2(s1, s1), make_float2(bf16lo(bw[y]), bf16hi(bw[y])));
                            if (EPI == FP4_GELU) a = f4_gelu2(a);
                            if (EPI == FP4_RELU) a = make_float2(f4_relu(a.x), f4_relu(a.y));
                            v[x] = a.x;
                            v[x + 1] = a.y;
                        }
                    }
                    if (EPI == FP4_BIAS) {
                        if (valid) f4_store32(args.out + grow * args.n_out, v, gcol, args.n_out, args.wide);
                    } else {
                        put_hidden(v, gcol);
                    }
                }
            }
            __syncwarp();   // the bias slice is rewritten for the next tile
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
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS)
                     : "memory");
    }
}

// Scale tiles of `batches` x `row_tiles` rows of `ntiles`: boxes of kt tiles.
bool make_map_scales(CUtensorMap *map, const void *base, int64_t row_tiles, int64_t ntiles, int kt) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {128, (cuuint64_t)ntiles, (cuuint64_t)row_tiles};
    cuuint64_t strides[2] = {512, (cuuint64_t)ntiles * 512};
    cuuint32_t box[3] = {128, (cuuint32_t)kt, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct F4Operand {
    const void *q, *scale;
    const float *global;
};

template <int FMT, int EPI>
moe_status launch_fp4(const F4Operand &a, const F4Operand &b, const F4Operand &b3, const F4Args &args_in,
                      cudaStream_t stream) {
    F4Args args = args_in;
    args.a_global = a.global;
    args.b_global = b.global;
    args.b3_global = b3.global;
    args.stall = take_gemm_stall() ? 1 : 0;
    args.lag = take_gemm_lag() ? 1 : 0;
    args.wide = args.n_out % 16 == 0 && ((uintptr_t)args.out & 31) == 0;
    const int64_t e = args.e;
    const int64_t nt = fp4_scale_tiles(Fp4<FMT>::BLK, args.K);
    const int64_t a_tiles = (args.c_max + 127) / 128, b_tiles = (args.n_out + 127) / 128;
    constexpr int KT = F4Tiling<FMT>::KT;
    CUtensorMap mA, mB, mSA, mSB;
    if (!make_map_u8(&mA, a.q, (uint64_t)(e * args.c_max), (uint64_t)args.K / 2, 32) ||
        !make_map_u8(&mB, b.q, (uint64_t)(e * args.n_out), (uint64_t)args.K / 2, 64) ||
        !make_map_scales(&mSA, a.scale, e * a_tiles, nt, KT) || !make_map_scales(&mSB, b.scale, e * b_tiles, nt, KT))
        return MOE_ERR_CUDA;
    CUtensorMap mB3 = mB, mSB3 = mSB;   // SwiGLU: its own
    if (EPI == FP4_SWIGLU && (!make_map_u8(&mB3, b3.q, (uint64_t)(e * args.n_out), (uint64_t)args.K / 2, 64) ||
                              !make_map_scales(&mSB3, b3.scale, e * b_tiles, nt, KT)))
        return MOE_ERR_CUDA;
    auto kern = fp4_group_gemm<FMT, EPI>;
    constexpr size_t SMEM = f4_smem_bytes<FMT>();
    static int units[64] = {0};   // resident clusters per device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
    int nunits = dev >= 0 && dev < 64 ? units[dev] : 0;
    if (!nunits) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM) != cudaSuccess)
            return MOE_ERR_CUDA;
        nunits = max_clusters(kern, SMEM, 2);
        if (dev >= 0 && dev < 64) units[dev] = nunits;
    }
    constexpr int NOUT_TILE = EPI == FP4_SWIGLU ? BN / 2 : BN;
    const int64_t upper = e * ((args.c_max + 2 * UM - 1) / (2 * UM)) * ((args.n_out + NOUT_TILE - 1) / NOUT_TILE);
    const int64_t grid = upper < nunits ? upper : nunits;
    return launch_cluster_pdl(kern, dim3((unsigned)(2 * grid)), dim3(NUM_THREADS), SMEM, 2, stream, mA, mB, mB3, mSA,
                              mSB, mSB3, args);
}

template <int FMT>
moe_status fp4_fc(int epi, const F4Operand &a, const F4Operand &b, const F4Operand &b3, const F4Args &args,
                  cudaStream_t stream) {
    switch (epi) {
        case FP4_BIAS: return launch_fp4<FMT, FP4_BIAS>(a, b, b3, args, stream);
        case FP4_RELU: return launch_fp4<FMT, FP4_RELU>(a, b, b3, args, stream);
        case FP4_GELU: return launch_fp4<FMT, FP4_GELU>(a, b, b3, args, stream);
        default: return launch_fp4<FMT, FP4_SWIGLU>(a, b, b3, args, stream);
    }
}

moe_status fp4_fc(moe_fp4 fmt, int epi, const F4Operand &a, const F4Operand &b, const F4Operand &b3,
                  const F4Args &args, cudaStream_t stream) {
    return fmt == MOE_FP4_MX ? fp4_fc<MOE_FP4_MX>(epi, a, b, b3, args, stream)
                             : fp4_fc<MOE_FP4_NV>(epi, a, b, b3, args, stream);
}

}  // namespace

moe_status product_fp4_launch(const void *a_q, const void *a_scale, const float *a_global,
                              const int32_t *counts, const int32_t *c_dev, const void *b_q,
                              const void *b_scale, const float *b_global, const void *bias,
                              moe_fp4 fmt, int e, int64_t c_max, int k, int n, void *out,
                              int32_t *st, cudaStream_t stream) {
    F4Args g{};
    g.counts = counts; g.c_dev = c_dev; g.status = st;
    g.bias = (const __nv_bfloat16 *)bias;
    g.out = (__nv_bfloat16 *)out;
    g.c_max = c_max; g.e = e; g.K = k; g.n_out = n;
    const F4Operand b{b_q, b_scale, b_global};
    return fp4_fc(fmt, FP4_BIAS, F4Operand{a_q, a_scale, a_global}, b, b, g, stream);
}

moe_status ffn_fp4_launch(const void *buf_q, const void *buf_scale, const float *buf_global,
                          const float *hid_global, const int32_t *counts, const int32_t *c_dev,
                          const void *w1_q, const void *w1_scale, const float *w1_global,
                          const void *b1, const void *w3_q, const void *w3_scale,
                          const float *w3_global, const void *w2_q, const void *w2_scale,
                          const float *w2_global, const void *b2, moe_fp4 fmt, moe_act act, int e,
                          int64_t c_max, int m, int h, void *hid_q, void *hid_scale, void *out,
                          int32_t *st, cudaStream_t stream) {
    const F4Operand w1{w1_q, w1_scale, w1_global};
    const F4Operand w3 = act == MOE_ACT_SWIGLU ? F4Operand{w3_q, w3_scale, w3_global} : w1;
    F4Args g{};
    g.counts = counts; g.c_dev = c_dev; g.status = st;
    g.bias = (const __nv_bfloat16 *)b1;
    g.out_q = (uint8_t *)hid_q;
    g.out_scale = (uint8_t *)hid_scale;
    g.out_global = hid_global;
    g.c_max = c_max; g.e = e; g.K = m; g.n_out = h;
    const int epi = act == MOE_ACT_SWIGLU ? FP4_SWIGLU : act == MOE_ACT_GELU ? FP4_GELU : FP4_RELU;
    moe_status r = fp4_fc(fmt, epi, F4Operand{buf_q, buf_scale, buf_global}, w1, w3, g, stream);
    if (r != MOE_OK) return r;
    return product_fp4_launch(hid_q, hid_scale, hid_global, counts, c_dev, w2_q, w2_scale, w2_global, b2, fmt, e,
                              c_max, h, m, out, st, stream);
}

}  // namespace moe
