// C ABI entry points: synchronous argument checks, then kernel launches.
#include <atomic>

#include "common.cuh"
#include "fp4.cuh"

namespace moe {

static std::atomic<uint64_t> g_launches{0};
void note_launch() { g_launches.fetch_add(1, std::memory_order_relaxed); }

static std::atomic<int32_t> g_gemm_stalls{0}, g_gemm_lags{0};
static bool take_one(std::atomic<int32_t> &pending) {
    int32_t n = pending.load(std::memory_order_relaxed);
    while (n > 0 && !pending.compare_exchange_weak(n, n - 1, std::memory_order_relaxed)) {
    }
    return n > 0;
}
bool take_gemm_stall() { return take_one(g_gemm_stalls); }
bool take_gemm_lag() { return take_one(g_gemm_lags); }

// kernels (one translation unit each)
moe_status gate_topk_launch(const void *x, moe_dtype xdt, const float *wg, const float *bias,
                            int64_t s, int m, int e, int k, unsigned flags, int32_t *idx,
                            float *gates, int32_t *st, cudaStream_t stream);
moe_status gate_bwd_launch(const void *x, moe_dtype xdt, const float *wg, const float *bias,
                           int64_t s, int m, int e, int k, unsigned flags, const int32_t *idx,
                           const float *gates, const float *d_gates, float *d_logits, float *d_wg,
                           float *d_bias, float *d_x, int32_t *st, cudaStream_t stream);
int64_t capacity_bound_host(float f, int64_t s, int e, int k);
size_t capacity_workspace_bytes(int64_t s, int e, int k);
moe_status capacity_launch(const int32_t *idx, int64_t s, int e, int k, float f, int64_t c_max,
                           void *ws, int32_t *loc, int32_t *counts, int32_t *c_dev, int32_t *st,
                           cudaStream_t stream);
moe_status encode_launch(const void *x, moe_dtype dt, const int32_t *idx, const int32_t *loc,
                         const int32_t *counts, const int32_t *c_dev, int64_t s, int m, int e,
                         int k, int64_t c_max, unsigned flags, void *buf, int32_t *st,
                         cudaStream_t stream, int lo, int hi);
moe_status combine_launch(const void *src, moe_dtype dt, const int32_t *idx, const int32_t *loc,
                          const float *gates, const int32_t *c_dev, int64_t s, int m, int e, int k,
                          int64_t c_max, void *y, int32_t *st, cudaStream_t stream);
moe_status decode_bwd_launch(const void *dy, const void *out, moe_dtype dt, const int32_t *idx,
                             const int32_t *loc, const float *gates, const int32_t *counts,
                             const int32_t *c_dev, int64_t s, int m, int e, int k, int64_t c_max,
                             unsigned flags, void *d_out, float *d_gates, int32_t *st,
                             cudaStream_t stream);
moe_status capacity_noalloc_launch(const int32_t *idx, int64_t s, int e, int k, float f,
                                   int64_t c_max, int32_t *loc, int32_t *counts, int32_t *c_dev,
                                   int32_t *st, cudaStream_t stream);
moe_status probe_fp32_fma_launch(int packed, int blocks, int iters, float *out,
                                 cudaStream_t stream);
bool ffn_tc_supported(int e, int64_t c_max, int m, int h);
moe_status ffn_tc_launch(const void *buf, const int32_t *counts, const int32_t *c_dev,
                         const void *w1, const void *b1, const void *w3, const void *w2,
                         const void *b2, moe_act act, int e, int64_t c_max, int m, int h,
                         void *hid, void *out, int32_t *st, cudaStream_t stream, int row_lo,
                         int row_hi, void *pre = nullptr, SortedRows so = {});
size_t ffn_tc_bwd_workspace_bytes(moe_act act, int e, int64_t c_max, int m, int h);
moe_status quantize_rows_fp8_launch(const void *src, int64_t batches, int64_t rows_per_batch,
                                    int cols, const int32_t *counts, const int32_t *c_dev,
                                    void *q, float *scale, int32_t *st, cudaStream_t stream);
moe_status ffn_tc_fp8_launch(const void *buf_q, const float *buf_scale, const int32_t *counts,
                             const int32_t *c_dev, const void *w1_q, const float *w1_scale,
                             const void *b1, const void *w2_q, const float *w2_scale,
                             const void *b2, moe_act act, int e, int64_t c_max, int m, int h,
                             void *hid, void *hid_q, float *hid_scale, void *out, int32_t *st,
                             cudaStream_t stream);
moe_status route_topk_launch(const void *logits, moe_dtype ldt, const float *bias, int64_t s, int e,
                             int k, moe_score score, int groups, int topk_groups, int group_top,
                             float scale, unsigned flags, int32_t *idx, float *gates, int32_t *st,
                             cudaStream_t stream);
moe_status route_bwd_launch(const void *logits, moe_dtype ldt, const int32_t *idx,
                            const float *d_gates, int64_t s, int e, int k, moe_score score,
                            float scale, unsigned flags, void *d_logits, moe_dtype ddt, int32_t *st,
                            cudaStream_t stream);
moe_status quantize_fp4_launch(const void *src, moe_dtype sdt, int64_t batches, int64_t rpb, int cols,
                               moe_fp4 fmt, const float *global, const int32_t *counts,
                               const int32_t *c_dev, void *q, void *scale, int32_t *st,
                               cudaStream_t stream);
moe_status dequantize_fp4_launch(const void *q, const void *scale, int64_t batches, int64_t rpb,
                                 int cols, moe_fp4 fmt, const float *global, const int32_t *counts,
                                 const int32_t *c_dev, void *dst, moe_dtype ddt, int32_t *st,
                                 cudaStream_t stream);
moe_status product_fp4_launch(const void *a_q, const void *a_scale, const float *a_global,
                              const int32_t *counts, const int32_t *c_dev, const void *b_q,
                              const void *b_scale, const float *b_global, const void *bias,
                              moe_fp4 fmt, int e, int64_t c_max, int k, int n, void *out,
                              int32_t *st, cudaStream_t stream);
moe_status ffn_fp4_launch(const void *buf_q, const void *buf_scale, const float *buf_global,
                          const float *hid_global, const int32_t *counts, const int32_t *c_dev,
                          const void *w1_q, const void *w1_scale, const float *w1_global,
                          const void *b1, const void *w3_q, const void *w3_scale,
                          const float *w3_global, const void *w2_q, const void *w2_scale,
                          const float *w2_global, const void *b2, moe_fp4 fmt, moe_act act, int e,
                          int64_t c_max, int m, int h, void *hid_q, void *hid_scale, void *out,
                          int32_t *st, cudaStream_t stream);
moe_status ffn_tc_bwd_launch(const void *buf, const void *hid, const int32_t *counts,
                             const int32_t *c_dev, const void *w1, const void *b1, const void *w3,
                             const void *w2, moe_act act, int e, int64_t c_max, int m, int h,
                             const void *d_out, void *ws, void *d_buf, void *d_w1, void *d_w3,
                             void *d_w2, void *d_b1, void *d_b2, int32_t *st, cudaStream_t stream,
                             const void *pre = nullptr, bool wgrad_f32 = false,
                             SortedRows so = {});
size_t ffn_tc_sorted_bwd_workspace_bytes(moe_act act, int e, int64_t n, int m, int h);
moe_status quantize_rows_int8_launch(const void *src, moe_dtype sdt, const int32_t *rows, int64_t s, int cols, int k,
                                     int64_t n, void *q, float *scale, int32_t *st, cudaStream_t stream);
size_t product_int8_workspace_bytes(int e, int64_t n, int k);
moe_status product_int8_launch(const void *a_q, const float *a_scale, const SortedRows &so, const void *b_q,
                               const float *b_scale, const void *bias, int e, int k, int n_out, void *ws, void *out,
                               bool f32, int32_t *st, cudaStream_t stream);
size_t ffn_int8_workspace_bytes(int e, int64_t n, int m, int h);
moe_status ffn_int8_launch(const void *x_q, const float *x_scale, const SortedRows &so, const void *w1_q,
                           const float *w1_scale, const void *b1, const void *w3_q, const float *w3_scale,
                           const void *w2_q, const float *w2_scale, const void *b2, moe_act act, int e, int m, int h,
                           void *ws, void *out, int32_t *st, cudaStream_t stream);
bool few_rows(int64_t n, int e);
moe_status ffn_few_launch(const void *x, const SortedRows &so, const void *w1, const void *b1, const void *w3,
                          const void *w2, const void *b2, moe_act act, int e, int m, int h, void *hid, void *pre,
                          void *out, int32_t *st, cudaStream_t stream);
size_t sort_workspace_bytes(int64_t s, int e, int k);
moe_status sort_routes_launch(const int32_t *idx, int64_t s, int e, int k, int32_t *rows, int32_t *offsets,
                              int32_t *source, void *ws, int32_t *st, cudaStream_t stream);
moe_status encode_sorted_launch(const void *x, moe_dtype dt, const int32_t *rows, const float *gates, int64_t s, int m,
                                int k, int64_t n, void *out, int32_t *st, cudaStream_t stream);
moe_status decode_sorted_launch(const void *xs, moe_dtype dt, const int32_t *rows, const float *gates, int64_t s,
                                int m, int k, int64_t n, void *y, int32_t *st, cudaStream_t stream);
moe_status decode_sorted_bwd_launch(const void *dy, const void *xs, moe_dtype dt, const int32_t *rows,
                                    const float *gates, int64_t s, int m, int k, int64_t n, void *d_xs,
                                    float *d_gates, int32_t *st, cudaStream_t stream);
moe_status encode_sorted_bwd_launch(const void *d_out, const void *x, moe_dtype dt, const int32_t *rows,
                                    const float *gates, int64_t s, int m, int k, int64_t n, void *d_x,
                                    float *d_gates, int32_t *st, cudaStream_t stream);
moe_status ffn_simt_launch(const void *buf, moe_dtype dt, const int32_t *counts,
                           const int32_t *c_dev, const void *w1, const void *b1, const void *w3,
                           const void *w2, const void *b2, moe_act act, int e, int64_t c_max,
                           int m, int h, void *hid, void *out, int32_t *st, cudaStream_t stream);

}  // namespace moe

using namespace moe;

namespace {

constexpr int kMaxE = 1024;
constexpr int kMaxK = 32;

inline bool ok16(const void *p) { return p != nullptr && aligned16(p); }
inline bool ok4(const void *p) { return p != nullptr && ((uintptr_t)p & 3u) == 0; }
inline bool opt16(const void *p) { return p == nullptr || aligned16(p); }
inline bool valid_dt(moe_dtype dt) { return dt == MOE_F32 || dt == MOE_BF16; }
inline int vec_of(moe_dtype dt) { return dt == MOE_BF16 ? 8 : 4; }
inline size_t esize(moe_dtype dt) { return dt == MOE_BF16 ? 2 : 4; }
inline size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

bool routing_shape_ok(int64_t s, int e, int k) {
    return s >= 1 && s <= (int64_t)1 << 30 && e >= 1 && e <= kMaxE && k >= 1 && k <= e &&
           k <= kMaxK && s * (int64_t)k < ((int64_t)1 << 31);
}

bool rows_ok(moe_dtype dt, int m) { return valid_dt(dt) && m >= 1 && m % vec_of(dt) == 0; }

cudaStream_t as_stream(void *s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace

extern "C" {

const char *moe_status_str(moe_status st) {
    switch (st) {
        case MOE_OK: return "ok";
        case MOE_ERR_INVALID_ARG: return "invalid argument";
        case MOE_ERR_UNSUPPORTED: return "unsupported combination";
        case MOE_ERR_CUDA: return "CUDA error";
        case MOE_ERR_CAPACITY: return "capacity exceeds c_max";
        case MOE_ERR_TIMEOUT: return "bounded wait timed out";
    }
    return "unknown status";
}

uint64_t moe_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

moe_status moe_debug_stall_gemms(int32_t n) {
    if (n < 0) return MOE_ERR_INVALID_ARG;
    g_gemm_stalls.store(n, std::memory_order_relaxed);
    return MOE_OK;
}

moe_status moe_debug_lag_gemms(int32_t n) {
    if (n < 0) return MOE_ERR_INVALID_ARG;
    g_gemm_lags.store(n, std::memory_order_relaxed);
    return MOE_OK;
}

moe_status moe_gate_topk(const void *x, moe_dtype xdt, const float *wg, const float *bias,
                         int64_t s, int m, int e, int k, unsigned flags, int32_t *idx,
                         float *gates, int32_t *dev_status, void *stream) {
    if (!routing_shape_ok(s, e, k) || !rows_ok(xdt, m) || !ok16(x) || !ok16(wg) || !opt16(bias) ||
        !ok4(idx) || !ok4(gates) || !ok4(dev_status) || (flags & ~3u))
        return MOE_ERR_INVALID_ARG;
    if (e > 256) return MOE_ERR_UNSUPPORTED;
    return gate_topk_launch(x, xdt, wg, bias, s, m, e, k, flags, idx, gates, dev_status,
                            as_stream(stream));
}

moe_status moe_gate_bwd(const void *x, moe_dtype xdt, const float *wg, const float *bias,
                        int64_t s, int m, int e, int k, unsigned flags, const int32_t *idx,
                        const float *gates, const float *d_gates, float *d_logits, float *d_wg,
                        float *d_bias, float *d_x, int32_t *dev_status, void *stream) {
    if (!routing_shape_ok(s, e, k) || !rows_ok(xdt, m) || !ok16(x) || !ok16(wg) ||
        !opt16(bias) || !ok4(idx) || !ok4(gates) || !ok4(d_gates) || !ok4(d_logits) ||
        !opt16(d_wg) || !opt16(d_bias) || !opt16(d_x) || !ok4(dev_status) || (flags & ~3u))
        return MOE_ERR_INVALID_ARG;
    if (e > 256) return MOE_ERR_UNSUPPORTED;
    return gate_bwd_launch(x, xdt, wg, bias, s, m, e, k, flags, idx, gates, d_gates, d_logits,
                           d_wg, d_bias, d_x, dev_status, as_stream(stream));
}

int64_t moe_capacity_bound(float capacity_factor, int64_t s, int e, int k) {
    if (!routing_shape_ok(s, e, k) || capacity_factor != capacity_factor) return -1;
    return capacity_bound_host(capacity_factor, s, e, k);
}

size_t moe_capacity_workspace_size(int64_t s, int e, int k) {
    if (!routing_shape_ok(s, e, k)) return 0;
    return capacity_workspace_bytes(s, e, k);
}

moe_status moe_capacity_locations(const int32_t *idx, int64_t s, int e, int k,
                                  float capacity_factor, int64_t c_max, void *workspace,
                                  size_t workspace_bytes, int32_t *loc, int32_t *counts,
                                  int32_t *c_dev, int32_t *dev_status, void *stream) {
    if (!routing_shape_ok(s, e, k) || c_max < 1 || c_max > 0x7fffffff ||
        capacity_factor != capacity_factor || !ok4(idx) || !ok4(loc) || !ok4(counts) ||
        !ok4(c_dev) || !ok4(dev_status) || !ok16(workspace) ||
        workspace_bytes < capacity_workspace_bytes(s, e, k))
        return MOE_ERR_INVALID_ARG;
    return capacity_launch(idx, s, e, k, capacity_factor, c_max, workspace, loc, counts, c_dev,
                           dev_status, as_stream(stream));
}

moe_status moe_capacity_locations_noalloc(const int32_t *idx, int64_t s, int e, int k,
                                          float capacity_factor, int64_t c_max, int32_t *loc,
                                          int32_t *counts, int32_t *c_dev, int32_t *dev_status,
                                          void *stream) {
    if (!routing_shape_ok(s, e, k) || c_max < 1 || c_max > 0x7fffffff ||
        capacity_factor != capacity_factor || !ok4(idx) || !ok4(loc) || !ok4(counts) ||
        !ok4(c_dev) || !ok4(dev_status))
        return MOE_ERR_INVALID_ARG;
    return capacity_noalloc_launch(idx, s, e, k, capacity_factor, c_max, loc, counts, c_dev,
                                   dev_status, as_stream(stream));
}

moe_status moe_encode(const void *x, moe_dtype dt, const int32_t *idx, const int32_t *loc,
                      const int32_t *counts, const int32_t *c_dev, int64_t s, int m, int e, int k,
                      int64_t c_max, unsigned flags, void *buf, int32_t *dev_status,
                      void *stream) {
    if (!routing_shape_ok(s, e, k) || !rows_ok(dt, m) || c_max < 1 || c_max > 0x7fffffff ||
        !ok16(x) || !ok4(idx) || !ok4(loc) || !ok4(c_dev) || !ok16(buf) || !ok4(dev_status) ||
        (flags & ~3u) || ((flags & MOE_FLAG_ZERO_FILL) && !ok4(counts)))
        return MOE_ERR_INVALID_ARG;
    return encode_launch(x, dt, idx, loc, counts, c_dev, s, m, e, k, c_max, flags, buf, dev_status,
                         as_stream(stream), 0, 0x7fffffff);
}

size_t moe_expert_ffn_workspace_size(moe_dtype dt, moe_act act, int e, int64_t c_max, int m,
                                     int h) {
    (void)act;
    (void)m;
    if (!valid_dt(dt) || e < 1 || c_max < 1 || h < 1) return 0;
    return up256((size_t)e * (size_t)c_max * (size_t)h * esize(dt));
}

static moe_status expert_ffn(const void *buf, moe_dtype dt, const int32_t *counts,
                             const int32_t *c_dev, const void *w1, const void *b1, const void *w3,
                             const void *w2, const void *b2, moe_act act, int e, int64_t c_max,
                             int m, int h, void *workspace, size_t workspace_bytes, void *out,
                             void *pre, int32_t *dev_status, void *stream) {
    if (!rows_ok(dt, m) || !rows_ok(dt, h) || e < 1 || e > kMaxE || c_max < 1 ||
        c_max > 0x7fffffff || !ok16(buf) || !ok4(counts) || !ok4(c_dev) || !ok16(w1) ||
        !ok16(w2) || !opt16(b1) || !opt16(b2) || !ok16(out) || !ok4(dev_status) ||
        !ok16(workspace) ||
        workspace_bytes < moe_expert_ffn_workspace_size(dt, act, e, c_max, m, h))
        return MOE_ERR_INVALID_ARG;
    if (act != MOE_ACT_RELU && act != MOE_ACT_GELU && act != MOE_ACT_SWIGLU)
        return MOE_ERR_INVALID_ARG;
    if (act == MOE_ACT_SWIGLU && (!ok16(w3) || b1 != nullptr || b2 != nullptr))
        return MOE_ERR_INVALID_ARG;
    if (pre && dt != MOE_BF16) return MOE_ERR_UNSUPPORTED;
    if (pre && !ok16(pre)) return MOE_ERR_INVALID_ARG;
    if (dt == MOE_BF16) {
        if (!ffn_tc_supported(e, c_max, m, h)) return MOE_ERR_UNSUPPORTED;
        return ffn_tc_launch(buf, counts, c_dev, w1, b1, w3, w2, b2, act, e, c_max, m, h,
                             workspace, out, dev_status, as_stream(stream), 0, 0, pre);
    }
    return ffn_simt_launch(buf, dt, counts, c_dev, w1, b1, w3, w2, b2, act, e, c_max, m, h,
                           workspace, out, dev_status, as_stream(stream));
}

moe_status moe_expert_ffn(const void *buf, moe_dtype dt, const int32_t *counts,
                          const int32_t *c_dev, const void *w1, const void *b1, const void *w3,
                          const void *w2, const void *b2, moe_act act, int e, int64_t c_max, int m,
                          int h, void *workspace, size_t workspace_bytes, void *out,
                          int32_t *dev_status, void *stream) {
    return expert_ffn(buf, dt, counts, c_dev, w1, b1, w3, w2, b2, act, e, c_max, m, h, workspace,
                      workspace_bytes, out, nullptr, dev_status, stream);
}

moe_status moe_expert_ffn_train(const void *buf, moe_dtype dt, const int32_t *counts,
                                const int32_t *c_dev, const void *w1, const void *b1,
                                const void *w3, const void *w2, const void *b2, moe_act act, int e,
                                int64_t c_max, int m, int h, void *workspace,
                                size_t workspace_bytes, void *out, void *pre, int32_t *dev_status,
                                void *stream) {
    if (!pre) return MOE_ERR_INVALID_ARG;
    return expert_ffn(buf, dt, counts, c_dev, w1, b1, w3, w2, b2, act, e, c_max, m, h, workspace,
                      workspace_bytes, out, pre, dev_status, stream);
}

moe_status moe_decode(const void *out, moe_dtype dt, const int32_t *idx, const int32_t *loc,
                      const float *gates, const int32_t *c_dev, int64_t s, int m, int e, int k,
                      int64_t c_max, void *y, int32_t *dev_status, void *stream) {
    if (!routing_shape_ok(s, e, k) || !rows_ok(dt, m) || c_max < 1 || c_max > 0x7fffffff ||
        !ok16(out) || !ok4(idx) || !ok4(loc) || !ok4(gates) || !ok4(c_dev) || !ok16(y) ||
        !ok4(dev_status))
        return MOE_ERR_INVALID_ARG;
    return combine_launch(out, dt, idx, loc, gates, c_dev, s, m, e, k, c_max, y, dev_status,
                          as_stream(stream));
}

moe_status moe_decode_bwd(const void *dy, const void *out, moe_dtype dt, const int32_t *idx,
                          const int32_t *loc, const float *gates, const int32_t *counts,
                          const int32_t *c_dev, int64_t s, int m, int e, int k, int64_t c_max,
                          unsigned flags, void *d_out, float *d_gates, int32_t *dev_status,
                          void *stream) {
    if (!routing_shape_ok(s, e, k) || !rows_ok(dt, m) || c_max < 1 || c_max > 0x7fffffff ||
        !ok16(dy) || !ok16(out) || !ok4(idx) || !ok4(loc) || !ok4(gates) || !ok4(c_dev) ||
        !ok16(d_out) || !ok4(d_gates) || !ok4(dev_status) || (flags & ~3u) ||
        ((flags & MOE_FLAG_ZERO_FILL) && !ok4(counts)))
        return MOE_ERR_INVALID_ARG;
    return decode_bwd_launch(dy, out, dt, idx, loc, gates, counts, c_dev, s, m, e, k, c_max, flags,
                             d_out, d_gates, dev_status, as_stream(stream));
}

moe_status moe_encode_bwd(const void *d_buf, moe_dtype dt, const int32_t *idx, const int32_t *loc,
                          const int32_t *c_dev, int64_t s, int m, int e, int k, int64_t c_max,
                          void *dx, int32_t *dev_status, void *stream) {
    if (!routing_shape_ok(s, e, k) || !rows_ok(dt, m) || c_max < 1 || c_max > 0x7fffffff ||
        !ok16(d_buf) || !ok4(idx) || !ok4(loc) || !ok4(c_dev) || !ok16(dx) || !ok4(dev_status))
        return MOE_ERR_INVALID_ARG;
    return combine_launch(d_buf, dt, idx, loc, nullptr, c_dev, s, m, e, k, c_max, dx, dev_status,
                          as_stream(stream));
}

size_t moe_expert_ffn_bwd_workspace_size(moe_dtype dt, moe_act act, int e, int64_t c_max, int m,
                                         int h) {
    if (dt != MOE_BF16 || e < 1 || e > kMaxE || c_max < 1 || m < 1 || h < 1) return 0;
    if (act != MOE_ACT_RELU && act != MOE_ACT_GELU && act != MOE_ACT_SWIGLU) return 0;
    return ffn_tc_bwd_workspace_bytes(act, e, c_max, m, h);
}

static moe_status expert_ffn_bwd(const void *buf, const void *hid, const void *pre, moe_dtype dt,
                                 const int32_t *counts, const int32_t *c_dev, const void *w1,
                                 const void *b1, const void *w3, const void *w2, moe_act act, int e,
                                 int64_t c_max, int m, int h, const void *d_out, void *workspace,
                                 size_t workspace_bytes, void *d_buf, moe_dtype wgrad_dt,
                                 void *d_w1, void *d_w3, void *d_w2, void *d_b1, void *d_b2,
                                 int32_t *dev_status, void *stream) {
    if (wgrad_dt != MOE_BF16 && wgrad_dt != MOE_F32) return MOE_ERR_INVALID_ARG;
    if (!rows_ok(dt, m) || !rows_ok(dt, h) || e < 1 || e > kMaxE || c_max < 1 ||
        c_max > 0x7fffffff || !ok16(buf) || !ok16(hid) || !ok4(counts) || !ok4(c_dev) ||
        !ok16(w1) || !ok16(w2) || !opt16(b1) || !ok16(d_out) || !ok16(workspace) ||
        !ok16(d_buf) || !ok16(d_w1) || !ok16(d_w2) || !opt16(d_b1) || !opt16(d_b2) ||
        !ok4(dev_status))
        return MOE_ERR_INVALID_ARG;
    if (act != MOE_ACT_RELU && act != MOE_ACT_GELU && act != MOE_ACT_SWIGLU)
        return MOE_ERR_INVALID_ARG;
    if (act == MOE_ACT_SWIGLU &&
        (!ok16(w3) || !ok16(d_w3) || b1 != nullptr || d_b1 != nullptr || d_b2 != nullptr))
        return MOE_ERR_INVALID_ARG;
    if (dt != MOE_BF16) return MOE_ERR_UNSUPPORTED;
    if (workspace_bytes < moe_expert_ffn_bwd_workspace_size(dt, act, e, c_max, m, h))
        return MOE_ERR_INVALID_ARG;
    const int64_t h2 = act == MOE_ACT_SWIGLU ? 2 * (int64_t)h : h;
    // every operand of the products within the grouped GEMM's index range
    if (!ffn_tc_supported(e, c_max, m, h) || !ffn_tc_supported(e, h2, m, h) ||
        (int64_t)e * h2 >= ((int64_t)1 << 31) || (int64_t)e * ((c_max + 7) / 8 * 8) >= ((int64_t)1 << 31))
        return MOE_ERR_UNSUPPORTED;
    if (pre && !ok16(pre)) return MOE_ERR_INVALID_ARG;
    return ffn_tc_bwd_launch(buf, hid, counts, c_dev, w1, b1, w3, w2, act, e, c_max, m, h, d_out,
                             workspace, d_buf, d_w1, d_w3, d_w2, d_b1, d_b2, dev_status,
                             as_stream(stream), pre, wgrad_dt == MOE_F32);
}

moe_status moe_expert_ffn_bwd(const void *buf, const void *hid, moe_dtype dt,
                              const int32_t *counts, const int32_t *c_dev, const void *w1,
                              const void *b1, const void *w3, const void *w2, moe_act act, int e,
                              int64_t c_max, int m, int h, const void *d_out, void *workspace,
                              size_t workspace_bytes, void *d_buf, void *d_w1, void *d_w3,
                              void *d_w2, void *d_b1, void *d_b2, int32_t *dev_status,
                              void *stream) {
    return expert_ffn_bwd(buf, hid, nullptr, dt, counts, c_dev, w1, b1, w3, w2, act, e, c_max, m, h,
                          d_out, workspace, workspace_bytes, d_buf, dt, d_w1, d_w3, d_w2, d_b1, d_b2,
                          dev_status, stream);
}

moe_status moe_expert_ffn_bwd_saved(const void *buf, const void *hid, const void *pre,
                                    moe_dtype dt, const int32_t *counts, const int32_t *c_dev,
                                    const void *w1, const void *w3, const void *w2, moe_act act,
                                    int e, int64_t c_max, int m, int h, const void *d_out,
                                    void *workspace, size_t workspace_bytes, void *d_buf,
                                    moe_dtype wgrad_dt, void *d_w1, void *d_w3, void *d_w2,
                                    void *d_b1, void *d_b2, int32_t *dev_status, void *stream) {
    if (!pre) return MOE_ERR_INVALID_ARG;
    return expert_ffn_bwd(buf, hid, pre, dt, counts, c_dev, w1, nullptr, w3, w2, act, e, c_max, m, h,
                          d_out, workspace, workspace_bytes, d_buf, wgrad_dt, d_w1, d_w3, d_w2, d_b1,
                          d_b2, dev_status, stream);
}

// ------------------------------------------------- rows sorted by expert
namespace {

constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1024;

bool sort_shape_ok(int64_t s, int e, int k) {
    return s >= 1 && e >= 1 && e <= kMaxE && k >= 1 && k <= kMaxK && s <= kMaxRows / k;
}

bool move_ok(const void *read, const void *written, moe_dtype dt, const int32_t *rows, int64_t s, int m,
             int k, int64_t n, const int32_t *dev_status) {
    return s >= 1 && k >= 1 && k <= kMaxK && s <= kMaxRows / k && rows_ok(dt, m) && n >= 1 && n <= kMaxRows &&
           ok16(read) && ok16(written) && ok4(rows) && ok4(dev_status);
}

bool act_ok(moe_act act) { return act == MOE_ACT_RELU || act == MOE_ACT_GELU || act == MOE_ACT_SWIGLU; }

bool sorted_ffn_shape_ok(moe_act act, int e, int64_t n, int m, int h) {
    return act_ok(act) && e >= 1 && e <= kMaxE && n >= 1 && m >= 1 && m % 8 == 0 && h >= 1 && h % 8 == 0;
}

// within the grouped products' index range
bool sorted_ffn_supported(moe_act act, int e, int64_t n, int m, int h) {
    const int64_t lim = (int64_t)1 << 31, h2 = act == MOE_ACT_SWIGLU ? 2 * (int64_t)h : h;
    return n <= kMaxRows && (int64_t)e * h2 < lim && (int64_t)e * m < lim && h2 < lim;
}

}  // namespace

size_t moe_sort_workspace_size(int64_t s, int e, int k) {
    return sort_shape_ok(s, e, k) ? sort_workspace_bytes(s, e, k) : 0;
}

moe_status moe_sort_routes(const int32_t *idx, int64_t s, int e, int k, int32_t *rows, int32_t *offsets,
                           int32_t *source, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                           void *stream) {
    if (!sort_shape_ok(s, e, k) || !ok4(idx) || !ok4(rows) || !ok4(offsets) || (source && !ok4(source)) ||
        !ok16(workspace) || workspace_bytes < sort_workspace_bytes(s, e, k) || !ok4(dev_status))
        return MOE_ERR_INVALID_ARG;
    return sort_routes_launch(idx, s, e, k, rows, offsets, source, workspace, dev_status, as_stream(stream));
}

moe_status moe_encode_sorted(const void *x, moe_dtype dt, const int32_t *rows, const float *gates, int64_t s, int m,
                             int k, int64_t n, void *out, int32_t *dev_status, void *stream) {
    if (!move_ok(x, out, dt, rows, s, m, k, n, dev_status) || (gates && !ok4(gates))) return MOE_ERR_INVALID_ARG;
    return encode_sorted_launch(x, dt, rows, gates, s, m, k, n, out, dev_status, as_stream(stream));
}

moe_status moe_encode_sorted_bwd(const void *d_out, const void *x, moe_dtype dt, const int32_t *rows,
                                 const float *gates, int64_t s, int m, int k, int64_t n, void *d_x, float *d_gates,
                                 int32_t *dev_status, void *stream) {
    if (!move_ok(d_out, d_x, dt, rows, s, m, k, n, dev_status) || (gates && !ok4(gates)) || (d_gates && !ok4(d_gates)) ||
        (d_gates && (!gates || !ok16(x))))
        return MOE_ERR_INVALID_ARG;
    return encode_sorted_bwd_launch(d_out, x, dt, rows, gates, s, m, k, n, d_x, d_gates, dev_status,
                                    as_stream(stream));
}

moe_status moe_decode_sorted(const void *xs, moe_dtype dt, const int32_t *rows, const float *gates, int64_t s, int m,
                             int k, int64_t n, void *y, int32_t *dev_status, void *stream) {
    if (!move_ok(xs, y, dt, rows, s, m, k, n, dev_status) || (gates && !ok4(gates))) return MOE_ERR_INVALID_ARG;
    return decode_sorted_launch(xs, dt, rows, gates, s, m, k, n, y, dev_status, as_stream(stream));
}

moe_status moe_decode_sorted_bwd(const void *dy, const void *xs, moe_dtype dt, const int32_t *rows,
                                 const float *gates, int64_t s, int m, int k, int64_t n, void *d_xs, float *d_gates,
                                 int32_t *dev_status, void *stream) {
    if (!move_ok(dy, d_xs, dt, rows, s, m, k, n, dev_status) || !ok16(xs) || !ok4(gates) || !ok4(d_gates))
        return MOE_ERR_INVALID_ARG;
    return decode_sorted_bwd_launch(dy, xs, dt, rows, gates, s, m, k, n, d_xs, d_gates, dev_status,
                                    as_stream(stream));
}

moe_status moe_expert_ffn_sorted(const void *x, moe_dtype dt, const int32_t *offsets, const void *w1, const void *b1,
                                 const void *w3, const void *w2, const void *b2, moe_act act, int e, int64_t n, int m,
                                 int h, void *hid, void *pre, void *out, int32_t *dev_status, void *stream) {
    if (!valid_dt(dt) || !sorted_ffn_shape_ok(act, e, n, m, h) || !ok16(x) || !ok4(offsets) || !ok16(w1) ||
        !ok16(w2) || !opt16(b1) || !opt16(b2) || !ok16(hid) || !opt16(pre) || !ok16(out) || !ok4(dev_status))
        return MOE_ERR_INVALID_ARG;
    if (act == MOE_ACT_SWIGLU && (!ok16(w3) || b1 || b2)) return MOE_ERR_INVALID_ARG;
    if (dt != MOE_BF16 || !sorted_ffn_supported(act, e, n, m, h)) return MOE_ERR_UNSUPPORTED;
    if (few_rows(n, e))
        return ffn_few_launch(x, SortedRows{offsets, n}, w1, b1, w3, w2, b2, act, e, m, h, hid, pre, out, dev_status,
                              as_stream(stream));
    return ffn_tc_launch(x, nullptr, nullptr, w1, b1, w3, w2, b2, act, e, n, m, h, hid, out, dev_status,
                         as_stream(stream), 0, 0, pre, SortedRows{offsets, n});
}

size_t moe_expert_ffn_sorted_bwd_workspace_size(moe_act act, int e, int64_t n, int m, int h) {
    if (!sorted_ffn_shape_ok(act, e, n, m, h) || !sorted_ffn_supported(act, e, n, m, h)) return 0;
    return ffn_tc_sorted_bwd_workspace_bytes(act, e, n, m, h);
}

moe_status moe_expert_ffn_sorted_bwd(const void *x, const void *hid, const void *pre, moe_dtype dt,
                                     const int32_t *offsets, const void *w1, const void *w3, const void *w2,
                                     moe_act act, int e, int64_t n, int m, int h, const void *d_out, void *workspace,
                                     size_t workspace_bytes, void *d_x, moe_dtype wgrad_dt, void *d_w1, void *d_w3,
                                     void *d_w2, void *d_b1, void *d_b2, int32_t *dev_status, void *stream) {
    if (!valid_dt(dt) || !valid_dt(wgrad_dt) || !sorted_ffn_shape_ok(act, e, n, m, h) || !ok16(x) || !ok16(hid) ||
        !ok16(pre) || !ok4(offsets) || !ok16(w1) || !ok16(w2) || !ok16(d_out) || !ok16(workspace) || !ok16(d_x) ||
        !ok16(d_w1) || !ok16(d_w2) || !opt16(d_b1) || !opt16(d_b2) || !ok4(dev_status))
        return MOE_ERR_INVALID_ARG;
    if (act == MOE_ACT_SWIGLU && (!ok16(w3) || !ok16(d_w3) || d_b1 || d_b2)) return MOE_ERR_INVALID_ARG;
    if (dt != MOE_BF16 || !sorted_ffn_supported(act, e, n, m, h)) return MOE_ERR_UNSUPPORTED;
    if (workspace_bytes < ffn_tc_sorted_bwd_workspace_bytes(act, e, n, m, h)) return MOE_ERR_INVALID_ARG;
    return ffn_tc_bwd_launch(x, hid, nullptr, nullptr, w1, nullptr, w3, w2, act, e, n, m, h, d_out, workspace, d_x,
                             d_w1, d_w3, d_w2, d_b1, d_b2, dev_status, as_stream(stream), pre, wgrad_dt == MOE_F32,
                             SortedRows{offsets, n});
}

// --------------------------------------------------- 8-bit integer experts
namespace {

bool int8_shape_ok(int e, int64_t n, int k, int n_out) {
    return e >= 1 && e <= kMaxE && n >= 1 && k >= 16 && k % 16 == 0 && n_out >= 8 && n_out % 8 == 0;
}

// k: int32 holds any sum of 8-bit products; the rest within the grouped product's indexes (the
// last tile of channels may reach past the end)
bool int8_supported(int e, int64_t n, int k, int n_out) {
    return k < 1 << 17 && n <= kMaxRows && (int64_t)e * n_out <= kMaxRows &&
           (n / 192 + e) * ((n_out + 127) / 128) < (int64_t)1 << 31;
}

}  // namespace

moe_status moe_quantize_rows_int8(const void *src, moe_dtype sdt, const int32_t *rows, int64_t s, int cols, int k,
                                  int64_t n, void *q, float *scale, int32_t *dev_status, void *stream) {
    if (!valid_dt(sdt) || s < 1 || s > kMaxRows || cols < 16 || cols % 16 || n < 1 || n > kMaxRows || !ok16(src) ||
        !ok16(q) || !ok4(scale) || !ok4(dev_status))
        return MOE_ERR_INVALID_ARG;
    if (rows ? !ok4(rows) || k < 1 || k > kMaxK || s > kMaxRows / k : k != 0 || n != s) return MOE_ERR_INVALID_ARG;
    return quantize_rows_int8_launch(src, sdt, rows, s, cols, k, n, q, scale, dev_status, as_stream(stream));
}

size_t moe_product_int8_workspace_size(int e, int64_t n, int k, int n_out) {
    if (!int8_shape_ok(e, n, k, n_out) || !int8_supported(e, n, k, n_out)) return 0;
    return product_int8_workspace_bytes(e, n, k);
}

moe_status moe_product_int8(const void *a_q, const float *a_scale, const int32_t *offsets, const void *b_q,
                            const float *b_scale, const void *bias, int e, int64_t n, int k, int n_out,
                            void *workspace, size_t workspace_bytes, void *out, moe_dtype odt, int32_t *dev_status,
                            void *stream) {
    if (!int8_shape_ok(e, n, k, n_out) || !valid_dt(odt) || !ok16(a_q) || !ok4(a_scale) ||
        (offsets ? !ok4(offsets) : e != 1) || !ok16(b_q) || !ok4(b_scale) || !opt16(bias) || !ok16(workspace) ||
        !ok16(out) || !ok4(dev_status))
        return MOE_ERR_INVALID_ARG;
    if (!int8_supported(e, n, k, n_out)) return MOE_ERR_UNSUPPORTED;
    if (workspace_bytes < product_int8_workspace_bytes(e, n, k)) return MOE_ERR_INVALID_ARG;
    return product_int8_launch(a_q, a_scale, SortedRows{offsets, n}, b_q, b_scale, bias, e, k, n_out, workspace, out,
                               odt == MOE_F32, dev_status, as_stream(stream));
}

size_t moe_expert_ffn_int8_workspace_size(moe_act act, int e, int64_t n, int m, int h) {
    if (!act_ok(act) || m % 16 || !int8_shape_ok(e, n, m, h) || !int8_shape_ok(e, n, h, m) ||
        !int8_supported(e, n, m, h) || !int8_supported(e, n, h, m))
        return 0;
    return ffn_int8_workspace_bytes(e, n, m, h);
}

moe_status moe_expert_ffn_int8(const void *x_q, const float *x_scale, const int32_t *offsets, const void *w1_q,
                               const float *w1_scale, const void *b1, const void *w3_q, const float *w3_scale,
                               const void *w2_q, const float *w2_scale, const void *b2, moe_act act, int e, int64_t n,
                               int m, int h, void *workspace, size_t workspace_bytes, void *out, int32_t *dev_status,
                               void *stream) {
    if (!act_ok(act) || !int8_shape_ok(e, n, m, h) || !int8_shape_ok(e, n, h, m) || !ok16(x_q) || !ok4(x_scale) ||
        (offsets ? !ok4(offsets) : e != 1) || !ok16(w1_q) || !ok4(w1_scale) || !opt16(b1) || !ok16(w2_q) ||
        !ok4(w2_scale) || !opt16(b2) || !ok16(workspace) || !ok16(out) || !ok4(dev_status))
        return MOE_ERR_INVALID_ARG;
    if (act == MOE_ACT_SWIGLU ? !ok16(w3_q) || !ok4(w3_scale) || b1 || b2 : w3_q || w3_scale)
        return MOE_ERR_INVALID_ARG;
    if (!int8_supported(e, n, m, h) || !int8_supported(e, n, h, m)) return MOE_ERR_UNSUPPORTED;
    if (workspace_bytes < ffn_int8_workspace_bytes(e, n, m, h)) return MOE_ERR_INVALID_ARG;
    return ffn_int8_launch(x_q, x_scale, SortedRows{offsets, n}, w1_q, w1_scale, b1, w3_q, w3_scale, w2_q, w2_scale, b2,
                           act, e, m, h, workspace, out, dev_status, as_stream(stream));
}

size_t moe_layer_workspace_size(moe_dtype dt, moe_act act, int64_t s, int m, int e, int k,
                                int64_t c_max, int h) {
    size_t a = moe_capacity_workspace_size(s, e, k);
    size_t b = moe_expert_ffn_workspace_size(dt, act, e, c_max, m, h);
    if (a == 0 || b == 0) return 0;
    return up256(a) + up256(b);
}

moe_status moe_layer_forward(const void *x, moe_dtype dt, const float *wg, const float *gate_bias,
                             const void *w1, const void *b1, const void *w3, const void *w2,
                             const void *b2, moe_act act, int64_t s, int m, int e, int k, int h,
                             float capacity_factor, int64_t c_max, unsigned flags, int32_t *idx,
                             float *gates, int32_t *loc, int32_t *counts, int32_t *c_dev,
                             void *buf, void *out, void *y, void *workspace,
                             size_t workspace_bytes, int32_t *dev_status, void *stream) {
    size_t need = moe_layer_workspace_size(dt, act, s, m, e, k, c_max, h);
    if (need == 0 || workspace_bytes < need || !ok16(workspace)) return MOE_ERR_INVALID_ARG;
    size_t cap_b = up256(moe_capacity_workspace_size(s, e, k));
    char *ws = (char *)workspace;
    moe_status st;
    st = moe_gate_topk(x, dt, wg, gate_bias, s, m, e, k, flags & MOE_FLAG_NORMALIZE_GATES, idx,
                       gates, dev_status, stream);
    if (st != MOE_OK) return st;
    st = moe_capacity_locations(idx, s, e, k, capacity_factor, c_max, ws, cap_b, loc, counts, c_dev,
                                dev_status, stream);
    if (st != MOE_OK) return st;
    st = moe_encode(x, dt, idx, loc, counts, c_dev, s, m, e, k, c_max, flags & MOE_FLAG_ZERO_FILL,
                    buf, dev_status, stream);
    if (st != MOE_OK) return st;
    st = moe_expert_ffn(buf, dt, counts, c_dev, w1, b1, w3, w2, b2, act, e, c_max, m, h,
                        ws + cap_b, workspace_bytes - cap_b, out, dev_status, stream);
    if (st != MOE_OK) return st;
    return moe_decode(out, dt, idx, loc, gates, c_dev, s, m, e, k, c_max, y, dev_status, stream);
}

moe_status moe_layer_forward_host(const void *x_host, void *y_host, const void *x, moe_dtype dt,
                                  const float *wg, const float *gate_bias, const void *w1,
                                  const void *b1, const void *w3, const void *w2, const void *b2,
                                  moe_act act, int64_t s, int m, int e, int k, int h,
                                  float capacity_factor, int64_t c_max, unsigned flags,
                                  int32_t *idx, float *gates, int32_t *loc, int32_t *counts,
                                  int32_t *c_dev, void *buf, void *out, void *y, void *workspace,
                                  size_t workspace_bytes, int32_t *dev_status, void *stream) {
    if (x_host == nullptr || y_host == nullptr || !valid_dt(dt) || s < 1 || m < 1 || !ok16(x) ||
        !ok16(y))
        return MOE_ERR_INVALID_ARG;
    if (moe_layer_workspace_size(dt, act, s, m, e, k, c_max, h) == 0) return MOE_ERR_INVALID_ARG;
    const size_t bytes = (size_t)s * (size_t)m * esize(dt);
    cudaStream_t st = as_stream(stream);
    if (cudaMemcpyAsync(const_cast<void *>(x), x_host, bytes, cudaMemcpyHostToDevice, st) !=
        cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    moe_status r = moe_layer_forward(x, dt, wg, gate_bias, w1, b1, w3, w2, b2, act, s, m, e, k, h,
                                     capacity_factor, c_max, flags, idx, gates, loc, counts,
                                     c_dev, buf, out, y, workspace, workspace_bytes, dev_status,
                                     stream);
    if (r != MOE_OK) return r;
    if (cudaMemcpyAsync(y_host, y, bytes, cudaMemcpyDeviceToHost, st) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    return MOE_OK;
}

moe_status moe_layer_forward_pipelined(const void *x, moe_dtype dt, const float *wg,
                                       const float *gate_bias, const void *w1, const void *b1,
                                       const void *w3, const void *w2, const void *b2, moe_act act,
                                       int64_t s, int m, int e, int k, int h, float capacity_factor,
                                       int64_t c_max, unsigned flags, int32_t *idx, float *gates,
                                       int32_t *loc, int32_t *counts, int32_t *c_dev, void *buf,
                                       void *out, void *y, void *workspace, size_t workspace_bytes,
                                       int32_t *dev_status, int chunks, void *stream,
                                       void *aux_stream, void *const *events) {
    if (chunks < 1 || chunks > 64 || events == nullptr) return MOE_ERR_INVALID_ARG;
    for (int i = 0; i <= chunks; i++)
        if (events[i] == nullptr) return MOE_ERR_INVALID_ARG;
    if (dt != MOE_BF16 || chunks == 1)
        return moe_layer_forward(x, dt, wg, gate_bias, w1, b1, w3, w2, b2, act, s, m, e, k, h,
                                 capacity_factor, c_max, flags, idx, gates, loc, counts, c_dev, buf,
                                 out, y, workspace, workspace_bytes, dev_status, stream);
    size_t need = moe_layer_workspace_size(dt, act, s, m, e, k, c_max, h);
    if (need == 0 || workspace_bytes < need || !ok16(workspace)) return MOE_ERR_INVALID_ARG;
    // every stage's own checks, by the calls below, before anything is launched
    if (!routing_shape_ok(s, e, k) || !rows_ok(dt, m) || !rows_ok(dt, h) || c_max < 1 ||
        c_max > 0x7fffffff || !ok16(x) || !ok16(wg) || !opt16(gate_bias) || !ok4(idx) ||
        !ok4(gates) || !ok4(loc) || !ok4(counts) || !ok4(c_dev) || !ok16(buf) || !ok16(out) ||
        !ok16(y) || !ok4(dev_status) || !ok16(w1) || !ok16(w2) || !opt16(b1) || !opt16(b2) ||
        (flags & ~3u) || (act != MOE_ACT_RELU && act != MOE_ACT_GELU && act != MOE_ACT_SWIGLU) ||
        (act == MOE_ACT_SWIGLU && (!ok16(w3) || b1 != nullptr || b2 != nullptr)))
        return MOE_ERR_INVALID_ARG;
    if (e > 256 || !ffn_tc_supported(e, c_max, m, h)) return MOE_ERR_UNSUPPORTED;
    const size_t cap_b = up256(moe_capacity_workspace_size(s, e, k));
    char *ws = (char *)workspace;
    cudaStream_t st = as_stream(stream), aux = as_stream(aux_stream);
    cudaEvent_t *ev = (cudaEvent_t *)events;
    moe_status r;
    r = moe_gate_topk(x, dt, wg, gate_bias, s, m, e, k, flags & MOE_FLAG_NORMALIZE_GATES, idx, gates,
                      dev_status, stream);
    if (r != MOE_OK) return r;
    r = moe_capacity_locations(idx, s, e, k, capacity_factor, c_max, ws, cap_b, loc, counts, c_dev,
                               dev_status, stream);
    if (r != MOE_OK) return r;
    if (cudaEventRecord(ev[0], st) != cudaSuccess || cudaStreamWaitEvent(aux, ev[0], 0) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    // slot chunks [lo, hi) of the expert buffer, in whole 256-row FFN tiles
    const int64_t step = ((c_max + chunks - 1) / chunks + 255) / 256 * 256;
    for (int i = 0; i < chunks; i++) {
        const int64_t lo = (int64_t)i * step, hi = lo + step;
        if (lo >= c_max) break;
        const int ihi = hi >= c_max ? 0x7fffffff : (int)hi;
        // encode of chunk i on the side stream (zero fill, if asked, with the first)
        r = encode_launch(x, dt, idx, loc, counts, c_dev, s, m, e, k, c_max,
                          i == 0 ? (flags & MOE_FLAG_ZERO_FILL) : 0u, buf, dev_status, aux, (int)lo,
                          ihi);
        if (r != MOE_OK) return r;
        if (cudaEventRecord(ev[1 + i], aux) != cudaSuccess ||
            cudaStreamWaitEvent(st, ev[1 + i], 0) != cudaSuccess) {
            cudaGetLastError();
            return MOE_ERR_CUDA;
        }
        // the FFN of chunk i on the main stream, while chunk i+1 is encoded
        r = ffn_tc_launch(buf, counts, c_dev, w1, b1, w3, w2, b2, act, e, c_max, m, h, ws + cap_b,
                          out, dev_status, st, (int)lo, hi >= c_max ? 0 : (int)hi);
        if (r != MOE_OK) return r;
    }
    return moe_decode(out, dt, idx, loc, gates, c_dev, s, m, e, k, c_max, y, dev_status, stream);
}

size_t moe_expert_ffn_fp8_workspace_size(int e, int64_t c_max, int m, int h) {
    if (e < 1 || e > kMaxE || c_max < 1 || m < 16 || h < 16 || m % 16 || h % 16) return 0;
    const int64_t rows = (int64_t)e * c_max;
    return up256((size_t)rows * h * 2) + up256((size_t)rows * h) + up256((size_t)rows * 4);
}

moe_status moe_quantize_rows_fp8(const void *src, int64_t batches, int64_t rows_per_batch,
                                 int cols, const int32_t *counts, const int32_t *c_dev, void *q,
                                 float *scale, int32_t *dev_status, void *stream) {
    if (batches < 1 || batches > 0x7fffffff || rows_per_batch < 1 || cols < 16 || cols % 16 ||
        batches * rows_per_batch > ((int64_t)1 << 40) || !ok16(src) || !ok16(q) || !ok4(scale) ||
        !ok4(dev_status) || (counts == nullptr) != (c_dev == nullptr) ||
        (counts && (!ok4(counts) || !ok4(c_dev))))
        return MOE_ERR_INVALID_ARG;
    return quantize_rows_fp8_launch(src, batches, rows_per_batch, cols, counts, c_dev, q, scale,
                                    dev_status, as_stream(stream));
}

moe_status moe_expert_ffn_fp8(const void *buf_q, const float *buf_scale, const int32_t *counts,
                              const int32_t *c_dev, const void *w1_q, const float *w1_scale,
                              const void *b1, const void *w2_q, const float *w2_scale,
                              const void *b2, moe_act act, int e, int64_t c_max, int m, int h,
                              void *workspace, size_t workspace_bytes, void *out,
                              int32_t *dev_status, void *stream) {
    const size_t need = moe_expert_ffn_fp8_workspace_size(e, c_max, m, h);
    if (need == 0 || c_max > 0x7fffffff || !ok16(buf_q) || !ok4(buf_scale) || !ok4(counts) ||
        !ok4(c_dev) || !ok16(w1_q) || !ok16(w1_scale) || !opt16(b1) || !ok16(w2_q) ||
        !ok16(w2_scale) || !opt16(b2) || !ok16(workspace) || workspace_bytes < need ||
        !ok16(out) || !ok4(dev_status))
        return MOE_ERR_INVALID_ARG;
    if (act != MOE_ACT_RELU && act != MOE_ACT_GELU) return MOE_ERR_UNSUPPORTED;
    if (!ffn_tc_supported(e, c_max, m, h)) return MOE_ERR_UNSUPPORTED;
    const int64_t rows = (int64_t)e * c_max;
    char *w = (char *)workspace;
    void *hid = w;
    void *hid_q = w + up256((size_t)rows * h * 2);
    float *hid_scale = (float *)(w + up256((size_t)rows * h * 2) + up256((size_t)rows * h));
    return ffn_tc_fp8_launch(buf_q, buf_scale, counts, c_dev, w1_q, w1_scale, b1, w2_q, w2_scale, b2,
                             act, e, c_max, m, h, hid, hid_q, hid_scale, out, dev_status,
                             as_stream(stream));
}

moe_status moe_route_topk(const void *logits, moe_dtype ldt, const float *bias, int64_t s, int e,
                          int k, moe_score score, int groups, int topk_groups, int group_top,
                          float scale, unsigned flags, int32_t *idx, float *gates,
                          int32_t *dev_status, void *stream) {
    if (!routing_shape_ok(s, e, k) || !valid_dt(ldt) || !ok16(logits) || !opt16(bias) ||
        (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) || groups < 1 || groups > e ||
        e % groups || topk_groups < 1 || topk_groups > groups ||
        (int64_t)topk_groups * (e / groups) < k || (group_top != 1 && group_top != 2) ||
        scale != scale || !ok4(idx) || !ok4(gates) || !ok4(dev_status) ||
        (flags & ~MOE_FLAG_NORMALIZE_GATES))
        return MOE_ERR_INVALID_ARG;
    if (groups > 32) return MOE_ERR_UNSUPPORTED;
    return route_topk_launch(logits, ldt, bias, s, e, k, score, groups, topk_groups, group_top, scale,
                             flags, idx, gates, dev_status, as_stream(stream));
}

moe_status moe_route_bwd(const void *logits, moe_dtype ldt, const int32_t *idx,
                         const float *d_gates, int64_t s, int e, int k, moe_score score,
                         float scale, unsigned flags, void *d_logits, moe_dtype ddt,
                         int32_t *dev_status, void *stream) {
    if (!routing_shape_ok(s, e, k) || !valid_dt(ldt) || !valid_dt(ddt) || !ok16(logits) ||
        (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) || scale != scale || !ok4(idx) ||
        !ok4(d_gates) || !ok16(d_logits) || !ok4(dev_status) || (flags & ~MOE_FLAG_NORMALIZE_GATES))
        return MOE_ERR_INVALID_ARG;
    return route_bwd_launch(logits, ldt, idx, d_gates, s, e, k, score, scale, flags, d_logits, ddt,
                            dev_status, as_stream(stream));
}

static bool fp4_ok(moe_fp4 fmt, int64_t rows, int cols) {
    return (fmt == MOE_FP4_MX || fmt == MOE_FP4_NV) && rows >= 1 && rows <= 0x7fffffff && cols >= 32 &&
           cols % 32 == 0;
}

size_t moe_fp4_scale_bytes(moe_fp4 fmt, int64_t rows, int cols) {
    return fp4_ok(fmt, rows, cols) ? (size_t)fp4_scale_bytes(fp4_blk(fmt), rows, cols) : 0;
}

// What both directions of the conversion check alike.
static bool fp4_rows_ok(const void *wide, moe_dtype dt, int64_t batches, int64_t rows, int cols,
                        moe_fp4 fmt, const float *global, const int32_t *counts,
                        const int32_t *c_dev, const void *q, const void *scale, const int32_t *st) {
    return fp4_ok(fmt, rows, cols) && batches >= 1 && batches <= 0x7fffffff && valid_dt(dt) &&
           batches * rows <= ((int64_t)1 << 40) && ok16(wide) && ok16(q) && ok16(scale) && ok4(st) &&
           (global == nullptr || (fmt == MOE_FP4_NV && ok4(global))) &&
           (counts == nullptr) == (c_dev == nullptr) && (!counts || (ok4(counts) && ok4(c_dev)));
}

moe_status moe_quantize_fp4(const void *src, moe_dtype sdt, int64_t batches,
                            int64_t rows_per_batch, int cols, moe_fp4 fmt,
                            const float *global_scale, const int32_t *counts,
                            const int32_t *c_dev, void *q, void *scale, int32_t *dev_status,
                            void *stream) {
    if (!fp4_rows_ok(src, sdt, batches, rows_per_batch, cols, fmt, global_scale, counts, c_dev, q, scale,
                     dev_status))
        return MOE_ERR_INVALID_ARG;
    return quantize_fp4_launch(src, sdt, batches, rows_per_batch, cols, fmt, global_scale, counts, c_dev,
                               q, scale, dev_status, as_stream(stream));
}

moe_status moe_dequantize_fp4(const void *q, const void *scale, int64_t batches,
                              int64_t rows_per_batch, int cols, moe_fp4 fmt,
                              const float *global_scale, const int32_t *counts,
                              const int32_t *c_dev, void *dst, moe_dtype ddt, int32_t *dev_status,
                              void *stream) {
    if (!fp4_rows_ok(dst, ddt, batches, rows_per_batch, cols, fmt, global_scale, counts, c_dev, q, scale,
                     dev_status))
        return MOE_ERR_INVALID_ARG;
    return dequantize_fp4_launch(q, scale, batches, rows_per_batch, cols, fmt, global_scale, counts,
                                 c_dev, dst, ddt, dev_status, as_stream(stream));
}

// Rows and columns within the 32-bit coordinates of the operands' tensor maps.
static bool fp4_range_ok(int e, int64_t c_max, int64_t k, int64_t n) {
    return (int64_t)e * c_max < ((int64_t)1 << 31) && (int64_t)e * n < ((int64_t)1 << 31) &&
           (int64_t)e * k < ((int64_t)1 << 31);
}

static bool fp4_factor_ok(moe_fp4 fmt, const float *g) {
    return g == nullptr || (fmt == MOE_FP4_NV && ok4(g));
}

moe_status moe_product_fp4(const void *a_q, const void *a_scale, const float *a_global,
                           const int32_t *counts, const int32_t *c_dev, const void *b_q,
                           const void *b_scale, const float *b_global, const void *bias,
                           moe_fp4 fmt, int e, int64_t c_max, int k, int n, void *out,
                           int32_t *dev_status, void *stream) {
    if (!fp4_ok(fmt, c_max, k) || e < 1 || e > kMaxE || n < 8 || n % 8 || !ok16(a_q) ||
        !ok16(a_scale) || !fp4_factor_ok(fmt, a_global) || !ok4(counts) || !ok4(c_dev) || !ok16(b_q) ||
        !ok16(b_scale) || !fp4_factor_ok(fmt, b_global) || !opt16(bias) || !ok16(out) || !ok4(dev_status))
        return MOE_ERR_INVALID_ARG;
    if (!fp4_range_ok(e, c_max, k, n)) return MOE_ERR_UNSUPPORTED;
    return product_fp4_launch(a_q, a_scale, a_global, counts, c_dev, b_q, b_scale, b_global, bias, fmt, e,
                              c_max, k, n, out, dev_status, as_stream(stream));
}

size_t moe_expert_ffn_fp4_workspace_size(moe_fp4 fmt, moe_act act, int e, int64_t c_max, int m,
                                         int h) {
    if (!fp4_ok(fmt, c_max, m) || !fp4_ok(fmt, c_max, h) || e < 1 || e > kMaxE ||
        (act != MOE_ACT_RELU && act != MOE_ACT_GELU && act != MOE_ACT_SWIGLU))
        return 0;
    return up256((size_t)e * c_max * (h / 2)) + up256((size_t)e * moe_fp4_scale_bytes(fmt, c_max, h));
}

moe_status moe_expert_ffn_fp4(const void *buf_q, const void *buf_scale, const float *buf_global,
                              const float *hid_global, const int32_t *counts,
                              const int32_t *c_dev, const void *w1_q, const void *w1_scale,
                              const float *w1_global, const void *b1, const void *w3_q,
                              const void *w3_scale, const float *w3_global, const void *w2_q,
                              const void *w2_scale, const float *w2_global, const void *b2,
                              moe_fp4 fmt, moe_act act, int e, int64_t c_max, int m, int h,
                              void *workspace, size_t workspace_bytes, void *out,
                              int32_t *dev_status, void *stream) {
    const size_t need = moe_expert_ffn_fp4_workspace_size(fmt, act, e, c_max, m, h);
    if (need == 0 || !ok16(buf_q) || !ok16(buf_scale) || !fp4_factor_ok(fmt, buf_global) ||
        !fp4_factor_ok(fmt, hid_global) || !ok4(counts) || !ok4(c_dev) || !ok16(w1_q) ||
        !ok16(w1_scale) || !fp4_factor_ok(fmt, w1_global) || !opt16(b1) || !ok16(w2_q) ||
        !ok16(w2_scale) || !fp4_factor_ok(fmt, w2_global) || !opt16(b2) || !ok16(workspace) ||
        workspace_bytes < need || !ok16(out) || !ok4(dev_status))
        return MOE_ERR_INVALID_ARG;
    if (act == MOE_ACT_SWIGLU) {
        if (!ok16(w3_q) || !ok16(w3_scale) || !fp4_factor_ok(fmt, w3_global) || b1 || b2)
            return MOE_ERR_INVALID_ARG;
    } else if (w3_q || w3_scale || w3_global) {
        return MOE_ERR_INVALID_ARG;
    }
    if (!fp4_range_ok(e, c_max, m, h) || !fp4_range_ok(e, c_max, h, m)) return MOE_ERR_UNSUPPORTED;
    char *w = (char *)workspace;
    return ffn_fp4_launch(buf_q, buf_scale, buf_global, hid_global, counts, c_dev, w1_q, w1_scale,
                          w1_global, b1, w3_q, w3_scale, w3_global, w2_q, w2_scale, w2_global, b2, fmt,
                          act, e, c_max, m, h, w, w + up256((size_t)e * c_max * (h / 2)), out,
                          dev_status, as_stream(stream));
}

moe_status moe_probe_fp32_fma(int packed, int blocks, int iters, float *out, void *stream) {
    if (blocks < 1 || iters < 1 || !ok4(out)) return MOE_ERR_INVALID_ARG;
    return probe_fp32_fma_launch(packed, blocks, iters, out, as_stream(stream));
}

}  // extern "C"
