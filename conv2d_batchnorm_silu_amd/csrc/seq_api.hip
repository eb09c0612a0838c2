// seq_api.hip -- argument checks of the sequence operators and the C entry
// points declared in include/tg_sequence.h.
#include "seq_internal.hpp"
#include "tg_sequence.h"

using namespace tg;

namespace {

// Row numbers, and a strip or chunk past them, are ints in the kernels; a
// launch has fewer than 2^32 threads along x, so the scan's single waves, and the
// single token's workgroups of 256 threads, are limited.
constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr int kMaxChannels = 1 << 20;
constexpr int64_t kMaxGroups = ((int64_t)1 << 26) - 1;
constexpr int64_t kMaxStepGroups = ((int64_t)1 << 24) - 1;
// The scan addresses 16 rows by 31-bit byte offsets.
constexpr int64_t kMaxScanStride = (int64_t)1 << 25;

bool dtype_ok(int d) { return d == TG_F16 || d == TG_BF16 || d == TG_F32; }
bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
// A launcher finds sizes that no launch holds before it launches anything.
tg_status of(hipError_t e) {
    return e == hipSuccess ? TG_OK
           : e == hipErrorInvalidConfiguration ? TG_ERR_UNSUPPORTED : TG_ERR_HIP;
}

#define TG_REQUIRE(cond, status) \
    do {                         \
        if (!(cond)) return (status); \
    } while (0)

tg_status check_seqs(const tg_seqs& s) {
    TG_REQUIRE(s.seqs >= 1 && s.rows >= 0, TG_ERR_INVALID_ARGUMENT);
    TG_REQUIRE(s.offsets || s.rows % s.seqs == 0, TG_ERR_INVALID_ARGUMENT);
    TG_REQUIRE(s.rows < kMaxRows && s.seqs < kMaxRows, TG_ERR_UNSUPPORTED);
    TG_REQUIRE(aligned(s.offsets, 4), TG_ERR_ALIGNMENT);
    return TG_OK;
}

// A tensor of rows that has to be there (unless the batch has no row).
tg_status check_rows(const tg_rows& r, const tg_seqs& s, int64_t width, size_t elem,
                     bool written) {
    if (s.rows == 0) return TG_OK;
    TG_REQUIRE(r.p, TG_ERR_INVALID_ARGUMENT);
    // Inputs may repeat a row (stride 0); written rows must not overlap.
    const int64_t least = written ? width : 0;
    TG_REQUIRE(r.row_stride >= least || (written && s.rows == 1), TG_ERR_INVALID_ARGUMENT);
    if (!s.offsets)
        TG_REQUIRE(r.seq_stride >= least || (written && s.seqs == 1), TG_ERR_INVALID_ARGUMENT);
    TG_REQUIRE(aligned(r.p, elem), TG_ERR_ALIGNMENT);
    return TG_OK;
}
tg_status check_scan_rows(const tg_rows& r, const tg_seqs& s, int64_t width, size_t elem,
                          bool written) {
    TG_REQUIRE(s.rows == 0 || r.row_stride < kMaxScanStride, TG_ERR_UNSUPPORTED);
    return check_rows(r, s, width, elem, written);
}

#define TG_CHECK(expr)                     \
    do {                                   \
        const tg_status st_ = (expr);      \
        if (st_ != TG_OK) return st_;      \
    } while (0)

tg_status check_conv(const tg_causal_conv_args* a) {
    TG_REQUIRE(a, TG_ERR_INVALID_ARGUMENT);
    TG_CHECK(check_seqs(a->seqs));
    TG_REQUIRE(a->D >= 1 && a->K >= 1 && a->w, TG_ERR_INVALID_ARGUMENT);
    TG_REQUIRE(dtype_ok((int)a->dtype) && a->D <= kMaxChannels && a->K >= 2 && a->K <= 8,
               TG_ERR_UNSUPPORTED);
    TG_REQUIRE((int)a->act == TG_ACT_SILU || (int)a->act == TG_ACT_NONE, TG_ERR_UNSUPPORTED);
    const size_t e = elem_bytes(a->dtype);
    TG_REQUIRE(aligned(a->w, 4) && aligned(a->bias, 4) && aligned(a->initial, e) &&
                   aligned(a->final, e), TG_ERR_ALIGNMENT);
    return check_rows(a->x, a->seqs, a->D, e, false);
}

tg_status check_scan(const tg_scan_args* a) {
    TG_REQUIRE(a, TG_ERR_INVALID_ARGUMENT);
    TG_CHECK(check_seqs(a->seqs));
    TG_REQUIRE(a->D >= 1 && a->N >= 1 && a->G >= 1 && a->D % a->G == 0, TG_ERR_INVALID_ARGUMENT);
    TG_REQUIRE(dtype_ok((int)a->dtype) && a->D <= kMaxChannels && a->N <= 128, TG_ERR_UNSUPPORTED);
    return TG_OK;
}
// Workgroups: one for each sequence and (at least one) block of channels.
tg_status check_scan_groups(const tg_scan_args* a) {
    TG_REQUIRE(a->seqs.seqs * ceil_div(a->D / a->G, 16) * a->G <= kMaxGroups, TG_ERR_UNSUPPORTED);
    return TG_OK;
}
tg_status check_scan_inputs(const tg_scan_args* a) {
    const size_t e = elem_bytes(a->dtype);
    TG_REQUIRE(a->A, TG_ERR_INVALID_ARGUMENT);
    TG_REQUIRE(aligned(a->A, 4) && aligned(a->D_skip, 4) && aligned(a->dt_bias, 4) &&
                   aligned(a->initial, 4) && aligned(a->final, 4), TG_ERR_ALIGNMENT);
    TG_CHECK(check_scan_rows(a->x, a->seqs, a->D, e, false));
    TG_CHECK(check_scan_rows(a->dt, a->seqs, a->D, e, false));
    TG_CHECK(check_scan_rows(a->B, a->seqs, (int64_t)a->G * a->N, e, false));
    TG_CHECK(check_scan_rows(a->C, a->seqs, (int64_t)a->G * a->N, e, false));
    if (a->z.p) TG_CHECK(check_scan_rows(a->z, a->seqs, a->D, e, false));
    return TG_OK;
}

}  // namespace

extern "C" {

tg_status tg_layer_norm(const void* x, int64_t x_stride, const void* residual,
                        int64_t residual_stride, const float* gamma, const float* beta, float eps,
                        int64_t rows, int C, tg_dtype dtype, void* y, void* sum, float* mean,
                        float* rstd, void* stream) {
    TG_REQUIRE(rows >= 0 && C >= 1 && eps >= 0.0f && gamma, TG_ERR_INVALID_ARGUMENT);
    TG_REQUIRE(!residual == !sum && !mean == !rstd, TG_ERR_INVALID_ARGUMENT);
    TG_REQUIRE(dtype_ok((int)dtype) && C <= kMaxChannels && rows < kMaxRows, TG_ERR_UNSUPPORTED);
    if (rows == 0) return TG_OK;
    TG_REQUIRE(x && y, TG_ERR_INVALID_ARGUMENT);
    TG_REQUIRE(x_stride == 0 || x_stride >= C || rows == 1, TG_ERR_INVALID_ARGUMENT);
    TG_REQUIRE(!residual || residual_stride == 0 || residual_stride >= C || rows == 1,
               TG_ERR_INVALID_ARGUMENT);
    const size_t e = elem_bytes(dtype);
    TG_REQUIRE(aligned(x, e) && aligned(y, e) && aligned(residual, e) && aligned(sum, e) &&
                   aligned(gamma, 4) && aligned(beta, 4) && aligned(mean, 4) && aligned(rstd, 4),
               TG_ERR_ALIGNMENT);
    return of(launch_layer_norm(x, x_stride, residual, residual_stride, gamma, beta, eps, rows, C,
                                dtype, y, sum, mean, rstd, (hipStream_t)stream));
}

tg_status tg_layer_norm_backward_workspace(int64_t rows, int C, tg_dtype dtype, size_t* bytes) {
    TG_REQUIRE(bytes && rows >= 0 && C >= 1, TG_ERR_INVALID_ARGUMENT);
    TG_REQUIRE(dtype_ok((int)dtype) && C <= kMaxChannels && rows < kMaxRows, TG_ERR_UNSUPPORTED);
    *bytes = layer_norm_backward_bytes(rows, C);
    return TG_OK;
}

tg_status tg_layer_norm_backward(const void* dy, int64_t dy_stride, const void* s, int64_t s_stride,
                                 const float* gamma, const float* mean, const float* rstd,
                                 const void* dsum, int64_t dsum_stride, int64_t rows, int C,
                                 tg_dtype dtype, void* dx, float* dgamma, float* dbeta,
                                 void* workspace, size_t workspace_bytes, void* stream) {
    TG_REQUIRE(rows >= 0 && C >= 1 && gamma && dgamma, TG_ERR_INVALID_ARGUMENT);
    TG_REQUIRE(dtype_ok((int)dtype) && C <= kMaxChannels && rows < kMaxRows, TG_ERR_UNSUPPORTED);
    const size_t e = elem_bytes(dtype);
    if (rows > 0) {
        TG_REQUIRE(dy && s && mean && rstd && dx, TG_ERR_INVALID_ARGUMENT);
        for (int64_t st : {dy_stride, s_stride, dsum ? dsum_stride : (int64_t)0})
            TG_REQUIRE(st == 0 || st >= C || rows == 1, TG_ERR_INVALID_ARGUMENT);
        TG_REQUIRE(aligned(dy, e) && aligned(s, e) && aligned(dsum, e) && aligned(dx, e) &&
                       aligned(gamma, 4) && aligned(mean, 4) && aligned(rstd, 4),
                   TG_ERR_ALIGNMENT);
        TG_REQUIRE(workspace && workspace_bytes >= layer_norm_backward_bytes(rows, C),
                   TG_ERR_WORKSPACE);
    }
    TG_REQUIRE(aligned(dgamma, 4) && aligned(dbeta, 4) && aligned(workspace, 16),
               TG_ERR_ALIGNMENT);
    return of(launch_layer_norm_backward(dy, dy_stride, s, s_stride, gamma, mean, rstd, dsum,
                                         dsum_stride, rows, C, dtype, dx, dgamma, dbeta, workspace,
                                         (hipStream_t)stream));
}

tg_status tg_causal_conv(const tg_causal_conv_args* a, void* stream) {
    TG_CHECK(check_conv(a));
    TG_CHECK(check_rows(a->y, a->seqs, a->D, elem_bytes(a->dtype), true));
    return of(launch_causal_conv(*a, (hipStream_t)stream));
}

tg_status tg_causal_conv_backward_workspace(const tg_causal_conv_args* a, size_t* bytes) {
    TG_REQUIRE(bytes, TG_ERR_INVALID_ARGUMENT);
    TG_CHECK(check_conv(a));
    *bytes = causal_conv_backward_bytes(*a);
    return TG_OK;
}

tg_status tg_causal_conv_backward(const tg_causal_conv_args* a, tg_rows dy, tg_rows dx, float* dw,
                                  float* dbias, const void* dfinal, void* dinitial,
                                  void* workspace, size_t workspace_bytes, void* stream) {
    TG_CHECK(check_conv(a));
    const size_t e = elem_bytes(a->dtype), need = causal_conv_backward_bytes(*a);
    TG_REQUIRE(dw, TG_ERR_INVALID_ARGUMENT);
    TG_CHECK(check_rows(dy, a->seqs, a->D, e, false));
    TG_CHECK(check_rows(dx, a->seqs, a->D, e, true));
    TG_REQUIRE(aligned(dw, 4) && aligned(dbias, 4) && aligned(dfinal, e) && aligned(dinitial, e) &&
                   aligned(workspace, 16), TG_ERR_ALIGNMENT);
    TG_REQUIRE(need == 0 || (workspace && workspace_bytes >= need), TG_ERR_WORKSPACE);
    return of(launch_causal_conv_backward(*a, dy, dx, dw, dbias, dfinal, dinitial, workspace,
                                          (hipStream_t)stream));
}

tg_status tg_causal_conv_step(const void* x, int64_t x_stride, void* state, int64_t num_slots,
                              const int32_t* slots, const float* w, const float* bias, int64_t n,
                              int D, int K, tg_dtype dtype, tg_activation act, void* y,
                              void* stream) {
    TG_REQUIRE(n >= 0 && num_slots >= 0 && D >= 1 && K >= 1 && w && (slots || n <= num_slots),
               TG_ERR_INVALID_ARGUMENT);
    TG_REQUIRE(dtype_ok((int)dtype) && D <= kMaxChannels && K >= 2 && K <= 8 && n < kMaxRows &&
                   num_slots < kMaxRows, TG_ERR_UNSUPPORTED);
    TG_REQUIRE((int)act == TG_ACT_SILU || (int)act == TG_ACT_NONE, TG_ERR_UNSUPPORTED);
    if (n == 0) return TG_OK;
    TG_REQUIRE(x && y && (state || num_slots == 0) && (x_stride == 0 || x_stride >= D || n == 1),
               TG_ERR_INVALID_ARGUMENT);
    const size_t e = elem_bytes(dtype);
    TG_REQUIRE(aligned(x, e) && aligned(y, e) && aligned(state, e) && aligned(slots, 4) &&
                   aligned(w, 4) && aligned(bias, 4), TG_ERR_ALIGNMENT);
    return of(launch_causal_conv_step(x, x_stride, state, num_slots, slots, w, bias, n, D, K,
                                      dtype, (int)act == TG_ACT_SILU, y, (hipStream_t)stream));
}

tg_status tg_selective_scan_sizes(const tg_scan_args* a, size_t* workspace_bytes,
                                  size_t* saved_bytes, size_t* backward_bytes) {
    TG_CHECK(check_scan(a));
    TG_CHECK(check_scan_groups(a));
    scan_sizes(*a, workspace_bytes, saved_bytes, backward_bytes);
    return TG_OK;
}

tg_status tg_selective_scan(const tg_scan_args* a, void* workspace, size_t workspace_bytes,
                            void* saved, size_t saved_bytes, void* stream) {
    TG_CHECK(check_scan(a));
    TG_CHECK(check_scan_groups(a));
    TG_CHECK(check_scan_inputs(a));
    TG_CHECK(check_scan_rows(a->y, a->seqs, a->D, elem_bytes(a->dtype), true));
    size_t work = 0, keep = 0;
    scan_sizes(*a, &work, &keep, nullptr);
    TG_REQUIRE(aligned(workspace, 16) && aligned(saved, 16), TG_ERR_ALIGNMENT);
    TG_REQUIRE(work == 0 || (workspace && workspace_bytes >= work), TG_ERR_WORKSPACE);
    TG_REQUIRE(!saved || saved_bytes >= keep, TG_ERR_WORKSPACE);
    return of(launch_scan(*a, workspace, saved, (hipStream_t)stream));
}

tg_status tg_selective_scan_backward(const tg_scan_args* a, const tg_scan_grads* g,
                                     const void* saved, size_t saved_bytes, void* workspace,
                                     size_t workspace_bytes, void* stream) {
    TG_CHECK(check_scan(a));
    TG_CHECK(check_scan_groups(a));
    TG_CHECK(check_scan_inputs(a));
    TG_REQUIRE(g && g->dA && (!g->dz.p == !a->z.p), TG_ERR_INVALID_ARGUMENT);
    TG_REQUIRE(scan_sum_groups(*a) < (int64_t)1 << 24, TG_ERR_UNSUPPORTED);  // of 256 threads
    const size_t e = elem_bytes(a->dtype);
    const int64_t gn = (int64_t)a->G * a->N;
    TG_CHECK(check_scan_rows(g->dy, a->seqs, a->D, e, false));
    TG_CHECK(check_scan_rows(g->dx, a->seqs, a->D, e, true));
    TG_CHECK(check_scan_rows(g->ddt, a->seqs, a->D, e, true));
    TG_CHECK(check_scan_rows(g->dB, a->seqs, gn, e, true));
    TG_CHECK(check_scan_rows(g->dC, a->seqs, gn, e, true));
    if (g->dz.p) TG_CHECK(check_scan_rows(g->dz, a->seqs, a->D, e, true));
    TG_REQUIRE(aligned(g->dA, 4) && aligned(g->dD, 4) && aligned(g->ddt_bias, 4) &&
                   aligned(g->dfinal, 4) && aligned(g->dinitial, 4) && aligned(saved, 16) &&
                   aligned(workspace, 16), TG_ERR_ALIGNMENT);
    size_t keep = 0, need = 0;
    scan_sizes(*a, nullptr, &keep, &need);
    TG_REQUIRE(saved && saved_bytes >= keep && workspace && workspace_bytes >= need,
               TG_ERR_WORKSPACE);
    return of(launch_scan_backward(*a, *g, saved, workspace, (hipStream_t)stream));
}

tg_status tg_selective_scan_step(const tg_scan_args* a, float* state, int64_t num_slots,
                                 const int32_t* slots, void* stream) {
    TG_REQUIRE(a && a->seqs.seqs >= 0 && num_slots >= 0, TG_ERR_INVALID_ARGUMENT);
    if (a->seqs.seqs == 0) return TG_OK;
    TG_REQUIRE(a->seqs.rows == a->seqs.seqs && !a->seqs.offsets, TG_ERR_INVALID_ARGUMENT);
    TG_CHECK(check_scan(a));
    TG_REQUIRE(a->seqs.seqs * ceil_div(a->D, 64) <= kMaxStepGroups, TG_ERR_UNSUPPORTED);
    // Rows are a step's sequences: only the row strides count.
    tg_scan_args b = *a;
    for (tg_rows* r : {&b.x, &b.dt, &b.B, &b.C, &b.z, &b.y}) r->seq_stride = r->row_stride;
    TG_CHECK(check_scan_inputs(&b));
    TG_CHECK(check_scan_rows(b.y, b.seqs, b.D, elem_bytes(b.dtype), true));
    TG_REQUIRE((slots || a->seqs.seqs <= num_slots) && (state || num_slots == 0),
               TG_ERR_INVALID_ARGUMENT);
    TG_REQUIRE(num_slots < kMaxRows, TG_ERR_UNSUPPORTED);
    TG_REQUIRE(aligned(state, 4) && aligned(slots, 4), TG_ERR_ALIGNMENT);
    return of(launch_scan_step(b, state, num_slots, slots, (hipStream_t)stream));
}

}  // extern "C"
