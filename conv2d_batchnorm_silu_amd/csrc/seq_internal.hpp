// seq_internal.hpp -- launchers of the sequence operators (tg_sequence.h),
// called by seq_api.hip with checked arguments.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "tg_sequence.h"

namespace tg {

inline size_t elem_bytes(tg_dtype d) { return d == TG_F32 ? 4 : 2; }
inline size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The widest vector of `cap` elements or fewer (a power of two) that divides
// every length or stride, and whose bytes divide every address.
struct Widest {
    uint64_t bits = 0;  // or of all lengths (elements) and addresses (elements)
    void len(int64_t n) { bits |= (uint64_t)n; }
    void ptr(const void* p, size_t elem) { bits |= (uint64_t)((uintptr_t)p / elem); }
    int width(int cap) const {
        int v = cap;
        while (v > 1 && (bits & (uint64_t)(v - 1))) v >>= 1;
        return v;
    }
};

hipError_t launch_layer_norm(const void* x, int64_t xs, const void* res, int64_t rs,
                             const float* gamma, const float* beta, float eps, int64_t rows, int C,
                             tg_dtype dt, void* y, void* sum, float* mean, float* rstd,
                             hipStream_t st);
size_t layer_norm_backward_bytes(int64_t rows, int C);
hipError_t launch_layer_norm_backward(const void* dy, int64_t dys, const void* s, int64_t ss,
                                      const float* gamma, const float* mean, const float* rstd,
                                      const void* dsum, int64_t dss, int64_t rows, int C,
                                      tg_dtype dt, void* dx, float* dgamma, float* dbeta, void* ws,
                                      hipStream_t st);

hipError_t launch_causal_conv(const tg_causal_conv_args& a, hipStream_t st);
size_t causal_conv_backward_bytes(const tg_causal_conv_args& a);
hipError_t launch_causal_conv_backward(const tg_causal_conv_args& a, const tg_rows& dy,
                                       const tg_rows& dx, float* dw, float* dbias,
                                       const void* dfinal, void* dinitial, void* ws,
                                       hipStream_t st);
hipError_t launch_causal_conv_step(const void* x, int64_t xs, void* state, int64_t num_slots,
                                   const int32_t* slots, const float* w, const float* bias,
                                   int64_t n, int D, int K, tg_dtype dt, bool silu, void* y,
                                   hipStream_t st);

void scan_sizes(const tg_scan_args& a, size_t* work, size_t* saved, size_t* backward);
int64_t scan_sum_groups(const tg_scan_args& a);  // workgroups of the backward pass's sums
hipError_t launch_scan(const tg_scan_args& a, void* ws, void* saved, hipStream_t st);
hipError_t launch_scan_backward(const tg_scan_args& a, const tg_scan_grads& g, const void* saved,
                                void* ws, hipStream_t st);
hipError_t launch_scan_step(const tg_scan_args& a, float* state, int64_t num_slots,
                            const int32_t* slots, hipStream_t st);

// out[m] = sum over p < P of part[p*M + m], in a fixed order (seq_norm.hip).
// Columns from `split` on go to out2; either may be NULL (dropped).
hipError_t launch_column_sums(const float* part, int P, int64_t M, float* out, int64_t split,
                              float* out2, hipStream_t st);

}  // namespace tg
