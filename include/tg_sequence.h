/*
 * tg_sequence.h -- C ABI of the sequence operators of libtgconv.so for AMD
 * Instinct MI355X (gfx950): layer norm, group norm, the short causal convolution
 * with SiLU, the selective state space scan and the gated delta rule, each for
 * prompts, for training (forward and backward) and, where there is a state, for
 * single tokens.
 *
 * Tensors. Activations (x, y, z, dt, B, C, q, k, v, beta and their gradients) share
 * one dtype: TG_F16, TG_BF16 or TG_F32. Parameters, statistics and states of the scan
 * and the delta rule are fp32. All arithmetic and all sums are fp32 or wider (but where
 * the delta rule's text names fewer bits); every activation result is rounded once, to
 * nearest even. Channels are contiguous; a row is one token.
 *
 * Sequences. A batch is dense or packed (tg_seqs):
 *   dense   offsets == NULL: rows = seqs * L, and row l of sequence s of a
 *           tensor t starts at t.p + s*t.seq_stride + l*t.row_stride elements;
 *   packed  offsets = device int32 [seqs + 1], non-decreasing, first 0, last
 *           rows: sequence s is rows offsets[s] .. offsets[s+1]-1 of [rows],
 *           row r at t.p + r*t.row_stride (seq_stride is not read).
 * Sequences of no row and of one row are allowed in a packed batch. The
 * offsets are read on the device only and cut to 0 .. rows there, so wrong
 * ones give wrong results but no access outside the tensors; rows that no
 * sequence covers are not written.
 *
 * Entry points never abort, never throw, never print and never read the
 * process environment. They launch kernels only (no memset, no allocation, no
 * synchronisation) on `stream` (a hipStream_t passed as void*), so they may be
 * captured into a graph. The caller owns every buffer. Outputs must not
 * alias inputs unless the function says so. Results do not depend on
 * scheduling: the same call gives the same bits.
 *
 * Limits, for every function: rows, sequences and state slots below 2^30, up to 2^20
 * channels; more are TG_ERR_UNSUPPORTED, as is what an operator's own text names.
 *
 * Errors, for every function: TG_ERR_INVALID_ARGUMENT for a NULL required
 * pointer or a size, stride or eps out of its range; TG_ERR_UNSUPPORTED for a
 * dtype other than the three or sizes past the stated limits; TG_ERR_ALIGNMENT
 * for a pointer that is not a multiple of its element size;
 * TG_ERR_WORKSPACE for a missing or too small workspace; TG_ERR_HIP when a
 * launch fails. Nothing is launched on any error but the last.
 */
#ifndef TG_SEQUENCE_H
#define TG_SEQUENCE_H

#include <stdint.h>

#include "tg_conv_bn_silu.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows of a tensor; strides in elements. p == NULL: not given. */
typedef struct {
    void *p;
    int64_t seq_stride, row_stride;
} tg_rows;

typedef struct {
    int64_t seqs;           /* >= 1 */
    int64_t rows;           /* all sequences together, >= 0 */
    const int32_t *offsets; /* device [seqs + 1], or NULL: dense */
} tg_seqs;

/* ---- Layer norm -------------------------------------------------------
 *   s = x (+ residual, the sum rounded to dtype)
 *   mean = sum_c s / C, rstd = 1 / sqrt(sum_c (s - mean)^2 / C + eps)
 *   y = (s - mean) * rstd * gamma + beta
 * over each of `rows` rows of C >= 1 channels. x, residual: row strides >= C
 * (or 0: one row for all); y, sum: dense [rows][C]. residual and sum are given
 * together or not at all; sum may alias x or residual (same rows, dense), y
 * the other of the two (or, without a residual, x). beta, and mean with rstd
 * (fp32 [rows], for the backward pass) may be NULL. rows == 0 does nothing. */
tg_status tg_layer_norm(const void *x, int64_t x_stride, const void *residual,
                        int64_t residual_stride, const float *gamma, const float *beta, float eps,
                        int64_t rows, int C, tg_dtype dtype, void *y, void *sum, float *mean,
                        float *rstd, void *stream);

/* Gradients from dy [rows][C] (row stride), s (x, or sum where there was a
 * residual), mean and rstd of the forward pass: with h = (s - mean) * rstd and
 * g = dy * gamma,
 *   dx = rstd * (g - sum_c g / C - h * sum_c (g*h) / C) (+ dsum)
 *   dgamma = sum over rows of dy * h,   dbeta = sum over rows of dy
 * dsum (may be NULL): a gradient that reaches s past the norm. dx, dense
 * [rows][C], is the gradient of x and of the residual alike; it may alias dsum,
 * dy or s (dense). dgamma, dbeta: fp32 [C], written (not added to), dbeta may
 * be NULL. rows == 0 writes zeros there. workspace: from the size query,
 * 16-byte aligned. */
tg_status tg_layer_norm_backward_workspace(int64_t rows, int C, tg_dtype dtype, size_t *bytes);
tg_status tg_layer_norm_backward(const void *dy, int64_t dy_stride, const void *s, int64_t s_stride,
                                 const float *gamma, const float *mean, const float *rstd,
                                 const void *dsum, int64_t dsum_stride, int64_t rows, int C,
                                 tg_dtype dtype, void *dx, float *dgamma, float *dbeta,
                                 void *workspace, size_t workspace_bytes, void *stream);

/* ---- Short causal convolution -----------------------------------------
 * Depthwise over the rows of each sequence, K taps (2 .. 8):
 *   v[t,c] = bias[c] + sum_k w[k,c] * x[t-K+1+k, c],   y = act(v)
 * with act SiLU or none (TG_ACT_SILU, TG_ACT_NONE). x at t < 0 is the
 * sequence's state: initial [seqs][K-1][D], the K-1 rows before the sequence,
 * oldest first; NULL: zeros. final [seqs][K-1][D] (may be NULL) gets the last
 * K-1 rows in the same form; it must not alias initial. w: fp32 [K][D]
 * (taps outside, channels contiguous); bias: fp32 [D] or NULL.
 * Fewer than 2^23 sequences of fewer than 2^28 rows are always taken, as are fewer
 * than 2^24 single tokens; beyond that TG_ERR_UNSUPPORTED where one launch does not
 * hold them. */
typedef struct {
    tg_seqs seqs;
    int D, K;
    tg_dtype dtype;
    tg_activation act;
    tg_rows x, y;
    const float *w, *bias;
    const void *initial;
    void *final;
} tg_causal_conv_args;
tg_status tg_causal_conv(const tg_causal_conv_args *a, void *stream);

/* Gradients. a: the forward call's arguments (y and final are not read). dy,
 * dx: rows like x. dw fp32 [K][D] and dbias fp32 [D] (may be NULL) are written.
 * dfinal [seqs][K-1][D] (may be NULL): gradient of the final states; dinitial
 * [seqs][K-1][D] (may be NULL): gradient of the initial states. */
tg_status tg_causal_conv_backward_workspace(const tg_causal_conv_args *a, size_t *bytes);
tg_status tg_causal_conv_backward(const tg_causal_conv_args *a, tg_rows dy, tg_rows dx, float *dw,
                                  float *dbias, const void *dfinal, void *dinitial,
                                  void *workspace, size_t workspace_bytes, void *stream);

/* One token for each of n sequences, x [n][D] (row stride), y [n][D] dense:
 * y as above from the K-1 state rows and x, and the state moves on by one row
 * in place. state [num_slots][K-1][D] dense; sequence i keeps its state in
 * slot slots[i] (device int32 [n]; NULL: slot i, then n <= num_slots). Slots
 * below 0 or past the end mark rows without a sequence: y there is zero and
 * no state changes. Two sequences must not share a slot. y may alias x (dense). */
tg_status tg_causal_conv_step(const void *x, int64_t x_stride, void *state, int64_t num_slots,
                              const int32_t *slots, const float *w, const float *bias, int64_t n,
                              int D, int K, tg_dtype dtype, tg_activation act, void *y,
                              void *stream);

/* ---- Selective state space scan ---------------------------------------
 * For each sequence and channel c, with N (1 .. 128) states and h[-1] the
 * initial state (or zeros):
 *   d[t]   = dt[t,c] + dt_bias[c], through softplus log(1 + e^d) if softplus
 *   h[t,n] = exp(d[t] * A[c,n]) * h[t-1,n] + d[t] * B[t,g,n] * x[t,c]
 *   v[t]   = sum_n C[t,g,n] * h[t,n] + D[c] * x[t,c]
 *   y[t,c] = v[t] * silu(z[t,c])      (v[t] where z is not given)
 * A step d of 0 keeps the state for any A, -inf included. Decays exp(d*A) above 1
 * are taken as they are, those below 2^-126 as 0; a channel's state that is infinite
 * or NaN makes its y infinite or NaN from there on.
 * B and C are shared by the D/G channels of a group g = c / (D/G); a row of
 * B or C is [G][N], contiguous. A fp32 [D][N]; D_skip, dt_bias fp32 [D] or
 * NULL; initial, final fp32 [seqs][D][N] or NULL. TG_ERR_UNSUPPORTED for row
 * strides of 2^25 elements or more, 2^26 or more pairs of a sequence and 16
 * channels, and in the backward pass for 2^29 or more values of dB. */
typedef struct {
    tg_seqs seqs;
    int D, N, G;
    tg_dtype dtype;
    int softplus;
    tg_rows x, dt, B, C, z, y;
    const float *A, *D_skip, *dt_bias;
    const float *initial;
    float *final;
} tg_scan_args;

/* workspace_bytes: scratch of tg_selective_scan (may be 0). saved_bytes: what
 * the forward pass keeps for the backward pass (states at regular steps).
 * backward_bytes: scratch of tg_selective_scan_backward. Any may be NULL. */
tg_status tg_selective_scan_sizes(const tg_scan_args *a, size_t *workspace_bytes,
                                  size_t *saved_bytes, size_t *backward_bytes);
/* saved (fp32, may be NULL): filled for the backward pass. y may be x, dt or z
 * themselves (same address and strides), which a backward pass then lacks. */
tg_status tg_selective_scan(const tg_scan_args *a, void *workspace, size_t workspace_bytes,
                            void *saved, size_t saved_bytes, void *stream);

/* Gradients, all written: dx, ddt, dz as rows like x; dB, dC rows [G][N];
 * dA fp32 [D][N]; dD, ddt_bias fp32 [D] (NULL where not wanted; dz NULL iff z
 * is); dinitial fp32 [seqs][D][N] or NULL. dfinal (or NULL): the gradient of
 * the final states. a: the forward call's arguments (y, final are not read;
 * initial only enters through saved). */
typedef struct {
    tg_rows dy;
    const float *dfinal;
    tg_rows dx, ddt, dB, dC, dz;
    float *dA, *dD, *ddt_bias, *dinitial;
} tg_scan_grads;
tg_status tg_selective_scan_backward(const tg_scan_args *a, const tg_scan_grads *g,
                                     const void *saved, size_t saved_bytes, void *workspace,
                                     size_t workspace_bytes, void *stream);

/* One token for each of n sequences: x, dt, z [n][D] and B, C [n][G][N] by
 * row stride (seqs.seqs = seqs.rows = n, offsets NULL; seq_stride is not
 * read), y likewise; it may be x, dt or z themselves. state fp32
 * [num_slots][D][N], updated in place; slots as in tg_causal_conv_step. initial
 * and final are not read. TG_ERR_UNSUPPORTED for 2^24 or more pairs of a
 * sequence and 64 channels. */
tg_status tg_selective_scan_step(const tg_scan_args *a, float *state, int64_t num_slots,
                                 const int32_t *slots, void *stream);

/* ---- Gated delta rule --------------------------------------------------
 * For each sequence and value head h, with a K x V matrix S, the initial state
 * (or zeros) before the first token, and hk = h / (HV/HK) its key head:
 *   d  = dt[t,h] + dt_bias[h], through softplus if softplus;  b = beta[t,h],
 *        through the logistic function if sigmoid
 *   q, k = q[t,hk], k[t,hk], divided by sqrt(sum of squares + 1e-6) if normalize
 *   S  = exp(d * A[h]) * S;   u = b * (v[t,h] - k S);   S = S + k u^T
 *   y[t,h] = scale * q S
 * q and k rows [HK][K], v and y rows [HV][V], dt and beta rows [HV], each
 * contiguous; K 1 .. 256. A fp32 [HV]; dt_bias fp32 [HV] or NULL; initial, final
 * fp32 [seqs][HV][K][V] or NULL.
 * A sum of squares of q or k past fp32 is infinite and makes NaN.
 * A step d of 0 keeps the state for any A, -inf included; decays below 2^-126 are
 * taken as 0, and have no gradient; nor has an infinite A, or dt through it. Decays
 * above 1 are taken as they are while the product over any tokens in a row is within
 * fp32; past it results are infinite or NaN. States and what lies between enter the
 * products with 24 bits, what only reaches y, and the pairs of tokens in dq and dk, of
 * 16-bit tensors with 17.
 * A NaN or infinite value of a token makes its own y and, but for q, those of the later
 * tokens of its head infinite or NaN (of v: in its column), and no other. In the
 * gradients it may reach any token of its sequence and key head.
 * TG_ERR_UNSUPPORTED for K > 256, row strides of 2^25 elements or more, 2^24 or more
 * pairs of a value head and 64 tokens of a sequence (32 for fp16, fp32 and K > 128; 2^23
 * pairs for K > 128; a packed batch counts rows/64 + seqs for each head), and 2^23 or more of a sequence and value head (a multiple of 8 of
 * them) and 32 columns of V (16 for fp32 with K > 128); in a step 2^24 or more of a
 * sequence, value head and 32 columns. */
typedef struct {
    tg_seqs seqs;
    int HK, HV, K, V;
    tg_dtype dtype;
    int softplus, sigmoid, normalize;
    float scale;
    tg_rows q, k, v, dt, beta, y;
    const float *A, *dt_bias;
    const float *initial;
    float *final;
} tg_delta_args;

/* As tg_selective_scan_sizes. */
tg_status tg_gated_delta_rule_sizes(const tg_delta_args *a, size_t *workspace_bytes,
                                    size_t *saved_bytes, size_t *backward_bytes);
/* saved (fp32, may be NULL): filled for the backward pass with the state before
 * each 64 (32) tokens and their corrections. y may be v itself (same address and
 * strides), which a backward pass then lacks. */
tg_status tg_gated_delta_rule(const tg_delta_args *a, void *workspace, size_t workspace_bytes,
                              void *saved, size_t saved_bytes, void *stream);

/* Gradients, all written: dq, dk, dv, ddt, dbeta as rows like q, k, v, dt, beta;
 * dA, ddt_bias fp32 [HV] (ddt_bias may be NULL); dinitial fp32
 * [seqs][HV][K][V] or NULL. dfinal (or NULL): the gradient of the final states.
 * a: the forward call's arguments (y, final are not read; initial only enters
 * through saved). */
typedef struct {
    tg_rows dy;
    const float *dfinal;
    tg_rows dq, dk, dv, ddt, dbeta;
    float *dA, *ddt_bias, *dinitial;
} tg_delta_grads;
tg_status tg_gated_delta_rule_backward(const tg_delta_args *a, const tg_delta_grads *g,
                                       const void *saved, size_t saved_bytes, void *workspace,
                                       size_t workspace_bytes, void *stream);

/* One token for each of n sequences, rows by row stride as in
 * tg_selective_scan_step; state fp32 [num_slots][HV][K][V], updated in place; slots as in
 * tg_causal_conv_step. */
tg_status tg_gated_delta_rule_step(const tg_delta_args *a, float *state, int64_t num_slots,
                                   const int32_t *slots, void *stream);

/* ---- Group norm --------------------------------------------------------
 * Over each n and group g of C/G neighbouring channels of x [N][L][C], L rows (the
 * pixels of a map; 1: the heads of a token) for each n:
 *   mean = sum x / (L*C/G), rstd = 1 / sqrt(sum (x - mean)^2 / (L*C/G) + eps)
 *   v = (x - mean) * rstd * gamma[c] + beta[c]
 *   y = act(v) * silu(z)         (act(v) where z is not given)
 * with act SiLU or none (TG_ACT_SILU, TG_ACT_NONE). Rows of x and z are a row
 * stride >= C apart (or 0: one row for all); y is dense and may be x or z
 * themselves (dense). beta, and mean with rstd (fp32 [N][G], for the backward
 * pass) may be NULL. N == 0 does nothing; L >= 1. A group's sum of squared distances to
 * its mean past fp32 is infinite or NaN, as is a sum of x past it where L is 1. TG_ERR_UNSUPPORTED for more than
 * 4096 groups, or L or N*L of 2^30 or more, or N past 2^24 where a group has more than
 * 256 channels or L is not 1. */
typedef struct {
    int64_t N, L;
    int C, G;
    tg_dtype dtype;
    tg_activation act;
    float eps;
    const void *x;
    int64_t x_stride;
    const void *z;
    int64_t z_stride;
    const float *gamma, *beta;
    void *y;
    float *mean, *rstd;
} tg_group_norm_args;

/* Scratch of tg_group_norm (may be 0) and of its backward pass; either may be NULL. */
tg_status tg_group_norm_sizes(const tg_group_norm_args *a, size_t *workspace_bytes,
                              size_t *backward_bytes);
tg_status tg_group_norm(const tg_group_norm_args *a, void *workspace, size_t workspace_bytes,
                        void *stream);

/* Gradients. a: the forward call's arguments (y is not read), with its mean and
 * rstd, which are required. dy by row stride; dx, dz dense (dz NULL iff z is): dx may
 * be x or dy, dz may be z or the other of dx's two (dense). dgamma, dbeta fp32 [C],
 * written; dbeta may be NULL. N == 0 writes zeros there. */
typedef struct {
    const void *dy;
    int64_t dy_stride;
    void *dx, *dz;
    float *dgamma, *dbeta;
} tg_group_norm_grads;
tg_status tg_group_norm_backward(const tg_group_norm_args *a, const tg_group_norm_grads *g,
                                 void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TG_SEQUENCE_H */
