// seq_norm.hip -- layer norm, forward and backward (tg_layer_norm,
// tg_layer_norm_backward), with an optional residual sum before it.
//
// Both passes are bound by HBM: a few operations for each element read or
// written. So each element is read once and held in registers: TPR threads
// (one wave to sixteen) share a row, a thread holds NV vectors of V
// elements of it, V as wide (up to 16 bytes) as the alignment of C, the
// strides and the pointers allows. The statistics are two sums over the
// held values, the mean first and then the squared distances from it: the
// one-pass form (sum of squares minus square of the sum) cancels when the
// mean is large against the spread. Sums are fp32, over at most 16 values in a
// thread (C / 1024 where a row is too long to be held) and a tree over the threads.
//
// A workgroup walks over rows with gamma and beta in registers: reading them
// for every row would be four bytes each next to two of x. Rows too long for
// the held form take the looped kernels, which read
// the row again from the cache.
//
// Backward: the column sums (dgamma, dbeta) run down the rows while dx runs
// along them. Each thread owns the same columns of every row of its
// workgroup and adds them up in registers; the workgroup's partial sums go to the
// workspace and a second kernel adds the workgroups' in a fixed order, so the
// result does not depend on scheduling (atomics would).
#include <type_traits>

#include "seq_device.hpp"
#include "seq_internal.hpp"

namespace tg {
namespace {

constexpr int kColThreads = 16;  // row phases of the column sums

// Sum over the TPR threads of a row, in every thread. red: 16 floats of LDS
// for this use alone until the next barrier.
template <int TPR>
__device__ __forceinline__ float row_total(float v, float* red) {
    v = wave_sum(v);
    if constexpr (TPR > 64) {
        const int w = threadIdx.x >> 6, first = w & ~(TPR / 64 - 1);
        if ((threadIdx.x & 63) == 0) red[w] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) v += red[first + i];
    }
    return v;
}

// Two sums at once, in every thread of the row. red: two rows of 16 floats.
template <int TPR>
__device__ __forceinline__ void row_totals(float& u, float& v, float (*red)[16]) {
    u = wave_sum(u);
    v = wave_sum(v);
    if constexpr (TPR > 64) {
        const int w = threadIdx.x >> 6, first = w & ~(TPR / 64 - 1);
        if ((threadIdx.x & 63) == 0) red[0][w] = u, red[1][w] = v;
        __syncthreads();
        u = v = 0.0f;
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) u += red[0][first + i], v += red[1][first + i];
    }
}

struct NormFwd {
    const void *x, *res;
    int64_t xs, rs;
    const float *gamma, *beta;
    float eps;
    int64_t rows;
    int C;
    void *y, *sum;
    float *mean, *rstd;
};

template <typename T, int V, int TPR, int NV>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void norm_fwd(const NormFwd a) {
    constexpr int kBlock = TPR > 256 ? TPR : 256;
    constexpr int RPB = kBlock / TPR;
    __shared__ float red[2][16];
    const int i = threadIdx.x % TPR, C = a.C;
    float ga[NV][V], be[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * TPR + i) * V;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            ga[j][e] = c < C ? a.gamma[c + e] : 0.0f;
            be[j][e] = c < C && a.beta ? a.beta[c + e] : 0.0f;
        }
    }
    const float inv = 1.0f / (float)C;
    Vec<T, V> rx[NV], rr[NV];
    const auto fetch = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + i) * V;
            if (c < C) {
                rx[j].load((const T*)a.x + row * a.xs + c);
                if (a.res) rr[j].load((const T*)a.res + row * a.rs + c);
            }
        }
    };
    // The barriers of a row that several waves share have to match: all groups of the
    // workgroup go round as often as its first, those past the last row idly.
    const int64_t step = (int64_t)gridDim.x * RPB;
    const int grp = threadIdx.x / TPR;
    int64_t first = (int64_t)blockIdx.x * RPB;
    if (first + grp < a.rows) fetch(first + grp);
    for (; first < a.rows; first += step) {
        const int64_t row = first + grp;
        const int D = row < a.rows ? C : 0;  // this group's channels
        float v[NV][V], s = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + i) * V;
            if (c < D) {
                rx[j].values(v[j]);
                if (a.res) {
                    float r[V];
                    rr[j].values(r);
                    // The statistics are those of the rounded sum: it is what the next
                    // block and the backward pass read.
#pragma unroll
                    for (int e = 0; e < V; ++e) v[j][e] = (float)(T)(v[j][e] + r[e]);
                    store_f32<T, V>((T*)a.sum + row * C + c, v[j]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) v[j][e] = 0.0f;
            }
        }
        // The next row arrives while this one is reduced and written.
        if (row + step < a.rows) fetch(row + step);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) s += v[j][e];
        const float mean = row_total<TPR>(s, red[0]) * inv;
        float q = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const bool in = (j * TPR + i) * V < D;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float d = in ? v[j][e] - mean : 0.0f;
                v[j][e] = d;
                q = __builtin_fmaf(d, d, q);
            }
        }
        const float var = row_total<TPR>(q, red[1]) * inv;
        const float rstd = 1.0f / sqrtf(var + a.eps);
        if (i < D && i == 0 && a.mean) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + i) * V;
            if (c < D) {
                float o[V];
#pragma unroll
                for (int e = 0; e < V; ++e)
                    o[e] = __builtin_fmaf(v[j][e] * rstd, ga[j][e], be[j][e]);
                store_f32<T, V>((T*)a.y + row * C + c, o);
            }
        }
    }
}

// Rows of any length: 1024 threads read the row three times.
template <typename T>
__global__ __launch_bounds__(1024) void norm_fwd_long(const NormFwd a) {
    __shared__ float red[2][16];
    const int i = threadIdx.x, C = a.C;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* xp = (const T*)a.x + row * a.xs;
        const T* rp = (const T*)a.res + row * a.rs;
        T* sp = (T*)a.sum + row * C;
        float s = 0.0f;
        for (int c = i; c < C; c += 1024) {
            float v = (float)xp[c];
            if (a.res) {
                const T t = (T)(v + (float)rp[c]);
                sp[c] = t;
                v = (float)t;
            }
            s += v;
        }
        const T* vp = a.res ? sp : xp;  // each thread reads back what it wrote itself
        const float mean = row_total<1024>(s, red[0]) / (float)C;
        float q = 0.0f;
        for (int c = i; c < C; c += 1024) {
            const float d = (float)vp[c] - mean;
            q = __builtin_fmaf(d, d, q);
        }
        const float rstd = 1.0f / sqrtf(row_total<1024>(q, red[1]) / (float)C + a.eps);
        if (i == 0 && a.mean) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
        for (int c = i; c < C; c += 1024)
            ((T*)a.y)[row * C + c] = (T)__builtin_fmaf(((float)vp[c] - mean) * rstd, a.gamma[c],
                                                       a.beta ? a.beta[c] : 0.0f);
    }
}

struct NormBwd {
    const void *dy, *s, *dsum;
    int64_t dys, ss, dss;
    const float *gamma, *mean, *rstd;
    int64_t rows;
    int C;
    void* dx;
    float* part;  // [gridDim.x][2][C]: dgamma, dbeta of a workgroup's rows
};

template <typename T, int V, int TPR, int NV>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void norm_bwd(const NormBwd a) {
    constexpr int kBlock = TPR > 256 ? TPR : 256;
    constexpr int RPB = kBlock / TPR;
    __shared__ float red[4][16];
    const int i = threadIdx.x % TPR, grp = threadIdx.x / TPR, C = a.C;
    float ga[NV][V], dg[NV][V], db[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * TPR + i) * V;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            ga[j][e] = c < C ? a.gamma[c + e] : 0.0f;
            dg[j][e] = db[j][e] = 0.0f;
        }
    }
    const float inv = 1.0f / (float)C;
    int flip = 0;  // two sets of sums: one row's are read while the next's are written
    Vec<T, V> rg[NV], rs[NV], rd[NV];
    float rmean = 0.0f, rrstd = 0.0f;
    const auto fetch = [&](int64_t row) {
        rmean = a.mean[row];
        rrstd = a.rstd[row];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + i) * V;
            if (c < C) {
                rg[j].load((const T*)a.dy + row * a.dys + c);
                rs[j].load((const T*)a.s + row * a.ss + c);
                if (a.dsum) rd[j].load((const T*)a.dsum + row * a.dss + c);
            }
        }
    };
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t first = (int64_t)blockIdx.x * RPB;
    if (first + grp < a.rows) fetch(first + grp);
    for (; first < a.rows; first += step) {  // barriers as in the forward pass
        const int64_t row = first + grp;
        const int D = row < a.rows ? C : 0;
        const float mean = rmean, rstd = rrstd;
        float g[NV][V], h[NV][V], s1 = 0.0f, s2 = 0.0f;
        Vec<T, V> add[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + i) * V;
            add[j] = rd[j];
            if (c < D) {
                rg[j].values(g[j]);
                rs[j].values(h[j]);
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) g[j][e] = 0.0f, h[j][e] = mean;
            }
        }
        // The next row arrives while this one is reduced and written.
        if (row + step < a.rows) fetch(row + step);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                h[j][e] = (h[j][e] - mean) * rstd;
                dg[j][e] = __builtin_fmaf(g[j][e], h[j][e], dg[j][e]);
                db[j][e] += g[j][e];
                g[j][e] *= ga[j][e];
                s1 += g[j][e];
                s2 = __builtin_fmaf(g[j][e], h[j][e], s2);
            }
        row_totals<TPR>(s1, s2, red + flip);
        flip ^= 2;
        const float m1 = s1 * inv, m2 = s2 * inv;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + i) * V;
            if (c < D) {
                float o[V];
#pragma unroll
                for (int e = 0; e < V; ++e)
                    o[e] = rstd * (g[j][e] - __builtin_fmaf(h[j][e], m2, m1));
                if (a.dsum) {
                    float r[V];
                    add[j].values(r);
#pragma unroll
                    for (int e = 0; e < V; ++e) o[e] += r[e];
                }
                store_f32<T, V>((T*)a.dx + row * C + c, o);
            }
        }
    }
    // The row groups of the workgroup one after another, then one row of
    // partial sums for the workgroup.
    float* part = a.part + (int64_t)blockIdx.x * 2 * C;
    if constexpr (RPB > 1) {
        __shared__ float acc[RPB - 1][2 * V * TPR];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            __syncthreads();
            if (grp > 0)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    acc[grp - 1][(2 * e) * TPR + i] = dg[j][e];
                    acc[grp - 1][(2 * e + 1) * TPR + i] = db[j][e];
                }
            __syncthreads();
            if (grp == 0)
#pragma unroll
                for (int e = 0; e < V; ++e)
#pragma unroll
                    for (int r = 0; r < RPB - 1; ++r) {
                        dg[j][e] += acc[r][(2 * e) * TPR + i];
                        db[j][e] += acc[r][(2 * e + 1) * TPR + i];
                    }
        }
    }
    if (grp == 0)
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + i) * V;
            if (c < C)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    part[c + e] = dg[j][e];
                    part[C + c + e] = db[j][e];
                }
        }
}

// Rows of any length. The column sums live in the workspace: a workgroup
// owns its row of it, and a thread its columns.
template <typename T>
__global__ __launch_bounds__(1024) void norm_bwd_long(const NormBwd a) {
    __shared__ float red[2][16];
    const int i = threadIdx.x, C = a.C;
    float* part = a.part + (int64_t)blockIdx.x * 2 * C;
    for (int c = i; c < C; c += 1024) part[c] = part[C + c] = 0.0f;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* gp = (const T*)a.dy + row * a.dys;
        const T* sp = (const T*)a.s + row * a.ss;
        const float mean = a.mean[row], rstd = a.rstd[row];
        float s1 = 0.0f, s2 = 0.0f;
        for (int c = i; c < C; c += 1024) {
            const float d = (float)gp[c], h = ((float)sp[c] - mean) * rstd, g = d * a.gamma[c];
            part[c] = __builtin_fmaf(d, h, part[c]);
            part[C + c] += d;
            s1 += g;
            s2 = __builtin_fmaf(g, h, s2);
        }
        row_totals<1024>(s1, s2, red);
        const float m1 = s1 / (float)C, m2 = s2 / (float)C;
        for (int c = i; c < C; c += 1024) {
            const float d = (float)gp[c], h = ((float)sp[c] - mean) * rstd;
            float o = rstd * (d * a.gamma[c] - __builtin_fmaf(h, m2, m1));
            if (a.dsum) o += (float)((const T*)a.dsum)[row * a.dss + c];
            ((T*)a.dx)[row * C + c] = (T)o;
        }
        __syncthreads();  // red is written again by the next row
    }
}

// Column sums of [P][M]: 64 columns for each workgroup, 16 row phases.
__global__ __launch_bounds__(64 * kColThreads) void column_sums(const float* part, int P,
                                                                int64_t M, float* out,
                                                                int64_t split, float* out2) {
    __shared__ float red[kColThreads][64];
    const int l = threadIdx.x & 63, ph = threadIdx.x >> 6;
    const int64_t m = (int64_t)blockIdx.x * 64 + l;
    float s = 0.0f;
    if (m < M)
#pragma unroll 8
        for (int p = ph; p < P; p += kColThreads) s += part[(int64_t)p * M + m];
    red[ph][l] = s;
    __syncthreads();
    if (ph == 0 && m < M) {
        s = 0.0f;
#pragma unroll
        for (int k = 0; k < kColThreads; ++k) s += red[k][l];
        float* o = m < split ? out : out2;
        if (o) o[m < split ? m : m - split] = s;
    }
}

// Which numbers of threads for a row (tpr) and of vectors in a thread (nv) are
// built. A thread holds at most 8 values (16 for the longest rows): with their
// gamma and beta, or (backward) five such sets, and the next row on its way,
// that leaves five to eight waves on a SIMD, which counts for more than a row's
// barriers: 16384 x 2048 bf16 forward and backward took 165 us with a wave and 32
// values for each row, 113 us with 256 threads and 8 values.
constexpr bool shape_used(int V, int tpr, int nv, bool bwd) {
    if (V >= 4) return tpr < 1024 ? nv == 1 : nv * V <= (bwd ? 8 : 16);
    if (tpr == 128 || tpr == 512) return false;
    const int most = V == 1 ? 8 : tpr == 1024 && !bwd ? 8 : 4;
    return nv <= most && (tpr == 64 || nv >= (V == 1 ? 4 : 2));
}

// The fewest threads that hold C elements in vectors of V; tpr 0: too long
// for the held form.
struct Shape {
    int tpr, nv;
};
Shape norm_shape(int C, int V, bool bwd) {
    const int64_t n = ceil_div(C, V);
    for (int tpr : {64, 128, 256, 512, 1024})
        for (int nv = 1; nv <= 8; nv *= 2)
            if (shape_used(V, tpr, nv, bwd) && n <= (int64_t)tpr * nv) return {tpr, nv};
    return {0, 0};
}

// Workgroups of the forward pass: 2048 where a wave holds a row (25088 x 363
// fp32: 13 us; 1024 take 19), else 1024 threads on each compute unit (8192 x
// 4096 bf16: 57 us; half as many take 64, twice as many 61).
int norm_grid(int64_t rows, int tpr) {
    const int rpb = tpr >= 256 ? 1 : 256 / tpr;
    const int64_t need = ceil_div(rows, rpb), most = tpr == 64 ? 2048 : tpr < 256 ? 1024 : 256 * (1024 / tpr);
    return (int)(need < most ? need : most);
}

template <typename T, int V, int TPR, int NV>
void norm_one(int grid, const NormFwd& a, hipStream_t st) {
    norm_fwd<T, V, TPR, NV><<<grid, TPR > 256 ? TPR : 256, 0, st>>>(a);
}
template <typename T, int V, int TPR, int NV>
void norm_one(int grid, const NormBwd& a, hipStream_t st) {
    norm_bwd<T, V, TPR, NV><<<grid, TPR > 256 ? TPR : 256, 0, st>>>(a);
}
// The kernel for tpr threads and nv vectors, if it is built.
template <typename T, int V, int TPR, int NV, typename Args>
void norm_try(const Shape& sh, int grid, const Args& a, hipStream_t st) {
    if constexpr (shape_used(V, TPR, NV, std::is_same<Args, NormBwd>::value))
        if (sh.tpr == TPR && sh.nv == NV) norm_one<T, V, TPR, NV>(grid, a, st);
}
template <typename T, int V, int TPR, typename Args>
void norm_nv(const Shape& sh, int grid, const Args& a, hipStream_t st) {
    norm_try<T, V, TPR, 1>(sh, grid, a, st);
    norm_try<T, V, TPR, 2>(sh, grid, a, st);
    norm_try<T, V, TPR, 4>(sh, grid, a, st);
    norm_try<T, V, TPR, 8>(sh, grid, a, st);
}
template <typename T, int V, typename Args>
void norm_tpr(const Shape& sh, int grid, const Args& a, hipStream_t st) {
    norm_nv<T, V, 64>(sh, grid, a, st);
    norm_nv<T, V, 128>(sh, grid, a, st);
    norm_nv<T, V, 256>(sh, grid, a, st);
    norm_nv<T, V, 512>(sh, grid, a, st);
    norm_nv<T, V, 1024>(sh, grid, a, st);
}
template <typename T, typename Args>
void norm_launch(int V, const Shape& sh, int grid, const Args& a, hipStream_t st) {
    if constexpr (sizeof(T) == 2)
        if (V == 8) return norm_tpr<T, 8>(sh, grid, a, st);
    if (V == 4) norm_tpr<T, 4>(sh, grid, a, st);
    else if (V == 2) norm_tpr<T, 2>(sh, grid, a, st);
    else norm_tpr<T, 1>(sh, grid, a, st);
}

template <typename T>
void fwd_typed(int V, const NormFwd& a, hipStream_t st) {
    const Shape sh = norm_shape(a.C, V, false);
    if (!sh.tpr) {
        norm_fwd_long<T><<<norm_grid(a.rows, 1024), 1024, 0, st>>>(a);
        return;
    }
    const int grid = norm_grid(a.rows, sh.tpr);
    norm_launch<T>(V, sh, grid, a, st);
}
template <typename T>
void bwd_typed(int V, int grid, const NormBwd& a, hipStream_t st) {
    const Shape sh = norm_shape(a.C, V, true);
    if (!sh.tpr) norm_bwd_long<T><<<grid, 1024, 0, st>>>(a);
    else norm_launch<T>(V, sh, grid, a, st);
}

// Workgroups of the backward pass, one row of partial sums each (16384 x 2048
// bf16, forward and backward: 111 us; 384 workgroups 123, 768 and 1024: 115, 128).
int bwd_grid(int64_t rows) {
    const int64_t need = ceil_div(rows, 4);
    return (int)(need < 512 ? need : 512);
}

}  // namespace

hipError_t launch_column_sums(const float* part, int P, int64_t M, float* out, int64_t split,
                              float* out2, hipStream_t st) {
    column_sums<<<(unsigned)ceil_div(M, 64), 64 * kColThreads, 0, st>>>(part, P, M, out, split,
                                                                         out2);
    return hipGetLastError();
}

hipError_t launch_layer_norm(const void* x, int64_t xs, const void* res, int64_t rs,
                             const float* gamma, const float* beta, float eps, int64_t rows, int C,
                             tg_dtype dt, void* y, void* sum, float* mean, float* rstd,
                             hipStream_t st) {
    const size_t e = elem_bytes(dt);
    Widest w;
    w.len(C), w.len(xs), w.ptr(x, e), w.ptr(y, e);
    if (res) w.len(rs), w.ptr(res, e), w.ptr(sum, e);
    const int V = w.width((int)(16 / e));
    const NormFwd a{x, res, xs, rs, gamma, beta, eps, rows, C, y, sum, mean, rstd};
    if (dt == TG_F32) fwd_typed<float>(V, a, st);
    else if (dt == TG_BF16) fwd_typed<bf16>(V, a, st);
    else fwd_typed<f16>(V, a, st);
    return hipGetLastError();
}

size_t layer_norm_backward_bytes(int64_t rows, int C) {
    return (size_t)bwd_grid(rows) * 2 * C * sizeof(float);
}

hipError_t launch_layer_norm_backward(const void* dy, int64_t dys, const void* s, int64_t ss,
                                      const float* gamma, const float* mean, const float* rstd,
                                      const void* dsum, int64_t dss, int64_t rows, int C,
                                      tg_dtype dt, void* dx, float* dgamma, float* dbeta, void* ws,
                                      hipStream_t st) {
    const size_t e = elem_bytes(dt);
    Widest w;
    w.len(C), w.len(dys), w.len(ss), w.ptr(dy, e), w.ptr(s, e), w.ptr(dx, e);
    if (dsum) w.len(dss), w.ptr(dsum, e);
    const int V = w.width((int)(16 / e)), grid = bwd_grid(rows);
    const NormBwd a{dy, s, dsum, dys, ss, dss, gamma, mean, rstd, rows, C, dx, (float*)ws};
    if (rows > 0) {
        if (dt == TG_F32) bwd_typed<float>(V, grid, a, st);
        else if (dt == TG_BF16) bwd_typed<bf16>(V, grid, a, st);
        else bwd_typed<f16>(V, grid, a, st);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return launch_column_sums((const float*)ws, rows > 0 ? grid : 0, 2 * (int64_t)C, dgamma, C,
                              dbeta, st);
}

}  // namespace tg
