// seq_group_norm.hip -- group norm with an activation and a gate over rows of
// channels, forward and backward (tg_group_norm, tg_group_norm_backward).
//
// Bound by HBM: a dozen operations for each element read. Two forms:
//
// Heads (L == 1, a group no longer than 64 lanes hold): the lanes of a group
// hold it in registers, so x (in the backward pass dy, x and z) is read once. A lane
// keeps its channels from row to row, with gamma and beta in registers and, in the
// backward pass, the sums for their gradients.
//
// Maps (L > 1, or long groups): the rows of an n are cut into chunks, a workgroup
// for each. One kernel takes the chunks' statistics, the next joins those of its n
// (a few hundred bytes from L2) and normalises, reading x again from the caches
// where it is not larger than they are. Statistics: a thread adds up x - x0 and its
// square over up to 32 rows, x0 the first of them; as x0 is one of the samples, its
// distance from their mean is at most the root of the sum of squares that is
// wanted, so the subtraction costs at most a factor 32 of fp32's precision, and
// nothing where the mean is large. Sets are joined by their counts, means and squares.
//
// Sums across workgroups go through the workspace and are added in a fixed order.
//
// 16384 tokens of 16 heads of 128, gate, bf16: forward 50 us (4.0 TB/s), backward 70 (4.8).
// 32 maps of 56 x 56 x 256, fp16: statistics 12 us, the second sweep 31 (3.3 TB/s). Small maps
// are a chain of launches of 7 to 20 us, of which latency (joining the chunks, weights,
// first rows) is the most.
#include "seq_device.hpp"
#include "seq_internal.hpp"

namespace tg {
namespace {

constexpr int kBlockRows = 32;  // rows with one x0
constexpr int kThreads = 256;
constexpr int kAhead = 4;  // rows on their way in a thread
// Chunks of maps whose channels' sums are held at once, 8 bytes for each channel: those of
// all would be four times x for a million n of one row. 16384 rows of 4096 bf16 channels
// take 1045 us in eight launches of 2048 chunks, 968 in one; smaller ones 15 to 20% more,
// so that 64 MB are always held.
constexpr int64_t kMostSums = 2048, kSumBytes = (int64_t)64 << 20;

struct GroupArgs {
    const void *x, *z, *dy;
    int64_t xs, zs, ds;
    const float *gamma, *beta;
    float eps;
    int64_t N, L;
    int C, G, silu;
    void *y, *dz;  // y: dx in the backward pass
    float *mean, *rstd;
    int chunks, rows;      // of an n; rows of a chunk
    float *stats, *cols;   // [N][chunks][G][2]; [units][2][C], sums of dv h and of dv
    int64_t units;         // heads: rows in flight; maps: chunks of a launch of map_sums
    int64_t first;         // the first of these chunks
};

struct Moments {
    float n, mean, m2;
};
__device__ __forceinline__ void join(Moments& a, const Moments& b) {
    // An empty set is no set at mean 0: the distance to it may have no square in fp32.
    if (b.n == 0.0f) return;
    if (a.n == 0.0f) {
        a = b;
        return;
    }
    const float n = a.n + b.n, d = b.mean - a.mean, f = b.n / n;
    a.mean = __builtin_fmaf(d, f, a.mean);
    a.m2 += b.m2 + d * d * a.n * f;
    a.n = n;
}

// y and its factors: a = act(v), and what dy is multiplied by on its way to v.
__device__ __forceinline__ float activation(int silu, float v) {
    return silu ? silu_f32(v) : v;
}
__device__ __forceinline__ void activation_grad(int silu, float v, float& a, float& slope) {
    if (silu) {
        const float s = sigmoid_f32(v);
        a = v * s;
        slope = s * __builtin_fmaf(v, 1.0f - s, 1.0f);
    } else {
        a = v;
        slope = 1.0f;
    }
}

// Threads of a group (a power of two up to 64) when 256 share G groups.
__device__ __forceinline__ int lanes_of_group(int G) {
    int p = 1;
    while (p < 64 && p * 2 * G <= kThreads) p *= 2;
    return p;
}

// ---- maps

// Where a workgroup's threads are: n, the chunk's rows, columns of vectors from
// tx on, TX apart, rows from ty on, TY apart.
template <int V>
struct Place {
    int64_t n, first;
    int chunk, rows, TX, TY, tx, ty;
    __device__ __forceinline__ explicit Place(const GroupArgs& a, int64_t at = blockIdx.x) {
        n = at / a.chunks;
        chunk = (int)(at % a.chunks);
        first = (int64_t)chunk * a.rows;
        rows = (int)(a.L - first < a.rows ? a.L - first : a.rows);
        const int cols = a.C / V;
        TX = cols < kThreads ? cols : kThreads;
        TY = kThreads / TX;
        tx = threadIdx.x % TX;
        ty = threadIdx.x / TX;
    }
};

template <typename T, int V>
__global__ __launch_bounds__(kThreads) void map_stats(const GroupArgs a) {
    __shared__ float sm[3][kThreads];
    const Place<V> p(a);
    const int Cg = a.C / a.G, cols = a.C / V, gv = Cg / V;  // vectors of a group
    const T* x = (const T*)a.x + (p.n * a.L + p.first) * a.xs;
    float* out = a.stats + ((int64_t)blockIdx.x * a.G) * 2;
    // Whole groups at a time: of as many vectors as there are threads, or one group
    // in pieces.
    const int per = gv <= p.TX ? p.TX / gv * gv : p.TX;
    for (int base = 0; base < cols; base += gv <= p.TX ? per : gv) {
        const int width = gv <= p.TX ? imin(per, cols - base) : gv;
        Moments all = {0.0f, 0.0f, 0.0f};
        if (p.ty < p.TY)
            for (int v = p.tx; v < width; v += per) {
                if (p.tx >= per) break;
                const T* xc = x + (base + v) * V;
                for (int r0 = p.ty; r0 < p.rows; r0 += kBlockRows * p.TY) {
                    float k[V], s[V], q[V], t[V];
                    load_f32<T, V>(xc + r0 * a.xs, k);
#pragma unroll
                    for (int e = 0; e < V; ++e) s[e] = q[e] = 0.0f;
                    const int left = (p.rows - r0 + p.TY - 1) / p.TY, m = imin(kBlockRows, left);
                    int i = 1;
                    for (; i + 4 <= m; i += 4) {
                        Vec<T, V> w[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) w[u].load(xc + (int64_t)(r0 + (i + u) * p.TY) * a.xs);
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            w[u].values(t);
#pragma unroll
                            for (int e = 0; e < V; ++e) {
                                const float d = t[e] - k[e];
                                s[e] += d;
                                q[e] = __builtin_fmaf(d, d, q[e]);
                            }
                        }
                    }
                    for (; i < m; ++i) {
                        load_f32<T, V>(xc + (int64_t)(r0 + i * p.TY) * a.xs, t);
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            const float d = t[e] - k[e];
                            s[e] += d;
                            q[e] = __builtin_fmaf(d, d, q[e]);
                        }
                    }
                    // The channels' sets first with each other, all of the same count.
                    const float n = (float)m, inv = 1.0f / n;
                    Moments b = {n * V, 0.0f, 0.0f};
                    float mean[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        mean[e] = __builtin_fmaf(s[e], inv, k[e]);
                        b.mean += (mean[e] - mean[0]) * (1.0f / V);
                        // Not by fmaxf: where squares are infinite, NaN has to stay.
                        const float m2 = q[e] - s[e] * s[e] * inv;
                        b.m2 += m2 < 0.0f ? 0.0f : m2;
                    }
                    b.mean += mean[0];
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float d = mean[e] - b.mean;
                        b.m2 = __builtin_fmaf(d * d, n, b.m2);
                    }
                    join(all, b);
                }
            }
        __syncthreads();
        sm[0][threadIdx.x] = all.n;
        sm[1][threadIdx.x] = all.mean;
        sm[2][threadIdx.x] = all.m2;
        __syncthreads();
        // Threads of a group join what its columns' threads found.
        const int groups = gv <= p.TX ? width / gv : 1, wide = gv <= p.TX ? gv : p.TX;
        const int P = lanes_of_group(groups), lane = threadIdx.x % P;
        for (int g0 = 0; g0 < groups; g0 += kThreads / P) {
            const int g = g0 + threadIdx.x / P;
            Moments m = {0.0f, 0.0f, 0.0f};
            if (g < groups)
                for (int i = lane; i < wide * p.TY; i += P) {
                    const int at = (i / wide) * p.TX + g * wide + i % wide;
                    join(m, Moments{sm[0][at], sm[1][at], sm[2][at]});
                }
            for (int d = 1; d < P; d *= 2)
                join(m, Moments{__shfl_xor(m.n, d), __shfl_xor(m.mean, d), __shfl_xor(m.m2, d)});
            if (g < groups && lane == 0) {
                out[(base / gv + g) * 2] = m.mean;
                out[(base / gv + g) * 2 + 1] = m.m2;
            }
        }
        __syncthreads();
    }
}

// The chunks' statistics of an n joined, by all threads: mean and rstd of group g in
// lds[2g], lds[2g + 1].
__device__ __forceinline__ void join_chunks(const GroupArgs& a, int64_t n, float* lds) {
    const float per = (float)(a.C / a.G);
    const int P = lanes_of_group(a.G), lane = threadIdx.x % P;
    for (int g0 = 0; g0 < a.G; g0 += kThreads / P) {
        const int g = g0 + threadIdx.x / P;
        Moments m = {0.0f, 0.0f, 0.0f};
        if (g < a.G)
            for (int c0 = lane; c0 < a.chunks; c0 += 4 * P) {
                float2 s[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    s[u] = ((const float2*)a.stats)[(n * a.chunks + imin(c0 + u * P, a.chunks - 1)) * a.G + g];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int c = c0 + u * P;
                    const int64_t left = a.L - (int64_t)c * a.rows;
                    if (c < a.chunks)
                        join(m, Moments{per * (float)(left < a.rows ? left : a.rows), s[u].x, s[u].y});
                }
            }
        for (int d = 1; d < P; d *= 2)
            join(m, Moments{__shfl_xor(m.n, d), __shfl_xor(m.mean, d), __shfl_xor(m.m2, d)});
        if (g < a.G && lane == 0) {
            lds[2 * g] = m.mean;
            lds[2 * g + 1] = 1.0f / sqrtf(m.m2 / m.n + a.eps);
        }
    }
    __syncthreads();
}

template <typename T, int V>
__global__ __launch_bounds__(kThreads) void map_apply(const GroupArgs a) {
    extern __shared__ float stat[];
    const Place<V> p(a);
    const int64_t row0 = p.n * a.L + p.first;
    Vec<T, V> x[kAhead], z[kAhead];
    const auto fetch = [&](int v, int r) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (r + u * p.TY < p.rows) {
                const int64_t row = row0 + r + u * p.TY;
                x[u].load((const T*)a.x + row * a.xs + v * V);
                if (a.z) z[u].load((const T*)a.z + row * a.zs + v * V);
            }
    };
    float gamma[V], beta[V];
    const auto weights = [&](int v) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            gamma[e] = a.gamma[v * V + e];
            beta[e] = a.beta ? a.beta[v * V + e] : 0.0f;
        }
    };
    // The first rows and weights are on their way while the statistics are joined.
    fetch(p.tx, p.ty);
    weights(p.tx);
    join_chunks(a, p.n, stat);
    if (p.chunk == 0 && a.mean)
        for (int g = threadIdx.x; g < a.G; g += kThreads) {
            a.mean[p.n * a.G + g] = stat[2 * g];
            a.rstd[p.n * a.G + g] = stat[2 * g + 1];
        }
    if (p.ty >= p.TY) return;
    const int Cg = a.C / a.G;
    for (int v = p.tx; v < a.C / V; v += p.TX) {
        const int c = v * V;
        float mean[V], ga[V], be[V];
        int g = c / Cg, left = (g + 1) * Cg - c;  // the group, and its channels from c + e on
#pragma unroll
        for (int e = 0; e < V; ++e, --left) {
            if (left == 0) ++g, left = Cg;
            mean[e] = stat[2 * g];
            ga[e] = gamma[e] * stat[2 * g + 1];
            be[e] = beta[e];
        }
        if (v + p.TX < a.C / V) weights(v + p.TX);
        for (int r = p.ty; r < p.rows; r += kAhead * p.TY) {
            float o[kAhead][V];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                float xv[V], zv[V];
                x[u].values(xv);
                if (a.z) z[u].values(zv);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    o[u][e] = activation(a.silu, __builtin_fmaf(xv[e] - mean[e], ga[e], be[e]));
                    if (a.z) o[u][e] *= silu_f32(zv[e]);
                }
            }
            // The next ones, of this column or the thread's next.
            if (r + kAhead * p.TY < p.rows) fetch(v, r + kAhead * p.TY);
            else if (v + p.TX < a.C / V) fetch(v + p.TX, p.ty);
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (r + u * p.TY < p.rows)
                    store_f32<T, V>((T*)a.y + (row0 + r + u * p.TY) * a.C + c, o[u]);
        }
    }
}

// dv and h of V values.
template <int V>
struct Slopes {
    float dv[V], h[V], dz[V];
    __device__ __forceinline__ void make(const GroupArgs& a, const float (&x)[V], const float (&z)[V],
                                         const float (&dy)[V], const float (&mean)[V],
                                         const float (&rstd)[V], const float (&ga)[V],
                                         const float (&be)[V]) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            h[e] = (x[e] - mean[e]) * rstd[e];
            float act, slope, d = dy[e];
            activation_grad(a.silu, __builtin_fmaf(h[e], ga[e], be[e]), act, slope);
            if (a.z) {
                const float s = sigmoid_f32(z[e]);
                dz[e] = d * act * s * __builtin_fmaf(z[e], 1.0f - s, 1.0f);
                d *= z[e] * s;
            }
            dv[e] = d * slope;
        }
    }
};

template <typename T, int V>
__global__ __launch_bounds__(kThreads) void map_sums(const GroupArgs a) {
    __shared__ float sm[2 * V][kThreads];
    const int64_t at = a.first + blockIdx.x;
    const Place<V> p(a, at);
    const int Cg = a.C / a.G;
    const int64_t row0 = p.n * a.L + p.first;
    float* cols = a.cols + (int64_t)blockIdx.x * 2 * a.C;
    for (int base = 0; base < a.C / V; base += p.TX) {
        const int v = base + p.tx;
        float s[V] = {}, q[V] = {};
        if (p.ty < p.TY && v < a.C / V) {
            const int c = v * V;
            float ga[V], be[V], mean[V], rstd[V];
            int g = c / Cg, left = (g + 1) * Cg - c;
#pragma unroll
            for (int e = 0; e < V; ++e, --left) {
                if (left == 0) ++g, left = Cg;
                mean[e] = a.mean[p.n * a.G + g];
                rstd[e] = a.rstd[p.n * a.G + g];
                ga[e] = a.gamma[c + e];
                be[e] = a.beta ? a.beta[c + e] : 0.0f;
            }
            const auto one = [&](const Vec<T, V>& xr, const Vec<T, V>& zr, const Vec<T, V>& dr) {
                float x[V], z[V], dy[V];
                xr.values(x);
                dr.values(dy);
                if (a.z) zr.values(z);
                Slopes<V> t;
                t.make(a, x, z, dy, mean, rstd, ga, be);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    s[e] += t.dv[e];
                    q[e] = __builtin_fmaf(t.dv[e], t.h[e], q[e]);
                }
            };
            const auto fetch = [&](int r, Vec<T, V>& x, Vec<T, V>& z, Vec<T, V>& d) {
                x.load((const T*)a.x + (row0 + r) * a.xs + c);
                d.load((const T*)a.dy + (row0 + r) * a.ds + c);
                if (a.z) z.load((const T*)a.z + (row0 + r) * a.zs + c);
            };
            int r = p.ty;
            for (; r + p.TY < p.rows; r += 2 * p.TY) {
                Vec<T, V> x[2], z[2], d[2];
                fetch(r, x[0], z[0], d[0]);
                fetch(r + p.TY, x[1], z[1], d[1]);
                one(x[0], z[0], d[0]);
                one(x[1], z[1], d[1]);
            }
            if (r < p.rows) {
                Vec<T, V> x, z, d;
                fetch(r, x, z, d);
                one(x, z, d);
            }
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < V; ++e) sm[2 * e][threadIdx.x] = s[e], sm[2 * e + 1][threadIdx.x] = q[e];
        __syncthreads();
        for (int i = threadIdx.x; i < p.TX * 2 * V; i += kThreads) {
            const int col = i / (2 * V), k = i % (2 * V), cv = base + col;
            if (cv < a.C / V) {
                float t = 0.0f;
                for (int y = 0; y < p.TY; ++y) t += sm[k][y * p.TX + col];
                // dgamma's sums (of dv h) first, then dbeta's.
                cols[(k & 1 ? 0 : a.C) + cv * V + k / 2] = t;
            }
        }
    }
    // The groups' sums of gamma times these, which the workgroup wrote itself.
    __threadfence_block();
    __syncthreads();
    const int P = lanes_of_group(a.G), lane = threadIdx.x % P;
    for (int g0 = 0; g0 < a.G; g0 += kThreads / P) {
        const int g = g0 + threadIdx.x / P;
        float s = 0.0f, q = 0.0f;
        if (g < a.G)
            for (int c = g * Cg + lane; c < (g + 1) * Cg; c += P) {
                s = __builtin_fmaf(cols[a.C + c], a.gamma[c], s);
                q = __builtin_fmaf(cols[c], a.gamma[c], q);
            }
        for (int d = 1; d < P; d *= 2) s += __shfl_xor(s, d), q += __shfl_xor(q, d);
        if (g < a.G && lane == 0) {
            float* out = a.stats + (at * a.G + g) * 2;
            out[0] = s;
            out[1] = q;
        }
    }
}

template <typename T, int V>
__global__ __launch_bounds__(kThreads) void map_grads(const GroupArgs a) {
    extern __shared__ float stat[];  // [G][2]: the groups' means of g and of g h
    const Place<V> p(a);
    const int Cg = a.C / a.G;
    const int64_t row0 = p.n * a.L + p.first;
    Vec<T, V> x[2], z[2], d[2];
    const auto fetch = [&](int v, int r) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
            if (r + u * p.TY < p.rows) {
                const int64_t row = row0 + r + u * p.TY;
                x[u].load((const T*)a.x + row * a.xs + v * V);
                d[u].load((const T*)a.dy + row * a.ds + v * V);
                if (a.z) z[u].load((const T*)a.z + row * a.zs + v * V);
            }
    };
    float mean[V], rstd[V], ga[V], be[V];
    const auto weights = [&](int v) {
        const int c = v * V;
        int g = c / Cg, left = (g + 1) * Cg - c;  // the group, and its channels from c + e on
#pragma unroll
        for (int e = 0; e < V; ++e, --left) {
            if (left == 0) ++g, left = Cg;
            mean[e] = a.mean[p.n * a.G + g];
            rstd[e] = a.rstd[p.n * a.G + g];
            ga[e] = a.gamma[c + e];
            be[e] = a.beta ? a.beta[c + e] : 0.0f;
        }
    };
    // On their way while the sums are joined.
    fetch(p.tx, p.ty);
    weights(p.tx);
    {
        const float inv = 1.0f / ((float)Cg * (float)a.L);
        const int P = lanes_of_group(a.G), lane = threadIdx.x % P;
        for (int g0 = 0; g0 < a.G; g0 += kThreads / P) {
            const int g = g0 + threadIdx.x / P;
            float s = 0.0f, q = 0.0f;
            if (g < a.G)
                for (int c0 = lane; c0 < a.chunks; c0 += 4 * P) {
                    float2 t[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        t[u] = ((const float2*)a.stats)[(p.n * a.chunks + imin(c0 + u * P, a.chunks - 1)) * a.G + g];
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        if (c0 + u * P < a.chunks) s += t[u].x, q += t[u].y;
                }
            for (int d = 1; d < P; d *= 2) s += __shfl_xor(s, d), q += __shfl_xor(q, d);
            if (g < a.G && lane == 0) stat[2 * g] = s * inv, stat[2 * g + 1] = q * inv;
        }
        __syncthreads();
    }
    if (p.ty >= p.TY) return;
    for (int v = p.tx; v < a.C / V; v += p.TX) {
        const int c = v * V;
        if (v != p.tx) weights(v);
        float m1[V], m2[V];
        int g = c / Cg, left = (g + 1) * Cg - c;
#pragma unroll
        for (int e = 0; e < V; ++e, --left) {
            if (left == 0) ++g, left = Cg;
            m1[e] = stat[2 * g];
            m2[e] = stat[2 * g + 1];
        }
        for (int r = p.ty; r < p.rows; r += 2 * p.TY) {
            Slopes<V> t[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float xv[V], zv[V], dv[V];
                x[u].values(xv);
                d[u].values(dv);
                if (a.z) z[u].values(zv);
                t[u].make(a, xv, zv, dv, mean, rstd, ga, be);
            }
            // The next ones, of this column or the thread's next.
            if (r + 2 * p.TY < p.rows) fetch(v, r + 2 * p.TY);
            else if (v + p.TX < a.C / V) fetch(v + p.TX, p.ty);
#pragma unroll
            for (int u = 0; u < 2; ++u)
                if (r + u * p.TY < p.rows) {
                    const int64_t at = (row0 + r + u * p.TY) * a.C + c;
                    float o[V];
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        o[e] = rstd[e] * (__builtin_fmaf(t[u].dv[e], ga[e], -m1[e]) - t[u].h[e] * m2[e]);
                    store_f32<T, V>((T*)a.y + at, o);
                    if (a.z) store_f32<T, V>((T*)a.dz + at, t[u].dz);
                }
        }
    }
}

// ---- heads

// Sum over the P lanes of a group, in each of them.
template <int P>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int d = 1; d < P; d *= 2) v += __shfl_xor(v, d);
    return v;
}

// P lanes hold a group as NV vectors each. Lane group u of the launch has group u % G
// of rows u / G, u / G + units, ...
template <typename T, int V, int P, int NV, bool BACK>
__global__ __launch_bounds__(kThreads) void heads(const GroupArgs a) {
    const int64_t u = (int64_t)blockIdx.x * (kThreads / P) + threadIdx.x / P;
    const int g = (int)(u % a.G), lane = threadIdx.x % P, Cg = a.C / a.G;
    const int64_t first = u / a.G;
    const bool live = first < a.units;
    float ga[NV][V], be[NV][V], dg[NV][V] = {}, db[NV][V] = {};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * P + lane) * V;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            ga[j][e] = live && c < Cg ? a.gamma[g * Cg + c + e] : 0.0f;
            be[j][e] = live && c < Cg && a.beta ? a.beta[g * Cg + c + e] : 0.0f;
        }
    }
    const float inv = 1.0f / (float)Cg;
    Vec<T, V> rx[NV], rz[NV], rd[NV];
    float rmean = 0.0f, rrstd = 0.0f;
    const auto fetch = [&](int64_t n) {
        if constexpr (BACK) rmean = a.mean[n * a.G + g], rrstd = a.rstd[n * a.G + g];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * P + lane) * V, at = g * Cg + c;
            if (c < Cg) {
                rx[j].load((const T*)a.x + n * a.xs + at);
                if (a.z) rz[j].load((const T*)a.z + n * a.zs + at);
                if constexpr (BACK) rd[j].load((const T*)a.dy + n * a.ds + at);
            }
        }
    };
    if (live && first < a.N) fetch(first);
    // All lanes of a wave go round as often as its first group: sums cross lanes.
    for (int64_t n = first; __any(live && n < a.N); n += a.units) {
        const bool in = live && n < a.N;
        const int D = in ? Cg : 0;
        float x[NV][V], z[NV][V], dy[NV][V];
        const float mean0 = rmean, rstd0 = rrstd;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const bool ok = (j * P + lane) * V < D;
            rx[j].values(x[j]);
            if (a.z) rz[j].values(z[j]);
            if constexpr (BACK) rd[j].values(dy[j]);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (!ok) x[j][e] = BACK ? mean0 : 0.0f;
                if (!ok && BACK) dy[j][e] = 0.0f;
            }
        }
        if (in && n + a.units < a.N) fetch(n + a.units);
        if constexpr (!BACK) {
            float s = 0.0f, q = 0.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < V; ++e) s += x[j][e];
            const float mean = lanes_sum<P>(s) * inv;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const bool ok = (j * P + lane) * V < D;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    x[j][e] = ok ? x[j][e] - mean : 0.0f;
                    q = __builtin_fmaf(x[j][e], x[j][e], q);
                }
            }
            const float rstd = 1.0f / sqrtf(lanes_sum<P>(q) * inv + a.eps);
            if (in && lane == 0 && a.mean) {
                a.mean[n * a.G + g] = mean;
                a.rstd[n * a.G + g] = rstd;
            }
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (j * P + lane) * V;
                if (c < D) {
                    float o[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        o[e] = activation(a.silu, __builtin_fmaf(x[j][e] * rstd, ga[j][e], be[j][e]));
                        if (a.z) o[e] *= silu_f32(z[j][e]);
                    }
                    store_f32<T, V>((T*)a.y + n * a.C + g * Cg + c, o);
                }
            }
        } else {
            Slopes<V> t[NV];
            float s = 0.0f, q = 0.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                float m[V], q_[V];
#pragma unroll
                for (int e = 0; e < V; ++e) m[e] = mean0, q_[e] = rstd0;
                t[j].make(a, x[j], z[j], dy[j], m, q_, ga[j], be[j]);
                const bool ok = (j * P + lane) * V < D;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    if (!ok) t[j].dv[e] = t[j].h[e] = 0.0f;
                    db[j][e] += t[j].dv[e];
                    dg[j][e] = __builtin_fmaf(t[j].dv[e], t[j].h[e], dg[j][e]);
                    t[j].dv[e] *= ga[j][e];
                    s += t[j].dv[e];
                    q = __builtin_fmaf(t[j].dv[e], t[j].h[e], q);
                }
            }
            const float m1 = lanes_sum<P>(s) * inv, m2 = lanes_sum<P>(q) * inv;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (j * P + lane) * V;
                if (c < D) {
                    float o[V];
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        o[e] = rstd0 * (t[j].dv[e] - __builtin_fmaf(t[j].h[e], m2, m1));
                    store_f32<T, V>((T*)a.y + n * a.C + g * Cg + c, o);
                    if (a.z) store_f32<T, V>((T*)a.dz + n * a.C + g * Cg + c, t[j].dz);
                }
            }
        }
    }
    if constexpr (BACK) {
        if (!live) return;
        float* out = a.cols + first * 2 * a.C + g * Cg;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * P + lane) * V;
            if (c < Cg)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    out[c + e] = dg[j][e];
                    out[a.C + c + e] = db[j][e];
                }
        }
    }
}

// The form and its numbers, from the sizes alone (the vector width may be less than
// V where an address or stride is not a multiple of it).
struct GroupPlan {
    bool heads;
    int lanes, vectors;  // heads: P, NV at the width V
    int64_t units;       // heads: rows in flight; maps: chunks of a launch of map_sums
    int chunks, rows;    // maps
};

// Lanes and vectors of a group: as few vectors as 64 lanes allow.
bool heads_shape(int vectors, int* lanes, int* each) {
    for (int p = 1; p <= 64; p *= 2)
        for (int nv = 1; nv <= (p == 64 ? 4 : 1); nv *= 2)
            if (vectors <= p * nv) {
                *lanes = p, *each = nv;
                return true;
            }
    return false;
}
GroupPlan group_plan(const tg_group_norm_args& a, bool back) {
    GroupPlan p{};
    const int64_t Cg = a.C / a.G;
    // By scalars: what the narrowest vectors hold, any address serves.
    if (a.L == 1 && Cg <= 256) {
        p.heads = true;
        // Rows in flight: 2048 workgroups of them; in the backward pass no more than 512, each
        // a row of partial sums. That is a row of 2048 channels for a workgroup; narrower
        // ones leave compute units idle (16384 rows of 128 channels: 49 us).
        const int64_t row_threads = ceil_div(a.C, 8);
        int64_t most = (back ? 512 : 2048) * kThreads / row_threads;
        if (most < 1) most = 1;
        if (back && most > 512) most = 512;
        p.units = a.N < most ? a.N : most;
        return p;
    }
    // About 1024 workgroups, none of less than 2048 elements if there are enough rows, in
    // whole rounds of their threads (16-byte vectors); at most 256 chunks to join.
    const int64_t cols = ceil_div(a.C, 16 / (int64_t)elem_bytes(a.dtype));
    const int64_t round = kThreads / (cols < kThreads ? cols : kThreads), most = ceil_div(a.L, 256);
    int64_t rows = ceil_div(a.L * a.N, 1024), least = ceil_div(2048, a.C);
    if (rows < least) rows = least;
    if (rows < most) rows = most;
    rows = ceil_div(rows, round) * round;
    if (rows > a.L) rows = a.L;
    p.rows = (int)rows;
    p.chunks = (int)ceil_div(a.L, rows);
    const int64_t held = kSumBytes / (8 * (int64_t)a.C);
    p.units = held > kMostSums ? held : kMostSums;
    if (p.units > a.N * p.chunks) p.units = a.N * p.chunks;
    return p;
}

GroupArgs args_of(const tg_group_norm_args& a, const GroupPlan& p) {
    GroupArgs b{};
    b.x = a.x, b.xs = a.x_stride, b.z = a.z, b.zs = a.z_stride;
    b.gamma = a.gamma, b.beta = a.beta, b.eps = a.eps;
    b.N = a.N, b.L = a.L, b.C = a.C, b.G = a.G, b.silu = a.act == TG_ACT_SILU;
    b.y = a.y, b.mean = a.mean, b.rstd = a.rstd;
    b.chunks = p.chunks, b.rows = p.rows, b.units = p.units;
    return b;
}

template <typename T, int V, bool BACK>
hipError_t heads_typed(const GroupArgs& a, hipStream_t st) {
    int P = 0, NV = 0;
    if (!heads_shape((int)ceil_div(a.C / a.G, V), &P, &NV)) return hipErrorInvalidConfiguration;
    const int64_t grid = ceil_div(a.units * a.G, kThreads / P);
    if (grid >= (int64_t)1 << 24) return hipErrorInvalidConfiguration;
#define TG_X(P_, NV_) \
    if (P == P_ && NV == NV_) heads<T, V, P_, NV_, BACK><<<(unsigned)grid, kThreads, 0, st>>>(a)
    TG_X(1, 1);
    TG_X(2, 1);
    TG_X(4, 1);
    TG_X(8, 1);
    TG_X(16, 1);
    TG_X(32, 1);
    TG_X(64, 1);
    if constexpr (V <= 2) TG_X(64, 2);
    if constexpr (V == 1) TG_X(64, 4);
#undef TG_X
    return hipGetLastError();
}

// V: of what lies in one group (heads, statistics); W: of a row.
template <typename T, int V>
hipError_t stats_typed(const GroupArgs& a, const GroupPlan& p, bool back, hipStream_t st) {
    if (p.heads) return back ? heads_typed<T, V, true>(a, st) : heads_typed<T, V, false>(a, st);
    if (!back) map_stats<T, V><<<(unsigned)(a.N * a.chunks), kThreads, 0, st>>>(a);
    return hipGetLastError();
}
template <typename T, int W>
hipError_t sweeps_typed(const GroupArgs& a, bool back, hipStream_t st) {
    const unsigned grid = (unsigned)(a.N * a.chunks);
    if (back) {
        // Of several launches, each one's sums become a row behind the partial ones.
        GroupArgs b = a;
        float* row = a.cols + a.units * 2 * a.C;
        for (; b.first < grid; b.first += a.units, row += 2 * a.C) {
            const int64_t left = grid - b.first, now = left < a.units ? left : a.units;
            map_sums<T, W><<<(unsigned)now, kThreads, 0, st>>>(b);
            hipError_t e = hipGetLastError();
            if (e == hipSuccess && grid > a.units)
                e = launch_column_sums(a.cols, (int)now, 2 * (int64_t)a.C, row, 2 * (int64_t)a.C, nullptr, st);
            if (e != hipSuccess) return e;
        }
        map_grads<T, W><<<grid, kThreads, 2 * a.G * sizeof(float), st>>>(a);
    } else {
        map_apply<T, W><<<grid, kThreads, 2 * a.G * sizeof(float), st>>>(a);
    }
    return hipGetLastError();
}
#define TG_WIDTHS(N, X)                     \
    do {                                    \
        if constexpr (sizeof(T) == 2)       \
            if (N == 8) X(8);               \
        if (N == 4) X(4);                   \
        if (N == 2) X(2);                   \
        if (N == 1) X(1);                   \
    } while (0)
template <typename T>
hipError_t group_typed(int V, int W, const GroupArgs& a, const GroupPlan& p, bool back, hipStream_t st) {
    hipError_t e = hipErrorInvalidConfiguration;
#define TG_X(N) e = stats_typed<T, N>(a, p, back, st)
    TG_WIDTHS(V, TG_X);
#undef TG_X
    if (e != hipSuccess || p.heads) return e;
#define TG_X(N) e = sweeps_typed<T, N>(a, back, st)
    TG_WIDTHS(W, TG_X);
#undef TG_X
    return e;
}
#undef TG_WIDTHS
hipError_t group_run(tg_dtype dt, const GroupArgs& a, const GroupPlan& p, bool back, hipStream_t st) {
    const size_t e = elem_bytes(dt);
    Widest w;
    w.len(a.C), w.len(a.xs), w.ptr(a.x, e), w.ptr(a.y, e);
    if (a.z) w.len(a.zs), w.ptr(a.z, e);
    if (back) w.len(a.ds), w.ptr(a.dy, e);
    if (back && a.z) w.ptr(a.dz, e);
    const int W = w.width((int)(16 / e));
    w.len(a.C / a.G);
    const int V = w.width((int)(16 / e));
    if (dt == TG_F32) return group_typed<float>(V, W, a, p, back, st);
    if (dt == TG_BF16) return group_typed<bf16>(V, W, a, p, back, st);
    return group_typed<f16>(V, W, a, p, back, st);
}

// The maps' scratch in the backward pass: the groups' sums, then the channels' of one launch
// of map_sums, and where there are several launches a row of sums for each.
size_t stats_bytes(const tg_group_norm_args& a, const GroupPlan& p) {
    return up256((size_t)(a.N * p.chunks) * a.G * 2 * sizeof(float));
}
int64_t launch_sums(const tg_group_norm_args& a, const GroupPlan& p) {
    return a.N * p.chunks > p.units ? ceil_div(a.N * p.chunks, p.units) : 0;
}

}  // namespace

int64_t group_norm_groups(const tg_group_norm_args& a) {
    const GroupPlan p = group_plan(a, true);
    return p.heads ? p.units : a.N * p.chunks;
}

void group_norm_sizes(const tg_group_norm_args& a, size_t* work, size_t* backward) {
    const GroupPlan f = group_plan(a, false), b = group_plan(a, true);
    if (work) *work = f.heads ? 0 : (size_t)(a.N * f.chunks) * a.G * 2 * sizeof(float);
    if (backward)
        *backward = b.heads ? (size_t)b.units * 2 * a.C * sizeof(float)
                            : stats_bytes(a, b) +
                                  (size_t)(b.units + launch_sums(a, b)) * 2 * a.C * sizeof(float);
}

hipError_t launch_group_norm(const tg_group_norm_args& a, void* ws, hipStream_t st) {
    const GroupPlan p = group_plan(a, false);
    GroupArgs b = args_of(a, p);
    b.stats = (float*)ws;
    return group_run(a.dtype, b, p, false, st);
}

hipError_t launch_group_norm_backward(const tg_group_norm_args& a, const tg_group_norm_grads& g,
                                      void* ws, hipStream_t st) {
    const GroupPlan p = group_plan(a, true);
    GroupArgs b = args_of(a, p);
    b.stats = (float*)ws;
    b.cols = p.heads ? (float*)ws : (float*)((char*)ws + stats_bytes(a, p));
    b.dy = g.dy, b.ds = g.dy_stride, b.y = g.dx, b.dz = g.dz;
    if (a.N > 0) {
        const hipError_t e = group_run(a.dtype, b, p, true, st);
        if (e != hipSuccess) return e;
    }
    const int64_t sums = p.heads ? 0 : launch_sums(a, p);
    return launch_column_sums(sums ? b.cols + p.units * 2 * a.C : b.cols,
                              a.N > 0 ? (int)(sums ? sums : p.units) : 0, 2 * (int64_t)a.C, g.dgamma,
                              a.C, g.dbeta, st);
}

}  // namespace tg
