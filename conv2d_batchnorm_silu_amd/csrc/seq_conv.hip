// seq_conv.hip -- the short causal convolution with SiLU: prompts
// (tg_causal_conv), gradients (tg_causal_conv_backward) and single tokens
// (tg_causal_conv_step).
//
//   v[t] = bias + sum_k w[k] * x[t-K+1+k],  y[t] = v[t] * sigmoid(v[t])
//
// for each channel by itself: 2K operations for each element read and
// written, so the kernels are bound by memory. A thread owns V neighbouring
// channels (16 bytes where the alignment allows it) and walks down a strip
// of rows with the K-1 rows before it in registers, so each row is read once
// but for the K-1 rows in front of the strip. Strips are cut from the
// batch's rows as they lie, whatever the sequences' lengths; a strip that
// spans a sequence's end goes on with the next sequence's state.
#include "seq_device.hpp"
#include "seq_internal.hpp"

namespace tg {
namespace {

constexpr int kBlock = 256;

struct ConvFwd {
    SeqMap seqs;
    int D, K, silu, strip;
    Rows<const void> x;
    Rows<void> y;
    const float *w, *bias;
    const void* initial;
    void* final;
};

// Row l of sequence s, or for l < 0 its state row K-1+l (zeros without one).
template <typename T, int V, int K, typename A>
__device__ __forceinline__ void row_or_state(const A& a, int s, int start, int l, int c,
                                             float (&v)[V]) {
    if (l >= 0) {
        load_f32<T, V>(row_of<const T>(a.x, a.seqs, s, start, l) + c, v);
    } else if (a.initial) {
        load_f32<T, V>((const T*)a.initial + ((int64_t)s * (K - 1) + (K - 1) + l) * a.D + c, v);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = 0.0f;
    }
}

template <int V>
__device__ __forceinline__ void load_consts(const float* p, int c, float (&v)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = p ? p[c + e] : 0.0f;
}

// Rows that a thread has on their way while it computes: one row of a wave is 512
// bytes, and some thousand waves of one row each do not fill the memory's pipe.
constexpr int kAhead = 4;
template <typename T, int V>
struct Ahead {
    Vec<T, V> r[kAhead];
    // Rows l .. l+3 of the sequence, the last one (end - 1) again past the end.
    __device__ __forceinline__ void load(const Rows<const void>& x, const SeqMap& m, int s, int b,
                                         int l, int end, int c) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            r[k].load(row_of<const T>(x, m, s, b, imin(l + k, end - 1)) + c);
    }
};

// A wave's threads share a strip, so what goes by it is uniform.
__device__ __forceinline__ int wave_piece() {
    return __builtin_amdgcn_readfirstlane(blockIdx.x * blockDim.y + threadIdx.y);
}

// blockIdx.x: strips, then (with final) one more block row for each sequence.
// threadIdx.x: channel vectors, threadIdx.y: strips.
template <typename T, int V, int K>
__global__ __launch_bounds__(kBlock) void conv_fwd(const ConvFwd a, int strips) {
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    const SeqMap& m = a.seqs;
    const int piece = wave_piece();
    int t = piece * a.strip, s = piece < strips ? m.holder(t) : 0;
    if (c >= a.D) return;
    if (piece >= strips) {
        // The last K-1 rows of a sequence, as its next state.
        s = piece - strips;
        if (!a.final || s >= m.seqs) return;
        const int b = m.start(s), n = m.end(s) - b;
        for (int r = 0; r < K - 1; ++r) {
            float v[V];
            row_or_state<T, V, K>(a, s, b, n - (K - 1) + r, c, v);
            store_f32<T, V>((T*)a.final + ((int64_t)s * (K - 1) + r) * a.D + c, v);
        }
        return;
    }
    float w[K][V], bias[V], win[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k) load_consts<V>(a.w + (int64_t)k * a.D, c, w[k]);
    load_consts<V>(a.bias, c, bias);
    const int stop = imin(t + a.strip, m.rows);
    while (t < stop && s < m.seqs) {
        const int b = m.start(s), e = imin(m.end(s), stop);
        if (t < b) t = b;
        if (t < e) {
            Ahead<T, V> next;
            next.load(a.x, m, s, b, t - b, e - b, c);
#pragma unroll
            for (int k = 0; k < K - 1; ++k)
                row_or_state<T, V, K>(a, s, b, t - b - (K - 1) + k, c, win[k]);
            for (; t < e; t += kAhead) {
                const Ahead<T, V> cur = next;
                if (t + kAhead < e) next.load(a.x, m, s, b, t + kAhead - b, e - b, c);
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    if (t + u >= e) break;
                    cur.r[u].values(win[K - 1]);
                    float o[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        float v = bias[i];
#pragma unroll
                        for (int k = 0; k < K; ++k) v = __builtin_fmaf(w[k][i], win[k][i], v);
                        o[i] = a.silu ? silu_f32(v) : v;
                    }
                    store_f32<T, V>(row_of<T>(a.y, m, s, b, t + u - b) + c, o);
#pragma unroll
                    for (int k = 0; k < K - 1; ++k)
#pragma unroll
                        for (int i = 0; i < V; ++i) win[k][i] = win[k + 1][i];
                }
            }
            t = e;
        }
        ++s;
    }
}

struct ConvBwd {
    SeqMap seqs;
    int D, silu, strip;
    Rows<const void> x, dy;
    Rows<void> dx;
    const float *w, *bias;
    const void *initial, *dfinal;
    void* dinitial;
    float* part;  // [strips][K+1][D]: dw, dbias of a strip
};

// dL/dv of the row whose window is win.
template <int V, int K>
__device__ __forceinline__ void dpre(const float (&w)[K][V], const float (&bias)[V],
                                     const float (&win)[K][V], int silu, float (&g)[V]) {
    if (!silu) return;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float v = bias[i];
#pragma unroll
        for (int k = 0; k < K; ++k) v = __builtin_fmaf(w[k][i], win[k][i], v);
        const float sg = sigmoid_f32(v);
        g[i] *= sg * __builtin_fmaf(v, 1.0f - sg, 1.0f);
    }
}

// The gradient of the state row for position p (which may be negative) from
// that of the final states; zero where p is not among the last K-1.
template <typename T, int V, int K>
__device__ __forceinline__ void add_dfinal(const ConvBwd& a, int s, int n, int p, int c,
                                           float (&v)[V]) {
    const int r = p - (n - (K - 1));
    if (!a.dfinal || r < 0 || r >= K - 1) return;
    float f[V];
    load_f32<T, V>((const T*)a.dfinal + ((int64_t)s * (K - 1) + r) * a.D + c, f);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] += f[i];
}

// dx[t] = sum_j w[K-1-j] * dv[t+j]: the walk runs K-1 rows past the strip (or
// to the sequence's end) and sends dx[t] off when dv[t+K-1] is known. The
// ring acc[j] holds the sum so far of row t-j.
template <typename T, int V, int K>
__global__ __launch_bounds__(kBlock) void conv_bwd(const ConvBwd a, int strips) {
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    const SeqMap& m = a.seqs;
    const int piece = wave_piece();
    int t = piece * a.strip, s = piece < strips ? m.holder(t) : 0;
    if (c >= a.D) return;
    float w[K][V], bias[V], win[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k) load_consts<V>(a.w + (int64_t)k * a.D, c, w[k]);
    load_consts<V>(a.bias, c, bias);
    if (piece >= strips) {
        // The gradient of a sequence's initial state: position q < 0 takes w[k] * dv[t]
        // for t = q + K-1-k >= 0, and passes on what reaches it as a final state.
        s = piece - strips;
        if (!a.dinitial || s >= m.seqs) return;
        const int b = m.start(s), n = m.end(s) - b;
        float acc[K - 1][V];
#pragma unroll
        for (int r = 0; r < K - 1; ++r) {
#pragma unroll
            for (int i = 0; i < V; ++i) acc[r][i] = 0.0f;
            add_dfinal<T, V, K>(a, s, n, r - (K - 1), c, acc[r]);
        }
#pragma unroll
        for (int t = 0; t < K - 1; ++t) {
            if (t >= n) break;
#pragma unroll
            for (int k = 0; k < K; ++k) row_or_state<T, V, K>(a, s, b, t - (K - 1) + k, c, win[k]);
            float g[V];
            load_f32<T, V>(row_of<const T>(a.dy, m, s, b, t) + c, g);
            dpre<V, K>(w, bias, win, a.silu, g);
#pragma unroll
            for (int k = 0; k < K - 1 - t; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i)
                    acc[t + k][i] = __builtin_fmaf(w[k][i], g[i], acc[t + k][i]);
        }
#pragma unroll
        for (int r = 0; r < K - 1; ++r)
            store_f32<T, V>((T*)a.dinitial + ((int64_t)s * (K - 1) + r) * a.D + c, acc[r]);
        return;
    }
    float dw[K][V], db[V], acc[K][V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        db[i] = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) dw[k][i] = 0.0f;
    }
    const int stop = imin(t + a.strip, m.rows);
    while (t < stop && s < m.seqs) {
        const int b = m.start(s), end = m.end(s), n = end - b, e = imin(end, stop);
        if (t < b) t = b;
        if (t < e) {
            const int first = t, far = imin(e + K - 1, end);
            Ahead<T, V> nx, ng;
            nx.load(a.x, m, s, b, t - b, far - b, c);
            ng.load(a.dy, m, s, b, t - b, far - b, c);
#pragma unroll
            for (int k = 0; k < K - 1; ++k)
                row_or_state<T, V, K>(a, s, b, t - b - (K - 1) + k, c, win[k]);
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) acc[k][i] = 0.0f;
            // Up to K-1 steps past the last row with dv: they only send rows off.
            for (; t < e + K - 1; t += kAhead) {
                const Ahead<T, V> cx = nx, cg = ng;
                if (t + kAhead < far) {
                    nx.load(a.x, m, s, b, t + kAhead - b, far - b, c);
                    ng.load(a.dy, m, s, b, t + kAhead - b, far - b, c);
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int r = t + u;
                    if (r >= e + K - 1) break;
                    float g[V];
                    if (r < far) {
                        cx.r[u].values(win[K - 1]);
                        cg.r[u].values(g);
                        dpre<V, K>(w, bias, win, a.silu, g);
                    } else {
#pragma unroll
                        for (int i = 0; i < V; ++i) g[i] = 0.0f, win[K - 1][i] = 0.0f;
                    }
                    if (r < e) {
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            db[i] += g[i];
#pragma unroll
                            for (int k = 0; k < K; ++k)
                                dw[k][i] = __builtin_fmaf(g[i], win[k][i], dw[k][i]);
                        }
                    }
                    // Row r-j takes w[K-1-j] * dv[r].
#pragma unroll
                    for (int j = 0; j < K; ++j)
#pragma unroll
                        for (int i = 0; i < V; ++i)
                            acc[j][i] = __builtin_fmaf(w[K - 1 - j][i], g[i], acc[j][i]);
                    const int done = r - (K - 1);
                    if (done >= first && done < e) {
                        add_dfinal<T, V, K>(a, s, n, done - b, c, acc[K - 1]);
                        store_f32<T, V>(row_of<T>(a.dx, m, s, b, done - b) + c, acc[K - 1]);
                    }
#pragma unroll
                    for (int j = K - 1; j > 0; --j)
#pragma unroll
                        for (int i = 0; i < V; ++i) acc[j][i] = acc[j - 1][i];
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[0][i] = 0.0f;
#pragma unroll
                    for (int k = 0; k < K - 1; ++k)
#pragma unroll
                        for (int i = 0; i < V; ++i) win[k][i] = win[k + 1][i];
                }
            }
            t = e;
        }
        ++s;
    }
    float* part = a.part + (int64_t)piece * (K + 1) * a.D + c;
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int k = 0; k < K; ++k) part[(int64_t)k * a.D + i] = dw[k][i];
        part[(int64_t)K * a.D + i] = db[i];
    }
}

struct ConvStep {
    const void* x;
    int64_t xs;
    void* state;
    int64_t num_slots;
    const int32_t* slots;
    const float *w, *bias;
    int64_t n;
    int D, silu;
    void* y;
};

// All K rows are read before the state moves: the loads do not wait for the
// stores.
template <typename T, int V, int K>
__global__ __launch_bounds__(kBlock) void conv_step(const ConvStep a) {
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    const int64_t i = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (c >= a.D || i >= a.n) return;
    const int64_t slot = a.slots ? a.slots[i] : i;
    float win[K][V], o[V];
    T* yp = (T*)a.y + i * a.D + c;
    if (slot < 0 || slot >= a.num_slots) {
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = 0.0f;
        store_f32<T, V>(yp, o);
        return;
    }
    T* st = (T*)a.state + slot * (K - 1) * a.D + c;
#pragma unroll
    for (int k = 0; k < K - 1; ++k) load_f32<T, V>(st + (int64_t)k * a.D, win[k]);
    load_f32<T, V>((const T*)a.x + i * a.xs + c, win[K - 1]);
    load_consts<V>(a.bias, c, o);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float w[V];
        load_consts<V>(a.w + (int64_t)k * a.D, c, w);
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = __builtin_fmaf(w[e], win[k][e], o[e]);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = a.silu ? silu_f32(o[e]) : o[e];
    store_f32<T, V>(yp, o);
#pragma unroll
    for (int k = 0; k < K - 1; ++k) store_f32<T, V>(st + (int64_t)k * a.D, win[k + 1]);
}

// X(T, V, K) for the element type, vector width and number of taps.
#define TG_CONV_K(X, T, V)                     \
    do {                                       \
        switch (K) {                           \
            case 2: X(T, V, 2); break;         \
            case 3: X(T, V, 3); break;         \
            case 4: X(T, V, 4); break;         \
            case 5: X(T, V, 5); break;         \
            case 6: X(T, V, 6); break;         \
            case 7: X(T, V, 7); break;         \
            default: X(T, V, 8); break;        \
        }                                      \
    } while (0)
#define TG_CONV_T(X, T, W)                     \
    do {                                       \
        if (V == W) TG_CONV_K(X, T, W);        \
        else TG_CONV_K(X, T, 1);               \
    } while (0)
// The full width (8 bytes) or single elements: 8 halves would need 100 registers for
// the window and the taps alone.
#define TG_CONV_DISPATCH(X)                            \
    do {                                               \
        if (dtype == TG_F32) TG_CONV_T(X, float, 2);   \
        else if (dtype == TG_BF16) TG_CONV_T(X, bf16, 4); \
        else TG_CONV_T(X, f16, 4);                     \
    } while (0)

int vec_for(tg_dtype dt, const Widest& w) {
    const int full = (int)(8 / elem_bytes(dt));
    return w.width(full) == full ? full : 1;
}

// Block of bx channel vectors by by strips.
struct Block {
    dim3 block;
    unsigned cblocks;
};
Block conv_block(int D, int V) {
    const int64_t n = ceil_div(D, V);
    unsigned bx = 64;
    while (bx < 256 && bx < n) bx *= 2;
    return {dim3(bx, kBlock / bx), (unsigned)ceil_div(n, bx)};
}

// The grid for `pieces` strips or rows; false where a launch does not hold them:
// fewer than 2^32 threads along x (16 to 256 for each piece, by D).
bool conv_grid(const Block& bl, int64_t pieces, dim3& grid) {
    const int64_t x = ceil_div(pieces, bl.block.y);
    grid = dim3((unsigned)x, bl.cblocks);
    return x * bl.block.x < (int64_t)1 << 32;
}

void widest_rows(Widest& w, const tg_causal_conv_args& a, const tg_rows& r) {
    w.ptr(r.p, elem_bytes(a.dtype));
    w.len(r.row_stride);
    if (!a.seqs.offsets) w.len(r.seq_stride);
}

// Rows for each strip: the K-1 rows in front of a strip are read twice (from
// the cache), so no more strips than `waves` waves want, of 4 to `most` rows.
// Forward 4096 waves (16384 x 2048 bf16: 28 us, 9001 x 1000 f16: 12; 8192 waves 30 and
// 14), backward 2048 (9001 x 1000 f16 with its sums: 28 us; 1536 waves 30, 3072: 29).
int strip_of(int64_t rows, int D, int V, int most, int waves) {
    const int64_t strip = ceil_div(rows * ceil_div(ceil_div(D, V), 64), waves);
    return (int)(strip < 4 ? 4 : strip > most ? most : strip);
}

}  // namespace

hipError_t launch_causal_conv(const tg_causal_conv_args& a, hipStream_t st) {
    const tg_dtype dtype = a.dtype;
    const int K = a.K;
    const size_t e = elem_bytes(dtype);
    Widest w;
    w.len(a.D);
    widest_rows(w, a, a.x);
    widest_rows(w, a, a.y);
    if (a.initial) w.ptr(a.initial, e);
    if (a.final) w.ptr(a.final, e);
    const int V = vec_for(dtype, w);
    const Block bl = conv_block(a.D, V);
    const int strip = strip_of(a.seqs.rows, a.D, V, 32, 4096);
    const int strips = (int)ceil_div(a.seqs.rows, strip);
    const ConvFwd f{map_of(a.seqs), a.D, K, a.act == TG_ACT_SILU, strip, rows_of<const void>(a.x),
                    rows_of<void>(a.y), a.w, a.bias, a.initial, a.final};
    const int64_t pieces = strips + (a.final ? a.seqs.seqs : 0);
    if (pieces == 0) return hipSuccess;
    dim3 grid;
    if (!conv_grid(bl, pieces, grid)) return hipErrorInvalidConfiguration;
#define TG_X(T, V, K) conv_fwd<T, V, K><<<grid, bl.block, 0, st>>>(f, strips)
    TG_CONV_DISPATCH(TG_X);
#undef TG_X
    return hipGetLastError();
}

namespace {
int bwd_vec(const tg_causal_conv_args& a, const tg_rows* dy, const tg_rows* dx, const void* dfinal,
            const void* dinitial) {
    Widest w;
    const size_t e = elem_bytes(a.dtype);
    w.len(a.D);
    widest_rows(w, a, a.x);
    if (dy) widest_rows(w, a, *dy);
    if (dx) widest_rows(w, a, *dx);
    if (a.initial) w.ptr(a.initial, e);
    if (dfinal) w.ptr(dfinal, e);
    if (dinitial) w.ptr(dinitial, e);
    return vec_for(a.dtype, w);
}
// Strips of the backward pass by the sizes alone (the workspace is asked for
// before all pointers are known).
int bwd_strip(const tg_causal_conv_args& a) {
        return strip_of(a.seqs.rows, a.D, (int)(8 / elem_bytes(a.dtype)), 64, 2048);
}
}  // namespace

size_t causal_conv_backward_bytes(const tg_causal_conv_args& a) {
    return (size_t)ceil_div(a.seqs.rows, bwd_strip(a)) * (a.K + 1) * a.D * sizeof(float);
}

hipError_t launch_causal_conv_backward(const tg_causal_conv_args& a, const tg_rows& dy,
                                       const tg_rows& dx, float* dw, float* dbias,
                                       const void* dfinal, void* dinitial, void* ws,
                                       hipStream_t st) {
    const tg_dtype dtype = a.dtype;
    const int K = a.K, V = bwd_vec(a, &dy, &dx, dfinal, dinitial);
    const Block bl = conv_block(a.D, V);
    const int strip = bwd_strip(a);
    const int strips = (int)ceil_div(a.seqs.rows, strip);
    const ConvBwd f{map_of(a.seqs), a.D, a.act == TG_ACT_SILU, strip, rows_of<const void>(a.x),
                    rows_of<const void>(dy), rows_of<void>(dx), a.w, a.bias, a.initial, dfinal,
                    dinitial, (float*)ws};
    const int64_t pieces = strips + (dinitial ? a.seqs.seqs : 0);
    if (pieces > 0) {
        dim3 grid;
        if (!conv_grid(bl, pieces, grid)) return hipErrorInvalidConfiguration;
#define TG_X(T, V, K) conv_bwd<T, V, K><<<grid, bl.block, 0, st>>>(f, strips)
        TG_CONV_DISPATCH(TG_X);
#undef TG_X
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return launch_column_sums((const float*)ws, strips, (int64_t)(K + 1) * a.D, dw,
                              (int64_t)K * a.D, dbias, st);
}

hipError_t launch_causal_conv_step(const void* x, int64_t xs, void* state, int64_t num_slots,
                                   const int32_t* slots, const float* w, const float* bias,
                                   int64_t n, int D, int K, tg_dtype dtype, bool silu, void* y,
                                   hipStream_t st) {
    const size_t e = elem_bytes(dtype);
    Widest wd;
    wd.len(D), wd.len(xs), wd.ptr(x, e), wd.ptr(state, e), wd.ptr(y, e);
    const int V = vec_for(dtype, wd);
    const Block bl = conv_block(D, V);
    const ConvStep f{x, xs, state, num_slots, slots, w, bias, n, D, silu, y};
    dim3 grid;
    if (!conv_grid(bl, n, grid)) return hipErrorInvalidConfiguration;
#define TG_X(T, V, K) conv_step<T, V, K><<<grid, bl.block, 0, st>>>(f)
    TG_CONV_DISPATCH(TG_X);
#undef TG_X
    return hipGetLastError();
}

}  // namespace tg
