// seq_scan.hip -- the selective state space scan: prompts (tg_selective_scan),
// gradients (tg_selective_scan_backward) and single tokens
// (tg_selective_scan_step).
//
//   d = softplus(dt + dt_bias),  a[n] = exp(d * A[n]) = 2^(d * A[n]*log2 e)
//   h[n] = a[n] * h[n] + (d * x) * B[n],  v = sum_n C[n] * h[n] + D * x,  y = v * silu(z)
//
// Per channel and state one exponential and four multiplications or
// additions for every token: with N = 16 states that is far more than the
// eight bytes a token and channel move, so the scan is bound by the vector
// units, not by HBM.
//
// A wave holds 16 channels, each by 4 lanes of NS states (4*NS >= N; states
// past N have A = B = C = 0). It takes TT tokens at a time: the lanes first
// share out the TT x 16 (token, channel) items, so that softplus is computed
// once for each, and put d, d*x and the tokens' B and C into LDS in fp32; then
// every lane runs its states through the TT tokens; the sums over n are
// joined over the 4 lanes.
//
// Tokens past the end count as d = x = B = C = 0: a = 1, and the state stays.
#include "seq_device.hpp"
#include "seq_internal.hpp"

namespace tg {
namespace {

constexpr int kCh = 16;  // channels of a wave
constexpr float kLn2 = 0.69314718055994531f;

struct ScanArgs {
    SeqMap seqs;
    int D, N, G, Dg, bpg;  // Dg: channels of a group, in bpg blocks of 16
    int softplus;
    Rows<const void> x, dt, B, C, z;
    Rows<void> y;
    const float *A, *D_skip, *dt_bias, *initial;
    float *final, *saved;
};

__device__ __forceinline__ float quad_sum(float v) {
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0xB1, 0xF, 0xF, false));
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x4E, 0xF, 0xF, false));
    return v;
}

// What a wave keeps in LDS of TT tokens.
template <int NS, int TT>
struct Tile {
    float2 d[TT][kCh];     // d, d*x
    float B[TT][4 * NS];
    float C[TT][4 * NS];
    float dy[TT][kCh];     // backward only
};

// The wave's place: its sequence, block of channels and states. Neighbouring
// blocks share the cache lines of x, dt, z and y (16 channels are a quarter of
// one), so they run on one XCD.
struct Place {
    int s, start, len, block, g, cl, q, ch;
    bool in;
    __device__ __forceinline__ Place(const SeqMap& m, int G, int Dg, int bpg) {
        const int tile = xcd_contiguous_tile(blockIdx.x, gridDim.x);
        s = tile / (G * bpg);
        block = tile - s * (G * bpg);
        start = m.start(s);
        len = m.end(s) - start;
        g = block / bpg;
        const int c0 = (block - g * bpg) * kCh;
        cl = (threadIdx.x & 63) >> 2;
        q = threadIdx.x & 3;
        in = c0 + cl < Dg;
        ch = g * Dg + c0 + (in ? cl : 0);
    }
};

template <typename T, int NS, int TT>
__device__ __forceinline__ void stage_bc(const ScanArgs& a, const Place& p, int l0,
                                         Tile<NS, TT>& tile) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int k = 0; k < TT * NS * 4; k += 64) {
        const int i = k + lane, t = i / (4 * NS), n = i % (4 * NS), l = l0 + t;
        if (TT * NS * 4 % 64 == 0 || t < TT) {
            float b = 0.0f, c = 0.0f;
            if (n < a.N && l < p.len) {
                b = (float)row_of<const T>(a.B, a.seqs, p.s, p.start, l)[p.g * a.N + n];
                c = (float)row_of<const T>(a.C, a.seqs, p.s, p.start, l)[p.g * a.N + n];
            }
            tile.B[t][n] = b;
            tile.C[t][n] = c;
        }
    }
}

template <typename T, int NS, int TT>
__global__ __launch_bounds__(64) void scan_fwd(const ScanArgs a) {
    constexpr int kItems = TT / 4;
    __shared__ Tile<NS, TT> tile;
    const Place p(a.seqs, a.G, a.Dg, a.bpg);
    float A2[NS], h[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        const int n = p.q * NS + j;
        const bool in = p.in && n < a.N;
        A2[j] = in ? a.A[(int64_t)p.ch * a.N + n] * kLog2e : 0.0f;
        h[j] = in && a.initial ? a.initial[((int64_t)p.s * a.D + p.ch) * a.N + n] : 0.0f;
    }
    const float skip = a.D_skip ? a.D_skip[p.ch] : 0.0f;
    const float bias = a.dt_bias ? a.dt_bias[p.ch] : 0.0f;
    int64_t slot = a.seqs.slot0(p.s, TT);
    for (int l0 = 0; l0 < p.len; l0 += TT, ++slot) {
        float x[kItems], z[kItems], v[kItems];
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int t = p.q + 4 * i, l = l0 + t;
            float d = 0.0f;
            x[i] = z[i] = v[i] = 0.0f;
            if (l < p.len) {
                x[i] = (float)row_of<const T>(a.x, a.seqs, p.s, p.start, l)[p.ch];
                d = (float)row_of<const T>(a.dt, a.seqs, p.s, p.start, l)[p.ch] + bias;
                if (a.z.p) z[i] = (float)row_of<const T>(a.z, a.seqs, p.s, p.start, l)[p.ch];
                if (a.softplus) d = softplus_f32(d);
            }
            tile.d[t][p.cl] = make_float2(d, d * x[i]);
        }
        stage_bc<T, NS, TT>(a, p, l0, tile);
        __syncthreads();
        if (a.saved && p.in)
#pragma unroll
            for (int j = 0; j < NS; ++j)
                a.saved[(slot * a.D + p.ch) * (4 * NS) + p.q * NS + j] = h[j];
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const float2 d = tile.d[t][p.cl];
            float y = 0.0f;
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                const float e = __builtin_amdgcn_exp2f(d.x * A2[j]);
                h[j] = __builtin_fmaf(e, h[j], d.y * tile.B[t][p.q * NS + j]);
                y = __builtin_fmaf(h[j], tile.C[t][p.q * NS + j], y);
            }
            y = quad_sum(y);
            if ((t & 3) == p.q) v[t >> 2] = y;
        }
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int l = l0 + p.q + 4 * i;
            if (l < p.len && p.in) {
                float o = __builtin_fmaf(skip, x[i], v[i]);
                if (a.z.p) o *= silu_f32(z[i]);
                row_of<T>(a.y, a.seqs, p.s, p.start, l)[p.ch] = (T)o;
            }
        }
        __syncthreads();
    }
    if (a.final && p.in)
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            const int n = p.q * NS + j;
            if (n < a.N) a.final[((int64_t)p.s * a.D + p.ch) * a.N + n] = h[j];
        }
}

struct ScanGrads {
    Rows<const void> dy;
    const float *dfinal, *saved;
    Rows<void> dx, ddt, dz;
    float* dinitial;
    float* part_bc;   // [blocks of channels][rows][2][4*NS]: dB, dC of a block
    float* part_a;    // [seqs][D][N]
    float* part_d;    // [seqs][2][D]: dD, ddt_bias
};

// The chunks of a sequence from the last to the first. In each, the states
// are computed again from the one the forward pass saved at its start and held
// in registers with the decays, and then the adjoint runs backwards:
//   g[t] = dv[t]*C[t] + a[t+1]*g[t+1]                 (dL/dh[t])
//   dd[t]  = sum_n g*(A*a[t]*h[t-1] + B*x),  dx[t] = d * sum_n g*B + D*dv
//   dA += g*a[t]*h[t-1]*d,   dB = sum_c g*d*x,   dC = sum_c dv*h
template <typename T, int NS, int TT>
__global__ __launch_bounds__(64) void scan_bwd(const ScanArgs a, const ScanGrads b) {
    constexpr int kItems = TT / 4;
    __shared__ Tile<NS, TT> tile;
    const Place p(a.seqs, a.G, a.Dg, a.bpg);
    float A2[NS], dA[NS], carry[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        const int n = p.q * NS + j;
        const bool in = p.in && n < a.N;
        A2[j] = in ? a.A[(int64_t)p.ch * a.N + n] * kLog2e : 0.0f;
        carry[j] = in && b.dfinal ? b.dfinal[((int64_t)p.s * a.D + p.ch) * a.N + n] : 0.0f;
        dA[j] = 0.0f;
    }
    const float skip = a.D_skip ? a.D_skip[p.ch] : 0.0f;
    const float bias = a.dt_bias ? a.dt_bias[p.ch] : 0.0f;
    float dD = 0.0f, dbias = 0.0f;
    const int64_t slot0 = a.seqs.slot0(p.s, TT);
    const int row0 = p.start;  // of the flat rows, dense or packed
    for (int l0 = (p.len - 1) / TT * TT; l0 >= 0 && p.len > 0; l0 -= TT) {
        float x[kItems], raw[kItems], dl[kItems], z[kItems], dout[kItems];
        float v[kItems], e1[kItems], e2[kItems];
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int t = p.q + 4 * i, l = l0 + t;
            x[i] = raw[i] = z[i] = dout[i] = dl[i] = 0.0f;
            v[i] = e1[i] = e2[i] = 0.0f;
            if (l < p.len && p.in) {
                x[i] = (float)row_of<const T>(a.x, a.seqs, p.s, p.start, l)[p.ch];
                raw[i] = (float)row_of<const T>(a.dt, a.seqs, p.s, p.start, l)[p.ch] + bias;
                if (a.z.p) z[i] = (float)row_of<const T>(a.z, a.seqs, p.s, p.start, l)[p.ch];
                dout[i] = (float)row_of<const T>(b.dy, a.seqs, p.s, p.start, l)[p.ch];
                dl[i] = a.softplus ? softplus_f32(raw[i]) : raw[i];
            }
            tile.d[t][p.cl] = make_float2(dl[i], dl[i] * x[i]);
            tile.dy[t][p.cl] = a.z.p ? dout[i] * silu_f32(z[i]) : dout[i];
        }
        stage_bc<T, NS, TT>(a, p, l0, tile);
        __syncthreads();
        float h0[NS], dec[TT][NS], h[TT][NS];
        const int64_t slot = slot0 + l0 / TT;
#pragma unroll
        for (int j = 0; j < NS; ++j)
            h0[j] = p.in ? b.saved[(slot * a.D + p.ch) * (4 * NS) + p.q * NS + j] : 0.0f;
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const float2 d = tile.d[t][p.cl];
            float y = 0.0f;
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                dec[t][j] = __builtin_amdgcn_exp2f(d.x * A2[j]);
                h[t][j] = __builtin_fmaf(dec[t][j], t ? h[t - 1][j] : h0[j],
                                         d.y * tile.B[t][p.q * NS + j]);
                y = __builtin_fmaf(h[t][j], tile.C[t][p.q * NS + j], y);
            }
            y = quad_sum(y);
            if ((t & 3) == p.q) v[t >> 2] = y;
        }
#pragma unroll
        for (int t = TT - 1; t >= 0; --t) {
            const float2 d = tile.d[t][p.cl];
            const float dy = tile.dy[t][p.cl];
            float f1 = 0.0f, f2 = 0.0f, dB[NS], dC[NS];
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                const float g = __builtin_fmaf(dy, tile.C[t][p.q * NS + j], carry[j]);
                carry[j] = g * dec[t][j];
                const float gu = carry[j] * (t ? h[t - 1][j] : h0[j]);
                f1 = __builtin_fmaf(gu, A2[j], f1);
                f2 = __builtin_fmaf(g, tile.B[t][p.q * NS + j], f2);
                dA[j] = __builtin_fmaf(gu, d.x, dA[j]);
                dB[j] = g * d.y;
                dC[j] = dy * h[t][j];
            }
            f1 = quad_sum(f1);
            f2 = quad_sum(f2);
            if ((t & 3) == p.q) e1[t >> 2] = f1, e2[t >> 2] = f2;
#pragma unroll
            for (int j = 0; j < NS; ++j)
#pragma unroll
                for (int o = 4; o < 64; o *= 2) {
                    dB[j] += __shfl_xor(dB[j], o);
                    dC[j] += __shfl_xor(dC[j], o);
                }
            if (p.cl == 0 && l0 + t < p.len) {
                float* o = b.part_bc +
                           (((int64_t)p.block * a.seqs.rows + row0 + l0 + t) * 2) * (4 * NS) +
                           p.q * NS;
#pragma unroll
                for (int j = 0; j < NS; ++j) o[j] = dB[j], o[4 * NS + j] = dC[j];
            }
        }
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int t = p.q + 4 * i, l = l0 + t;
            const float dy = tile.dy[t][p.cl];
            if (l < p.len && p.in) {
                float ddl = __builtin_fmaf(e2[i], x[i], e1[i] * kLn2);
                if (a.softplus) ddl *= sigmoid_f32(raw[i]);
                row_of<T>(b.ddt, a.seqs, p.s, p.start, l)[p.ch] = (T)ddl;
                row_of<T>(b.dx, a.seqs, p.s, p.start, l)[p.ch] =
                    (T)__builtin_fmaf(e2[i], dl[i], skip * dy);
                if (a.z.p) {
                    const float sg = sigmoid_f32(z[i]), y = __builtin_fmaf(skip, x[i], v[i]);
                    row_of<T>(b.dz, a.seqs, p.s, p.start, l)[p.ch] =
                        (T)(dout[i] * y * sg * __builtin_fmaf(z[i], 1.0f - sg, 1.0f));
                }
                dbias += ddl;
                dD = __builtin_fmaf(dy, x[i], dD);
            }
        }
        __syncthreads();
    }
    dD = quad_sum(dD);
    dbias = quad_sum(dbias);
    if (!p.in) return;
    if (p.q == 0) {
        b.part_d[(int64_t)p.s * 2 * a.D + p.ch] = dD;
        b.part_d[((int64_t)p.s * 2 + 1) * a.D + p.ch] = dbias;
    }
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        const int n = p.q * NS + j;
        if (n < a.N) {
            const int64_t o = ((int64_t)p.s * a.D + p.ch) * a.N + n;
            b.part_a[o] = dA[j];
            if (b.dinitial) b.dinitial[o] = carry[j];
        }
    }
}

// dB and dC of the rows that the sequences cover: sums over a group's blocks
// of channels.
template <typename T>
__global__ __launch_bounds__(256) void scan_bc_sums(const ScanArgs a, const float* part, int NP,
                                                    Rows<void> dB, Rows<void> dC) {
    const SeqMap& m = a.seqs;
    const int64_t per = (int64_t)a.G * 2 * NP, last = m.end(m.seqs - 1) * per;
    for (int64_t i = m.start(0) * per + (int64_t)blockIdx.x * 256 + threadIdx.x; i < last;
         i += (int64_t)gridDim.x * 256) {
        const int row = (int)(i / per), r = (int)(i - row * per);
        const int g = r / (2 * NP), k = r - g * 2 * NP, c = k / NP, n = k - c * NP;
        if (n >= a.N) continue;
        float v = 0.0f;
        for (int blk = 0; blk < a.bpg; ++blk)
            v += part[(((int64_t)(g * a.bpg + blk) * m.rows + row) * 2 + c) * NP + n];
        const int s = m.offsets ? 0 : row / m.L;
        row_of<T>(c ? dC : dB, m, s, 0, m.offsets ? row : row - s * m.L)[g * a.N + n] = (T)v;
    }
}

struct StepArgs {
    ScanArgs a;
    float* state;
    int64_t num_slots;
    const int32_t* slots;
};

// One token: 4 lanes for each channel, VN states of a lane at a time.
template <typename T, int VN>
__global__ __launch_bounds__(256) void scan_step(const StepArgs b) {
    const ScanArgs& a = b.a;
    const int blocks = (a.D + 63) >> 6, i = blockIdx.x / blocks, q = threadIdx.x & 3;
    const int ch = (blockIdx.x - i * blocks) * 64 + (threadIdx.x >> 2);
    if (ch >= a.D) return;
    T* yp = (T*)a.y.p + (int64_t)i * a.y.row + ch;
    const int64_t slot = b.slots ? b.slots[i] : i;
    if (slot < 0 || slot >= b.num_slots) {
        if (q == 0) *yp = (T)0.0f;
        return;
    }
    const float x = (float)((const T*)a.x.p)[(int64_t)i * a.x.row + ch];
    float d = (float)((const T*)a.dt.p)[(int64_t)i * a.dt.row + ch];
    if (a.dt_bias) d += a.dt_bias[ch];
    if (a.softplus) d = softplus_f32(d);
    const int g = ch / a.Dg;
    const T* Bp = (const T*)a.B.p + (int64_t)i * a.B.row + g * a.N;
    const T* Cp = (const T*)a.C.p + (int64_t)i * a.C.row + g * a.N;
    float* hp = b.state + (slot * a.D + ch) * a.N;
    const float* Ap = a.A + (int64_t)ch * a.N;
    float v = 0.0f;
    for (int n = q * VN; n < a.N; n += 4 * VN) {
        float h[VN], A[VN];
        load_f32<float, VN>(hp + n, h);
        load_f32<float, VN>(Ap + n, A);
#pragma unroll
        for (int j = 0; j < VN; ++j) {
            const float e = __builtin_amdgcn_exp2f(d * (A[j] * kLog2e));
            h[j] = __builtin_fmaf(e, h[j], d * x * (float)Bp[n + j]);
            v = __builtin_fmaf(h[j], (float)Cp[n + j], v);
        }
        store_f32<float, VN>(hp + n, h);
    }
    v = quad_sum(v);
    if (q == 0) {
        if (a.D_skip) v = __builtin_fmaf(a.D_skip[ch], x, v);
        if (a.z.p) v *= silu_f32((float)((const T*)a.z.p)[(int64_t)i * a.z.row + ch]);
        *yp = (T)v;
    }
}

// States of a lane for N, and tokens of a chunk: as many as the registers
// hold decays for.
int states_for(int N) {
    int ns = 1;
    while (4 * ns < N) ns *= 2;
    return ns;
}
constexpr int chunk_for(int ns) { return ns <= 4 ? 16 : 64 / ns < 4 ? 4 : 64 / ns; }

ScanArgs args_of(const tg_scan_args& a, float* saved) {
    const int Dg = a.D / a.G;
    return {map_of(a.seqs), a.D, a.N, a.G, Dg, (int)ceil_div(Dg, kCh), a.softplus,
            rows_of<const void>(a.x), rows_of<const void>(a.dt), rows_of<const void>(a.B),
            rows_of<const void>(a.C), rows_of<const void>(a.z), rows_of<void>(a.y), a.A, a.D_skip,
            a.dt_bias, a.initial, a.final, saved};
}

#define TG_SCAN_NS(X, T)                           \
    do {                                           \
        switch (states_for(N)) {                   \
            case 1: X(T, 1); break;                \
            case 2: X(T, 2); break;                \
            case 4: X(T, 4); break;                \
            case 8: X(T, 8); break;                \
            case 16: X(T, 16); break;              \
            default: X(T, 32); break;              \
        }                                          \
    } while (0)
#define TG_SCAN_DISPATCH(X)                        \
    do {                                           \
        if (dtype == TG_F32) TG_SCAN_NS(X, float); \
        else if (dtype == TG_BF16) TG_SCAN_NS(X, bf16); \
        else TG_SCAN_NS(X, f16);                   \
    } while (0)

struct BackwardWs {
    size_t bc, a, d, total;
};
BackwardWs backward_ws(const tg_scan_args& a) {
    const int np = 4 * states_for(a.N), blocks = a.G * (int)ceil_div(a.D / a.G, kCh);
    BackwardWs w;
    w.bc = 0;
    w.a = up256((size_t)blocks * a.seqs.rows * 2 * np * sizeof(float));
    w.d = w.a + up256((size_t)a.seqs.seqs * a.D * a.N * sizeof(float));
    w.total = w.d + up256((size_t)a.seqs.seqs * 2 * a.D * sizeof(float));
    return w;
}

}  // namespace

void scan_sizes(const tg_scan_args& a, size_t* work, size_t* saved, size_t* backward) {
    const int ns = states_for(a.N);
    const int64_t slots = a.seqs.rows / chunk_for(ns) + a.seqs.seqs;
    if (work) *work = 0;
    if (saved) *saved = (size_t)slots * a.D * 4 * ns * sizeof(float);
    if (backward) *backward = backward_ws(a).total;
}

hipError_t launch_scan(const tg_scan_args& a, void*, void* saved, hipStream_t st) {
    const tg_dtype dtype = a.dtype;
    const int N = a.N;
    const ScanArgs f = args_of(a, (float*)saved);
    const unsigned grid = (unsigned)(f.G * f.bpg * a.seqs.seqs);
#define TG_X(T, NS) scan_fwd<T, NS, chunk_for(NS)><<<grid, 64, 0, st>>>(f)
    TG_SCAN_DISPATCH(TG_X);
#undef TG_X
    return hipGetLastError();
}

hipError_t launch_scan_backward(const tg_scan_args& a, const tg_scan_grads& g, const void* saved,
                                void* ws, hipStream_t st) {
    const tg_dtype dtype = a.dtype;
    const int N = a.N, np = 4 * states_for(N);
    const BackwardWs w = backward_ws(a);
    const ScanArgs f = args_of(a, nullptr);
    const ScanGrads b{rows_of<const void>(g.dy), g.dfinal, (const float*)saved,
                      rows_of<void>(g.dx), rows_of<void>(g.ddt), rows_of<void>(g.dz), g.dinitial,
                      (float*)ws, (float*)((char*)ws + w.a), (float*)((char*)ws + w.d)};
    const unsigned grid = (unsigned)(f.G * f.bpg * a.seqs.seqs);
#define TG_X(T, NS) scan_bwd<T, NS, chunk_for(NS)><<<grid, 64, 0, st>>>(f, b)
    TG_SCAN_DISPATCH(TG_X);
#undef TG_X
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.seqs.rows > 0) {
        const int64_t need = ceil_div(a.seqs.rows * a.G * 2 * np, 256);
        const unsigned sums = (unsigned)(need < 4096 ? need : 4096);
        const Rows<void> dB = rows_of<void>(g.dB), dC = rows_of<void>(g.dC);
        if (dtype == TG_F32) scan_bc_sums<float><<<sums, 256, 0, st>>>(f, b.part_bc, np, dB, dC);
        else if (dtype == TG_BF16) scan_bc_sums<bf16><<<sums, 256, 0, st>>>(f, b.part_bc, np, dB, dC);
        else scan_bc_sums<f16><<<sums, 256, 0, st>>>(f, b.part_bc, np, dB, dC);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const int seqs = (int)a.seqs.seqs;
    e = launch_column_sums(b.part_a, seqs, (int64_t)a.D * N, g.dA, (int64_t)a.D * N, nullptr, st);
    if (e != hipSuccess || (!g.dD && !g.ddt_bias)) return e;
    return launch_column_sums(b.part_d, seqs, 2 * (int64_t)a.D, g.dD, a.D, g.ddt_bias, st);
}

hipError_t launch_scan_step(const tg_scan_args& a, float* state, int64_t num_slots,
                            const int32_t* slots, hipStream_t st) {
    const StepArgs b{args_of(a, nullptr), state, num_slots, slots};
    const unsigned grid = (unsigned)(ceil_div(a.D, 64) * a.seqs.seqs);
    const bool v4 = a.N % 4 == 0 && ((uintptr_t)state & 15) == 0 && ((uintptr_t)a.A & 15) == 0;
#define TG_X(T)                                                  \
    do {                                                         \
        if (v4) scan_step<T, 4><<<grid, 256, 0, st>>>(b);        \
        else scan_step<T, 1><<<grid, 256, 0, st>>>(b);           \
    } while (0)
    if (a.dtype == TG_F32) TG_X(float);
    else if (a.dtype == TG_BF16) TG_X(bf16);
    else TG_X(f16);
#undef TG_X
    return hipGetLastError();
}

}  // namespace tg
