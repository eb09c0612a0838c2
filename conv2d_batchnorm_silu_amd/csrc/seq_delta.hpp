// seq_delta.hpp -- what the gated delta rule's kernels share: numbers held as
// sums of bf16 parts, their fragments for the matrix instructions, the staging
// of rows in LDS, and the layout of a chunk's prepared matrices.
//
// Every product goes through v_mfma_f32_16x16x32_bf16. A bf16 input is its own first
// part, an fp16 input two parts (exactly), an fp32 input three (24 bits). What lies
// between is split into two parts for prompts of 16-bit tensors (off by at most
// 2^-18; the product of two low parts, as small, is dropped), so that states,
// which are fp32, keep 17 bits at two or three matrix instructions a product; fp16
// instructions would take one, but have 11 bits and not the range of states. In
// training, and for fp32, it is three parts: the gradients of A and dt_bias are
// fp32 sums over all tokens that cancel (17 bits left them off by up to 6e-5).
// Six instructions a product are fewer than the fp32 matrix instructions' sixteen.
// Products that only reach an output of the tensors' type take as many parts as an
// input has.
//
// Fragments. Lane l of a wave holds row (of the left operand) or column (of the
// right) l % 16 and, with g = l / 16, the eight inner indices 4g .. 4g+3 and
// 16 + 4g .. 16 + 4g+3 of a block of 32, in both operands alike. That is the
// order in which two accumulators of 16 x 16 (lane: column l % 16, rows 4g ..
// 4g+3) lie one below the other, so a product's result is the next product's
// operand without leaving its registers.
#pragma once

#include "seq_device.hpp"
#include "seq_internal.hpp"

namespace tg {

typedef bf16 bf16x4_t __attribute__((ext_vector_type(4)));
typedef bf16 bf16x8_t __attribute__((ext_vector_type(8)));

constexpr float kUnitEps = 1e-6f;  // added to the squared length of a normalised q or k

template <typename T>
inline constexpr int kIn = sizeof(T) == 4 ? 3 : 2;  // parts of an input
template <>
inline constexpr int kIn<bf16> = 1;
template <typename T>
inline constexpr int kMid = sizeof(T) == 4 ? 3 : 2;  // parts of an intermediate in a prompt
constexpr int kTrain = 3;                            // and in training

// Tokens of a chunk: 64, or 32 where two chunks' parts of q and k (padded to KP) and
// the matrices made from them would not fit LDS together.
constexpr int delta_chunk(int in, int KP) { return in == 1 && KP <= 128 ? 64 : 32; }

template <int N>
struct Frag {
    bf16x8_t p[N];
};

template <int N>
__device__ __forceinline__ void split(float x, bf16 (&p)[N]) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
        p[n] = (bf16)x;
        x -= (float)p[n];
    }
}
template <int N>
__device__ __forceinline__ Frag<N> frag_of(const float (&v)[8]) {
    Frag<N> f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        bf16 p[N];
        split<N>(v[j], p);
#pragma unroll
        for (int n = 0; n < N; ++n) f.p[n][j] = p[n];
    }
    return f;
}
template <int N>
__device__ __forceinline__ Frag<N> frag_of(const float4_t& a, const float4_t& b) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = a[j], v[4 + j] = b[j];
    return frag_of<N>(v);
}
// The inner index of a fragment's element j in its block of 32.
__device__ __forceinline__ int frag_at(int g, int j) { return 16 * (j >> 2) + 4 * g + (j & 3); }

// c += a b, the products of parts i and j with i + j < N, small ones first.
template <int N, int NA, int NB>
__device__ __forceinline__ void mma(float4_t& c, const Frag<NA>& a, const Frag<NB>& b) {
#pragma unroll
    for (int s = N - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i <= s; ++i)
            if (i < NA && s - i < NB)
                c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[i], b.p[s - i], c, 0, 0, 0);
}

// A matrix in LDS, in N planes of parts: row r of a plane at r * ld elements.
template <int N>
struct Planes {
    bf16* p;
    int ld, plane;
    // Rows row0 .. +15 as the outer index, columns k0 .. +31 as the inner one.
    __device__ __forceinline__ Frag<N> rows(int row0, int k0) const {
        const int l = threadIdx.x & 63;
        const bf16* at = p + (row0 + (l & 15)) * ld + k0 + 4 * (l >> 4);
        Frag<N> f;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const bf16x4_t a = *(const bf16x4_t*)(at + n * plane);
            const bf16x4_t b = *(const bf16x4_t*)(at + n * plane + 16);
            f.p[n] = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        }
        return f;
    }
    // Columns col0 .. +15 as the outer index, rows k0 .. +31 as the inner one: the
    // transposing read gives lane i of 16 the four rows of column i when lane i
    // points at columns 4(i%4) .. +3 of row i/4.
    __device__ __forceinline__ Frag<N> cols(int k0, int col0) const {
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        const int l = threadIdx.x & 63, i = l & 15;
        bf16* at = p + (k0 + 4 * (l >> 4) + (i >> 2)) * ld + col0 + 4 * (i & 3);
        Frag<N> f;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + n * plane));
            const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_s16x4*)(at + n * plane + 16 * ld));
            f.p[n] = __builtin_bit_cast(bf16x8_t,
                                        __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
        }
        return f;
    }
    __device__ __forceinline__ float at(int r, int c) const {
        float v = 0.0f;
#pragma unroll
        for (int n = N - 1; n >= 0; --n) v += (float)p[n * plane + r * ld + c];
        return v;
    }
    __device__ __forceinline__ void put(int r, int c, float v) const {
        bf16 q[N];
        split<N>(v, q);
#pragma unroll
        for (int n = 0; n < N; ++n) p[n * plane + r * ld + c] = q[n];
    }
};

// Eight elements of a row on their way through registers.
template <typename T>
struct Eight {
    typename VecOf<T, 8>::type r;
    // Up to n from p on (n <= 0: none), zeros behind; wide: all eight are there and
    // lie on 16 bytes where n > 0.
    __device__ __forceinline__ void load(const T* p, int n, bool wide) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = (T)0.0f;
        if (wide) {
            if (n > 0) r = *(const typename VecOf<T, 8>::type*)p;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) r[j] = p[j];
        }
    }
    template <int N>
    __device__ __forceinline__ void put(const Planes<N>& d, int row, int c) const {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = (float)r[j];
        const Frag<N> f = frag_of<N>(x);
#pragma unroll
        for (int q = 0; q < N; ++q) *(bf16x8_t*)(d.p + q * d.plane + row * d.ld + c) = f.p[q];
    }
};

// R rows of W columns of T from src (rows `stride` apart) as eights, by `THREADS`
// threads: fetch() starts the loads, put() writes them as parts; zeros past n
// rows and m columns. More than one batch in flight where COUNT is more than one.
template <typename T, int R, int W, int THREADS>
struct Tile {
    static constexpr int total = R * W / 8, COUNT = (total + THREADS - 1) / THREADS;
    Eight<T> e[COUNT];
    __device__ __forceinline__ void fetch(int tid, const T* src, int64_t stride, int n, int m,
                                          bool wide) {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            const int at = i * THREADS + tid, r = at / (W / 8), c = at % (W / 8) * 8;
            const bool in = total % THREADS == 0 || at < total;
            e[i].load(src + r * stride + c, in && r < n ? m - c : 0, wide);
        }
    }
    template <int N>
    __device__ __forceinline__ void put(int tid, const Planes<N>& d) const {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            const int at = i * THREADS + tid;
            if (total % THREADS == 0 || at < total) e[i].put(d, at / (W / 8), at % (W / 8) * 8);
        }
    }
};
// The same in one go.
template <typename T, int R, int W, int THREADS, int N>
__device__ __forceinline__ void stage(const Planes<N>& d, const T* src, int64_t stride, int n, int m,
                                      bool wide) {
    Tile<T, R, W, THREADS> t;
    t.fetch(threadIdx.x, src, stride, n, m, wide);
    t.put(threadIdx.x, d);
}

// What a chunk's tokens scale by (rows of `scal`, C floats each); G the decays'
// logarithms added up from the chunk's first token, rk and rq the inverse lengths.
enum DeltaScale {
    kReadK,   // e^G rk: the state before the chunk, read by k
    kWrite,   // e^(G_last - G) rk b: what a correction adds to the state after it
    kBeta,    // b
    kReadQ,   // e^G rq scale
    kTailK,   // e^(G_last - G) rk
    kUnitK,   // rk
    kUnitQ,   // rq
    kDecay,   // e^G
    kScales
};

// A chunk's prepared matrices: its scales, then fragments (1 KB each part) of
// X = (I + N)^-1 and of P. Below the diagonal blocks of 16 x 32 there are
// frag_count() of them; transposed, the same number.
constexpr int frag_count(int C) { return C == 64 ? 6 : 2; }
// Fragment of rows 16 mt .. of the lower triangle and columns 32 kt ..; of
// the upper triangle for a transposed one.
constexpr int frag_index(int C, int mt, int kt, bool upper) {
    return C == 32 ? mt : upper ? (kt == 1 ? mt : 4 + mt) : (kt == 0 ? mt : 2 + mt);
}
constexpr bool frag_used(int C, int mt, int kt, bool upper) {
    return C == 32 || (upper ? kt == 1 || mt < 2 : kt == 0 || mt >= 2);
}
constexpr int prep_bytes(int C, int parts) { return kScales * C * 4 + frag_count(C) * 1024 * parts; }

struct DeltaArgs {
    SeqMap map;
    int HK, HV, K, V;
    int softplus, sigmoid, normalize;
    float scale;
    Rows<const void> q, k, v, dt, beta;
    Rows<void> y;
    const float *A, *dt_bias, *initial;
    float* final;
    bool wide_qk, wide_v, wide_y, wide_s;  // 16-byte rows of q and k, of v, of y (4 values), of saved states
    char* prep;    // [slots][HV] of prep_bytes
    float* saved;  // [slots][HV] of K*V + C*V, or null
    // The backward pass.
    Rows<const void> dy;
    Rows<void> dq, dk, dv, ddt, dbeta;
    bool wide_dy;
    const float* dfinal;
    float *dinitial, *back;  // back: like saved
    float* part;             // [slots][2][HV]
};

inline int64_t delta_slots(const tg_seqs& s, int C) {
    return s.offsets ? s.rows / C + s.seqs : s.seqs * ceil_div(s.rows / s.seqs, C);
}
inline int delta_padded(int K) { return K <= 64 ? 64 : K <= 128 ? 128 : 256; }
inline int delta_in(tg_dtype d) { return d == TG_BF16 ? 1 : d == TG_F16 ? 2 : 3; }
inline int delta_chunk_of(const tg_delta_args& a) {
    return delta_chunk(delta_in(a.dtype), delta_padded(a.K));
}

// The chunk of (sequence, slice of the columns) that a workgroup of the serial
// kernels has: slices of one head on one XCD (workgroups go round the 8 XCDs),
// whose L2 then holds that head's q and k once.
struct HeadSlice {
    int pair, slice;
};
__device__ __forceinline__ HeadSlice head_slice(int slices) {
    const int b = blockIdx.x;
    return {(b / 8 / slices) * 8 + b % 8, (b / 8) % slices};
}
inline int64_t head_slice_grid(int64_t pairs, int slices) { return ceil_div(pairs, 8) * 8 * slices; }

// The step size, its slope, the decay's logarithm to base 2 and b of a token.
struct DeltaGate {
    float d, slope, g2, b;
};
__device__ __forceinline__ DeltaGate delta_gate(const DeltaArgs& a, float dt, float beta, int h) {
    DeltaGate o;
    const float raw = dt + (a.dt_bias ? a.dt_bias[h] : 0.0f);
    if (a.softplus) softplus_grad_f32(raw, o.d, o.slope);
    else o.d = raw, o.slope = 1.0f;
    // A step of zero keeps the state for any rate. Decays are taken as 0 long before
    // 2^-150 and as infinite long before 2^1000: infinite sums have no differences.
    float g = o.d == 0.0f ? 0.0f : a.A[h] * o.d * kLog2e;
    g = g < -150.0f ? -150.0f : g > 1000.0f ? 1000.0f : g;
    o.g2 = g;
    o.b = a.sigmoid ? sigmoid_f32(beta) : beta;
    return o;
}
__device__ __forceinline__ double wave_prefix(double v) {
    const int l = threadIdx.x & 63;
#pragma unroll
    for (int s = 1; s < 64; s *= 2) {
        const double u = __shfl_up(v, s);
        if (l >= s) v += u;
    }
    return v;
}
__device__ __forceinline__ float decay_between(double hi, double lo) {
    return __builtin_amdgcn_exp2f((float)(hi - lo));
}

// The serial kernels: a workgroup has up to two waves that compute, 16 columns each,
// and loaders before them that bring the next chunk's rows and matrices to LDS
// (through registers: rows of any stride, split into parts once for all columns)
// while the first work on this one's; the loads of the one after that are then on
// their way. With one set of buffers (stages == 1, where two do not fit) loads still
// are a chunk ahead, but their writing waits for the computation.
constexpr int kMaxColumns = 2;
// Four loading waves; two where a computing wave needs more than 256 registers, half of
// its SIMD's.
constexpr int delta_loaders(int KP) { return KP == 256 ? 2 : 4; }

// One chunk on its way: q, k, the prepared matrices (PREP bytes) and rows of 16
// or 32 columns of a V-wide tensor.
template <typename T, int KP, int C, int PREP>
struct ChunkLoad {
    static constexpr int kLoadThreads = delta_loaders(KP) * 64;
    static constexpr int NP = (PREP / 16 + kLoadThreads - 1) / kLoadThreads;
    Tile<T, C, KP, kLoadThreads> q, k;
    float4 p[NP];
    Tile<T, C, kMaxColumns * 16, kLoadThreads> v;
    __device__ __forceinline__ void fetch(const DeltaArgs& a, const Rows<const void>& vr, bool wide_v,
                                          int s, int start, int lo, int n, int hk, int h, int v0,
                                          int64_t chunk) {
        const int tid = threadIdx.x % kLoadThreads;
        k.fetch(tid, row_of<const T>(a.k, a.map, s, start, lo) + (int64_t)hk * a.K, a.k.row, n, a.K,
                a.wide_qk);
        q.fetch(tid, row_of<const T>(a.q, a.map, s, start, lo) + (int64_t)hk * a.K, a.q.row, n, a.K,
                a.wide_qk);
        const float4* src = (const float4*)(a.prep + chunk * PREP);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int at = i * kLoadThreads + tid;
            if (PREP / 16 % kLoadThreads == 0 || at < PREP / 16) p[i] = src[at];
        }
        v.fetch(tid, row_of<const T>(vr, a.map, s, start, lo) + (int64_t)h * a.V + v0, vr.row, n,
                a.V - v0, wide_v);
    }
    template <int N>
    __device__ __forceinline__ void put(float4* prep, const Planes<N>& kp, const Planes<N>& qp) const {
        const int tid = threadIdx.x % kLoadThreads;
        k.put(tid, kp);
        q.put(tid, qp);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int at = i * kLoadThreads + tid;
            if (PREP / 16 % kLoadThreads == 0 || at < PREP / 16) prep[at] = p[i];
        }
    }
};

// One fragment of the prepared matrices, N parts, from LDS.
template <int N>
__device__ __forceinline__ Frag<N> prepared(const bf16* f, int index) {
    Frag<N> o;
#pragma unroll
    for (int q = 0; q < N; ++q)
        o.p[q] = *(const bf16x8_t*)(f + (index * N + q) * 512 + (threadIdx.x & 63) * 8);
    return o;
}

// NM: parts of X; BACK: the transposed matrices.
template <typename T, int NM, bool BACK>
hipError_t launch_delta_prep(const DeltaArgs& a, int KP, int64_t slots, hipStream_t st);
extern template hipError_t launch_delta_prep<float, kTrain, true>(const DeltaArgs&, int, int64_t, hipStream_t);
extern template hipError_t launch_delta_prep<f16, kTrain, true>(const DeltaArgs&, int, int64_t, hipStream_t);
extern template hipError_t launch_delta_prep<bf16, kTrain, true>(const DeltaArgs&, int, int64_t, hipStream_t);

DeltaArgs delta_args(const tg_delta_args& a);
// Waves that compute (16 columns each) in a serial kernel's workgroups.
inline int delta_waves(int V) { return V > 16 ? 2 : 1; }

}  // namespace tg
