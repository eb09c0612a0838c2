// seq_delta.hpp -- what the gated delta rule's kernels share: numbers held as
// sums of bf16 parts, their fragments for the matrix instructions, the staging
// of rows in LDS, and the layout of a chunk's prepared matrices.
//
// Every product goes through v_mfma_f32_16x16x32_bf16. A bf16 input is its own first
// part, an fp16 input two parts (exactly), an fp32 input three (24 bits). What lies
// between is split into three, so that states and the gradients of parameters, which
// are fp32, are as exact as fp32 products would leave them: at three to six
// instructions a product, fewer than the fp32 matrix instructions' sixteen, and with
// fp32's range, which fp16 parts would not have.
//
// That holds for prompts too, where two parts (17 bits) left the fp32 states off by 2 to
// 5e-6 of their norm, ten times as much, for a walk of 185 us in place of 225 (4 x 4096
// tokens of 16 heads). Products that only reach y, or only the gradients of q and k, take two parts of
// 16-bit tensors: a single one left bf16 outputs off by 1.6 times their rounding, dq and
// dk by 1.3, and by any share where most of them is taken off again along q and k.
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
inline constexpr int kOut = kIn<T> > 2 ? 3 : 2;  // of what only reaches y, dq or dk
constexpr int kParts = 3;                        // of what lies between

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

// c[m] += a[m] b, or a b[m], where m is used, the same products: independent
// accumulators in turn, as one has to wait for its last product.
template <int N, int M, int NA, int NB, typename Used>
__device__ __forceinline__ void mma_rows(float4_t (&c)[M], const Frag<NA> (&a)[M], const Frag<NB>& b,
                                         Used used) {
#pragma unroll
    for (int s = N - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i <= s; ++i)
            if (i < NA && s - i < NB)
#pragma unroll
                for (int m = 0; m < M; ++m)
                    if (used(m))
                        c[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[m].p[i], b.p[s - i], c[m], 0,
                                                                       0, 0);
}
template <int N, int M, int NA, int NB, typename Used>
__device__ __forceinline__ void mma_cols(float4_t (&c)[M], const Frag<NA>& a, const Frag<NB> (&b)[M],
                                         Used used) {
#pragma unroll
    for (int s = N - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i <= s; ++i)
            if (i < NA && s - i < NB)
#pragma unroll
                for (int m = 0; m < M; ++m)
                    if (used(m))
                        c[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[i], b[m].p[s - i], c[m], 0,
                                                                       0, 0);
}
struct All {
    __device__ __forceinline__ constexpr bool operator()(int) const { return true; }
};

// Whether any of these is infinite or NaN, found by a sum: then it is not 0.
__device__ __forceinline__ float strange(float sum, const float4_t& v) {
#pragma unroll
    for (int j = 0; j < 4; ++j) sum = __builtin_fmaf(v[j], 0.0f, sum);
    return sum;
}
// A right operand's block of 32 tokens t without what is infinite or NaN (a first part
// tells): products with zeros above a diagonal would take it to tokens before its own.
// `from` becomes the first such token of the lane's column.
template <int N>
__device__ __forceinline__ void put_aside(Frag<N>& f, int t, int& from) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int j = 7; j >= 0; --j) {
        const float v = (float)f.p[0][j];
        if (v - v == 0.0f) continue;
        from = imin(from, t * 32 + frag_at(g, j));
#pragma unroll
        for (int n = 0; n < N; ++n) f.p[n][j] = (bf16)0.0f;
    }
}
__device__ __forceinline__ int column_least(int v) {
    v = imin(v, __shfl_xor(v, 16));
    return imin(v, __shfl_xor(v, 32));
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

// R rows of W columns of T on their way through the registers of THREADS threads,
// eight elements in each: fetch() starts the loads, put() writes them as parts, with
// zeros past n >= 0 rows and m >= 1 columns. WIDE: m and all addresses are multiples of
// eight elements (of 16 bytes for fp32). What lies outside is loaded from the last
// row and column inside and dropped in put(): a load under a condition, into
// registers that would have to be zeroed before, would wait for all loads on
// their way. A thread's offsets are 32-bit and found once, its addresses are a
// uniform pointer and an offset.
template <typename T, int R, int W, int THREADS, bool WIDE>
struct Tile {
    typedef typename VecOf<T, 8>::type eight;
    static constexpr int total = R * W / 8, COUNT = (total + THREADS - 1) / THREADS;
    eight e[COUNT];
    uint32_t off[COUNT];
    uint32_t stride;
    int n, m;
    __device__ __forceinline__ static int tid() { return threadIdx.x % THREADS; }
    __device__ __forceinline__ static int row(int i) { return (i * THREADS + tid()) / (W / 8); }
    __device__ __forceinline__ static int column(int i) { return (i * THREADS + tid()) % (W / 8) * 8; }
    __device__ __forceinline__ static bool inside(int i) {
        return total % THREADS == 0 || i * THREADS + tid() < total;
    }
    __device__ __forceinline__ void shape(int64_t row_stride, int cols) {
        stride = (uint32_t)row_stride;
        m = cols;
#pragma unroll
        for (int i = 0; i < COUNT; ++i)
            off[i] = (uint32_t)imin(row(i), R - 1) * stride +
                     (uint32_t)(WIDE ? imin(column(i), m - 8) : imin(column(i), m - 1));
    }
    __device__ __forceinline__ void fetch(const T* src, int rows) {
        n = imin(rows, R);
        if (WIDE && n == R) {
#pragma unroll
            for (int i = 0; i < COUNT; ++i) e[i] = *(const eight*)(src + off[i]);
            return;
        }
        const int last = n > 0 ? n - 1 : 0;
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            const int r = imin(row(i), R - 1);
            const T* p = src + (off[i] - (uint32_t)(r - imin(r, last)) * stride);
            if constexpr (WIDE) {
                e[i] = *(const eight*)p;
            } else {
                const int left = m - 1 - imin(column(i), m - 1);
#pragma unroll
                for (int j = 0; j < 8; ++j) e[i][j] = p[imin(j, left)];
            }
        }
    }
    __device__ __forceinline__ eight value(int i) const {
        if (WIDE && n == R && m == W) return e[i];
        const int r = row(i), c = column(i);
        eight o;
        if constexpr (WIDE) {
            const bool ok = r < n && c < m;
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = ok ? e[i][j] : (T)0.0f;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = r < n && c + j < m ? e[i][j] : (T)0.0f;
        }
        return o;
    }
    template <int N>
    __device__ __forceinline__ void put(const Planes<N>& d) const {
        if (WIDE && n == R && m == W) put_values<N, true>(d);
        else put_values<N, false>(d);
    }
    template <int N, bool FULL>
    __device__ __forceinline__ void put_values(const Planes<N>& d) const {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            if (!inside(i)) continue;
            const eight v = FULL ? e[i] : value(i);
            bf16* at = d.p + row(i) * d.ld + column(i);
            if constexpr (sizeof(T) == 2 && N == 1) {
                *(eight*)at = v;
            } else {
                float x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = (float)v[j];
                const Frag<N> f = frag_of<N>(x);
#pragma unroll
                for (int q = 0; q < N; ++q) *(bf16x8_t*)(at + q * d.plane) = f.p[q];
            }
        }
    }
    // As they are, into rows of ld elements.
    __device__ __forceinline__ void put_raw(T* d, int ld) const {
#pragma unroll
        for (int i = 0; i < COUNT; ++i)
            if (inside(i)) *(eight*)(d + row(i) * ld + column(i)) = value(i);
    }
};

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

// What the passes keep for a chunk (`saved`: the state before it and its corrections;
// `back`: the gradient of the state after it and of v): for each 16 columns of V the
// accumulators of KP/16 and C/16 tiles as they are, four floats of a lane after the
// other, so that a wave writes a kilobyte at a time (2 x 2048 tokens of 16 heads: the
// backward walk takes 107 us, with rows of V 178). In floats:
inline __host__ __device__ int64_t kept_floats(int V, int KP, int C) {
    return (int64_t)((V + 15) / 16) * (KP / 16 + C / 16) * 256;
}
// Tile `tile` (S's first) of 16 columns vt.
__device__ __forceinline__ float4_t* kept_at(float* chunk, int KP, int C, int vt, int tile) {
    return (float4_t*)(chunk + ((int64_t)vt * (KP / 16 + C / 16) + tile) * 256) + (threadIdx.x & 63);
}

struct DeltaArgs {
    SeqMap map;
    int HK, HV, K, V;
    int softplus, sigmoid, normalize;
    float scale;
    Rows<const void> q, k, v, dt, beta;
    Rows<void> y;
    const float *A, *dt_bias, *initial;
    float* final;
    bool wide_qk, wide_v, wide_y;  // rows of 16 bytes of q and k, of v, of 4 values of y
    // Long sequences in segments (0: whole sequences) of whole chunks, a workgroup for
    // each: see seq_delta_segments.hip.
    int segment;
    int units;      // sequences, or the segments of all
    bool through;   // what a segment makes of a state is wanted, not y
    float* maps;    // [units][HV][KP][map_columns()]
    char* prep;    // [slots][HV] of prep_bytes
    float* saved;  // [slots][HV] of kept_floats(), or null
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
inline int delta_out(tg_dtype d) { return d == TG_F32 ? 3 : 2; }
inline int delta_in(tg_dtype d) { return d == TG_BF16 ? 1 : d == TG_F16 ? 2 : 3; }
inline int delta_chunk_of(const tg_delta_args& a) {
    return delta_chunk(delta_in(a.dtype), delta_padded(a.K));
}

// The segment (or sequence) that a workgroup of the serial kernels has: sequence s,
// rows lo .. hi-1 of its len.
struct Segment {
    int s, start, len, lo, hi;
    __device__ __forceinline__ bool find(const DeltaArgs& a, int unit) {
        s = a.segment ? a.map.owner(unit, a.segment) : unit;
        start = a.map.start(s);
        len = a.map.end(s) - start;
        lo = 0;
        hi = len;
        return !a.segment || SeqMap::piece(unit, a.map.slot0(s, a.segment), len, a.segment, lo, hi);
    }
};
// Columns of a segment's map of states: those of V, rounded up to a slice, and KP.
inline __host__ __device__ int map_columns(int V, int KP, int slice) {
    return (V + slice - 1) / slice * slice + KP;
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
// Within each 16 lanes: the value N lanes below (0 where there is none), and the sum of
// the lanes up to one's own.
template <int N>
__device__ __forceinline__ float row_shift16(float v) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x110 + N, 0xF, 0xF, false));
}
__device__ __forceinline__ float row_prefix16(float v) {
    v += row_shift16<1>(v);
    v += row_shift16<2>(v);
    v += row_shift16<4>(v);
    v += row_shift16<8>(v);
    return v;
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

// The serial kernels. A workgroup has 32 columns of V (16 where more do not fit LDS) and
// for each 16 of them two waves that carry S, and two that help. Wave (ct, hf) of the
// first has the 16 columns of ct, the half hf of S's K rows (in its accumulators)
// and the half hf of a chunk's tokens. What a product sums over all K rows is formed
// as two halves for all tokens and joined through LDS; what a token has found is given
// to the other half as fragments. So a chunk takes three barriers more than with
// a wave for 16 whole columns, but half the instructions one after another, and each
// SIMD has such a wave.
//
// The helpers bring rows of q, k and v to LDS through registers (rows of any stride,
// split into parts once for all columns), a chunk ahead and the loads another
// chunk ahead, and form what the recurrence does not wait for. A wave loads the
// prepared fragments of its own tokens to registers as soon as it has used the last
// chunk's. 4 x 4096 tokens of 16 heads of 128 x 128, bf16: a wave for 16 whole columns and
// four that load 215 us, four waves that share S and everything else 230, with helpers
// 164 (185 since y is made of two parts, 225 since the states always take three): 3.5 us a
// chunk, half of all wave cycles waits for LDS, matrix results and barriers.
constexpr int slice_of(int in, int KP) { return in * KP > 512 ? 16 : 32; }

// A barrier for what lies in LDS: __syncthreads would also wait for the loads and
// stores of global memory that are on their way.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Half fragments (the four rows that a lane has of a tile of 16) of N parts in LDS.
template <int N>
struct HalfFrags {
    bf16* p;
    __device__ __forceinline__ bf16x4_t* at(int tile, int n) const {
        return (bf16x4_t*)(p + ((tile * N + n) * 64 + (threadIdx.x & 63)) * 4);
    }
    __device__ __forceinline__ void put(int tile, const float4_t& v) const {
        bf16x4_t o[N];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            bf16 q[N];
            split<N>(v[j], q);
#pragma unroll
            for (int n = 0; n < N; ++n) o[n][j] = q[n];
        }
#pragma unroll
        for (int n = 0; n < N; ++n) *at(tile, n) = o[n];
    }
    // Of tiles 2t and 2t + 1.
    __device__ __forceinline__ Frag<N> frag(int t) const {
        Frag<N> f;
#pragma unroll
        for (int n = 0; n < N; ++n)
            f.p[n] = __builtin_shufflevector(*at(2 * t, n), *at(2 * t + 1, n), 0, 1, 2, 3, 4, 5, 6, 7);
        return f;
    }
};
__device__ __forceinline__ float4_t* sum_at(float* p, int tile) {
    return (float4_t*)(p + (tile * 64 + (threadIdx.x & 63)) * 4);
}

// One fragment of the prepared matrices, N parts, from the workspace.
template <int N>
__device__ __forceinline__ void prepared(Frag<N>& o, const bf16* f, int index) {
#pragma unroll
    for (int q = 0; q < N; ++q)
        o.p[q] = *(const bf16x8_t*)(f + (index * N + q) * 512 + (threadIdx.x & 63) * 8);
}

// A scale of the four rows that a lane has of tile mt.
__device__ __forceinline__ float4_t scales(const float* scal, int C, DeltaScale which, int mt) {
    return *(const float4_t*)(scal + which * C + mt * 16 + 4 * ((threadIdx.x & 63) >> 4));
}

// The kernels' launches; BACK: the transposed matrices.
template <typename T, bool BACK>
hipError_t launch_delta_prep(const DeltaArgs& a, int KP, int64_t slots, hipStream_t st);
template <typename T>
hipError_t launch_delta_forward(const DeltaArgs& a, int KP, hipStream_t st);
template <typename T>
hipError_t launch_delta_states(const DeltaArgs& a, int KP, hipStream_t st);
// The states before (reverse: their gradients after) each segment from those before the
// first (after the last): [units][HV][K][V].
hipError_t launch_delta_join(const DeltaArgs& a, const float* first, bool reverse, float* states, int KP,
                             int slice, hipStream_t st);
template <typename T>
hipError_t launch_delta_grads(const DeltaArgs& a, int KP, int64_t slots, hipStream_t st);

DeltaArgs delta_args(const tg_delta_args& a);

}  // namespace tg
