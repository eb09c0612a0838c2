// seq_delta.hip -- the gated delta rule's forward pass: prompts in chunks, and
// single tokens (tg_gated_delta_rule, tg_gated_delta_rule_step).
//
// In a chunk of C tokens, with S0 the K x V state before it, G the logarithms of
// the decays added up from its first token and D[i,j] = e^(G[i]-G[j]), the
// corrections E[i] = v[i] - k[i] S (S decayed to token i) solve
//     (I + N) E = v - e^G k S0,   N[i,j] = D[i,j] (k[i].k[j]) b[j] for j < i
// and  y = e^G q S0 + P b E,      P[i,j] = D[i,j] (q[i].k[j]) for j <= i
//      S = e^(G[C-1]) S0 + (e^(G[C-1]-G) k)^T b E.
// X = (I + N)^-1 and P need no state: one kernel makes them for all chunks at
// once. The other walks down a sequence's chunks; the V columns of S are
// independent, so each wave carries 16 of them, S in its accumulators, with q, k
// and the prepared matrices shared in LDS.
//
// q and k enter the products as they are; their inverse lengths, the decays, b
// and the scale are factors of rows, applied to accumulators in fp32.
//
// The matrices take 66 us for 4 x 4096 tokens of 16 heads of 128 (4.1 TB/s of q and k read
// and matrices written), 22 us for a quarter of them in training.
#include "seq_delta.hpp"
#include "tg_internal.hpp"

namespace tg {
namespace {

// c += A B over a block of 16: fp32 matrix instructions on 16 x 16 blocks of a
// matrix in LDS (the inverse is formed in fp32 throughout: its entries multiply
// each other up to C times). b: an accumulator as the right operand.
__device__ __forceinline__ void mm16(float4_t& c, const float* A, int ld, const float4_t& b) {
    const int l = threadIdx.x & 63, g = l >> 4;
#pragma unroll
    for (int s = 0; s < 4; ++s)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(A[(l & 15) * ld + 4 * g + s], b[s], c, 0, 0, 0);
}
__device__ __forceinline__ float4_t block16(const float* B, int ld) {
    const int l = threadIdx.x & 63, g = l >> 4;
    float4_t b;
#pragma unroll
    for (int s = 0; s < 4; ++s) b[s] = B[(4 * g + s) * ld + (l & 15)];
    return b;
}
__device__ __forceinline__ void put16(float* B, int ld, const float4_t& b, float sign) {
    const int l = threadIdx.x & 63, g = l >> 4;
#pragma unroll
    for (int s = 0; s < 4; ++s) B[(4 * g + s) * ld + (l & 15)] = sign * b[s];
}

// X = (I + N)^-1 in place of N (strictly lower, zeros above) by four waves:
// the diagonal blocks of 16 row by row, a lane for each column; then
// [[A, 0], [B, D]]^-1 = [[A', 0], [-D' B A', D']] for blocks of 16 and of 32.
template <int C, int LD>
__device__ __forceinline__ void invert(float* m) {
    const int w = threadIdx.x >> 6, l = threadIdx.x & 63, c = l & 15;
    float* d = m + w * 16 * (LD + 1);
    if (w < C / 16) {
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = i == c ? 1.0f : 0.0f;
#pragma unroll
            for (int j = 0; j < i; ++j) s = __builtin_fmaf(-d[i * LD + j], x[j], s);
            x[i] = s;
        }
        // All of the wave's reads are done before these writes: one wave's LDS
        // operations are in order.
        if (l < 16)
#pragma unroll
            for (int i = 0; i < 16; ++i) d[i * LD + c] = x[i];
    }
    lds_barrier();
    if (w < C / 32) {
        float* b = m + w * 32 * (LD + 1) + 16 * LD;  // the block below the first diagonal one
        float4_t t = {0, 0, 0, 0}, u = {0, 0, 0, 0};
        mm16(t, b, LD, block16(b - 16 * LD, LD));
        mm16(u, b + 16, LD, t);
        put16(b, LD, u, -1.0f);
    }
    lds_barrier();
    if constexpr (C == 64) {
        float4_t u[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
        float* b = m + 32 * LD;
        if (w < 2) {  // a wave for each column of blocks
            float4_t t[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (k < w) continue;
                const float4_t a = block16(m + k * 16 * LD + w * 16, LD);
                mm16(t[0], b + k * 16, LD, a);
                mm16(t[1], b + 16 * LD + k * 16, LD, a);
            }
            mm16(u[0], b + 32, LD, t[0]);
            mm16(u[1], b + 16 * LD + 32, LD, t[0]);
            mm16(u[1], b + 16 * LD + 48, LD, t[1]);
        }
        lds_barrier();
        if (w < 2) {
            put16(b + w * 16, LD, u[0], -1.0f);
            put16(b + 16 * LD + w * 16, LD, u[1], -1.0f);
        }
        lds_barrier();
    }
}

template <typename T, int KP>
struct PrepShape {
    static constexpr int NI = kIn<T>, C = delta_chunk(NI, KP), LD = KP + 8, ML = C + 4;
    // The matrices take the place of q and k.
    static constexpr int square = 2 * C * ML * 4, rows = 2 * NI * C * LD * 2;
    static constexpr int lds = kScales * C * 4 + C * 8 + (square > rows ? square : rows) + 16;
};

// One workgroup for a chunk and value head. BACK: the transposed matrices.
template <typename T, int KP, bool BACK, bool WIDE>
__global__ __launch_bounds__(256) void delta_prep(const DeltaArgs a) {
    using Sh = PrepShape<T, KP>;
    constexpr int NI = Sh::NI, C = Sh::C, LD = Sh::LD, ML = Sh::ML, NT = C / 16;
    constexpr int PP = BACK ? kParts : kOut<T>;  // parts of P
    extern __shared__ float4 lds[];
    float* scal = (float*)lds;
    double* G = (double*)(scal + kScales * C);
    float* mat = (float*)(G + C);
    float* pm = mat + C * ML;
    int* odd = (int*)((char*)lds + Sh::lds - 16);  // the first token whose row of N is not finite
    const Planes<NI> kp{(bf16*)mat, LD, C * LD}, qp{kp.p + NI * C * LD, LD, C * LD};
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, g = l >> 4, col = l & 15;
    const int slot = blockIdx.x / a.HV, h = blockIdx.x % a.HV, hk = h / (a.HV / a.HK);
    const int s = a.map.owner(slot, C), start = a.map.start(s);
    int lo, hi;
    if (!SeqMap::piece(slot, a.map.slot0(s, C), a.map.end(s) - start, C, lo, hi)) return;
    const int n = hi - lo;
    if (n <= 0) return;

    // With the chunk's last tokens all rows are written: those past the sequence's
    // end are zero, with a decay of 1.
    Tile<T, C, KP, 256, WIDE> kt, qt;
    kt.shape(a.k.row, a.K);
    qt.shape(a.q.row, a.K);
    kt.fetch(row_of<const T>(a.k, a.map, s, start, lo) + (int64_t)hk * a.K, n);
    qt.fetch(row_of<const T>(a.q, a.map, s, start, lo) + (int64_t)hk * a.K, n);
    if (w == 0) {
        DeltaGate t = {0.0f, 0.0f, 0.0f, 0.0f};
        if (l < n)
            t = delta_gate(a, (float)row_of<const T>(a.dt, a.map, s, start, lo + l)[h],
                           (float)row_of<const T>(a.beta, a.map, s, start, lo + l)[h], h);
        const double p = wave_prefix((double)t.g2);
        if (l < C) {
            G[l] = p;
            scal[kBeta * C + l] = t.b;
        }
    }
    if (tid == 0) *odd = C;
    kt.put(kp);
    qt.put(qp);
    lds_barrier();

    // k k^T and q k^T, a wave for each 16 rows (and product, where there are only 32).
    const int tile = C == 64 ? w : w & 1;
    const bool kk_here = C == 64 || w < 2, qk_here = C == 64 || w >= 2;
    float4_t kk[NT] = {}, qk[NT] = {}, qq = {0, 0, 0, 0};
#pragma unroll 2
    for (int k0 = 0; k0 < KP; k0 += 32) {
        const Frag<NI> kf = kp.rows(tile * 16, k0), qf = qp.rows(tile * 16, k0);
#pragma unroll
        for (int jt = 0; jt < NT; ++jt) {
            if (jt > tile) continue;
            const Frag<NI> bf = kp.rows(jt * 16, k0);
            if (kk_here) mma<kParts>(kk[jt], kf, bf);
            if (qk_here) mma<kParts>(qk[jt], qf, bf);
        }
        if (qk_here) mma<kParts>(qq, qf, qf);
    }
#pragma unroll
    for (int jt = 0; jt < NT; ++jt)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (jt == tile && col == 4 * g + r) {
                const int i = tile * 16 + col;
                if (kk_here)
                    scal[kUnitK * C + i] = a.normalize ? rsqrtf(kk[jt][r] + kUnitEps) : 1.0f;
                if (qk_here) scal[kUnitQ * C + i] = a.normalize ? rsqrtf(qq[r] + kUnitEps) : 1.0f;
            }
    lds_barrier();
    char* out = a.prep + (int64_t)blockIdx.x * prep_bytes(C, kParts + PP);
    if (tid < C) {
        const float e = __builtin_amdgcn_exp2f((float)G[tid]), t = decay_between(G[C - 1], G[tid]);
        const float rk = scal[kUnitK * C + tid], rq = scal[kUnitQ * C + tid];
        const float b = scal[kBeta * C + tid];
        float* o = (float*)out + tid;
        o[kReadK * C] = e * rk;
        o[kWrite * C] = t * rk * b;
        o[kBeta * C] = b;
        o[kReadQ * C] = e * rq * a.scale;
        o[kTailK * C] = t * rk;
        o[kUnitK * C] = rk;
        o[kUnitQ * C] = rq;
        o[kDecay * C] = e;
    }
    float bad = 0.0f;
#pragma unroll
    for (int jt = 0; jt < NT; ++jt) {
        const int j = jt * 16 + col;
        const float rk = scal[kUnitK * C + j], b = scal[kBeta * C + j];
        float4_t m;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = tile * 16 + 4 * g + r;
            const float D = j <= i ? decay_between(G[i], G[j]) : 0.0f;
            m[r] = j < i ? D * kk[jt][r] * scal[kUnitK * C + i] * rk * b : 0.0f;
            if (kk_here) mat[i * ML + j] = m[r];
            if (qk_here)
                pm[i * ML + j] = j <= i ? D * qk[jt][r] * scal[kUnitQ * C + i] * rk * a.scale : 0.0f;
        }
        bad = strange(bad, m);
    }
    // A row of N that is infinite or NaN makes its own row of X and the later ones NaN, not
    // the ones before it: the inverse is formed without it.
    if (kk_here && !(bad == 0.0f))
        for (int jt = 0; jt < NT; ++jt)
            for (int r = 0; r < 4; ++r) {
                const int i = tile * 16 + 4 * g + r;
                float* at = mat + i * ML + jt * 16 + col;
                if (*at - *at == 0.0f) continue;
                *at = 0.0f;
                atomicMin(odd, i);
            }
    lds_barrier();
    invert<C, ML>(mat);
    if (*odd < C) {
        for (int i = tid; i < C * C; i += 256)
            if (i / C >= *odd && i % C <= i / C) mat[i / C * ML + i % C] = __builtin_nanf("");
        lds_barrier();
    }

    // As fragments, in the order in which the serial kernel reads them.
    bf16* fx = (bf16*)(out + kScales * C * 4);
    bf16* fp = fx + frag_count(C) * 512 * kParts;
#pragma unroll
    for (int mt = 0; mt < NT; ++mt)
#pragma unroll
        for (int kt = 0; kt < C / 32; ++kt) {
            if (!frag_used(C, mt, kt, BACK)) continue;
            const int f = frag_index(C, mt, kt, BACK);
            if (f % 4 != w) continue;
            float x[8], p[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int o = mt * 16 + col, i = kt * 32 + frag_at(g, j);
                x[j] = BACK ? mat[i * ML + o] : mat[o * ML + i];
                p[j] = BACK ? pm[i * ML + o] : pm[o * ML + i];
            }
            const Frag<kParts> xf = frag_of<kParts>(x);
            const Frag<PP> pf = frag_of<PP>(p);
#pragma unroll
            for (int q = 0; q < kParts; ++q) *(bf16x8_t*)(fx + (f * kParts + q) * 512 + l * 8) = xf.p[q];
#pragma unroll
            for (int q = 0; q < PP; ++q) *(bf16x8_t*)(fp + (f * PP + q) * 512 + l * 8) = pf.p[q];
        }
}

// ---- single tokens
//
// Bound by the states, read and written once: 8 KV bytes for each sequence and
// head (64 sequences of 16 heads of 128 x 128: 23 us, 5.9 TB/s). 256 threads hold a slice of 32 columns or vectors of columns; thread
// (ty, tx) has rows ty, ty + 8, .. of vector tx in registers between the two
// products with k and q.
struct DeltaStep {
    DeltaArgs a;
    float* state;
    int64_t num_slots;
    const int32_t* slots;
};

template <typename T, int VEC, int KR>
__global__ __launch_bounds__(256) void delta_step(const DeltaStep p) {
    const DeltaArgs& a = p.a;
    __shared__ float kq[2][8 * KR];
    __shared__ float norm[2];
    __shared__ float sums[8][32 * VEC];
    const int tid = threadIdx.x, tx = tid & 31, ty = tid >> 5;
    const int slices = (a.V + 32 * VEC - 1) / (32 * VEC);
    const int slice = blockIdx.x % slices, pair = blockIdx.x / slices;
    const int i = pair / a.HV, h = pair % a.HV, hk = h / (a.HV / a.HK);
    const int v = (slice * 32 + tx) * VEC;
    const int64_t at = p.slots ? p.slots[i] : i;
    T* y = (T*)a.y.p + i * a.y.row + (int64_t)h * a.V;
    if (at < 0 || at >= p.num_slots) {
        if (ty == 0)
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (v + e < a.V) y[v + e] = (T)0.0f;
        return;
    }
    float* S = p.state + (at * a.HV + h) * a.K * a.V + v;
    float st[KR][VEC];
#pragma unroll
    for (int j = 0; j < KR; ++j) {
        const int k = j * 8 + ty;
        if (k < a.K && v < a.V) load_f32<float, VEC>(S + (int64_t)k * a.V, st[j]);
        else
#pragma unroll
            for (int e = 0; e < VEC; ++e) st[j][e] = 0.0f;
    }
    const T* kr = (const T*)a.k.p + i * a.k.row + (int64_t)hk * a.K;
    const T* qr = (const T*)a.q.p + i * a.q.row + (int64_t)hk * a.K;
    const DeltaGate t = delta_gate(a, (float)((const T*)a.dt.p)[i * a.dt.row + h],
                                   (float)((const T*)a.beta.p)[i * a.beta.row + h], h);
    float vv[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e)
        vv[e] = v + e < a.V ? (float)((const T*)a.v.p)[i * a.v.row + (int64_t)h * a.V + v + e] : 0.0f;
    if (tid < 128) {  // a wave for each of k and q
        const T* x = tid < 64 ? kr : qr;
        float sq = 0.0f;
        for (int k = tid & 63; k < 8 * KR; k += 64) {
            const float f = k < a.K ? (float)x[k] : 0.0f;
            kq[tid >> 6][k] = f;
            sq = __builtin_fmaf(f, f, sq);
        }
        sq = wave_sum(sq);
        if ((tid & 63) == 0) norm[tid >> 6] = a.normalize ? rsqrtf(sq + kUnitEps) : 1.0f;
    }
    __syncthreads();
    // The sum over all rows of x times the held state, for the thread's columns.
    const auto product = [&](const float* x, float (&o)[VEC]) {
        float s[VEC] = {};
#pragma unroll
        for (int j = 0; j < KR; ++j) {
            const float f = x[j * 8 + ty];
#pragma unroll
            for (int e = 0; e < VEC; ++e) s[e] = __builtin_fmaf(f, st[j][e], s[e]);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) sums[ty][e * 32 + tx] = s[e];
        __syncthreads();
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            o[e] = 0.0f;
#pragma unroll
            for (int r = 0; r < 8; ++r) o[e] += sums[r][e * 32 + tx];
        }
        __syncthreads();
    };
    const float decay = __builtin_amdgcn_exp2f(t.g2), rk = norm[0], rq = norm[1];
    float u[VEC], o[VEC];
    product(kq[0], u);
#pragma unroll
    for (int e = 0; e < VEC; ++e) u[e] = rk * t.b * __builtin_fmaf(-decay * rk, u[e], vv[e]);
#pragma unroll
    for (int j = 0; j < KR; ++j) {
        const int k = j * 8 + ty;
        const float f = kq[0][k];
#pragma unroll
        for (int e = 0; e < VEC; ++e) st[j][e] = __builtin_fmaf(f, u[e], decay * st[j][e]);
        if (k < a.K && v < a.V) store_f32<float, VEC>(S + (int64_t)k * a.V, st[j]);
    }
    product(kq[1], o);
    if (ty == 0)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (v + e < a.V) y[v + e] = (T)(a.scale * rq * o[e]);
}

template <typename T>
hipError_t step_typed(const DeltaStep& p, bool v4, unsigned n, hipStream_t st) {
    const DeltaArgs& a = p.a;
    const unsigned grid = (unsigned)(n * a.HV * ceil_div(a.V, v4 ? 128 : 32));
#define TG_X(KR)                                                       \
    do {                                                               \
        if (v4) delta_step<T, 4, KR><<<grid, 256, 0, st>>>(p);         \
        else delta_step<T, 1, KR><<<grid, 256, 0, st>>>(p);            \
    } while (0)
    if (a.K <= 64) TG_X(8);
    else if (a.K <= 128) TG_X(16);
    else TG_X(32);
#undef TG_X
    return hipGetLastError();
}

// The maps of all segments, the states between them, and the walk from those.
template <typename Walk>
hipError_t in_segments(const DeltaArgs& a, const float* first, bool reverse, float* states, int KP,
                       int slice, hipStream_t st, Walk walk) {
    DeltaArgs b = a;
    b.through = true;
    hipError_t e = walk(b);
    if (e == hipSuccess) e = launch_delta_join(a, first, reverse, states, KP, slice, st);
    if (e != hipSuccess) return e;
    b.through = false;
    (reverse ? b.dfinal : b.initial) = states;
    return walk(b);
}

template <typename T>
hipError_t forward_typed(const DeltaArgs& a, int64_t slots, float* states, hipStream_t st) {
    const int KP = delta_padded(a.K);
    const hipError_t e = launch_delta_prep<T, false>(a, KP, slots, st);
    if (e != hipSuccess || !a.segment) return e == hipSuccess ? launch_delta_forward<T>(a, KP, st) : e;
    return in_segments(a, a.initial, false, states, KP, slice_of(kIn<T>, KP), st, [&](const DeltaArgs& b) {
        return launch_delta_forward<T>(b, KP, st);
    });
}
template <typename T>
hipError_t backward_typed(const DeltaArgs& a, int64_t slots, float* states, hipStream_t st) {
    const int KP = delta_padded(a.K);
    hipError_t e = launch_delta_prep<T, true>(a, KP, slots, st);
    if (e != hipSuccess) return e;
    if (a.segment)
        e = in_segments(a, a.dfinal, true, states, KP, slice_of(kIn<T>, KP), st,
                        [&](const DeltaArgs& b) { return launch_delta_states<T>(b, KP, st); });
    else e = launch_delta_states<T>(a, KP, st);
    return e == hipSuccess ? launch_delta_grads<T>(a, KP, slots, st) : e;
}

}  // namespace

template <typename T, bool BACK>
hipError_t launch_delta_prep(const DeltaArgs& a, int KP, int64_t slots, hipStream_t st) {
    const unsigned grid = (unsigned)(slots * a.HV);
    if (grid == 0) return hipSuccess;
#define TG_X(KP_)                                                                               \
    do {                                                                                        \
        constexpr int bytes = PrepShape<T, KP_>::lds;                                           \
        const auto kernel = a.wide_qk ? delta_prep<T, KP_, BACK, true>                          \
                                      : delta_prep<T, KP_, BACK, false>;                        \
        const hipError_t e = ensure_dynamic_lds((const void*)kernel, bytes);                    \
        if (e != hipSuccess) return e;                                                          \
        kernel<<<grid, 256, bytes, st>>>(a);                                                    \
    } while (0)
    if (KP == 64) TG_X(64);
    else if (KP == 128) TG_X(128);
    else TG_X(256);
#undef TG_X
    return hipGetLastError();
}

DeltaArgs delta_args(const tg_delta_args& a) {
    DeltaArgs b{};
    b.map = map_of(a.seqs);
    b.HK = a.HK, b.HV = a.HV, b.K = a.K, b.V = a.V;
    b.softplus = a.softplus, b.sigmoid = a.sigmoid, b.normalize = a.normalize, b.scale = a.scale;
    b.q = rows_of<const void>(a.q), b.k = rows_of<const void>(a.k), b.v = rows_of<const void>(a.v);
    b.dt = rows_of<const void>(a.dt), b.beta = rows_of<const void>(a.beta);
    b.y = rows_of<void>(a.y);
    b.A = a.A, b.dt_bias = a.dt_bias, b.initial = a.initial, b.final = a.final;
    const size_t e = elem_bytes(a.dtype);
    // seq strides mean nothing in a packed batch.
    const auto rows = [&](Widest& w, const tg_rows& r) {
        w.len(r.row_stride), w.ptr(r.p, e);
        if (!a.seqs.offsets) w.len(r.seq_stride);
    };
    Widest qk, v, y;
    qk.len(a.K), rows(qk, a.q), rows(qk, a.k);
    v.len(a.V), rows(v, a.v);
    y.len(a.V), rows(y, a.y);
    b.wide_qk = qk.width(8) == 8, b.wide_v = v.width(8) == 8, b.wide_y = y.width(4) == 4;
    return b;
}

namespace {

// What a pass keeps for the segments: their maps and the states between them.
struct SegmentRoom {
    int segment;
    int64_t units;
    size_t maps, states;
    explicit SegmentRoom(const tg_delta_args& a) {
        const int in = delta_in(a.dtype), KP = delta_padded(a.K);
        segment = delta_segment(a);
        units = segment ? delta_slots(a.seqs, segment) : a.seqs.seqs;
        maps = segment ? up256((size_t)(units * a.HV * KP * map_columns(a.V, KP, slice_of(in, KP))) * 4) : 0;
        states = segment ? up256((size_t)(units * a.HV * a.K * a.V) * 4) : 0;
    }
};
size_t kept_bytes(const tg_delta_args& a) {
    const int C = delta_chunk_of(a);
    return (size_t)(delta_slots(a.seqs, C) * a.HV * kept_floats(a.V, delta_padded(a.K), C)) * 4;
}
size_t prep_room(const tg_delta_args& a, int parts) {
    const int C = delta_chunk_of(a);
    return up256((size_t)(delta_slots(a.seqs, C) * a.HV) * prep_bytes(C, parts));
}

}  // namespace

// In workgroups of 256 threads.
int64_t delta_groups(const tg_delta_args& a) {
    const int KP = delta_padded(a.K), slice = slice_of(delta_in(a.dtype), KP);
    const int64_t chunks = delta_slots(a.seqs, delta_chunk_of(a)) * a.HV * (KP == 256 ? 2 : 1);
    const SegmentRoom room(a);
    const int slices = (int)ceil_div(a.V, slice) + (room.segment ? KP / slice : 0);
    const int64_t serial = 2 * head_slice_grid(room.units * a.HV, slices);
    return chunks > serial ? chunks : serial;
}

void delta_sizes(const tg_delta_args& a, size_t* work, size_t* saved, size_t* backward) {
    const SegmentRoom room(a);
    const size_t kept = kept_bytes(a), between = room.maps + room.states;
    if (work) *work = prep_room(a, kParts + delta_out(a.dtype)) + between;
    if (saved) *saved = kept;
    if (backward)
        *backward = prep_room(a, 2 * kParts) + up256(kept) + between +
                    (size_t)(delta_slots(a.seqs, delta_chunk_of(a)) * a.HV) * 2 * sizeof(float);
}

hipError_t launch_delta(const tg_delta_args& a, void* ws, void* saved, hipStream_t st) {
    DeltaArgs b = delta_args(a);
    const SegmentRoom room(a);
    b.prep = (char*)ws;
    b.saved = (float*)saved;
    b.segment = room.segment, b.units = (int)room.units;
    b.maps = (float*)(b.prep + prep_room(a, kParts + delta_out(a.dtype)));
    float* states = (float*)((char*)b.maps + room.maps);
    const int64_t slots = delta_slots(a.seqs, delta_chunk_of(a));
    if (a.dtype == TG_F32) return forward_typed<float>(b, slots, states, st);
    if (a.dtype == TG_BF16) return forward_typed<bf16>(b, slots, states, st);
    return forward_typed<f16>(b, slots, states, st);
}

hipError_t launch_delta_backward(const tg_delta_args& a, const tg_delta_grads& gr,
                                 const void* saved, void* ws, hipStream_t st) {
    DeltaArgs b = delta_args(a);
    const int64_t slots = delta_slots(a.seqs, delta_chunk_of(a));
    const SegmentRoom room(a);
    b.segment = room.segment, b.units = (int)room.units;
    b.saved = (float*)saved;
    b.prep = (char*)ws;
    b.back = (float*)(b.prep + prep_room(a, 2 * kParts));
    b.maps = (float*)((char*)b.back + up256(kept_bytes(a)));
    float* states = (float*)((char*)b.maps + room.maps);
    b.part = (float*)((char*)states + room.states);
    b.dy = rows_of<const void>(gr.dy);
    b.dq = rows_of<void>(gr.dq), b.dk = rows_of<void>(gr.dk), b.dv = rows_of<void>(gr.dv);
    b.ddt = rows_of<void>(gr.ddt), b.dbeta = rows_of<void>(gr.dbeta);
    b.dfinal = gr.dfinal, b.dinitial = gr.dinitial;
    const size_t e = elem_bytes(a.dtype);
    Widest dy;
    dy.len(a.V), dy.len(gr.dy.row_stride), dy.ptr(gr.dy.p, e);
    if (!a.seqs.offsets) dy.len(gr.dy.seq_stride);
    b.wide_dy = dy.width(8) == 8;
    hipError_t err = a.dtype == TG_F32   ? backward_typed<float>(b, slots, states, st)
                     : a.dtype == TG_BF16 ? backward_typed<bf16>(b, slots, states, st)
                                          : backward_typed<f16>(b, slots, states, st);
    if (err != hipSuccess) return err;
    return launch_column_sums(b.part, (int)slots, 2 * (int64_t)a.HV, gr.dA, a.HV, gr.ddt_bias, st);
}

hipError_t launch_delta_step(const tg_delta_args& a, float* state, int64_t num_slots,
                             const int32_t* slots, hipStream_t st) {
    const DeltaStep p{delta_args(a), state, num_slots, slots};
    const bool v4 = a.V % 4 == 0 && ((uintptr_t)state & 15) == 0;
    const unsigned n = (unsigned)a.seqs.seqs;
    if (a.dtype == TG_F32) return step_typed<float>(p, v4, n, st);
    if (a.dtype == TG_BF16) return step_typed<bf16>(p, v4, n, st);
    return step_typed<f16>(p, v4, n, st);
}

}  // namespace tg
