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
// joined over the 4 lanes, which leaves each lane the results of its own items.
//
// The recurrence is linear, so tokens can be split up: a segment's last state is
//   P * (state before it) + (last state from zero),  P[n] = 2^(A[n] log2 e * sum d).
// The W waves of a workgroup take TT tokens each side by side: every wave
// runs its segment from zero, they exchange P and the last states through LDS, and
// each adds what the state before it gives. With few sequences and channels the
// workgroups split the tokens in the same way (parts of PL tokens): a first
// kernel computes the parts' P and last states.
//
// A decay P over a segment may be past fp32 (a rate above zero, a negative step) where
// the states that it carries are not: a state of zero, above all. Multiplying twice by
// the root of P, held at fp32's largest, is right for those: P past the square of that
// makes any state but zero infinite. The backward pass takes the roots always. The forward
// pass, where the second multiplication counts for more (prompts 208 us for 192), takes P, and
// where such decays may be sees a state come out infinite or NaN and goes over the
// segments again by the roots.
//
// Tokens past the end count as d = 0 (and dL/dv = 0): a = 1, and the state stays.
#include <float.h>

#include "seq_device.hpp"
#include "seq_internal.hpp"
#include "tg_internal.hpp"

namespace tg {
namespace {

constexpr int kCh = 16;  // channels of a wave
constexpr float kLn2 = 0.69314718055994531f;

// Tokens that a wave takes at a time. The backward pass holds TT tokens'
// decays and states: for NS = 4 two waves on a SIMD with 16 tokens. With 8 its kernel took
// as long on three waves (163 us against 167, 2 x 2048 tokens, 2048 channels), the
// training step 5% more, saving twice the states. The split kernels go to scratch even so:
// 6 registers for NS = 4, 16 for 8, over 100 for 32. The forward pass holds decays only,
// without scratch: 8 tokens leave room for four waves on a SIMD, which took
// 203 us where two waves of 16 tokens took 241 (4 x 4096 tokens, 2048 channels, bf16).
constexpr int chunk_for(int ns) { return ns <= 4 ? 16 : 64 / ns < 4 ? 4 : 64 / ns; }
constexpr int fwd_chunk_for(int ns) { return ns <= 4 ? 8 : chunk_for(ns); }
// Waves of a workgroup side by side: what they exchange (2*NS values for each lane, in
// two buffers) takes 12 to 38 KiB of LDS for NS up to 4 and 72 to 81 above, 148 with the
// backward pass's tiles at most (NS = 8), of a compute unit's 160.
constexpr int waves_for(int ns) { return ns <= 8 ? 8 : 64 / ns; }

struct ScanArgs {
    SeqMap seqs;
    int D, N, G, Dg, bpg;  // Dg: channels of a group, in bpg blocks of 16
    int softplus, PL;      // PL: tokens of a part; 0: sequences are not split
    Rows<const void> x, dt, B, C, z;
    Rows<void> y;
    const float *A, *D_skip, *dt_bias, *initial;
    float *final, *saved;
    float* parts;  // [slots of PL tokens][2][D][4*NS]: P (or its root) and last state
};

// Value k of a pair over two lanes: the lane whose bit is clear keeps a, the
// other b, each summed over both lanes. o is what the other lane wants.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                         0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kRor4 = 0x124, kRor8 = 0x128, kRor12 = 0x12C;

__device__ __forceinline__ float quad_sum(float v) {
    v += dpp<kXor1>(v);
    v += dpp<kXor2>(v);
    return v;
}
// The sums of v[0..3] over the 4 lanes of a quad, v[q] in lane q.
__device__ __forceinline__ float quad_sums(float v0, float v1, float v2, float v3, int q) {
    const bool b0 = q & 1, b1 = q & 2;
    const float a = (b0 ? v1 : v0) + dpp<kXor1>(b0 ? v0 : v1);
    const float b = (b0 ? v3 : v2) + dpp<kXor1>(b0 ? v2 : v3);
    return (b1 ? b : a) + dpp<kXor2>(b1 ? a : b);
}
// The sums over the 16 channels (lane bits 2 to 5) in levels, each of which
// joins two lanes and halves the values a lane holds: of a pair, the lane whose
// bit is clear keeps the first and the other the second.
template <int BIT>
__device__ __forceinline__ float join(float v0, float v1, int lane) {
    if constexpr (BIT == 5 || BIT == 4) {
        const unsigned u0 = __builtin_bit_cast(unsigned, v0), u1 = __builtin_bit_cast(unsigned, v1);
        const auto w = BIT == 5 ? __builtin_amdgcn_permlane32_swap(u0, u1, false, false)
                                : __builtin_amdgcn_permlane16_swap(u0, u1, false, false);
        // (A bit cast of a vector's element itself would take element 0.)
        const unsigned r0 = w[0], r1 = w[1];
        return __builtin_bit_cast(float, r0) + __builtin_bit_cast(float, r1);
    } else {
        const bool up = lane & (1 << BIT);
        const float o = up ? v0 : v1;
        if constexpr (BIT == 3) return (up ? v1 : v0) + dpp<kRor8>(o);
        // Lane i ^ 4 is 4 up or down within the row. Both moves by all lanes: in a
        // branch they would read lanes that are switched off.
        const float down = dpp<kRor4>(o), above = dpp<kRor12>(o);
        return (up ? v1 : v0) + (up ? down : above);
    }
}
// Of n values v[0..n) (n a power of two), the level of BIT; n/2 remain.
template <int BIT, int N>
__device__ __forceinline__ void join_all(float* v, int lane) {
#pragma unroll
    for (int k = 0; k < N / 2; ++k) v[k] = join<BIT>(v[2 * k], v[2 * k + 1], lane);
}
// How many of the levels (bits 5, 4, 3, 2) a token's own NS values take.
constexpr int levels_of(int ns) { return ns >= 4 ? 2 : ns == 2 ? 1 : 0; }
// The levels of one token's values ...
template <int NS>
__device__ __forceinline__ void join_token(float (&v)[NS], int lane) {
    if constexpr (NS >= 2) join_all<5, NS>(v, lane);
    if constexpr (NS >= 4) join_all<4, NS / 2>(v, lane);
}
// ... and the rest over the tokens of a group, which leave a lane value
// b5 + 2*b4 + 4*b3 + 8*b2 of each 16 in token order.
template <int NS>
__device__ __forceinline__ float join_group(float* v, int lane) {
    if constexpr (NS == 1) join_all<5, 16>(v, lane);
    if constexpr (NS <= 2) join_all<4, 8>(v, lane);
    join_all<3, 4>(v, lane);
    return join<2>(v[0], v[1], lane);
}

// What a wave keeps in LDS of TT tokens.
template <int NS, int TT>
struct alignas(16) Tile {
    float2 d[TT][kCh];  // d, d*x
    float B[TT][4 * NS];
    float C[TT][4 * NS];
};
// The backward pass: dL/dv too, and the items' x, slope of softplus and dz for
// v = 1, which would take registers until the end of the chunk.
template <int NS, int TT>
struct alignas(16) BackTile {
    Tile<NS, TT> f;
    float dv[TT][kCh];
    float4 item[TT / 4][64];
    float dA[2][64][NS];  // a lane's sum so far, and what its additions dropped
};
// NS consecutive floats of LDS or memory (NS floats aligned).
template <int NS>
__device__ __forceinline__ void get(const float* p, float (&v)[NS]) {
    constexpr int V = NS < 4 ? NS : 4;
#pragma unroll
    for (int j = 0; j < NS; j += V) load_f32<float, V>(p + j, *(float (*)[V])(v + j));
}
template <int NS>
__device__ __forceinline__ void put(float* p, const float (&v)[NS]) {
    constexpr int V = NS < 4 ? NS : 4;
#pragma unroll
    for (int j = 0; j < NS; j += V) store_f32<float, V>(p + j, *(const float (*)[V])(v + j));
}

// The long loops start at 256 bytes: the same instructions took 194 or 201 us
// (4 x 4096 tokens, 2048 channels), 234 or 244 with the backward pass, as they happened to lie.
__device__ __forceinline__ void align_loop() { asm volatile(".p2align 8"); }

// Computes v here: the compiler would move a sum to its use further down and
// keep all of its operands for that long.
__device__ __forceinline__ void pin(float& v) { asm volatile("" : "+v"(v)); }

// One token of a tile as a lane reads it.
template <int NS>
struct Token {
    float2 d;
    float B[NS], C[NS];
};
// Run body(t, token) over the TT tokens, up or down, each token's LDS reads
// issued one token ahead. Without the scheduling fence the compiler hoists the
// reads of all TT tokens to the front, and without the opaque lane indices it
// keeps what one pass over the tile read for the next; both spill.
template <int NS, int TT, bool WITH_B, bool WITH_C, bool UP, typename Body>
__device__ __forceinline__ void for_tokens(const Tile<NS, TT>& tile, int cl, int q, Body body) {
    asm volatile("" : "+v"(cl), "+v"(q));
    const auto read = [&](int t) {
        Token<NS> k;
        k.d = tile.d[t][cl];
        if constexpr (WITH_B) get<NS>(&tile.B[t][q * NS], k.B);
        if constexpr (WITH_C) get<NS>(&tile.C[t][q * NS], k.C);
        return k;
    };
    Token<NS> cur = read(UP ? 0 : TT - 1);
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        const int t = UP ? i : TT - 1 - i;
        Token<NS> next;
        if (i + 1 < TT) next = read(UP ? t + 1 : t - 1);
        body(t, cur);
        __builtin_amdgcn_sched_barrier(0);
        if (i + 1 < TT) cur = next;
    }
}

// Order LDS accesses of one wave among its lanes: the hardware keeps a wave's
// LDS accesses in order, so only the compiler has to.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// A workgroup's place: its sequence, part of it (tokens lo to hi) and block of
// channels; a lane's channel and states. Neighbouring blocks share the cache lines of
// x, dt, z and y (16 channels are a quarter of one), so they run on one XCD.
struct Place {
    int slot, s, start, len, lo, hi, block, g, cl, q, ch, w;
    int64_t part0;  // the slot of the sequence's first part
    bool in;
    // by_rows: lane q*16 + channel (what the matrix instructions give), else
    // lane channel*4 + q (what the sums over channels join best).
    __device__ __forceinline__ Place(const ScanArgs& a, bool by_rows) {
        const SeqMap& m = a.seqs;
        const int tile = xcd_contiguous_tile(blockIdx.x, gridDim.x), nb = a.G * a.bpg;
        slot = tile / nb;
        block = tile - slot * nb;
        s = a.PL ? m.owner(slot, a.PL) : slot;
        start = m.start(s);
        len = m.end(s) - start;
        lo = 0, hi = len, part0 = 0;
        if (a.PL) {
            part0 = m.slot0(s, a.PL);
            if (!SeqMap::piece(slot, (int)part0, len, a.PL, lo, hi)) lo = -1;
        }
        g = block / a.bpg;
        const int c0 = (block - g * a.bpg) * kCh;
        w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int lane = threadIdx.x & 63;
        cl = by_rows ? lane & 15 : lane >> 2;
        q = by_rows ? lane >> 4 : lane & 3;
        in = c0 + cl < a.Dg;
        ch = g * a.Dg + c0 + (in ? cl : 0);
    }
    __device__ __forceinline__ int part(int PL) const { return PL ? lo / PL : 0; }
};

// A tensor's rows of one sequence. A chunk's rows are read and written through a
// buffer descriptor that ends with the last token: what lies past it reads
// as zero and is not written, so the tail of a sequence takes no branch. (Rows
// that are one row for all tokens, with a stride of 0, read as that row
// there: what has to be zero past the end, d and dv, is set so by itself.) The host
// keeps row strides below 2^25 elements, so that a chunk's offsets fit 31 bits.
constexpr uint32_t kNowhere = 0x80000000u;  // an offset past any chunk
struct Col {
    char* base;
    uint32_t row, width;  // bytes from row to row, bytes of a row
    template <typename P>
    __device__ __forceinline__ Col(const Rows<P>& r, const SeqMap& m, const Place& p, int elem,
                                   int width_)
        : base((char*)r.p + (m.offsets ? (int64_t)p.start * r.row : (int64_t)p.s * r.seq) * elem),
          row((uint32_t)r.row * elem),
          width((uint32_t)width_ * elem) {}
    // Up to n rows from token l, not past hi.
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t rows(int l, int hi, int n) const {
        const int have = imin(hi - l, n);
        const uint32_t bytes = have > 0 ? (uint32_t)(have - 1) * row + width : 0;
        return __builtin_amdgcn_make_buffer_rsrc(base + (int64_t)l * row, 0, bytes, 0x00027000);
    }
};
// An element as loaded, and its value.
template <typename T>
struct Raw {
    typedef uint16_t type;
};
template <>
struct Raw<float> {
    typedef uint32_t type;
};
template <typename T>
__device__ __forceinline__ typename Raw<T>::type buf_load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    if constexpr (sizeof(T) == 2) return __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
    else return __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
}
template <typename T>
__device__ __forceinline__ float raw_value(typename Raw<T>::type v) {
    return (float)__builtin_bit_cast(T, v);
}
template <typename T>
__device__ __forceinline__ void buf_store(__amdgpu_buffer_rsrc_t r, uint32_t off, float v) {
    const T t = (T)v;
    const typename Raw<T>::type u = __builtin_bit_cast(typename Raw<T>::type, t);
    if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b16(u, r, off, 0, 0);
    else __builtin_amdgcn_raw_buffer_store_b32(u, r, off, 0, 0);
}

// The items of a lane in one tensor: token q + 4*i of the chunk at l, the
// lane's channel.
template <typename T>
__device__ __forceinline__ uint32_t item_offset(const Col& c, const Place& p) {
    return p.in ? (uint32_t)p.q * c.row + (uint32_t)p.ch * (uint32_t)sizeof(T) : kNowhere;
}
// An offset that is added up where it is used: the compiler would keep every sum.
__device__ __forceinline__ uint32_t here(uint32_t off) {
    asm volatile("" : "+v"(off));
    return off;
}
template <typename T, int TT>
struct Items {
    typename Raw<T>::type v[TT / 4];
    __device__ __forceinline__ void load(const Col& c, const Place& p, int l) {
        const __amdgpu_buffer_rsrc_t r = c.rows(l, p.hi, TT);
        const uint32_t off = here(item_offset<T>(c, p));
#pragma unroll
        for (int i = 0; i < TT / 4; ++i) v[i] = buf_load<T>(r, off + i * (4 * c.row));
    }
    __device__ __forceinline__ float operator[](int i) const { return raw_value<T>(v[i]); }
};
template <typename T, int TT>
__device__ __forceinline__ void store_items(const Col& c, const Place& p, int l,
                                            const float (&v)[TT / 4]) {
    const __amdgpu_buffer_rsrc_t r = c.rows(l, p.hi, TT);
    const uint32_t off = here(item_offset<T>(c, p));
#pragma unroll
    for (int i = 0; i < TT / 4; ++i) buf_store<T>(r, off + i * (4 * c.row), v[i]);
}

// A wave's share of TT tokens' B or C: element lane + 64*k of [TT][4*NS].
template <typename T, int NS, int TT>
struct Shared {
    static constexpr int kN = 4 * NS, kPer = TT * kN / 64;
    typename Raw<T>::type v[kPer];
    __device__ __forceinline__ void load(const Col& c, const Place& p, int N, int l) {
        const __amdgpu_buffer_rsrc_t r = c.rows(l, p.hi, TT);
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            // Rows k*64/kN (the same for all lanes) and lane/kN (for short rows).
            const int t0 = k * 64 / kN, t = kN < 64 ? lane / kN : 0;
            const int n = kN < 64 ? lane % kN : (k * 64 % kN) + lane;
            const uint32_t off = n < N ? (uint32_t)t * c.row +
                                             (uint32_t)(p.g * N + n) * (uint32_t)sizeof(T)
                                       : kNowhere;
            v[k] = buf_load<T>(r, here(off) + t0 * c.row);
        }
    }
    __device__ __forceinline__ void put(float (&to)[TT][kN]) const {
#pragma unroll
        for (int k = 0; k < kPer; ++k)
            (&to[0][0])[k * 64 + (threadIdx.x & 63)] = raw_value<T>(v[k]);
    }
};

// A wave's states (or their adjoints) after its segment from zero, and the decay over it
// (or its root): LDS [W][2][64][NS] floats, and after them [64][NS]: the true state that the round
// before left; then [W][64], the segments' sums of step sizes.
template <int NS>
__device__ __forceinline__ float* exchange_at(float* ex, int w, int which) {
    return ex + ((w * 2 + which) * 64 + (threadIdx.x & 63)) * NS;
}
template <int NS>
__device__ __forceinline__ float* sum_at(float* ex, int W, int w) {
    return ex + (2 * W + 1) * 64 * NS + w * 64 + (threadIdx.x & 63);
}
constexpr int exchange_floats(int W, int ns) { return (2 * W + 1) * 64 * ns + W * 64; }

// State j of a lane, with lanes by rows: the rows of a 16 x 16 matrix that the
// lane holds, 4q to 4q+3 (with NS < 4 only NS of them are used).
template <int NS, bool ROWS>
__device__ __forceinline__ int state_of(int q, int j) {
    return !ROWS || NS < 4 ? q * NS + j : (j & ~3) * 4 + q * 4 + (j & 3);
}

// A * log2(e), held within fp32: a rate past it would make NaN of a step of zero, as
// tokens past the end have, and forgets the state at any other step either way.
__device__ __forceinline__ float rate2(float A) {
    const float v = A * kLog2e;
    return v < -FLT_MAX ? -FLT_MAX : v > FLT_MAX ? FLT_MAX : v;  // NaN stays
}

// log2(a) = d * A2 of the lane's states, zero past N and for lanes without a
// channel.
template <int NS, bool ROWS>
__device__ __forceinline__ void load_A2(const ScanArgs& a, const Place& p, float (&A2)[NS]) {
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        const int n = state_of<NS, ROWS>(p.q, j);
        A2[j] = p.in && n < a.N ? rate2(a.A[(int64_t)p.ch * a.N + n]) : 0.0f;
    }
}
template <int NS, bool ROWS>
__device__ __forceinline__ void load_state(const float* st, const ScanArgs& a, const Place& p,
                                           float (&h)[NS]) {
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        const int n = state_of<NS, ROWS>(p.q, j);
        h[j] = st && p.in && n < a.N ? st[((int64_t)p.s * a.D + p.ch) * a.N + n] : 0.0f;
    }
}
template <int NS, bool ROWS>
__device__ __forceinline__ void store_state(float* st, const ScanArgs& a, const Place& p,
                                            const float (&h)[NS]) {
    if (!st || !p.in) return;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        const int n = state_of<NS, ROWS>(p.q, j);
        if (n < a.N) st[((int64_t)p.s * a.D + p.ch) * a.N + n] = h[j];
    }
}
// The root of a decay 2^L.
__device__ __forceinline__ float root_decay(float L) {
    return fminf(__builtin_amdgcn_exp2f(0.5f * L), FLT_MAX);
}
// The state (or adjoint) h over a segment of that root which leaves e from zero.
__device__ __forceinline__ float carried(float root, float h, float e) {
    return __builtin_fmaf(root, root * h, e);
}
// Whether a segment's decay can be more than 1, by whole waves: the same in all waves
// that hold these channels.
template <int NS>
__device__ __forceinline__ bool may_grow(const ScanArgs& a, const float (&A2)[NS]) {
    float most = 0.0f;
#pragma unroll
    for (int j = 0; j < NS; ++j) most = fmaxf(most, A2[j]);
    return !a.softplus || __ballot(most > 0.0f) != 0;
}
// The state h after the exchange's first n segments: if it came out infinite or NaN, as
// a decay past fp32 makes any state and more decays keep it, again by the roots.
template <int NS>
__device__ __forceinline__ void carry_grown(float* ex, int W, int n, const float (&A2)[NS],
                                            float (&h)[NS]) {
    float nan = 0.0f;
#pragma unroll
    for (int j = 0; j < NS; ++j) nan = __builtin_fmaf(h[j], 0.0f, nan);
    if (__ballot(nan != 0.0f) == 0) return;
    get<NS>(exchange_at<NS>(ex, W, 0), h);
#pragma clang loop unroll(disable)
    for (int k = 0; k < n; ++k) {
        float e[NS];
        const float sum = *sum_at<NS>(ex, W, k);
        get<NS>(exchange_at<NS>(ex, k, 1), e);
#pragma unroll
        for (int j = 0; j < NS; ++j) h[j] = carried(root_decay(sum * A2[j]), h[j], e[j]);
    }
}
template <int NS>
__device__ __forceinline__ float* part_at(const ScanArgs& a, const Place& p, int part, int which) {
    return a.parts + (((p.part0 + part) * 2 + which) * a.D + p.ch) * (4 * NS) + p.q * NS;
}

// h through parts first, first + step, ... (n of them), from memory four at a time.
template <int NS>
__device__ __forceinline__ void fold_parts(const ScanArgs& a, const Place& p, int first, int n,
                                           int step, bool grow, float (&h)[NS]) {
    for (int k = 0; k < n; k += 4) {
        float P[4][NS], e[4][NS];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int part = first + imin(k + u, n - 1) * step;
            get<NS>(part_at<NS>(a, p, part, 0), P[u]);
            get<NS>(part_at<NS>(a, p, part, 1), e[u]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (k + u < n)
#pragma unroll
                for (int j = 0; j < NS; ++j)
                    h[j] = grow ? carried(P[u][j], h[j], e[u][j])
                                : __builtin_fmaf(P[u][j], h[j], e[u][j]);
    }
}

__device__ __forceinline__ float step_size(const ScanArgs& a, float raw) {
    return a.softplus ? softplus_f32(raw) : raw;
}

// The forward kernels have lanes by rows: lane q*16 + c holds channel c and states
// 4q .. 4q+3 (and the same of each further 16). That is how
// v_mfma_f32_16x16x1_4b_f32 leaves four 16 x 16 outer products, one for each of four tokens:
// (d*x)[c] * B[n] of four tokens and four states comes from one matrix
// instruction (exact fp32 products), beside the vector units, with operands as the lanes loaded
// them: lane (token, channel) its own item's d*x, and lane (token, n) B. C in
// every lane that needs it is the product with ones.
typedef float f32x16 __attribute__((ext_vector_type(16)));
constexpr int blocks_of(int ns) { return ns <= 4 ? 1 : ns / 4; }  // of 16 states

// A lane's elements of B or C: token 4*g + (lane >> 4), state row lane & 15 of
// each block of 16 (zero where that is no state).
template <typename T, int NS, int TT>
struct RowVals {
    typename Raw<T>::type v[TT / 4][blocks_of(NS)];
    __device__ __forceinline__ void load(const Col& c, const Place& p, int N, int l) {
        const __amdgpu_buffer_rsrc_t r = c.rows(l, p.hi, TT);
        const int row = threadIdx.x & 15;
        const int n = NS >= 4 ? row : (row >> 2) * NS + (row & 3);
#pragma unroll
        for (int m = 0; m < blocks_of(NS); ++m) {
            const bool in = n + 16 * m < N && (NS >= 4 || (row & 3) < NS);
            const uint32_t off = in ? (uint32_t)p.q * c.row +
                                          (uint32_t)(p.g * N + n + 16 * m) * (uint32_t)sizeof(T)
                                    : kNowhere;
            const uint32_t o = here(off);
#pragma unroll
            for (int g = 0; g < TT / 4; ++g) v[g][m] = buf_load<T>(r, o + g * (4 * c.row));
        }
    }
    // out[token][j]: value of tokens 4*g to 4*g+3 times x (a lane's item of
    // token 4*g + q, or one) for the lane's states.
    __device__ __forceinline__ void outer(int g, float x, float (&out)[4][NS]) const {
        const f32x16 zero = {};
#pragma unroll
        for (int m = 0; m < blocks_of(NS); ++m) {
            const f32x16 d =
                __builtin_amdgcn_mfma_f32_16x16x1f32(raw_value<T>(v[g][m]), x, zero, 0, 0, 0);
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int j = 0; j < 4 && j < NS; ++j) out[t][4 * m + j] = d[4 * t + j];
        }
    }
};

// The step sizes of a wave's tokens, for all lanes of a channel.
template <int TT>
struct alignas(16) Steps {
    float d[kCh][TT + 4];
};

// The sums of y[0..3] over the 4 lanes of a channel, token q's in lane q.
__device__ __forceinline__ float row_sums(const float (&y)[4], int lane) {
    return join<4>(join<5>(y[0], y[2], lane), join<5>(y[1], y[3], lane), lane);
}

// Run body(g) over the groups of 4 tokens, in order, without moving work
// from one to another: otherwise all groups' products are held at once.
template <int TT, typename Body>
__device__ __forceinline__ void for_groups(Body body) {
#pragma unroll
    for (int g = 0; g < TT / 4; ++g) {
        body(g);
        __builtin_amdgcn_sched_barrier(0);
    }
}

template <typename T, int NS, int TT, bool SPLIT>
__global__ __launch_bounds__(SPLIT ? 64 * waves_for(NS) : 64)
    __attribute__((amdgpu_waves_per_eu(NS <= 4 ? 4 : 1))) void scan_fwd(const ScanArgs a) {
    constexpr int kItems = TT / 4;
    extern __shared__ float4 lds[];
    const int W = SPLIT ? blockDim.x >> 6 : 1;
    const Place p(a, true);
    if (p.lo < 0) return;
    const int lane = threadIdx.x & 63;
    Steps<TT>& steps = ((Steps<TT>*)lds)[p.w];
    float* const exchange = (float*)((Steps<TT>*)lds + W);
    float A2[NS], h[NS];
    load_A2<NS, true>(a, p, A2);
    const bool grow = SPLIT && may_grow<NS>(a, A2);
    load_state<NS, true>(a.initial, a, p, h);
    if (a.PL) fold_parts<NS>(a, p, 0, p.part(a.PL), 1, grow, h);
    const float skip = a.D_skip ? a.D_skip[p.ch] : 0.0f;
    const float bias = a.dt_bias ? a.dt_bias[p.ch] : 0.0f;
    constexpr int E = sizeof(T);
    const Col cx(a.x, a.seqs, p, E, a.D), cdt(a.dt, a.seqs, p, E, a.D), cz(a.z, a.seqs, p, E, a.D),
        cB(a.B, a.seqs, p, E, a.G * a.N), cC(a.C, a.seqs, p, E, a.G * a.N),
        cy(a.y, a.seqs, p, E, a.D);
    Items<T, TT> rx, rdt, rz;
    RowVals<T, NS, TT> rB, rC;
    const auto fetch = [&](int l) {
        rx.load(cx, p, l);
        rdt.load(cdt, p, l);
        if (a.z.p) rz.load(cz, p, l);
        rB.load(cB, p, a.N, l);
        rC.load(cC, p, a.N, l);
    };
    // The state at the start of a wave's tokens, for the backward pass.
    const auto save = [&](int l, const float (&r)[NS]) {
        constexpr int every = chunk_for(NS);
        if (!a.saved || !p.in || l >= p.hi || l % every) return;
        float* const to =
            a.saved + ((a.seqs.slot0(p.s, every) + (int64_t)(l / every)) * a.D + p.ch) * (4 * NS);
        constexpr int V = NS < 4 ? NS : 4;
#pragma unroll
        for (int j = 0; j < NS; j += V)
            store_f32<float, V>(to + state_of<NS, true>(p.q, j), *(const float (*)[V])(r + j));
    };
    int flip = 0;
    if (SPLIT && p.w == W - 1) put<NS>(exchange_at<NS>(exchange, W, 0), h);
    if (p.lo < p.hi) fetch(p.lo + p.w * TT);
    for (int l0 = p.lo; l0 < p.hi; l0 += W * TT) {
        align_loop();
        const int l = l0 + p.w * TT;
        float x[kItems], u[kItems], z[kItems], v[kItems];
        RowVals<T, NS, TT> tB = rB, tC = rC;
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            x[i] = rx[i];
            z[i] = a.z.p ? rz[i] : 0.0f;
            float d = step_size(a, rdt[i] + bias);
            if (l + TT > p.hi) d = l + p.q + 4 * i < p.hi ? d : 0.0f;
            u[i] = d * x[i];
            steps.d[p.cl][4 * i + p.q] = d;
        }
        wave_sync();
        // The next tokens arrive while these are computed.
        if (l0 + W * TT < p.hi) fetch(l + W * TT);
        if constexpr (SPLIT) {
            float dec[TT][NS], e[NS], sum = 0.0f;
#pragma unroll
            for (int j = 0; j < NS; ++j) e[j] = 0.0f;
            for_groups<TT>([&](int g) {
                float d[4], b[4][NS];
                load_f32<float, 4>(&steps.d[p.cl][4 * g], d);
                tB.outer(g, u[g], b);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    sum += d[t];
#pragma unroll
                    for (int j = 0; j < NS; ++j) {
                        dec[4 * g + t][j] = __builtin_amdgcn_exp2f(d[t] * A2[j]);
                        e[j] = __builtin_fmaf(dec[4 * g + t][j], e[j], b[t][j]);
                    }
                }
            });
            float P[NS], r[NS];
#pragma unroll
            for (int j = 0; j < NS; ++j) P[j] = __builtin_amdgcn_exp2f(sum * A2[j]);
            float* const ex = exchange + flip * exchange_floats(W, NS);
            flip ^= 1;
            put<NS>(exchange_at<NS>(ex, p.w, 0), P);
            put<NS>(exchange_at<NS>(ex, p.w, 1), e);
            *sum_at<NS>(ex, W, p.w) = sum;
            __syncthreads();
            // The other buffer is written next, past this barrier of the next
            // round: nobody still reads it then.
            get<NS>(exchange_at<NS>(ex, W, 0), r);
            // Two segments at a time: one by one the reads' latency adds up.
            int k = 0;
            for (; k + 1 < p.w; k += 2) {
                float P1[NS], e1[NS];
                get<NS>(exchange_at<NS>(ex, k, 0), P);
                get<NS>(exchange_at<NS>(ex, k, 1), e);
                get<NS>(exchange_at<NS>(ex, k + 1, 0), P1);
                get<NS>(exchange_at<NS>(ex, k + 1, 1), e1);
#pragma unroll
                for (int j = 0; j < NS; ++j)
                    r[j] = __builtin_fmaf(P1[j], __builtin_fmaf(P[j], r[j], e[j]), e1[j]);
            }
            if (k < p.w) {
                get<NS>(exchange_at<NS>(ex, k, 0), P);
                get<NS>(exchange_at<NS>(ex, k, 1), e);
#pragma unroll
                for (int j = 0; j < NS; ++j) r[j] = __builtin_fmaf(P[j], r[j], e[j]);
            }
            if (__builtin_expect(grow, 0)) carry_grown<NS>(ex, W, p.w, A2, r);
            save(l, r);
            // The second run, from the true state. Its products d*x*B are made
            // again: holding them would take as many registers as the decays.
            for_groups<TT>([&](int g) {
                float b[4][NS], C[4][NS], y[4];
                tB.outer(g, u[g], b);
                tC.outer(g, 1.0f, C);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    y[t] = 0.0f;
#pragma unroll
                    for (int j = 0; j < NS; ++j) {
                        r[j] = __builtin_fmaf(dec[4 * g + t][j], r[j], b[t][j]);
                        y[t] = __builtin_fmaf(r[j], C[t][j], y[t]);
                    }
                }
                v[g] = row_sums(y, lane);
            });
            // The last wave has reached the state that the next round starts from.
            if (p.w == W - 1) {
                put<NS>(exchange_at<NS>(exchange + flip * exchange_floats(W, NS), W, 0), r);
#pragma unroll
                for (int j = 0; j < NS; ++j) h[j] = r[j];
            }
        } else {
            save(l, h);
            for_groups<TT>([&](int g) {
                float d[4], b[4][NS], C[4][NS], y[4];
                load_f32<float, 4>(&steps.d[p.cl][4 * g], d);
                tB.outer(g, u[g], b);
                tC.outer(g, 1.0f, C);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    y[t] = 0.0f;
#pragma unroll
                    for (int j = 0; j < NS; ++j) {
                        const float e = __builtin_amdgcn_exp2f(d[t] * A2[j]);
                        h[j] = __builtin_fmaf(e, h[j], b[t][j]);
                        y[t] = __builtin_fmaf(h[j], C[t][j], y[t]);
                    }
                }
                v[g] = row_sums(y, lane);
            });
        }
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            v[i] = __builtin_fmaf(skip, x[i], v[i]);
            if (a.z.p) v[i] *= silu_f32(z[i]);
        }
        store_items<T, TT>(cy, p, l, v);
        wave_sync();
    }
    if (p.w == W - 1 && p.hi == p.len) store_state<NS, true>(a.final, a, p, h);
}

// The decay of one run (its root, if a decay can be more than 1) and its state h over
// n more, first, first + step, ...; sum: of the run's step sizes.
template <int NS>
__device__ __forceinline__ void join_runs(float* ex, int W, int first, int n, int step,
                                          const float (&A2)[NS], bool grow, float sum,
                                          float (&P)[NS], float (&h)[NS]) {
    for (int k = 0; k < n; ++k) {
        float Q[NS], e[NS];
        get<NS>(exchange_at<NS>(ex, first + k * step, 0), Q);
        get<NS>(exchange_at<NS>(ex, first + k * step, 1), e);
        sum += *sum_at<NS>(ex, W, first + k * step);
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            h[j] = grow ? carried(Q[j], h[j], e[j]) : __builtin_fmaf(Q[j], h[j], e[j]);
            P[j] *= Q[j];
        }
    }
    if (grow)
#pragma unroll
        for (int j = 0; j < NS; ++j) P[j] = root_decay(sum * A2[j]);
}

// The parts' decays and last states from zero, for all parts but a sequence's
// last. The waves take a part's tokens in W runs side by side.
template <typename T, int NS, int TT>
__global__ __launch_bounds__(64 * waves_for(NS)) void scan_parts(const ScanArgs a) {
    extern __shared__ float4 lds[];
    const int W = blockDim.x >> 6;
    const Place p(a, true);
    if (p.lo < 0 || p.hi == p.len) return;
    Steps<TT>& steps = ((Steps<TT>*)lds)[p.w];
    float* const ex = (float*)((Steps<TT>*)lds + W);
    float A2[NS], h[NS], sum = 0.0f;
    load_A2<NS, true>(a, p, A2);
    const bool grow = may_grow<NS>(a, A2);
#pragma unroll
    for (int j = 0; j < NS; ++j) h[j] = 0.0f;
    const float bias = a.dt_bias ? a.dt_bias[p.ch] : 0.0f;
    const int run = a.PL / W;  // PL is a multiple of W * TT
    constexpr int E = sizeof(T);
    const Col cx(a.x, a.seqs, p, E, a.D), cdt(a.dt, a.seqs, p, E, a.D),
        cB(a.B, a.seqs, p, E, a.G * a.N);
    Items<T, TT> rx, rdt;
    RowVals<T, NS, TT> rB;
    const auto fetch = [&](int l) {
        rx.load(cx, p, l);
        rdt.load(cdt, p, l);
        rB.load(cB, p, a.N, l);
    };
    const int first = p.lo + p.w * run;
    fetch(first);
    for (int l = first; l < first + run; l += TT) {
        float u[TT / 4];
        RowVals<T, NS, TT> tB = rB;
#pragma unroll
        for (int i = 0; i < TT / 4; ++i) {
            const float d = step_size(a, rdt[i] + bias);
            u[i] = d * rx[i];
            steps.d[p.cl][4 * i + p.q] = d;
        }
        wave_sync();
        if (l + TT < first + run) fetch(l + TT);
        for_groups<TT>([&](int g) {
            float d[4], b[4][NS];
            load_f32<float, 4>(&steps.d[p.cl][4 * g], d);
            tB.outer(g, u[g], b);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                sum += d[t];
#pragma unroll
                for (int j = 0; j < NS; ++j)
                    h[j] = __builtin_fmaf(__builtin_amdgcn_exp2f(d[t] * A2[j]), h[j], b[t][j]);
            }
        });
        wave_sync();
    }
    float P[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j)
        P[j] = grow ? root_decay(sum * A2[j]) : __builtin_amdgcn_exp2f(sum * A2[j]);
    put<NS>(exchange_at<NS>(ex, p.w, 0), P);
    put<NS>(exchange_at<NS>(ex, p.w, 1), h);
    *sum_at<NS>(ex, W, p.w) = sum;
    __syncthreads();
    if (p.w != 0) return;
    join_runs<NS>(ex, W, 1, W - 1, 1, A2, grow, sum, P, h);
    if (!p.in) return;
    put<NS>(part_at<NS>(a, p, p.part(a.PL), 0), P);
    put<NS>(part_at<NS>(a, p, p.part(a.PL), 1), h);
}

struct ScanGrads {
    Rows<const void> dy;
    const float *dfinal, *saved;
    Rows<void> dx, ddt, dz;
    float* dinitial;
    float* part_bc;  // [blocks of channels][rows][2][4*NS]: dB, dC of a block
    float* part_a;   // [slots][D*N + 2*D]: dA, dD, ddt_bias of a sequence or part
};

// The chunks of a sequence (or part) from the last to the first. In each, the states
// are computed again from the one the forward pass saved at its start and held
// in registers with the decays, and then the adjoint runs backwards:
//   g[t] = dv[t]*C[t] + a[t+1]*g[t+1]                 (dL/dh[t])
//   dd[t]  = sum_n g*(A*a[t]*h[t-1] + B*x),  dx[t] = d * sum_n g*B + D*dv
//   dA += g*a[t]*h[t-1]*d,   dB = sum_c g*d*x,   dC = sum_c dv*h
// Split over waves and workgroups like the forward pass: what a segment passes
// to the tokens before it, a[first]*g[first], is linear in what reaches it.
template <typename T, int NS, int TT, bool SPLIT>
__global__ __launch_bounds__(SPLIT ? 64 * waves_for(NS) : 64) void scan_bwd(const ScanArgs a,
                                                                            const ScanGrads b) {
    // dB and dC: values of a token after its own levels, and tokens of a group.
    constexpr int kItems = TT / 4, kHeld = NS >> levels_of(NS), GT = NS < 16 ? 16 / NS : 1;
    extern __shared__ float4 lds[];
    const int W = SPLIT ? blockDim.x >> 6 : 1;
    const Place p(a, false);
    float* const sums = b.part_a + (int64_t)p.slot * a.D * (a.N + 2);
    if (p.lo < 0) {  // nobody's slot adds nothing
        if (p.w == 0 && p.in) {
            if (p.q < 2) sums[(int64_t)a.D * a.N + p.q * a.D + p.ch] = 0.0f;
            for (int n = p.q; n < a.N; n += 4) sums[(int64_t)p.ch * a.N + n] = 0.0f;
        }
        return;
    }
    BackTile<NS, TT>& both = ((BackTile<NS, TT>*)lds)[p.w];
    Tile<NS, TT>& tile = both.f;
    float* const exchange = (float*)((BackTile<NS, TT>*)lds + W);
    const int lane = threadIdx.x & 63;
    // c: a[t+1]*g[t+1] of the next token.
    float A2[NS], c[NS], dA[NS];
    load_A2<NS, false>(a, p, A2);
    load_state<NS, false>(b.dfinal, a, p, c);
    if (a.PL) {
        const int last = p.len > 0 ? (p.len - 1) / a.PL : 0;
        fold_parts<NS>(a, p, last, last - p.part(a.PL), -1, true, c);
    }
#pragma unroll
    for (int j = 0; j < NS; ++j) dA[j] = 0.0f;
    put<NS>(both.dA[0][lane], dA);
    put<NS>(both.dA[1][lane], dA);
    const float skip = a.D_skip ? a.D_skip[p.ch] : 0.0f;
    const float bias = a.dt_bias ? a.dt_bias[p.ch] : 0.0f;
    float dD = 0.0f, dbias = 0.0f;
    const int64_t slot0 = a.seqs.slot0(p.s, TT);
    constexpr int E = sizeof(T);
    const Col cx(a.x, a.seqs, p, E, a.D), cdt(a.dt, a.seqs, p, E, a.D), cz(a.z, a.seqs, p, E, a.D),
        cdy(b.dy, a.seqs, p, E, a.D), cB(a.B, a.seqs, p, E, a.G * a.N),
        cC(a.C, a.seqs, p, E, a.G * a.N), cdx(b.dx, a.seqs, p, E, a.D),
        cddt(b.ddt, a.seqs, p, E, a.D), cdz(b.dz, a.seqs, p, E, a.D);
    Items<T, TT> rx, rdt, rz, rdy;
    Shared<T, NS, TT> rB, rC;
    float rh[NS];
    const auto fetch = [&](int l) {
        rx.load(cx, p, l);
        rdt.load(cdt, p, l);
        if (a.z.p) rz.load(cz, p, l);
        rdy.load(cdy, p, l);
        rB.load(cB, p, a.N, l);
        rC.load(cC, p, a.N, l);
#pragma unroll
        for (int j = 0; j < NS; ++j) rh[j] = 0.0f;
        if (p.in && l < p.hi)
            get<NS>(b.saved + ((slot0 + l / TT) * a.D + p.ch) * (4 * NS) + p.q * NS, rh);
    };
    int flip = 0;
    if (SPLIT && p.w == 0) put<NS>(exchange_at<NS>(exchange, W, 0), c);
    const int chunks = (p.hi - p.lo + W * TT - 1) / (W * TT);
    if (chunks > 0) fetch(p.lo + ((chunks - 1) * W + p.w) * TT);
    for (int chunk = chunks - 1; chunk >= 0; --chunk) {
        align_loop();
        const int l = p.lo + (chunk * W + p.w) * TT;
        float h0[NS];
#pragma unroll
        for (int j = 0; j < NS; ++j) h0[j] = rh[j];
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int t = p.q + 4 * i;
            const float x = rx[i], raw = rdt[i] + bias, dout = rdy[i];
            float d = raw, slope = 1.0f, dv = dout, w = 0.0f;  // w: dz for v = 1
            if (a.softplus) softplus_grad_f32(raw, d, slope);
            if (a.z.p) {
                const float z = rz[i], sg = sigmoid_f32(z);
                dv = dout * (z * sg);
                w = dout * (sg * __builtin_fmaf(z, 1.0f - sg, 1.0f));
            }
            if (l + TT > p.hi) {
                // Past the end the state and its adjoint only pass through, but
                // their product, which dL/dd holds, is not zero; and rows that are
                // one row for all tokens do not read as zero there.
                const bool real = l + t < p.hi;
                d = real ? d : 0.0f;
                slope = real ? slope : 0.0f;
                dv = real ? dv : 0.0f;
            }
            tile.d[t][p.cl] = make_float2(d, d * x);
            both.dv[t][p.cl] = dv;
            both.item[i][lane] = make_float4(x, slope, w, 0.0f);
        }
        rB.put(tile.B);
        rC.put(tile.C);
        wave_sync();
        float dec[TT][NS], h[TT][NS], v[kItems], e1[kItems], e2[kItems], sum = 0.0f;
        {
            float y[4];
            for_tokens<NS, TT, true, true, true>(tile, p.cl, p.q, [&](int t, const Token<NS>& k) {
                float s = 0.0f;
                sum += k.d.x;
#pragma unroll
                for (int j = 0; j < NS; ++j) {
                    dec[t][j] = __builtin_amdgcn_exp2f(k.d.x * A2[j]);
                    h[t][j] = __builtin_fmaf(dec[t][j], t ? h[t - 1][j] : h0[j], k.d.y * k.B[j]);
                    s = __builtin_fmaf(h[t][j], k.C[j], s);
                }
                y[t & 3] = s;
                pin(y[t & 3]);
                if ((t & 3) == 3) {
                    v[t >> 2] = quad_sums(y[0], y[1], y[2], y[3], p.q);
                    pin(v[t >> 2]);
                }
            });
        }
        if constexpr (SPLIT) {
            float P[NS], e[NS];
#pragma unroll
            for (int j = 0; j < NS; ++j) e[j] = 0.0f;
            // Two operations for each state: the reads go two tokens ahead (one
            // ahead 236 us, two or three 228: 2 x 2048 tokens, 2048 channels, both passes).
            constexpr int kLead = 2;
            float dv[kLead + 1], C[kLead + 1][NS];
            int q = p.q, cl = p.cl;
            asm volatile("" : "+v"(cl), "+v"(q));
            const auto read = [&](int t) {
                dv[t % (kLead + 1)] = both.dv[t][cl];
                get<NS>(&tile.C[t][q * NS], C[t % (kLead + 1)]);
            };
#pragma unroll
            for (int t = TT - 1; t >= TT - kLead; --t) read(t);
#pragma unroll
            for (int t = TT - 1; t >= 0; --t) {
                if (t >= kLead) read(t - kLead);
#pragma unroll
                for (int j = 0; j < NS; ++j)
                    e[j] = __builtin_fmaf(dv[t % (kLead + 1)], C[t % (kLead + 1)][j], e[j]) *
                           dec[t][j];
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int j = 0; j < NS; ++j) P[j] = root_decay(sum * A2[j]);
            float* const ex = exchange + flip * exchange_floats(W, NS);
            flip ^= 1;
            put<NS>(exchange_at<NS>(ex, p.w, 0), P);
            put<NS>(exchange_at<NS>(ex, p.w, 1), e);
            __syncthreads();
            get<NS>(exchange_at<NS>(ex, W, 0), c);
            // Two segments at a time: one by one the reads' latency adds up.
            int m = W - 1;
            for (; m > p.w + 1; m -= 2) {
                float P1[NS], e1[NS];
                get<NS>(exchange_at<NS>(ex, m, 0), P);
                get<NS>(exchange_at<NS>(ex, m, 1), e);
                get<NS>(exchange_at<NS>(ex, m - 1, 0), P1);
                get<NS>(exchange_at<NS>(ex, m - 1, 1), e1);
#pragma unroll
                for (int j = 0; j < NS; ++j)
                    c[j] = carried(P1[j], carried(P[j], c[j], e[j]), e1[j]);
            }
            if (m > p.w) {
                get<NS>(exchange_at<NS>(ex, m, 0), P);
                get<NS>(exchange_at<NS>(ex, m, 1), e);
#pragma unroll
                for (int j = 0; j < NS; ++j) c[j] = carried(P[j], c[j], e[j]);
            }
        }
        float dAc[NS];
#pragma unroll
        for (int j = 0; j < NS; ++j) dAc[j] = 0.0f;
        float gB[kHeld * GT], gC[kHeld * GT];
        for_tokens<NS, TT, true, true, false>(tile, p.cl, p.q, [&](int t, const Token<NS>& k) {
            const float dv = both.dv[t][p.cl];
            float f1 = 0.0f, f2 = 0.0f, dB[NS], dC[NS];
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                const float g = __builtin_fmaf(dv, k.C[j], c[j]);
                c[j] = g * dec[t][j];
                const float gu = c[j] * (t ? h[t - 1][j] : h0[j]);
                f1 = __builtin_fmaf(gu, A2[j], f1);
                f2 = __builtin_fmaf(g, k.B[j], f2);
                dAc[j] = __builtin_fmaf(gu, k.d.x, dAc[j]);
                dB[j] = g * k.d.y;
                dC[j] = dv * h[t][j];
            }
            join_token<NS>(dB, lane);
            join_token<NS>(dC, lane);
#pragma unroll
            for (int j = 0; j < kHeld; ++j) {
                pin(dB[j]);
                pin(dC[j]);
                gB[t % GT * kHeld + j] = dB[j];
                gC[t % GT * kHeld + j] = dC[j];
            }
            pin(f1);
            pin(f2);
            // In the places of this token's decay and state, which are done with.
            dec[t][0] = f1;
            h[t][0] = f2;
            if (t % GT == 0)
#pragma unroll
                for (int k0 = 0; k0 < kHeld * GT; k0 += 16 >> levels_of(NS)) {
                    const float sB = join_group<NS>(gB + k0, lane);
                    const float sC = join_group<NS>(gC + k0, lane);
                    const int i = (k0 << levels_of(NS)) + ((lane >> 5) & 1) + ((lane >> 3) & 2) +
                                  ((lane >> 1) & 4) + ((lane << 1) & 8);
                    const int u = t + i / NS, n = p.q * NS + i % NS;
                    if (l + u < p.hi) {
                        float* o = b.part_bc + (((int64_t)p.block * a.seqs.rows + p.start + l + u) *
                                                2) * (4 * NS) + n;
                        o[0] = sB;
                        o[4 * NS] = sC;
                    }
                }
            // The next tokens' loads, with enough time left to arrive and no
            // sooner: they take the registers of states that are done with.
            if (t == TT / 4 && chunk > 0) fetch(l - W * TT);
        });
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            e1[i] = quad_sums(dec[4 * i][0], dec[4 * i + 1][0], dec[4 * i + 2][0],
                              dec[4 * i + 3][0], p.q);
            e2[i] = quad_sums(h[4 * i][0], h[4 * i + 1][0], h[4 * i + 2][0], h[4 * i + 3][0], p.q);
        }
        // The sum over all tokens is long: what each addition drops is kept
        // (Kahan), so that it is as exact as a chunk's own sum.
        float lost[NS];
        get<NS>(both.dA[0][lane], dA);
        get<NS>(both.dA[1][lane], lost);
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            const float add = dAc[j] - lost[j], s = dA[j] + add;
            lost[j] = (s - dA[j]) - add;
            dA[j] = s;
        }
        put<NS>(both.dA[0][lane], dA);
        put<NS>(both.dA[1][lane], lost);
        if (SPLIT && p.w == 0)
            put<NS>(exchange_at<NS>(exchange + flip * exchange_floats(W, NS), W, 0), c);
        float dt[kItems], dx[kItems], dz[kItems];
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int t = p.q + 4 * i;
            const float4 it = both.item[i][lane];
            const float dv = both.dv[t][p.cl];
            dt[i] = __builtin_fmaf(e2[i], it.x, e1[i] * kLn2) * it.y;
            dx[i] = __builtin_fmaf(e2[i], tile.d[t][p.cl].x, skip * dv);
            dz[i] = it.z * __builtin_fmaf(skip, it.x, v[i]);
            dbias += dt[i];
            dD = __builtin_fmaf(dv, it.x, dD);
        }
        store_items<T, TT>(cddt, p, l, dt);
        store_items<T, TT>(cdx, p, l, dx);
        if (a.z.p) store_items<T, TT>(cdz, p, l, dz);
        wave_sync();
    }
    dD = quad_sum(dD);
    dbias = quad_sum(dbias);
    get<NS>(both.dA[0][lane], dA);
    if constexpr (SPLIT) {
        // The waves' sums, one after another.
        __syncthreads();
        float* const ex = exchange;
        put<NS>(exchange_at<NS>(ex, p.w, 0), dA);
        exchange_at<NS>(ex, p.w, 1)[0] = p.q == 0 ? dD : dbias;
        __syncthreads();
        if (p.w == 0)
            for (int k = 1; k < W; ++k) {
                float e[NS];
                get<NS>(exchange_at<NS>(ex, k, 0), e);
#pragma unroll
                for (int j = 0; j < NS; ++j) dA[j] += e[j];
                const float o = exchange_at<NS>(ex, k, 1)[0];
                dD += o;
                dbias += o;
            }
    }
    if (p.w != 0 || !p.in) return;
    if (p.q < 2) sums[(int64_t)a.D * a.N + p.q * a.D + p.ch] = p.q == 0 ? dD : dbias;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        const int n = p.q * NS + j;
        if (n < a.N) sums[(int64_t)p.ch * a.N + n] = dA[j];
    }
    if (p.lo == 0) store_state<NS, false>(b.dinitial, a, p, c);
}

// What the parts but a sequence's first pass to the tokens before them, from
// zero, and their decays.
template <typename T, int NS, int TT>
__global__ __launch_bounds__(64 * waves_for(NS)) void scan_bwd_parts(const ScanArgs a,
                                                                     const ScanGrads b) {
    extern __shared__ float4 lds[];
    const int W = blockDim.x >> 6;
    const Place p(a, false);
    if (p.lo <= 0) return;
    Tile<NS, TT>& tile = ((Tile<NS, TT>*)lds)[p.w];
    float* const ex = (float*)((Tile<NS, TT>*)lds + W);
    float A2[NS], c[NS], sum = 0.0f;
    load_A2<NS, false>(a, p, A2);
#pragma unroll
    for (int j = 0; j < NS; ++j) c[j] = 0.0f;
    const float bias = a.dt_bias ? a.dt_bias[p.ch] : 0.0f;
    const int run = a.PL / W;
    constexpr int E = sizeof(T);
    const Col cdt(a.dt, a.seqs, p, E, a.D), cz(a.z, a.seqs, p, E, a.D),
        cdy(b.dy, a.seqs, p, E, a.D), cC(a.C, a.seqs, p, E, a.G * a.N);
    Items<T, TT> rdt, rz, rdy;
    Shared<T, NS, TT> rC;
    const auto fetch = [&](int l) {
        rdt.load(cdt, p, l);
        if (a.z.p) rz.load(cz, p, l);
        rdy.load(cdy, p, l);
        rC.load(cC, p, a.N, l);
    };
    const int first = p.lo + p.w * run;
    fetch(first + run - TT);
    for (int l = first + run - TT; l >= first; l -= TT) {
#pragma unroll
        for (int i = 0; i < TT / 4; ++i) {
            const int t = p.q + 4 * i;
            float d = step_size(a, rdt[i] + bias);
            float dv = a.z.p ? rdy[i] * silu_f32(rz[i]) : rdy[i];
            if (l + TT > p.hi) {
                d = l + t < p.hi ? d : 0.0f;
                dv = l + t < p.hi ? dv : 0.0f;
            }
            tile.d[t][p.cl] = make_float2(d, dv);
        }
        rC.put(tile.C);
        wave_sync();
        if (l > first) fetch(l - TT);
        for_tokens<NS, TT, false, true, false>(tile, p.cl, p.q, [&](int, const Token<NS>& k) {
            sum += k.d.x;
#pragma unroll
            for (int j = 0; j < NS; ++j)
                c[j] = __builtin_fmaf(k.d.y, k.C[j], c[j]) * __builtin_amdgcn_exp2f(k.d.x * A2[j]);
        });
        wave_sync();
    }
    float P[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) P[j] = root_decay(sum * A2[j]);
    put<NS>(exchange_at<NS>(ex, p.w, 0), P);
    put<NS>(exchange_at<NS>(ex, p.w, 1), c);
    *sum_at<NS>(ex, W, p.w) = sum;
    __syncthreads();
    if (p.w != W - 1) return;
    join_runs<NS>(ex, W, W - 2, W - 1, -1, A2, true, sum, P, c);
    if (!p.in) return;
    put<NS>(part_at<NS>(a, p, p.part(a.PL), 0), P);
    put<NS>(part_at<NS>(a, p, p.part(a.PL), 1), c);
}

// The sums over workgroups, each by kPhases threads in a fixed order. The first
// `rows_blocks` workgroups: dB and dC of the rows that the sequences cover, over a
// group's blocks of channels; the others: dA, dD and ddt_bias over the slots.
constexpr int kPhases = 4;
struct ScanSums {
    const float *part_bc, *part_a;
    int NP, slots, rows_blocks;
    Rows<void> dB, dC;
    float *dA, *dD, *ddt_bias;
};
template <typename T>
__global__ __launch_bounds__(64 * kPhases) void scan_sums(const ScanArgs a, const ScanSums b) {
    __shared__ float red[kPhases][64];
    const SeqMap& m = a.seqs;
    const int lane = threadIdx.x & 63, ph = threadIdx.x >> 6, NP = b.NP;
    const bool rows = (int)blockIdx.x < b.rows_blocks;
    const int64_t M = (int64_t)a.D * (a.N + 2), per = (int64_t)a.G * 2 * NP;
    const float* p = nullptr;
    int64_t step = M, i = (int64_t)((int)blockIdx.x - b.rows_blocks) * 64 + lane;
    int row = 0, g = 0, c = 0, n = 0, count = b.slots;
    if (rows) {
        i = m.start(0) * per + (int64_t)blockIdx.x * 64 + lane;
        row = (int)(i / per);
        const int r = (int)(i - row * per), k = r % (2 * NP);
        g = r / (2 * NP), c = k / NP, n = k - c * NP;
        step = (int64_t)m.rows * 2 * NP;
        count = a.bpg;
        if (i < m.end(m.seqs - 1) * per && n < a.N)
            p = b.part_bc + (((int64_t)g * a.bpg * m.rows + row) * 2 + c) * NP + n;
    } else if (i < M) {
        p = b.part_a + i;
    }
    float v = 0.0f;
    if (p)
#pragma unroll 8
        for (int k = ph; k < count; k += kPhases) v += p[k * step];
    red[ph][lane] = v;
    __syncthreads();
    if (ph != 0 || !p) return;
#pragma unroll
    for (int j = 1; j < kPhases; ++j) v += red[j][lane];
    if (rows) {
        const int s = m.offsets ? 0 : row / m.L;
        row_of<T>(c ? b.dC : b.dB, m, s, 0, m.offsets ? row : row - s * m.L)[g * a.N + n] = (T)v;
        return;
    }
    const int64_t dn = (int64_t)a.D * a.N;
    if (i < dn) b.dA[i] = v;
    else if (i < dn + a.D && b.dD) b.dD[i - dn] = v;
    else if (i >= dn + a.D && b.ddt_bias) b.ddt_bias[i - dn - a.D] = v;
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
            const float e = __builtin_amdgcn_exp2f(d * rate2(A[j]));
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

// States of a lane: 4 lanes hold N.
int states_for(int N) {
    int ns = 1;
    while (4 * ns < N) ns *= 2;
    return ns;
}

// How a call is cut up, by its sizes alone.
struct Plan {
    int ns, tt, waves, PL;  // waves 1: whole sequences by single waves
    int64_t slots, nb;      // workgroups: slots * nb
};
Plan plan_of(const tg_scan_args& a, bool forward) {
    Plan p;
    p.ns = states_for(a.N);
    p.tt = forward ? fwd_chunk_for(p.ns) : chunk_for(p.ns);
    p.nb = (int64_t)a.G * ceil_div(a.D / a.G, kCh);
    const int64_t groups = a.seqs.seqs * p.nb;
    p.waves = groups >= 4096 ? 1 : waves_for(p.ns);
    p.PL = 0;
    p.slots = a.seqs.seqs;
    // Fewer than four waves for each compute unit: parts of the sequences, so
    // many that there are sixteen, and not shorter than two rounds of a workgroup.
    // The parts' own pass costs two thirds of the scan and a launch: 9 packed
    // sequences with 1728 waves take 24 to 33 us whole and 33 to 37 in parts. The rule
    // counts sequences, not their tokens, and does badly by one that is long: 16384
    // tokens take 396 us with 1920 channels, in parts, and 465 with 2048, whole (4 x
    // 4096: 194); 12000 packed with 15 of 10 each, 4096 channels, by single waves, 2026 us
    // (16 of 759: 261).
    if (p.waves > 1 && groups * p.waves < 1024) {
        const int64_t round = (int64_t)p.waves * p.tt;
        int64_t pl = a.seqs.rows * p.nb * p.waves / 4096 / round * round;
        if (pl < 2 * round) pl = 2 * round;
        const int64_t longest = a.seqs.offsets ? a.seqs.rows : a.seqs.rows / a.seqs.seqs;
        if (pl < longest) {
            p.PL = (int)pl;
            p.slots = a.seqs.offsets ? a.seqs.rows / pl + a.seqs.seqs
                                     : a.seqs.seqs * ceil_div(longest, pl);
        }
    }
    return p;
}
size_t parts_bytes(const tg_scan_args& a, const Plan& p) {
    return p.PL ? (size_t)p.slots * 2 * a.D * 4 * p.ns * sizeof(float) : 0;
}

// Written rows whose stride keeps the tokens past the end out of the one before:
// with a single row in the batch any stride is accepted, and none is used.
Rows<void> written_rows(const tg_rows& r, const tg_scan_args& a) {
    Rows<void> w = rows_of<void>(r);
    if (a.seqs.rows == 1) w.row = a.D;
    return w;
}

ScanArgs args_of(const tg_scan_args& a, const Plan& p, float* saved, void* parts) {
    const int Dg = a.D / a.G;
    return {map_of(a.seqs), a.D, a.N, a.G, Dg, (int)ceil_div(Dg, kCh), a.softplus, p.PL,
            rows_of<const void>(a.x), rows_of<const void>(a.dt), rows_of<const void>(a.B),
            rows_of<const void>(a.C), rows_of<const void>(a.z), written_rows(a.y, a), a.A, a.D_skip,
            a.dt_bias, a.initial, a.final, saved, (float*)parts};
}

#define TG_SCAN_NS(X, T)                           \
    do {                                           \
        switch (p.ns) {                            \
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

// Tiles of `tile` bytes for each wave, and `buffers` exchange buffers.
template <typename Kernel, typename... Args>
hipError_t launch_waves(Kernel kernel, const Plan& p, size_t tile, int buffers, hipStream_t st,
                        const Args&... args) {
    const size_t bytes = p.waves * tile + (p.waves > 1 ? buffers * exchange_floats(p.waves, p.ns) * sizeof(float) : 0);
    try {
        const hipError_t e = ensure_dynamic_lds((const void*)kernel, bytes);
        if (e != hipSuccess) return e;
    } catch (...) {  // its record of kernels could not grow
        return hipErrorOutOfMemory;
    }
    kernel<<<(unsigned)(p.slots * p.nb), 64 * p.waves, bytes, st>>>(args...);
    return hipGetLastError();
}

template <typename T, int NS>
hipError_t fwd_typed(const Plan& p, const ScanArgs& f, hipStream_t st) {
    constexpr int TT = fwd_chunk_for(NS);
    constexpr size_t tile = sizeof(Steps<TT>);
    if (p.PL) {
        const hipError_t e = launch_waves(scan_parts<T, NS, TT>, p, tile, 1, st, f);
        if (e != hipSuccess) return e;
    }
    if (p.waves > 1) return launch_waves(scan_fwd<T, NS, TT, true>, p, tile, 2, st, f);
    return launch_waves(scan_fwd<T, NS, TT, false>, p, tile, 0, st, f);
}
template <typename T, int NS>
hipError_t bwd_typed(const Plan& p, const ScanArgs& f, const ScanGrads& b, hipStream_t st) {
    constexpr int TT = chunk_for(NS);
    constexpr size_t tile = sizeof(Tile<NS, TT>), both = sizeof(BackTile<NS, TT>);
    if (p.PL) {
        const hipError_t e = launch_waves(scan_bwd_parts<T, NS, TT>, p, tile, 1, st, f, b);
        if (e != hipSuccess) return e;
    }
    if (p.waves > 1) return launch_waves(scan_bwd<T, NS, TT, true>, p, both, 2, st, f, b);
    return launch_waves(scan_bwd<T, NS, TT, false>, p, both, 0, st, f, b);
}

struct BackwardWs {
    size_t bc, parts, total;  // the sums of dA, dD and ddt_bias come first
};
BackwardWs backward_ws(const tg_scan_args& a, const Plan& p) {
    BackwardWs w;
    w.bc = up256((size_t)p.slots * a.D * (a.N + 2) * sizeof(float));
    w.parts = w.bc + up256((size_t)p.nb * a.seqs.rows * 2 * 4 * p.ns * sizeof(float));
    w.total = w.parts + parts_bytes(a, p);
    return w;
}

}  // namespace

static int64_t sum_row_groups(const tg_scan_args& a) {
    return ceil_div(a.seqs.rows * a.G * 2 * 4 * states_for(a.N), 64);
}
int64_t scan_sum_groups(const tg_scan_args& a) {
    return sum_row_groups(a) + ceil_div((int64_t)a.D * (a.N + 2), 64);
}

void scan_sizes(const tg_scan_args& a, size_t* work, size_t* saved, size_t* backward) {
    const Plan f = plan_of(a, true), p = plan_of(a, false);
    const int64_t slots = a.seqs.rows / p.tt + a.seqs.seqs;
    if (work) *work = parts_bytes(a, f);
    if (saved) *saved = (size_t)slots * a.D * 4 * p.ns * sizeof(float);
    if (backward) *backward = backward_ws(a, p).total;
}

hipError_t launch_scan(const tg_scan_args& a, void* ws, void* saved, hipStream_t st) {
    const tg_dtype dtype = a.dtype;
    const Plan p = plan_of(a, true);
    const ScanArgs f = args_of(a, p, (float*)saved, ws);
#define TG_X(T, NS) return fwd_typed<T, NS>(p, f, st)
    TG_SCAN_DISPATCH(TG_X);
#undef TG_X
    return hipErrorInvalidValue;
}

hipError_t launch_scan_backward(const tg_scan_args& a, const tg_scan_grads& g, const void* saved,
                                void* ws, hipStream_t st) {
    const tg_dtype dtype = a.dtype;
    const Plan p = plan_of(a, false);
    const BackwardWs w = backward_ws(a, p);
    char* const base = (char*)ws;
    const ScanArgs f = args_of(a, p, nullptr, base + w.parts);
    const ScanGrads b{rows_of<const void>(g.dy), g.dfinal, (const float*)saved,
                      written_rows(g.dx, a), written_rows(g.ddt, a), written_rows(g.dz, a), g.dinitial,
                      (float*)(base + w.bc), (float*)base};
    hipError_t e = hipSuccess;
#define TG_X(T, NS) e = bwd_typed<T, NS>(p, f, b, st)
    TG_SCAN_DISPATCH(TG_X);
#undef TG_X
    if (e != hipSuccess) return e;
    const int np = 4 * p.ns;
    const int64_t row_blocks = sum_row_groups(a);
    const ScanSums s{b.part_bc, b.part_a, np, (int)p.slots, (int)row_blocks,
                     rows_of<void>(g.dB), rows_of<void>(g.dC), g.dA, g.dD, g.ddt_bias};
    const unsigned grid = (unsigned)scan_sum_groups(a);
    constexpr int threads = 64 * kPhases;
    if (dtype == TG_F32) scan_sums<float><<<grid, threads, 0, st>>>(f, s);
    else if (dtype == TG_BF16) scan_sums<bf16><<<grid, threads, 0, st>>>(f, s);
    else scan_sums<f16><<<grid, threads, 0, st>>>(f, s);
    return hipGetLastError();
}

hipError_t launch_scan_step(const tg_scan_args& a, float* state, int64_t num_slots,
                            const int32_t* slots, hipStream_t st) {
    const StepArgs b{args_of(a, Plan{}, nullptr, nullptr), state, num_slots, slots};
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
