// seq_delta_backward.hip -- gradients of the gated delta rule
// (tg_gated_delta_rule_backward), in the notation of seq_delta.hip. With dS the
// gradient of the state after a chunk, w = dy and U = b E:
//     dU = P^T w + e^(G[C-1]-G) k dS,     R = dv = X^T (b dU)
//     dS0 = e^(G[C-1]) dS + (e^G scale q)^T w - (e^G k)^T R
// walks up the chunks like the forward pass walks down. The rest needs only S0
// and E (saved by the forward pass), dS and R of a chunk, for all chunks at once:
//     F = w E^T,  H = -R E^T,  Z = e^(G[C-1]-G) (k dS).E
//     dq = scale e^G w S0^T + (scale b D F) k
//     dk = (scale b D F)^T q + e^(G[C-1]-G) b E dS^T - e^G R S0^T + (M + M^T) k,
//          M = b D H, strictly lower
//     db[j] = Z[j] + sum_i T[i,j],        T = (D scale q k^T) F + (D k k^T) H
// and the logarithm of token t's decay gets what passes it:
//     dg[t] = sum_{j < t <= i} T[i,j] b[j] + sum_{j < t} b[j] Z[j] + e^(G[C-1]) <dS, S0>
//             + sum_{i >= t} e^G[i] (scale q[i].(w S0^T)[i] - k[i].(R S0^T)[i])
// Each term holds t's decay as a factor, so dg is small where the decay is strong. (As
// sums of dG[i] from t to the chunk's end, which are fewer, terms that do not pass
// t cancel but for their rounding, which a large rate would multiply.)
#include "seq_delta.hpp"
#include "tg_internal.hpp"

namespace tg {
namespace {

template <typename T, int KP>
struct BackShape {
    static constexpr int NI = kIn<T>, C = delta_chunk(NI, KP), LD = KP + 8, NT = C / 16;
    static constexpr int slice = slice_of(NI, KP), cols = slice / 16, WL = slice + 8;
    static constexpr int rows = NI * C * LD * 2;
    static constexpr int stage = kScales * C * 4 + 2 * rows + NI * C * WL * 2;
    // For 16 columns: sums of halves and P^T w; b dU, R for dS; q's part of dS.
    static constexpr int sums = NT * 1024, share = 2 * sums + NT * 512 * 2 * kParts + KP / 16 * 1024;
    static constexpr int stages = 2 * stage + cols * share <= 160 * 1024 ? 2 : 1;
    static constexpr int lds = stages * stage + cols * share, carriers = cols * 2, threads = carriers * 128;
    static_assert(lds <= 160 * 1024, "more LDS than a compute unit has");
};

// The states' gradients, from the last chunk to the first, divided among the waves
// like the forward pass; the helpers form P^T w and q's part of dS0.
template <typename T, int KP, bool WIDE, bool WIDE_V>
__global__ __launch_bounds__(slice_of(kIn<T>, KP) * 16, 1) void delta_backward(const DeltaArgs a) {
    using Sh = BackShape<T, KP>;
    constexpr int NI = Sh::NI, C = Sh::C, LD = Sh::LD, WL = Sh::WL, NT = Sh::NT, HT = NT / 2;
    constexpr int KH = KP / 2, KT = KH / 16, NK = KH / 32, CT = C / 32;
    extern __shared__ float4 lds[];
    const int w = (threadIdx.x >> 6) % Sh::carriers, l = threadIdx.x & 63, g = l >> 4, col = l & 15;
    const int ct = w % Sh::cols, hf = w / Sh::cols;
    const bool helper = threadIdx.x >= Sh::carriers * 64;
    const int slices = (a.V + Sh::slice - 1) / Sh::slice;
    const HeadSlice at = head_slice(a.through ? slices + KP / Sh::slice : slices);
    if (at.pair >= a.units * a.HV) return;
    const int unit = at.pair / a.HV, h = at.pair % a.HV, hk = h / (a.HV / a.HK);
    Segment seg;
    if (!seg.find(a, unit)) return;
    if (a.through && seg.lo == 0) return;  // nobody goes on from there
    const int s = seg.s, start = seg.start, first = seg.lo, len = seg.hi - seg.lo;
    const int slot0 = a.map.slot0(s, C) + first / C, chunks = (len + C - 1) / C;
    // The slices behind V's start from columns of the identity, with no dy.
    const bool unity = at.slice >= slices;
    const int v0 = unity ? 0 : at.slice * Sh::slice, k0 = hf * KH;
    char* share = (char*)lds + Sh::stages * Sh::stage + ct * Sh::share;
    float *xsum = (float*)share, *usum = (float*)(share + Sh::sums), *qsum = (float*)(share + 2 * Sh::sums);
    const HalfFrags<kParts> rx{(bf16*)(share + 2 * Sh::sums + KP / 16 * 1024)}, wx{rx.p + NT * kParts * 256};

    // A stage: scales, k, q, the slice of dy.
    const auto stage = [&](int c) { return (char*)lds + (c % Sh::stages) * Sh::stage; };
    const auto planes = [&](int c, int which) {
        return Planes<NI>{(bf16*)(stage(c) + kScales * C * 4 + which * Sh::rows), which < 2 ? LD : WL,
                          which < 2 ? C * LD : C * WL};
    };
    const auto record = [&](int c) {
        return a.prep + ((int64_t)(slot0 + c) * a.HV + h) * prep_bytes(C, 2 * kParts);
    };
    // Tiles hf * HT + i of X^T and P^T, blocks of 32 columns from theirs on.
    Frag<kParts> prep[HT][CT];
    const auto used = [&](int t) { return t == CT - 1 || hf == 0; };
    const auto fetch_prepared = [&](int c, int which) {
        const bf16* f = (const bf16*)(record(c < 0 ? 0 : c) + kScales * C * 4) +
                        which * frag_count(C) * 512 * kParts;
#pragma unroll
        for (int i = 0; i < HT; ++i)
#pragma unroll
            for (int t = 0; t < CT; ++t)
                prepared(prep[i][t], f, used(t) ? frag_index(C, hf * HT + i, t, true) : 0);
    };

    if (helper) {
        Tile<T, C, KP, Sh::carriers * 64, WIDE> kt, qt;
        Tile<T, C, Sh::slice, Sh::carriers * 64, WIDE_V> vt;
        kt.shape(a.k.row, a.K);
        qt.shape(a.q.row, a.K);
        vt.shape(a.dy.row, imin(Sh::slice, a.V - v0));
        constexpr int SC = kScales * C / 4, SN = (SC + Sh::carriers * 64 - 1) / (Sh::carriers * 64);
        float4 st[SN];
        const auto fetch = [&](int c) {
            c = c < 0 ? 0 : c;
            const int lo = c * C, n = imin(C, len - lo);
            kt.fetch(row_of<const T>(a.k, a.map, s, start, first + lo) + (int64_t)hk * a.K, n);
            qt.fetch(row_of<const T>(a.q, a.map, s, start, first + lo) + (int64_t)hk * a.K, n);
            vt.fetch(row_of<const T>(a.dy, a.map, s, start, first + lo) + (int64_t)h * a.V + v0,
                     unity ? 0 : n);
#pragma unroll
            for (int i = 0; i < SN; ++i)
                st[i] = ((const float4*)record(c))[(i * Sh::carriers * 64 + kt.tid()) % SC];
        };
        const auto put = [&](int c) {
            if (c < 0) return;
#pragma unroll
            for (int i = 0; i < SN; ++i)
                ((float4*)stage(c))[(i * Sh::carriers * 64 + kt.tid()) % SC] = st[i];
            kt.put(planes(c, 0));
            qt.put(planes(c, 1));
            vt.put(planes(c, 2));
        };
        if (chunks > 0) {
            fetch(chunks - 1);
            fetch_prepared(chunks - 1, 1);
            put(chunks - 1);
            fetch(chunks - 2);
        }
        for (int c = chunks - 1; c >= 0; --c) {
            lds_barrier();  // chunk c is there
            const float* scal = (const float*)stage(c);
            const Planes<NI> qp = planes(c, 1), wp = planes(c, 2);
            Frag<NI> wf[CT];
#pragma unroll
            for (int t = 0; t < CT; ++t) wf[t] = wp.cols(t * 32, ct * 16);
            float4_t u[HT] = {};  // P^T w
#pragma unroll
            for (int t = 0; t < CT; ++t)
                if (used(t)) {
                    Frag<kParts> f[HT];
#pragma unroll
                    for (int i = 0; i < HT; ++i) f[i] = prep[i][t];
                    mma_rows<kParts>(u, f, wf[t], All());
                }
#pragma unroll
            for (int i = 0; i < HT; ++i) *sum_at(usum, hf * HT + i) = u[i];
            if (Sh::stages == 2) {
                put(c - 1);
                fetch(c - 2);
            }
            lds_barrier();
            fetch_prepared(c - 1, 1);
            // Half of the tiles on each side of a barrier that the others come to soon.
            Frag<kParts> qw[CT];
#pragma unroll
            for (int b = 0; b < CT; ++b) {
                float y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    y[j] = 0.0f;
#pragma unroll
                    for (int q = NI - 1; q >= 0; --q) y[j] += (float)wf[b].p[q][j];
                }
                qw[b] =
                    frag_of<kParts>(float4_t{y[0], y[1], y[2], y[3]} * scales(scal, C, kReadQ, 2 * b),
                                    float4_t{y[4], y[5], y[6], y[7]} * scales(scal, C, kReadQ, 2 * b + 1));
            }
            const auto tiles = [&](int first) {
                float4_t D[KT / 2] = {};
#pragma unroll
                for (int b = 0; b < CT; ++b) {
                    Frag<NI> f[KT / 2];
#pragma unroll
                    for (int t = 0; t < KT / 2; ++t) f[t] = qp.cols(b * 32, k0 + (first + t) * 16);
                    mma_rows<kParts>(D, f, qw[b], All());
                }
#pragma unroll
                for (int t = 0; t < KT / 2; ++t) *sum_at(qsum, hf * KT + first + t) = D[t];
            };
            tiles(0);
            lds_barrier();
            tiles(KT / 2);
            lds_barrier();
            if (Sh::stages == 1) {
                lds_barrier();  // chunk c has been read
                put(c - 1);
                fetch(c - 2);
            }
        }
        return;
    }

    __builtin_amdgcn_s_setprio(2);  // the helpers have time
    const int v = v0 + ct * 16 + col;
    const int64_t KV = (int64_t)a.K * a.V;
    const float* after = a.dfinal ? a.dfinal + ((int64_t)(a.segment ? unit : s) * a.HV + h) * KV : nullptr;
    const auto tile_at = [&](int i) { return i < HT ? (1 - hf) * HT + i : hf * HT + i - HT; };
    if (chunks > 0) fetch_prepared(chunks - 1, 0);
    float4_t S[KT];  // dS
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int k = k0 + t * 16 + 4 * g + r;
            if (a.through) S[t][r] = unity && k == (at.slice - slices) * Sh::slice + v && k < a.K ? 1.0f : 0.0f;
            else S[t][r] = after && k < a.K && v < a.V ? after[(int64_t)k * a.V + v] : 0.0f;
        }
    for (int c = chunks - 1; c >= 0; --c) {
        lds_barrier();  // chunk c is there
        const float* scal = (const float*)stage(c);
        const Planes<NI> kp = planes(c, 0);
        float* keep = a.back + ((int64_t)(slot0 + c) * a.HV + h) * kept_floats(a.V, KP, C);
        const int vt = v0 / 16 + ct;
        if (vt * 16 < a.V && !a.through)
#pragma unroll
            for (int t = 0; t < KT; ++t) *kept_at(keep, KP, C, vt, hf * KT + t) = S[t];
        // k dS over this half's rows: the other half's tokens, then its own.
        float4_t x[NT] = {};
#pragma unroll
        for (int t = 0; t < NK; ++t) {
            const Frag<kParts> sf = frag_of<kParts>(S[2 * t], S[2 * t + 1]);
            Frag<NI> f[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i) f[i] = kp.rows(tile_at(i) * 16, k0 + t * 32);
            mma_rows<kParts>(x, f, sf, All());
        }
#pragma unroll
        for (int i = 0; i < HT; ++i) *sum_at(xsum, tile_at(i)) = x[i];
        lds_barrier();
        float4_t R[HT] = {};
#pragma unroll
        for (int i = 0; i < HT; ++i) {
            const int mt = hf * HT + i;
            const float4_t z = x[HT + i] + *sum_at(xsum, mt);
            rx.put(mt, (*sum_at(usum, mt) + z * scales(scal, C, kTailK, mt)) * scales(scal, C, kBeta, mt));
        }
        lds_barrier();
#pragma unroll
        for (int t = 0; t < CT; ++t)
            if (used(t)) {
                const Frag<kParts> bf = rx.frag(t);
                Frag<kParts> f[HT];
#pragma unroll
                for (int i = 0; i < HT; ++i) f[i] = prep[i][t];
                mma_rows<kParts>(R, f, bf, All());
            }
        fetch_prepared(c - 1, 0);
#pragma unroll
        for (int i = 0; i < HT; ++i)
            wx.put(hf * HT + i, -R[i] * scales(scal, C, kReadK, hf * HT + i));
        const float total = scal[kDecay * C + C - 1];
        lds_barrier();
#pragma unroll
        for (int t = 0; t < KT; ++t) S[t] = S[t] * total + *sum_at(qsum, hf * KT + t);
#pragma unroll
        for (int b = 0; b < CT; ++b) {
            const Frag<kParts> kr = wx.frag(b);
            Frag<NI> f[KT];
#pragma unroll
            for (int t = 0; t < KT; ++t) f[t] = kp.cols(b * 32, k0 + t * 16);
            mma_rows<kParts>(S, f, kr, All());
        }
        if (vt * 16 < a.V && !a.through)
#pragma unroll
            for (int i = 0; i < HT; ++i) *kept_at(keep, KP, C, vt, KP / 16 + hf * HT + i) = R[i];
        if (Sh::stages == 1) lds_barrier();
    }
    if (a.through) {
        const int columns = map_columns(a.V, KP, Sh::slice);
        float* out = a.maps + ((int64_t)unit * a.HV + h) * KP * columns + at.slice * Sh::slice + ct * 16 + col;
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) out[(int64_t)(k0 + t * 16 + 4 * g + r) * columns] = S[t][r];
    } else if (a.dinitial && seg.lo == 0 && v < a.V) {
        float* out = a.dinitial + ((int64_t)s * a.HV + h) * KV;
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int k = k0 + t * 16 + 4 * g + r;
                if (k < a.K) out[(int64_t)k * a.V + v] = S[t][r];
            }
    }
}

template <typename T, int KP>
hipError_t states_at(const DeltaArgs& a, hipStream_t st) {
    using Sh = BackShape<T, KP>;
    const auto kernel = !a.wide_qk   ? delta_backward<T, KP, false, false>
                        : a.wide_dy ? delta_backward<T, KP, true, true>
                                    : delta_backward<T, KP, true, false>;
    const hipError_t e = ensure_dynamic_lds((const void*)kernel, Sh::lds);
    if (e != hipSuccess) return e;
    const int slices = (int)ceil_div(a.V, Sh::slice) + (a.through ? KP / Sh::slice : 0);
    const int64_t grid = head_slice_grid((int64_t)a.units * a.HV, slices);
    kernel<<<(unsigned)grid, Sh::threads, Sh::lds, st>>>(a);
    return hipGetLastError();
}

}  // namespace

template <typename T>
hipError_t launch_delta_states(const DeltaArgs& a, int KP, hipStream_t st) {
    if (KP == 64) return states_at<T, 64>(a, st);
    if (KP == 128) return states_at<T, 128>(a, st);
    return states_at<T, 256>(a, st);
}
template hipError_t launch_delta_states<float>(const DeltaArgs&, int, hipStream_t);
template hipError_t launch_delta_states<bf16>(const DeltaArgs&, int, hipStream_t);
template hipError_t launch_delta_states<f16>(const DeltaArgs&, int, hipStream_t);

}  // namespace tg
