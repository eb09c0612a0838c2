// seq_delta_forward.hip -- the gated delta rule's walk down a sequence's chunks, in
// the notation of seq_delta.hip: the V columns of S are independent, so workgroups
// have slices of them, S in accumulators and one chunk after the other in LDS.
#include "seq_delta.hpp"
#include "tg_internal.hpp"

namespace tg {
namespace {

// Rows row0 + 4g .. +3 of column col0 + l % 16 of a tile of T in LDS.
template <typename T>
__device__ __forceinline__ float4_t values4(const T* p, int ld, int row0, int col0) {
    const int l = threadIdx.x & 63, g = l >> 4, i = l & 15;
    float4_t o;
    if constexpr (sizeof(T) == 2) {
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        const T* at = p + (row0 + 4 * g + (i >> 2)) * ld + col0 + 4 * (i & 3);
        const auto r = __builtin_bit_cast(typename VecOf<T, 4>::type,
                                          __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at));
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = (float)r[j];
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = (float)p[(row0 + 4 * g + j) * ld + col0 + i];
    }
    return o;
}

template <typename T, int KP>
struct FwdShape {
    static constexpr int NI = kIn<T>, NO = kOut<T>, C = delta_chunk(NI, KP), LD = KP + 8, NT = C / 16;
    static constexpr int slice = slice_of(NI, KP), cols = slice / 16, VL = slice + 8;
    static constexpr int rows = NI * C * LD * 2;
    static constexpr int stage = kScales * C * 4 + 2 * rows + C * VL * (int)sizeof(T);
    // For 16 columns: sums of halves; right sides, corrections for S and for y; S for y.
    static constexpr int sums = NT * 1024, share = sums + NT * 512 * (2 * kParts + NO) + KP / 32 * NO * 1024;
    static constexpr int stages = 2 * stage + cols * share <= 160 * 1024 ? 2 : 1;
    static constexpr int lds = stages * stage + cols * share, carriers = cols * 2, threads = carriers * 128;
    static_assert(lds <= 160 * 1024, "more LDS than a compute unit has");
};

template <typename T, int KP, bool WIDE, bool WIDE_V>
__global__ __launch_bounds__(slice_of(kIn<T>, KP) * 16, 1) void delta_forward(const DeltaArgs a) {
    using Sh = FwdShape<T, KP>;
    constexpr int NI = Sh::NI, NO = Sh::NO, C = Sh::C, LD = Sh::LD, VL = Sh::VL, NT = Sh::NT, HT = NT / 2;
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
    if (a.through && seg.hi == seg.len) return;  // nobody goes on from there
    const int s = seg.s, start = seg.start, first = seg.lo, len = seg.hi - seg.lo;
    const int slot0 = a.map.slot0(s, C) + first / C, chunks = (len + C - 1) / C;
    // The slices behind V's start from columns of the identity, with no v.
    const bool unity = at.slice >= slices;
    const int v0 = unity ? 0 : at.slice * Sh::slice;
    char* share = (char*)lds + Sh::stages * Sh::stage + ct * Sh::share;
    float* xsum = (float*)share;
    const HalfFrags<kParts> rx{(bf16*)(share + Sh::sums)}, wx{rx.p + NT * kParts * 256};
    const HalfFrags<NO> ux{wx.p + NT * kParts * 256};
    bf16* sx = ux.p + NT * NO * 256;  // S's fragments, NO parts

    // A stage: scales, k, q, the slice of v.
    const auto stage = [&](int c) { return (char*)lds + (c % Sh::stages) * Sh::stage; };
    const auto planes = [&](int c, int which) {
        return Planes<NI>{(bf16*)(stage(c) + kScales * C * 4 + which * Sh::rows), LD, C * LD};
    };
    const auto record = [&](int c) {
        return a.prep + ((int64_t)(slot0 + c) * a.HV + h) * prep_bytes(C, kParts + NO);
    };
    // Whether a half's corrections are not finite: in place of scales that this walk does
    // not read.
    const auto odd = [&](int c, int half) { return (int*)stage(c) + kTailK * C + ct * 2 + half; };
    // Tiles hf * HT + i of X and P, blocks of 32 columns up to theirs.
    const auto used = [&](int t) { return t == 0 || hf != 0; };

    if (helper) {
        const int vy = v0 + ct * 16 + 4 * g;
        const uint32_t at_y = (uint32_t)(hf * HT * 16 + col) * (uint32_t)a.y.row + ct * 16 + 4 * g;
        Tile<T, C, KP, Sh::carriers * 64, WIDE> kt, qt;
        Tile<T, C, Sh::slice, Sh::carriers * 64, WIDE_V> vt;
        kt.shape(a.k.row, a.K);
        qt.shape(a.q.row, a.K);
        vt.shape(a.v.row, imin(Sh::slice, a.V - v0));
        constexpr int SC = kScales * C / 4, SN = (SC + Sh::carriers * 64 - 1) / (Sh::carriers * 64);
        float4 st[SN];
        Frag<NO> pf[HT][CT];
        const auto fetch = [&](int c) {
            c = imin(c, chunks - 1);
            const int lo = c * C, n = imin(C, len - lo);
            kt.fetch(row_of<const T>(a.k, a.map, s, start, first + lo) + (int64_t)hk * a.K, n);
            qt.fetch(row_of<const T>(a.q, a.map, s, start, first + lo) + (int64_t)hk * a.K, n);
            vt.fetch(row_of<const T>(a.v, a.map, s, start, first + lo) + (int64_t)h * a.V + v0,
                     unity ? 0 : n);
#pragma unroll
            for (int i = 0; i < SN; ++i)
                st[i] = ((const float4*)record(c))[(i * Sh::carriers * 64 + kt.tid()) % SC];
        };
        const auto put = [&](int c) {
            if (c >= chunks) return;
#pragma unroll
            for (int i = 0; i < SN; ++i)
                ((float4*)stage(c))[(i * Sh::carriers * 64 + kt.tid()) % SC] = st[i];
            kt.put(planes(c, 0));
            qt.put(planes(c, 1));
            vt.put_raw((T*)(planes(c, 1).p + NI * C * LD), VL);
        };
        const auto fetch_p = [&](int c) {
            const bf16* f =
                (const bf16*)(record(imin(c, chunks - 1)) + kScales * C * 4) + frag_count(C) * 512 * kParts;
#pragma unroll
            for (int i = 0; i < HT; ++i)
#pragma unroll
                for (int t = 0; t < CT; ++t)
                    prepared(pf[i][t], f, used(t) ? frag_index(C, hf * HT + i, t, false) : 0);
        };
        if (chunks > 0) {
            fetch(0);
            fetch_p(0);
            put(0);
            fetch(1);
        }
        for (int c = 0; c < chunks; ++c) {
            lds_barrier();  // chunk c is there
            if (Sh::stages == 2) {
                put(c + 1);
                fetch(c + 2);
            }
            const int lo = c * C, n = imin(C, len - lo);
            const float* scal = (const float*)stage(c);
            const Planes<NI> qp = planes(c, 1);
            lds_barrier();  // so is S0 for y
            // y transposed, so that a lane holds four neighbouring columns of a token.
            // Half of it on each side of a barrier that the others come to soon.
            float4_t ys[HT] = {};
            const auto blocks = [&](int first) {
#pragma unroll
                for (int t = 0; t < KP / 64; ++t) {
                    Frag<NO> sf;
                    Frag<NI> f[HT];
                    prepared(sf, sx, first + t);
#pragma unroll
                    for (int i = 0; i < HT; ++i) f[i] = qp.rows((hf * HT + i) * 16, (first + t) * 32);
                    mma_cols<NO>(ys, sf, f, All());
                }
            };
            if (!a.through) blocks(0);
            lds_barrier();
            if (!a.through) blocks(KP / 64);
#pragma unroll
            for (int i = 0; i < HT; ++i) ys[i] *= scal[kReadQ * C + (hf * HT + i) * 16 + col];
            lds_barrier();  // the corrections are there
            if (a.through) {
                if (Sh::stages == 1) {
                    lds_barrier();
                    put(c + 1);
                    fetch(c + 2);
                }
                continue;
            }
            const bool bad = *odd(c, 0) | *odd(c, 1);
            int from = C;
#pragma unroll
            for (int t = 0; t < CT; ++t)
                if (used(t)) {
                    Frag<NO> uf = ux.frag(t);
                    if (bad) put_aside(uf, t, from);
                    Frag<NO> f[HT];
#pragma unroll
                    for (int i = 0; i < HT; ++i) f[i] = pf[i][t];
                    mma_cols<NO>(ys, uf, f, All());
                }
            fetch_p(c + 1);
            if (bad) {
                from = column_least(from);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int f = __shfl(from, 4 * g + r);
#pragma unroll
                    for (int i = 0; i < HT; ++i)
                        if ((hf * HT + i) * 16 + col >= f) ys[i][r] = __builtin_nanf("");
                }
            }
            T* yb = row_of<T>(a.y, a.map, s, start, first + lo) + (int64_t)h * a.V + v0;
#pragma unroll
            for (int t = 0; t < HT; ++t)
                if (n == C || (hf * HT + t) * 16 + col < n) {
                    T* yp = yb + (int64_t)t * 16 * a.y.row + at_y;
                    const float o[4] = {ys[t][0], ys[t][1], ys[t][2], ys[t][3]};
                    if (a.wide_y) {
                        if (vy < a.V) store_f32<T, 4>(yp, o);
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (vy + r < a.V) yp[r] = (T)o[r];
                    }
                }
            if (Sh::stages == 1) {
                lds_barrier();  // chunk c has been read
                put(c + 1);
                fetch(c + 2);
            }
        }
        return;
    }

    __builtin_amdgcn_s_setprio(2);  // the helpers have time
    const int v = v0 + ct * 16 + col, k0 = hf * KH;
    const int64_t KV = (int64_t)a.K * a.V;
    const float* before = a.initial ? a.initial + ((int64_t)(a.segment ? unit : s) * a.HV + h) * KV : nullptr;
    const auto tile_at = [&](int i) { return i < HT ? (1 - hf) * HT + i : hf * HT + i - HT; };
    Frag<kParts> xf[HT][CT];
    const auto fetch_x = [&](int c) {
        const bf16* f = (const bf16*)(record(imin(c, chunks - 1)) + kScales * C * 4);
#pragma unroll
        for (int i = 0; i < HT; ++i)
#pragma unroll
            for (int t = 0; t < CT; ++t)
                prepared(xf[i][t], f, used(t) ? frag_index(C, hf * HT + i, t, false) : 0);
    };
    if (chunks > 0) fetch_x(0);
    float4_t S[KT];
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int k = k0 + t * 16 + 4 * g + r;
            if (a.through) S[t][r] = unity && k == (at.slice - slices) * Sh::slice + v && k < a.K ? 1.0f : 0.0f;
            else S[t][r] = before && k < a.K && v < a.V ? before[(int64_t)k * a.V + v] : 0.0f;
        }
    for (int c = 0; c < chunks; ++c) {
        lds_barrier();  // chunk c is there
        const float* scal = (const float*)stage(c);
        const Planes<NI> kp = planes(c, 0);
        const T* vl = (const T*)(planes(c, 1).p + NI * C * LD);
        // k S0 over this half's rows of S: first the other half's tokens, then its own.
        float4_t x[NT] = {};
#pragma unroll
        for (int t = 0; t < NK; ++t) {
            const Frag<kParts> sf = frag_of<kParts>(S[2 * t], S[2 * t + 1]);
#pragma unroll
            for (int q = 0; q < NO; ++q)
                *(bf16x8_t*)(sx + ((hf * NK + t) * NO + q) * 512 + l * 8) = sf.p[q];
            Frag<NI> f[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i) f[i] = kp.rows(tile_at(i) * 16, k0 + t * 32);
            mma_rows<kParts>(x, f, sf, All());
        }
#pragma unroll
        for (int i = 0; i < HT; ++i) *sum_at(xsum, tile_at(i)) = x[i];
        lds_barrier();
        float4_t e[HT];
#pragma unroll
        for (int i = 0; i < HT; ++i) {
            const int mt = hf * HT + i;
            const float4_t f = scales(scal, C, kReadK, mt), o = values4(vl, VL, mt * 16, ct * 16);
            rx.put(mt, o - f * (x[HT + i] + *sum_at(xsum, mt)));
            e[i] = float4_t{0, 0, 0, 0};
        }
        lds_barrier();
        // The corrections of this half's tokens.
#pragma unroll
        for (int t = 0; t < CT; ++t)
            if (used(t)) {
                const Frag<kParts> rf = rx.frag(t);
                Frag<kParts> f[HT];
#pragma unroll
                for (int i = 0; i < HT; ++i) f[i] = xf[i][t];
                mma_rows<kParts>(e, f, rf, All());
            }
        fetch_x(c + 1);
        float4_t u[HT];
        float bad = 0.0f;
#pragma unroll
        for (int i = 0; i < HT; ++i) {
            u[i] = e[i] * scales(scal, C, kBeta, hf * HT + i);
            bad = strange(bad, u[i]);
        }
        const bool again = __any(!(bad == 0.0f));
        if (l == 0) *odd(c, hf) = again;
        if (again) {
            // Again, without what is infinite or NaN: that reaches its own and later tokens.
            const bf16* x = (const bf16*)(record(c) + kScales * C * 4);
            int from = C;
#pragma unroll
            for (int i = 0; i < HT; ++i) e[i] = float4_t{0, 0, 0, 0};
#pragma unroll
            for (int t = 0; t < CT; ++t)
                if (used(t)) {
                    Frag<kParts> rf = rx.frag(t), f[HT];
                    put_aside(rf, t, from);
#pragma unroll
                    for (int i = 0; i < HT; ++i) prepared(f[i], x, frag_index(C, hf * HT + i, t, false));
                    mma_rows<kParts>(e, f, rf, All());
                }
            from = column_least(from);
#pragma unroll
            for (int i = 0; i < HT; ++i) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if ((hf * HT + i) * 16 + 4 * g + r >= from) e[i][r] = __builtin_nanf("");
                u[i] = e[i] * scales(scal, C, kBeta, hf * HT + i);
            }
        }
#pragma unroll
        for (int i = 0; i < HT; ++i) {
            const int mt = hf * HT + i;
            wx.put(mt, e[i] * scales(scal, C, kWrite, mt));
            ux.put(mt, u[i]);
        }
        lds_barrier();
        if (a.saved && !a.through) {
            float* keep = a.saved + ((int64_t)(slot0 + c) * a.HV + h) * kept_floats(a.V, KP, C);
            const int vt = v0 / 16 + ct;
            if (vt * 16 < a.V) {
#pragma unroll
                for (int t = 0; t < KT; ++t) *kept_at(keep, KP, C, vt, hf * KT + t) = S[t];
#pragma unroll
                for (int i = 0; i < HT; ++i) *kept_at(keep, KP, C, vt, KP / 16 + hf * HT + i) = e[i];
            }
        }
        const float total = scal[kDecay * C + C - 1];
#pragma unroll
        for (int t = 0; t < KT; ++t) S[t] *= total;
#pragma unroll
        for (int u = 0; u < CT; ++u) {
            const Frag<kParts> wf = wx.frag(u);
            Frag<NI> f[KT];
#pragma unroll
            for (int t = 0; t < KT; ++t) f[t] = kp.cols(u * 32, k0 + t * 16);
            mma_rows<kParts>(S, f, wf, All());
        }
        if (Sh::stages == 1) lds_barrier();
    }
    if (a.through) {
        const int columns = map_columns(a.V, KP, Sh::slice);
        float* out = a.maps + ((int64_t)unit * a.HV + h) * KP * columns + at.slice * Sh::slice + ct * 16 + col;
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) out[(int64_t)(k0 + t * 16 + 4 * g + r) * columns] = S[t][r];
    } else if (a.final && seg.hi == seg.len && v < a.V) {
        float* out = a.final + ((int64_t)s * a.HV + h) * KV;
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
hipError_t forward_at(const DeltaArgs& a, hipStream_t st) {
    using Sh = FwdShape<T, KP>;
    const auto kernel = !a.wide_qk  ? delta_forward<T, KP, false, false>
                        : a.wide_v ? delta_forward<T, KP, true, true>
                                   : delta_forward<T, KP, true, false>;
    const hipError_t e = ensure_dynamic_lds((const void*)kernel, Sh::lds);
    if (e != hipSuccess) return e;
    const int slices = (int)ceil_div(a.V, Sh::slice) + (a.through ? KP / Sh::slice : 0);
    const int64_t grid = head_slice_grid((int64_t)a.units * a.HV, slices);
    kernel<<<(unsigned)grid, Sh::threads, Sh::lds, st>>>(a);
    return hipGetLastError();
}

}  // namespace

template <typename T>
hipError_t launch_delta_forward(const DeltaArgs& a, int KP, hipStream_t st) {
    if (KP == 64) return forward_at<T, 64>(a, st);
    if (KP == 128) return forward_at<T, 128>(a, st);
    return forward_at<T, 256>(a, st);
}
template hipError_t launch_delta_forward<float>(const DeltaArgs&, int, hipStream_t);
template hipError_t launch_delta_forward<bf16>(const DeltaArgs&, int, hipStream_t);
template hipError_t launch_delta_forward<f16>(const DeltaArgs&, int, hipStream_t);

}  // namespace tg
