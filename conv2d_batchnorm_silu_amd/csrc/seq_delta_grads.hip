// seq_delta_grads.hip -- the gradients of the gated delta rule that a chunk's own
// tokens make, from the states and their gradients on both sides of it
// (seq_delta_backward.hip has the formulas).
#include "seq_delta.hpp"
#include "tg_internal.hpp"

namespace tg {
namespace {

// ---- the chunks' own gradients
//
// 2 x 2048 tokens of 16 heads of 128 x 128, bf16: 147 us, a wave on each SIMD (120 KB of
// LDS), half of its time waiting. (137 before the pairs' factors took two parts and the
// decays' gradients each pair by itself; then the next block of V in registers while one is
// worked on took 133, but 34 for 22 on 64 columns, and eight waves 238, spilled.) For K of
// 129 to 256 all of dq and dk does not fit the registers: 80 to 250 are spilled.
//
// One workgroup for a chunk and key head; its value heads one after another, dq
// and dk added up in registers. Wave w has the 16 rows (tokens) of tile w % (C/16)
// and, of each KB columns of q and k, KW. V goes by in blocks of 32.
template <typename T, int KP>
struct GradShape {
    static constexpr int NI = kIn<T>, C = delta_chunk(NI, KP), LD = KP + 8, NT = C / 16;
    static constexpr int waves = KP == 256 ? 8 : 4;  // 256 registers for each, with all of dq and dk
    static constexpr int parts = waves / NT, KB = NI == 1 && KP == 128 ? 128 : 64, KW = KB / parts, NB = KP / KB;
    static constexpr int VB = 32, VL = VB + 8, ML = C + 8, CL = C + 8, KL = KB + 8;
    // A block of V: dy as rows of tokens; E, R, S0 and dS as rows of V.
    static constexpr int wide = NI * C * VL * 2 + 2 * kParts * VB * (CL + KL) * 2;
    static constexpr int NP = kOut<T>, square = 2 * NP * C * ML * 2;                    // C x C
    static constexpr int scratch = wide > square ? wide : square;
    static constexpr int floats = 8 * C + 2 * NT * C + 2 * parts * C + 2 * waves * 16 + 16;
    static constexpr int lds = C * 8 + floats * 4 + 2 * NI * C * LD * 2 + scratch;
};

template <typename T, int KP, bool WIDE>
__global__ __launch_bounds__(KP == 256 ? 512 : 256, 1) void delta_grads(const DeltaArgs a) {
    using Sh = GradShape<T, KP>;
    constexpr int kThreads = 64 * Sh::waves;
    constexpr int NI = Sh::NI, NP = Sh::NP, C = Sh::C, LD = Sh::LD, NT = Sh::NT, NB = Sh::NB, KB = Sh::KB;
    constexpr int KW = Sh::KW, WT = KW / 16, VB = Sh::VB, VL = Sh::VL, ML = Sh::ML, CL = Sh::CL, KL = Sh::KL;
    extern __shared__ float4 lds[];
    double* G = (double*)lds;
    float* gb = (float*)(G + C);     // b
    float* ge = gb + C;              // e^G
    float* gt = ge + C;              // e^(G[C-1] - G)
    float* gs = gt + C;              // the step sizes' slopes
    float* gd = gs + C;              // step sizes
    float* rk = gd + C;
    float* rq = rk + C;
    float* own = rq + C;             // T's diagonal
    float* colsum = own + C;         // [NT][C]: column sums of T by row tile
    float* across = colsum + NT * C;  // [NT][C]: by row tile, T b of the pairs on either side of a token
    float* dots = across + NT * C;    // [2][parts][C]: rows' sums by part: the S0 terms, Z
    float* inner = dots + 2 * Sh::parts * C;   // [2][waves][16]: dq.q and dk.k of a tile's rows
    float* red = inner + 2 * Sh::waves * 16;   // <dS, S0> by wave
    const Planes<NI> kp{(bf16*)((float*)(G + C) + Sh::floats), LD, C * LD};
    const Planes<NI> qp{kp.p + NI * C * LD, LD, C * LD};
    bf16* scratch = qp.p + NI * C * LD;
    const Planes<NI> wp{scratch, VL, C * VL};
    const Planes<kParts> ep{wp.p + NI * C * VL, CL, VB * CL}, rp{ep.p + kParts * VB * CL, CL, VB * CL};
    const Planes<kParts> sp{rp.p + kParts * VB * CL, KL, VB * KL}, dp{sp.p + kParts * VB * KL, KL, VB * KL};
    const Planes<NP> bm{scratch, ML, C * ML}, mm{bm.p + NP * C * ML, ML, C * ML};
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, g = l >> 4, col = l & 15;
    const int tile = w % NT, part = w / NT, row0 = tile * 16;
    const int slot = blockIdx.x / a.HK, hk = blockIdx.x % a.HK, rep = a.HV / a.HK;
    const int s = a.map.owner(slot, C), start = a.map.start(s);
    int lo = 0, hi = 0;
    const bool here = SeqMap::piece(slot, a.map.slot0(s, C), a.map.end(s) - start, C, lo, hi);
    const int n = here ? hi - lo : 0;
    float* sums = a.part + (int64_t)slot * 2 * a.HV;
    if (n <= 0) {
        for (int i = tid; i < rep; i += kThreads) sums[hk * rep + i] = sums[a.HV + hk * rep + i] = 0.0f;
        return;
    }
    {
        Tile<T, C, KP, kThreads, WIDE> kt, qt;
        kt.shape(a.k.row, a.K);
        qt.shape(a.q.row, a.K);
        kt.fetch(row_of<const T>(a.k, a.map, s, start, lo) + (int64_t)hk * a.K, n);
        qt.fetch(row_of<const T>(a.q, a.map, s, start, lo) + (int64_t)hk * a.K, n);
        kt.put(kp);
        qt.put(qp);
    }

    float4_t dq[NB][WT] = {}, dk[NB][WT] = {};
    for (int h = hk * rep; h < (hk + 1) * rep; ++h) {
        const int64_t chunk = (int64_t)slot * a.HV + h, size = kept_floats(a.V, KP, C);
        float *S0 = a.saved + chunk * size, *dS = a.back + chunk * size;
        T* dv = row_of<T>(a.dv, a.map, s, start, lo) + (int64_t)h * a.V;
        const T* dy = row_of<const T>(a.dy, a.map, s, start, lo) + (int64_t)h * a.V;
        lds_barrier();
        if (w == 0) {
            DeltaGate t = {0.0f, 0.0f, 0.0f, 0.0f};
            if (l < n)
                t = delta_gate(a, (float)row_of<const T>(a.dt, a.map, s, start, lo + l)[h],
                               (float)row_of<const T>(a.beta, a.map, s, start, lo + l)[h], h);
            const double p = wave_prefix((double)t.g2);
            const double last = __shfl(p, C - 1);
            if (l < C) {
                G[l] = p;
                gb[l] = t.b;
                gs[l] = t.slope;
                gd[l] = t.d;
                ge[l] = __builtin_amdgcn_exp2f((float)p);
                gt[l] = decay_between(last, p);
                const float* sc = (const float*)(a.prep + chunk * prep_bytes(C, 2 * kParts));
                rk[l] = sc[kUnitK * C + l];
                rq[l] = sc[kUnitQ * C + l];
            }
        }
        float4_t F[NT] = {}, H[NT] = {};
        float dot0[4] = {}, dotz[4] = {}, whole = 0.0f;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int kb = nb * KB, kw = kb + part * KW;
            float4_t qs[WT] = {}, rs[WT] = {}, es[WT] = {};
            for (int vb = 0; vb < a.V; vb += VB) {
                lds_barrier();
                Tile<T, C, VB, kThreads, WIDE> tw;
                tw.shape(a.dy.row, imin(VB, a.V - vb));
                tw.fetch(dy + vb, n);
                // Tiles of a wave's lanes: each lane four rows of one column of V.
                constexpr int EN = NT * 2 * 64 / kThreads, SN = KB / 16 * 2 * 64 / kThreads;
                constexpr int EC = EN ? EN : 1, SC = SN ? SN : 1;
                float4_t er[EC], rr[EC], sr[SC], dr[SC];
                const auto of = [&](float* kept, int i, int tiles, int first) {
                    const int q = (i * kThreads + tid) >> 6, vt = vb / 16 + q / tiles;
                    const float4_t* at =
                        kept_at(kept, KP, C, imin(vt, (a.V - 1) / 16), first + q % tiles);
                    return vt * 16 < a.V ? *at : float4_t{0, 0, 0, 0};
                };
                const auto there = [&](int i, int tiles) { return i * kThreads + tid < tiles * 128; };
#pragma unroll
                for (int i = 0; i < EC; ++i)
                    if (EN || there(i, NT)) {
                        er[i] = of(S0, i, NT, KP / 16);
                        rr[i] = of(dS, i, NT, KP / 16);
                    }
#pragma unroll
                for (int i = 0; i < SC; ++i)
                    if (SN || there(i, KB / 16)) {
                        sr[i] = of(S0, i, KB / 16, kb / 16);
                        dr[i] = of(dS, i, KB / 16, kb / 16);
                    }
                tw.put(wp);
                const auto give = [&](const Planes<kParts>& d, const float4_t& x, int i, int tiles) {
                    const int q = (i * kThreads + tid) >> 6;
                    bf16* at = d.p + (q / tiles * 16 + col) * d.ld + q % tiles * 16 + 4 * g;
                    bf16x4_t o[kParts];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        bf16 b[kParts];
                        split<kParts>(x[j], b);
#pragma unroll
                        for (int m = 0; m < kParts; ++m) o[m][j] = b[m];
                    }
#pragma unroll
                    for (int m = 0; m < kParts; ++m) *(bf16x4_t*)(at + m * d.plane) = o[m];
                };
#pragma unroll
                for (int i = 0; i < EC; ++i)
                    if (EN || there(i, NT)) {
                        give(ep, er[i], i, NT);
                        give(rp, rr[i], i, NT);
                        if (nb == 0) {  // R is the gradient of v
                            const int q = (i * kThreads + tid) >> 6, v = vb + q / NT * 16 + col;
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const int t = q % NT * 16 + 4 * g + r;
                                if (t < n && v < a.V) dv[t * a.dv.row + v] = (T)rr[i][r];
                            }
                        }
                    }
#pragma unroll
                for (int i = 0; i < SC; ++i)
                    if (SN || there(i, KB / 16)) {
                        give(sp, sr[i], i, KB / 16);
                        give(dp, dr[i], i, KB / 16);
#pragma unroll
                        for (int j = 0; j < 4; ++j) whole = __builtin_fmaf(sr[i][j], dr[i][j], whole);
                    }
                lds_barrier();
                const Frag<NI> wf = wp.rows(row0, 0);
                const Frag<kParts> rf = rp.cols(0, row0), ef = ep.cols(0, row0);
                if (nb == 0)
#pragma unroll
                    for (int jt = 0; jt < NT; ++jt)
                        if (jt <= tile) {
                            const Frag<kParts> o = ep.cols(0, jt * 16);
                            mma<kParts>(F[jt], wf, o);
                            mma<kParts>(H[jt], rf, o);
                        }
#pragma unroll
                for (int t = 0; t < WT; ++t) {
                    const Frag<kParts> x = sp.cols(0, part * KW + t * 16);
                    mma<kParts>(qs[t], wf, x);
                    mma<kParts>(rs[t], rf, x);
                    mma<kParts>(es[t], ef, dp.cols(0, part * KW + t * 16));
                }
            }
            // Rows' factors, and the rows' products with q and k.
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = row0 + 4 * g + r;
                const float fq = a.scale * ge[i] * rq[i], fr = -ge[i] * rk[i], fe = gt[i] * rk[i];
                const float b = gb[i];
#pragma unroll
                for (int t = 0; t < WT; ++t) {
                    const float q = qp.at(i, kw + t * 16 + col), k = kp.at(i, kw + t * 16 + col);
                    const float x = fq * qs[t][r], y = fr * rs[t][r], z = fe * es[t][r];
                    dot0[r] = __builtin_fmaf(x, q, __builtin_fmaf(y, k, dot0[r]));
                    dotz[r] = __builtin_fmaf(z, k, dotz[r]);
                    dq[nb][t][r] += x;
                    dk[nb][t][r] += __builtin_fmaf(z, b, y);
                }
            }
        }
        // The pairs of tokens: k k^T and q k^T again, T, and the matrices that
        // multiply q and k.
        float4_t kk[NT] = {}, qk[NT] = {};
#pragma unroll 2
        for (int k0 = 0; k0 < KP; k0 += 32) {
            const Frag<NI> kf = kp.rows(row0, k0), qf = qp.rows(row0, k0);
#pragma unroll
            for (int jt = 0; jt < NT; ++jt)
                if (jt <= tile) {
                    const Frag<NI> o = kp.rows(jt * 16, k0);
                    mma<kParts>(kk[jt], kf, o);
                    mma<kParts>(qk[jt], qf, o);
                }
        }
        lds_barrier();  // the last block of V has been read
        float before[4] = {};  // T b of each row, columns before the tile
#pragma unroll
        for (int jt = 0; jt < NT; ++jt) {
            const int j = jt * 16 + col;
            const float b = gb[j];
            float sum = 0.0f, over = 0.0f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = row0 + 4 * g + r;
                float f = 0.0f, m = 0.0f, pair = 0.0f;
                if (j <= i) {
                    const float D = decay_between(G[i], G[j]) * rk[j];
                    f = F[jt][r] * D * a.scale * rq[i];
                    m = j < i ? -H[jt][r] * D * rk[i] : 0.0f;
                    const float t = f * qk[jt][r] + m * kk[jt][r];
                    // A token's own term has no decay.
                    if (j < i) {
                        sum += t;
                        pair = t * b;
                    } else if (part == 0) {
                        own[i] = t;
                    }
                }
                // Row i's pairs with the tokens before j have j's decay if j <= i.
                if (jt <= tile) {
                    const float upto = row_prefix16(pair);
                    over += j <= i ? before[r] + row_shift16<1>(upto) : 0.0f;
                    before[r] += row_sum16(pair);
                }
                if (part == 0) {
                    bm.put(i, j, f * b);
                    mm.put(i, j, m * b);
                }
            }
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            over += __shfl_xor(over, 16);
            over += __shfl_xor(over, 32);
            if (part == 0 && g == 0) colsum[tile * C + j] = sum, across[tile * C + j] = over;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float u = row_sum16(dot0[r]), z = row_sum16(dotz[r]);
            if (col == 0) {
                dots[part * C + row0 + 4 * g + r] = u;
                dots[(Sh::parts + part) * C + row0 + 4 * g + r] = z;
            }
        }
        whole = wave_sum(whole);
        if (l == 0) red[w] = whole;
        lds_barrier();
        if (w == 0) {
            float db = 0.0f, dg = 0.0f, bz = 0.0f, pairs = 0.0f;
            if (l < C) {
                float z = 0.0f;
#pragma unroll
                for (int p = 0; p < Sh::parts; ++p)
                    dg += dots[p * C + l], z += dots[(Sh::parts + p) * C + l];
                db = z + own[l];
#pragma unroll
                for (int t = 0; t < NT; ++t) db += colsum[t * C + l], pairs += across[t * C + l];
                bz = gb[l] * z;
            }
            float both = 0.0f;
#pragma unroll
            for (int i = 0; i < Sh::waves; ++i) both += red[i];
            // The S0 terms from each token on, Z of the tokens before it.
            bz = __shfl_up(bz, 1);
            if (l == 0) bz = 0.0f;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const float o = __shfl_down(dg, d), z = __shfl_up(bz, d);
                if (l + d < 64) dg += o;
                if (l >= d) bz += z;
            }
            dg += pairs + bz + ge[C - 1] * both;
            float pa = 0.0f, pb = 0.0f;
            if (l < n) {
                // A decay that is taken as 0 has no gradient, whatever its rate and step; an
                // infinite rate has none beside its steps of zero either.
                const float A = a.A[h];
                const float dd = dg == 0.0f || __builtin_isinf(A) ? 0.0f : dg * A * gs[l];
                const float b = gb[l];
                row_of<T>(a.ddt, a.map, s, start, lo + l)[h] = (T)dd;
                row_of<T>(a.dbeta, a.map, s, start, lo + l)[h] =
                    (T)(a.sigmoid ? db * b * (1.0f - b) : db);
                pa = dg == 0.0f ? 0.0f : dg * gd[l];
                pb = dd;
            }
            pa = wave_sum(pa);
            pb = wave_sum(pb);
            if (l == 0) sums[h] = pa, sums[a.HV + h] = pb;
        }
#pragma unroll 1
        for (int t = 0; t < C / 32; ++t) {
            const bool low = t * 32 <= row0 + 15, high = t * 32 + 31 >= row0;
            const Frag<NP> br = bm.rows(row0, t * 32), mr = mm.rows(row0, t * 32);
            const Frag<NP> bc = bm.cols(t * 32, row0), mc = mm.cols(t * 32, row0);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int u = 0; u < WT; ++u) {
                    const int k = nb * KB + part * KW + u * 16;
                    const Frag<NI> kc = kp.cols(t * 32, k);
                    if (low) {
                        mma<NP>(dq[nb][u], br, kc);
                        mma<NP>(dk[nb][u], mr, kc);
                    }
                    if (high) {
                        mma<NP>(dk[nb][u], bc, qp.cols(t * 32, k));
                        mma<NP>(dk[nb][u], mc, kc);
                    }
                }
        }
    }
    // These are rq dq and rk dk of the unit vectors: from them those of q and k.
    float iq[4] = {}, ik[4] = {};
    if (a.normalize) {
        lds_barrier();
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = row0 + 4 * g + r;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int t = 0; t < WT; ++t) {
                    const int k = nb * KB + part * KW + t * 16 + col;
                    iq[r] = __builtin_fmaf(dq[nb][t][r], qp.at(i, k), iq[r]);
                    ik[r] = __builtin_fmaf(dk[nb][t][r], kp.at(i, k), ik[r]);
                }
            iq[r] = row_sum16(iq[r]);
            ik[r] = row_sum16(ik[r]);
            if (col == 0) inner[w * 16 + 4 * g + r] = iq[r], inner[(Sh::waves + w) * 16 + 4 * g + r] = ik[r];
        }
        lds_barrier();
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = row0 + 4 * g + r;
            float x = 0.0f, y = 0.0f;
#pragma unroll
            for (int p = 0; p < Sh::parts; ++p) {
                x += inner[(p * NT + tile) * 16 + 4 * g + r];
                y += inner[(Sh::waves + p * NT + tile) * 16 + 4 * g + r];
            }
            iq[r] = x * rq[i] * rq[i];
            ik[r] = y * rk[i] * rk[i];
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int i = row0 + 4 * g + r;
        if (i >= n) continue;
        T* oq = row_of<T>(a.dq, a.map, s, start, lo + i) + (int64_t)hk * a.K;
        T* ok = row_of<T>(a.dk, a.map, s, start, lo + i) + (int64_t)hk * a.K;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int t = 0; t < WT; ++t) {
                const int k = nb * KB + part * KW + t * 16 + col;
                if (k < a.K) {
                    oq[k] = (T)(dq[nb][t][r] - iq[r] * qp.at(i, k));
                    ok[k] = (T)(dk[nb][t][r] - ik[r] * kp.at(i, k));
                }
            }
    }
}

template <typename T, int KP>
hipError_t grads_at(const DeltaArgs& a, int64_t slots, hipStream_t st) {
    using Sh = GradShape<T, KP>;
    static_assert(Sh::lds <= 160 * 1024, "more LDS than a compute unit has");
    const auto kernel = a.wide_qk && a.wide_dy ? delta_grads<T, KP, true>
                                                           : delta_grads<T, KP, false>;
    const hipError_t e = ensure_dynamic_lds((const void*)kernel, Sh::lds);
    if (e != hipSuccess) return e;
    kernel<<<(unsigned)(slots * a.HK), 64 * Sh::waves, Sh::lds, st>>>(a);
    return hipGetLastError();
}

}  // namespace

template <typename T>
hipError_t launch_delta_grads(const DeltaArgs& a, int KP, int64_t slots, hipStream_t st) {
    if (slots == 0) return hipSuccess;
    if (KP == 64) return grads_at<T, 64>(a, slots, st);
    if (KP == 128) return grads_at<T, 128>(a, slots, st);
    return grads_at<T, 256>(a, slots, st);
}
template hipError_t launch_delta_grads<float>(const DeltaArgs&, int, int64_t, hipStream_t);
template hipError_t launch_delta_grads<bf16>(const DeltaArgs&, int, int64_t, hipStream_t);
template hipError_t launch_delta_grads<f16>(const DeltaArgs&, int, int64_t, hipStream_t);

}  // namespace tg
