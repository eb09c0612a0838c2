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
//     dG[i] = sum_j T[i,j] b[j] - b[i] db[i] + e^G[i] (scale q[i].(w S0^T)[i] - k[i].(R S0^T)[i])
//     dG[C-1] += e^(G[C-1]) <dS, S0> + sum_j b[j] Z[j]
// and a token's decay logarithm gets the sum of dG from it to the chunk's end:
// the pairs of tokens on either side of it, nothing that cancels but T's own
// row and column sums.
#include "seq_delta.hpp"
#include "tg_internal.hpp"

namespace tg {
namespace {

template <typename T, int KP>
struct BackShape {
    static constexpr int NI = kIn<T>, C = delta_chunk(NI, KP), LD = KP + 16, WL = kMaxColumns * 16 + 16;
    static constexpr int prep = prep_bytes(C, 2 * kTrain);
    static constexpr int stage = prep + 2 * NI * C * LD * 2 + NI * C * WL * 2;
    static constexpr int stages = 2 * stage <= 160 * 1024 ? 2 : 1, lds = stages * stage;
    static_assert(lds <= 160 * 1024, "more LDS than a compute unit has");
};

// The states' gradients, from the last chunk to the first: 16 columns in a wave.
template <typename T, int KP>
__global__ __launch_bounds__((kMaxColumns + delta_loaders(KP)) * 64) void delta_backward(const DeltaArgs a) {
    using Sh = BackShape<T, KP>;
    constexpr int NI = Sh::NI, C = Sh::C, LD = Sh::LD, WL = Sh::WL, NT = C / 16, KT = KP / 16, NK = KP / 32;
    constexpr int kLoaders = delta_loaders(KP);
    extern __shared__ float4 lds[];
    const int waves = (int)(blockDim.x >> 6) - kLoaders, w = (threadIdx.x >> 6) - kLoaders;
    const int l = threadIdx.x & 63, g = l >> 4, col = l & 15;
    const HeadSlice at = head_slice((a.V + waves * 16 - 1) / (waves * 16));
    if (at.pair >= a.map.seqs * a.HV) return;
    const int s = at.pair / a.HV, h = at.pair % a.HV, hk = h / (a.HV / a.HK);
    const int start = a.map.start(s), len = a.map.end(s) - start, slot0 = a.map.slot0(s, C);
    const int chunks = (len + C - 1) / C, v0 = at.slice * waves * 16, v = v0 + w * 16 + col;
    // A stage: the prepared matrices, k, q, the slice of dy.
    const auto planes = [&](int c, int which) {
        bf16* k = (bf16*)((char*)lds + (c % Sh::stages) * Sh::stage + Sh::prep);
        return Planes<NI>{k + which * NI * C * LD, which < 2 ? LD : WL, which < 2 ? C * LD : C * WL};
    };

    if (w < 0) {
        ChunkLoad<T, KP, C, Sh::prep> load;
        const auto fetch = [&](int c) {
            load.fetch(a, a.dy, a.wide_dy, s, start, c * C, imin(C, len - c * C), hk, h, v0,
                       (int64_t)(slot0 + c) * a.HV + h);
        };
        if (chunks > 0) fetch(chunks - 1);
        for (int c = chunks - 1; c >= 0; --c) {
            if (Sh::stages == 1 && c < chunks - 1) __syncthreads();
            load.put(lds + (c % Sh::stages) * (Sh::stage / 16), planes(c, 0), planes(c, 1));
            load.v.put(threadIdx.x, planes(c, 2));
            if (c > 0) fetch(c - 1);
            __syncthreads();
        }
        if (Sh::stages == 1 && chunks > 0) __syncthreads();
        return;
    }

    const int64_t KV = (int64_t)a.K * a.V, held = ((int64_t)s * a.HV + h) * KV;
    float4_t S[KT];  // dS
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int k = t * 16 + 4 * g + r;
            S[t][r] = a.dfinal && k < a.K && v < a.V ? a.dfinal[held + (int64_t)k * a.V + v] : 0.0f;
        }
    for (int c = chunks - 1; c >= 0; --c) {
        __syncthreads();  // chunk c has been brought
        const int lo = c * C, n = imin(C, len - lo);
        const int64_t chunk = (int64_t)(slot0 + c) * a.HV + h;
        const float* scal = (const float*)(lds + (c % Sh::stages) * (Sh::stage / 16));
        const bf16* fx = (const bf16*)(scal + kScales * C);
        const bf16* fp = fx + frag_count(C) * 512 * kTrain;
        const Planes<NI> kp = planes(c, 0), qp = planes(c, 1), wp = planes(c, 2);

        float* keep = a.back + chunk * (KV + (int64_t)C * a.V);
        if (v < a.V)
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int k = t * 16 + 4 * g + r;
                    if (k < a.K) keep[(int64_t)k * a.V + v] = S[t][r];
                }
        Frag<kTrain> sf[NK];
#pragma unroll
        for (int t = 0; t < NK; ++t) sf[t] = frag_of<kTrain>(S[2 * t], S[2 * t + 1]);
        Frag<NI> wf[C / 32];
#pragma unroll
        for (int t = 0; t < C / 32; ++t) wf[t] = wp.cols(t * 32, w * 16);
        float4_t R[NT];
#pragma unroll
        for (int mt = 0; mt < NT; ++mt) {
            float4_t x = {0, 0, 0, 0};
#pragma unroll
            for (int t = 0; t < NK; ++t) mma<kTrain>(x, kp.rows(mt * 16, t * 32), sf[t]);
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] *= scal[kTailK * C + mt * 16 + 4 * g + r];
#pragma unroll
            for (int t = 0; t < C / 32; ++t)
                if (frag_used(C, mt, t, true))
                    mma<kTrain>(x, prepared<kTrain>(fp, frag_index(C, mt, t, true)), wf[t]);
#pragma unroll
            for (int r = 0; r < 4; ++r) R[mt][r] = x[r] * scal[kBeta * C + mt * 16 + 4 * g + r];
        }
        Frag<kTrain> bf[C / 32];
#pragma unroll
        for (int t = 0; t < C / 32; ++t) bf[t] = frag_of<kTrain>(R[2 * t], R[2 * t + 1]);
#pragma unroll
        for (int mt = 0; mt < NT; ++mt) {
            R[mt] = float4_t{0, 0, 0, 0};
#pragma unroll
            for (int t = 0; t < C / 32; ++t)
                if (frag_used(C, mt, t, true))
                    mma<kTrain>(R[mt], prepared<kTrain>(fx, frag_index(C, mt, t, true)), bf[t]);
            if (v < a.V)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = mt * 16 + 4 * g + r;
                    keep[KV + (int64_t)i * a.V + v] = R[mt][r];
                    if (i < n)
                        row_of<T>(a.dv, a.map, s, start, lo + i)[(int64_t)h * a.V + v] = (T)R[mt][r];
                }
        }
        Frag<kTrain> qw[C / 32], kr[C / 32];
#pragma unroll
        for (int t = 0; t < C / 32; ++t) {
            float x[8], y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int i = t * 32 + frag_at(g, j);
                float f = 0.0f;
#pragma unroll
                for (int q = NI - 1; q >= 0; --q) f += (float)wf[t].p[q][j];
                x[j] = f * scal[kReadQ * C + i];
                y[j] = -R[2 * t + (j >> 2)][j & 3] * scal[kReadK * C + i];
            }
            qw[t] = frag_of<kTrain>(x);
            kr[t] = frag_of<kTrain>(y);
        }
        const float total = scal[kDecay * C + C - 1];
#pragma unroll
        for (int t = 0; t < KT; ++t) {
#pragma unroll
            for (int r = 0; r < 4; ++r) S[t][r] *= total;
#pragma unroll
            for (int u = 0; u < C / 32; ++u) {
                mma<kTrain>(S[t], qp.cols(u * 32, t * 16), qw[u]);
                mma<kTrain>(S[t], kp.cols(u * 32, t * 16), kr[u]);
            }
        }
        if (Sh::stages == 1) __syncthreads();
    }
    if (a.dinitial && v < a.V)
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int k = t * 16 + 4 * g + r;
                if (k < a.K) a.dinitial[held + (int64_t)k * a.V + v] = S[t][r];
            }
}

// ---- the chunks' own gradients
//
// One workgroup for a chunk and key head; its value heads one after another, dq
// and dk added up in registers. Wave w has the 16 rows (tokens) of tile w % (C/16)
// and, of each KB columns of q and k, KW. V goes by in blocks of 32.
template <typename T, int KP>
struct GradShape {
    static constexpr int NI = kIn<T>, C = delta_chunk(NI, KP), LD = KP + 16, NT = C / 16;
    static constexpr int waves = KP == 256 ? 8 : 4;  // 256 registers for each, with all of dq and dk
    static constexpr int parts = waves / NT, KB = NI == 1 && KP == 128 ? 128 : 64, KW = KB / parts, NB = KP / KB;
    static constexpr int VB = 32, VL = VB + 8, ML = C + 16;
    static constexpr int wide = (NI + 2 * kTrain) * C * VL * 2 + 2 * kTrain * KB * VL * 2;  // a block of V
    static constexpr int square = 2 * NI * C * ML * 2;                                  // C x C
    static constexpr int scratch = wide > square ? wide : square;
    static constexpr int floats = 8 * C + NT * C + 2 * parts * C + 2 * waves * 16 + 16;
    static constexpr int lds = C * 8 + floats * 4 + 2 * NI * C * LD * 2 + scratch;
};

template <typename T, int KP>
__global__ __launch_bounds__(KP == 256 ? 512 : 256, 1) void delta_grads(const DeltaArgs a) {
    using Sh = GradShape<T, KP>;
    constexpr int kThreads = 64 * Sh::waves;
    constexpr int NI = Sh::NI, C = Sh::C, LD = Sh::LD, NT = Sh::NT, NB = Sh::NB, KB = Sh::KB;
    constexpr int KW = Sh::KW, WT = KW / 16, VB = Sh::VB, VL = Sh::VL, ML = Sh::ML;
    extern __shared__ float4 lds[];
    double* G = (double*)lds;
    float* gb = (float*)(G + C);     // b
    float* ge = gb + C;              // e^G
    float* gt = ge + C;              // e^(G[C-1] - G)
    float* gs = gt + C;              // the step sizes' slopes
    float* gd = gs + C;              // step sizes
    float* rk = gd + C;
    float* rq = rk + C;
    float* colsum = rq + C;          // [NT][C]: column sums of T by row tile
    float* dots = colsum + NT * C;   // [2][parts][C]: rows' sums by part: the S0 terms and T, Z
    float* inner = dots + 2 * Sh::parts * C;   // [2][waves][16]: dq.q and dk.k of a tile's rows
    float* red = inner + 2 * Sh::waves * 16;   // <dS, S0> by wave
    const Planes<NI> kp{(bf16*)((float*)(G + C) + Sh::floats), LD, C * LD};
    const Planes<NI> qp{kp.p + NI * C * LD, LD, C * LD};
    bf16* scratch = qp.p + NI * C * LD;
    const Planes<NI> wp{scratch, VL, C * VL};
    const Planes<kTrain> ep{wp.p + NI * C * VL, VL, C * VL}, rp{ep.p + kTrain * C * VL, VL, C * VL};
    const Planes<kTrain> sp{rp.p + kTrain * C * VL, VL, KB * VL}, dp{sp.p + kTrain * KB * VL, VL, KB * VL};
    const Planes<NI> bm{scratch, ML, C * ML}, mm{bm.p + NI * C * ML, ML, C * ML};
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
    stage<T, C, KP, kThreads>(kp, row_of<const T>(a.k, a.map, s, start, lo) + (int64_t)hk * a.K,
                              a.k.row, n, a.K, a.wide_qk);
    stage<T, C, KP, kThreads>(qp, row_of<const T>(a.q, a.map, s, start, lo) + (int64_t)hk * a.K,
                              a.q.row, n, a.K, a.wide_qk);

    float4_t dq[NB][WT] = {}, dk[NB][WT] = {};
    for (int h = hk * rep; h < (hk + 1) * rep; ++h) {
        const int64_t KV = (int64_t)a.K * a.V;
        const int64_t chunk = (int64_t)slot * a.HV + h, size = KV + (int64_t)C * a.V;
        const float *S0 = a.saved + chunk * size, *E = S0 + KV, *dS = a.back + chunk * size, *R = dS + KV;
        const T* dy = row_of<const T>(a.dy, a.map, s, start, lo) + (int64_t)h * a.V;
        __syncthreads();
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
                const float* sc = (const float*)(a.prep + chunk * prep_bytes(C, 2 * kTrain));
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
                __syncthreads();
                Tile<T, C, VB, kThreads> tw;
                Tile<float, C, VB, kThreads> te, tr;
                Tile<float, KB, VB, kThreads> ts, td;
                tw.fetch(tid, dy + vb, a.dy.row, n, a.V - vb, a.wide_dy);
                te.fetch(tid, E + vb, a.V, C, a.V - vb, a.wide_s);
                tr.fetch(tid, R + vb, a.V, C, a.V - vb, a.wide_s);
                ts.fetch(tid, S0 + (int64_t)kb * a.V + vb, a.V, a.K - kb, a.V - vb, a.wide_s);
                td.fetch(tid, dS + (int64_t)kb * a.V + vb, a.V, a.K - kb, a.V - vb, a.wide_s);
                tw.put(tid, wp);
                te.put(tid, ep);
                tr.put(tid, rp);
                ts.put(tid, sp);
                td.put(tid, dp);
#pragma unroll
                for (int i = 0; i < ts.COUNT; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        whole = __builtin_fmaf(ts.e[i].r[j], td.e[i].r[j], whole);
                __syncthreads();
                const Frag<NI> wf = wp.rows(row0, 0);
                const Frag<kTrain> rf = rp.rows(row0, 0), ef = ep.rows(row0, 0);
                if (nb == 0)
#pragma unroll
                    for (int jt = 0; jt < NT; ++jt)
                        if (jt <= tile) {
                            const Frag<kTrain> o = ep.rows(jt * 16, 0);
                            mma<kTrain>(F[jt], wf, o);
                            mma<kTrain>(H[jt], rf, o);
                        }
#pragma unroll
                for (int t = 0; t < WT; ++t) {
                    const Frag<kTrain> x = sp.rows(part * KW + t * 16, 0);
                    mma<kTrain>(qs[t], wf, x);
                    mma<kTrain>(rs[t], rf, x);
                    mma<kTrain>(es[t], ef, dp.rows(part * KW + t * 16, 0));
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
                    mma<kTrain>(kk[jt], kf, o);
                    mma<kTrain>(qk[jt], qf, o);
                }
        }
        __syncthreads();  // the last block of V has been read
        float rowt[4] = {};
#pragma unroll
        for (int jt = 0; jt < NT; ++jt) {
            const int j = jt * 16 + col;
            const float b = gb[j];
            float sum = 0.0f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = row0 + 4 * g + r;
                float f = 0.0f, m = 0.0f;
                if (j <= i) {
                    const float D = decay_between(G[i], G[j]) * rk[j];
                    f = F[jt][r] * D * a.scale * rq[i];
                    m = j < i ? -H[jt][r] * D * rk[i] : 0.0f;
                    const float t = f * qk[jt][r] + m * kk[jt][r];
                    sum += t;
                    rowt[r] = __builtin_fmaf(t, b, rowt[r]);
                }
                if (part == 0) {
                    bm.put(i, j, f * b);
                    mm.put(i, j, m * b);
                }
            }
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            if (part == 0 && g == 0) colsum[tile * C + j] = sum;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            // Row sums of T once, of the S0 terms by every part.
            const float u = row_sum16(dot0[r] + (part == 0 ? rowt[r] : 0.0f)), z = row_sum16(dotz[r]);
            if (col == 0) {
                dots[part * C + row0 + 4 * g + r] = u;
                dots[(Sh::parts + part) * C + row0 + 4 * g + r] = z;
            }
        }
        whole = wave_sum(whole);
        if (l == 0) red[w] = whole;
        __syncthreads();
        if (w == 0) {
            float db = 0.0f, dg = 0.0f, bz = 0.0f;
            if (l < C) {
                float u = 0.0f, z = 0.0f;
#pragma unroll
                for (int p = 0; p < Sh::parts; ++p)
                    u += dots[p * C + l], z += dots[(Sh::parts + p) * C + l];
                db = z;
#pragma unroll
                for (int t = 0; t < NT; ++t) db += colsum[t * C + l];
                dg = u - gb[l] * db;
                bz = gb[l] * z;
            }
            bz = wave_sum(bz);
            float both = 0.0f;
#pragma unroll
            for (int i = 0; i < Sh::waves; ++i) both += red[i];
            const float after = ge[C - 1] * both + bz;
            // From each token to the chunk's end: sums over the lanes above.
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const float o = __shfl_down(dg, d);
                if (l + d < 64) dg += o;
            }
            dg += after;
            float pa = 0.0f, pb = 0.0f;
            if (l < n) {
                const float dd = dg * a.A[h] * gs[l];
                const float b = gb[l];
                row_of<T>(a.ddt, a.map, s, start, lo + l)[h] = (T)dd;
                row_of<T>(a.dbeta, a.map, s, start, lo + l)[h] =
                    (T)(a.sigmoid ? db * b * (1.0f - b) : db);
                pa = dg * gd[l];
                pb = dd;
            }
            pa = wave_sum(pa);
            pb = wave_sum(pb);
            if (l == 0) sums[h] = pa, sums[a.HV + h] = pb;
        }
#pragma unroll 1
        for (int t = 0; t < C / 32; ++t) {
            const bool low = t * 32 <= row0 + 15, high = t * 32 + 31 >= row0;
            const Frag<NI> br = bm.rows(row0, t * 32), mr = mm.rows(row0, t * 32);
            const Frag<NI> bc = bm.cols(t * 32, row0), mc = mm.cols(t * 32, row0);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int u = 0; u < WT; ++u) {
                    const int k = nb * KB + part * KW + u * 16;
                    const Frag<NI> kc = kp.cols(t * 32, k);
                    if (low) {
                        mma<NI>(dq[nb][u], br, kc);
                        mma<NI>(dk[nb][u], mr, kc);
                    }
                    if (high) {
                        mma<NI>(dk[nb][u], bc, qp.cols(t * 32, k));
                        mma<NI>(dk[nb][u], mc, kc);
                    }
                }
        }
    }
    // These are rq dq and rk dk of the unit vectors: from them those of q and k.
    float iq[4] = {}, ik[4] = {};
    if (a.normalize) {
        __syncthreads();
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
        __syncthreads();
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
hipError_t backward_at(const DeltaArgs& a, int64_t slots, hipStream_t st) {
    const int waves = delta_waves(a.V);
    hipError_t e = launch_delta_prep<T, kTrain, true>(a, KP, slots, st);
    if (e != hipSuccess) return e;
    constexpr int lds = BackShape<T, KP>::lds;
    e = ensure_dynamic_lds((const void*)delta_backward<T, KP>, lds);
    if (e != hipSuccess) return e;
    const int64_t grid = head_slice_grid((int64_t)a.map.seqs * a.HV, (int)ceil_div(a.V, waves * 16));
    delta_backward<T, KP><<<(unsigned)grid, (waves + delta_loaders(KP)) * 64, lds, st>>>(a);
    e = hipGetLastError();
    if (e != hipSuccess || slots == 0) return e;
    constexpr int bytes = GradShape<T, KP>::lds;
    static_assert(bytes <= 160 * 1024, "more LDS than a compute unit has");
    e = ensure_dynamic_lds((const void*)delta_grads<T, KP>, bytes);
    if (e != hipSuccess) return e;
    delta_grads<T, KP><<<(unsigned)(slots * a.HK), 64 * GradShape<T, KP>::waves, bytes, st>>>(a);
    return hipGetLastError();
}
template <typename T>
hipError_t backward_typed(const DeltaArgs& a, int64_t slots, hipStream_t st) {
    switch (delta_padded(a.K)) {
        case 64: return backward_at<T, 64>(a, slots, st);
        case 128: return backward_at<T, 128>(a, slots, st);
        default: return backward_at<T, 256>(a, slots, st);
    }
}

}  // namespace

hipError_t launch_delta_backward(const tg_delta_args& a, const tg_delta_grads& gr,
                                 const void* saved, void* ws, hipStream_t st) {
    DeltaArgs b = delta_args(a);
    const int C = delta_chunk_of(a);
    const int64_t slots = delta_slots(a.seqs, C), chunks = slots * a.HV;
    const size_t states = (size_t)chunks * ((size_t)a.K * a.V + (size_t)C * a.V) * 4;
    b.saved = (float*)saved;
    b.prep = (char*)ws;
    b.back = (float*)(b.prep + up256((size_t)chunks * prep_bytes(C, 2 * kTrain)));
    b.part = (float*)((char*)b.back + up256(states));
    b.dy = rows_of<const void>(gr.dy);
    b.dq = rows_of<void>(gr.dq), b.dk = rows_of<void>(gr.dk), b.dv = rows_of<void>(gr.dv);
    b.ddt = rows_of<void>(gr.ddt), b.dbeta = rows_of<void>(gr.dbeta);
    b.dfinal = gr.dfinal, b.dinitial = gr.dinitial;
    const size_t e = elem_bytes(a.dtype);
    Widest dy, s;
    dy.len(a.V), dy.len(gr.dy.row_stride), dy.ptr(gr.dy.p, e);
    if (!a.seqs.offsets) dy.len(gr.dy.seq_stride);
    s.len(a.V), s.ptr(saved, 4), s.ptr(b.back, 4);
    b.wide_dy = dy.width(8) == 8, b.wide_s = s.width(8) == 8;
    hipError_t err = a.dtype == TG_F32   ? backward_typed<float>(b, slots, st)
                     : a.dtype == TG_BF16 ? backward_typed<bf16>(b, slots, st)
                                          : backward_typed<f16>(b, slots, st);
    if (err != hipSuccess) return err;
    return launch_column_sums(b.part, (int)slots, 2 * (int64_t)a.HV, gr.dA, a.HV, gr.ddt_bias, st);
}

}  // namespace tg
