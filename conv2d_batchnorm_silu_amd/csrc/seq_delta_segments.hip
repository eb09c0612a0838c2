// seq_delta_segments.hip -- the gated delta rule over few long sequences: the walk down
// a sequence's chunks, cut into segments.
//
// What a segment of tokens makes of a state S is M S + N, with M the K x K product of
// its tokens' maps. N is the state that it leaves behind from zero, and M's columns are
// what it makes of those of the identity with v = 0: K more columns for the same
// kernel. So all segments at once make their N and M; this file's kernel goes from one
// segment to the next, S = M S + N, and then all segments at once walk again, each from
// its state. That is two to three walks' work in place of one, on as many times more
// workgroups as there are segments: one fp32 sequence of 16384 tokens, 8 heads of
// 64 x 64, 1000 us whole, 134 + 35 + 75 in segments of 1024, in both cases after the
// chunks' matrices (38 us). The gradients of the states go the same way from the last
// segment to the first.
#include "seq_delta.hpp"
#include "tg_internal.hpp"

namespace tg {
namespace {

constexpr int kJoinColumns = 32;

struct JoinArgs {
    SeqMap map;
    int HV, K, V, segment, columns, reverse;
    const float *maps, *first;
    float* states;
};

// A workgroup for a head's 32 columns: S in LDS, M's rows by fp32 matrix instructions
// (each product once for each segment: nothing to gain from parts).
template <int KP>
__global__ __launch_bounds__(256) void delta_join(const JoinArgs a) {
    constexpr int RT = KP / 64, LD = kJoinColumns + 4;  // tiles of 16 rows of a wave
    __shared__ float S[KP * LD];
    const int w = threadIdx.x >> 6, l = threadIdx.x & 63, g = l >> 4, col = l & 15;
    const int slices = (a.V + kJoinColumns - 1) / kJoinColumns;
    const int pair = blockIdx.x / slices, v0 = (int)(blockIdx.x % slices) * kJoinColumns;
    const int s = pair / a.HV, h = pair % a.HV;
    const int len = a.map.end(s) - a.map.start(s), unit0 = a.map.slot0(s, a.segment);
    const int count = len > 0 ? (len + a.segment - 1) / a.segment : 1;
    const int64_t KV = (int64_t)a.K * a.V;
    for (int i = threadIdx.x; i < KP * kJoinColumns; i += 256) {
        const int k = i / kJoinColumns, v = v0 + i % kJoinColumns;
        S[k * LD + i % kJoinColumns] =
            a.first && k < a.K && v < a.V ? a.first[((int64_t)s * a.HV + h) * KV + (int64_t)k * a.V + v] : 0.0f;
    }
    for (int j = 0; j < count; ++j) {
        const int64_t unit = unit0 + (a.reverse ? count - 1 - j : j);
        __syncthreads();
        float* out = a.states + (unit * a.HV + h) * KV;
        for (int i = threadIdx.x; i < a.K * kJoinColumns; i += 256) {
            const int k = i / kJoinColumns, v = v0 + i % kJoinColumns;
            if (v < a.V) out[(int64_t)k * a.V + v] = S[k * LD + i % kJoinColumns];
        }
        if (j == count - 1) break;
        const float* N = a.maps + (unit * a.HV + h) * KP * a.columns + v0;
        const float* M = a.maps + (unit * a.HV + h) * KP * a.columns + a.columns - KP;
        float4_t c[RT][2];
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    c[t][b][r] = v0 + b * 16 + col < a.V
                                     ? N[(int64_t)((t * 4 + w) * 16 + 4 * g + r) * a.columns + b * 16 + col]
                                     : 0.0f;
#pragma unroll 4
        for (int q = 0; q < KP / 16; ++q) {
            float4_t m[RT];
            float x[2][4];
#pragma unroll
            for (int t = 0; t < RT; ++t)
                m[t] = *(const float4_t*)(M + (int64_t)((t * 4 + w) * 16 + col) * a.columns + q * 16 + 4 * g);
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[b][i] = S[(q * 16 + 4 * g + i) * LD + b * 16 + col];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        c[t][b] = __builtin_amdgcn_mfma_f32_16x16x4f32(m[t][i], x[b][i], c[t][b], 0, 0, 0);
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    S[((t * 4 + w) * 16 + 4 * g + r) * LD + b * 16 + col] = c[t][b][r];
    }
}

}  // namespace

hipError_t launch_delta_join(const DeltaArgs& a, const float* first, bool reverse, float* states, int KP,
                             int slice, hipStream_t st) {
    const JoinArgs j{a.map, a.HV, a.K, a.V, a.segment, map_columns(a.V, KP, slice), reverse,
                     a.maps, first, states};
    const unsigned grid = (unsigned)((int64_t)a.map.seqs * a.HV * ceil_div(a.V, kJoinColumns));
    if (KP == 64) delta_join<64><<<grid, 256, 0, st>>>(j);
    else if (KP == 128) delta_join<128><<<grid, 256, 0, st>>>(j);
    else delta_join<256><<<grid, 256, 0, st>>>(j);
    return hipGetLastError();
}

// Tokens of a segment, or 0: the time of the walks in chunks, a workgroup for a unit,
// head and slice on one of 256 compute units at a time. The two walks' steps cost as much
// as the one's; going from a segment to the next about as much as a step, and three launches
// more about three. The lengths of packed sequences are on the device: the longest is
// taken to be three times the mean.
int delta_segment(const tg_delta_args& a) {
    const int in = delta_in(a.dtype), KP = delta_padded(a.K), C = delta_chunk(in, KP);
    const int64_t slice = slice_of(in, KP), vs = ceil_div(a.V, slice), ks = KP / slice;
    const int64_t mean = a.seqs.rows / a.seqs.seqs;
    const int64_t longest = ceil_div(a.seqs.offsets ? (3 * mean < a.seqs.rows ? 3 * mean : a.seqs.rows) : mean, C);
    const int64_t all = ceil_div(a.seqs.rows, C) * a.HV, cus = 256;
    const int64_t whole = longest > ceil_div(all * vs, cus) ? longest : ceil_div(all * vs, cus);
    int64_t best = whole * 3 / 4, chosen = 0;
    for (int64_t sc = 4; sc * 2 <= longest; sc *= 2) {
        const int64_t units = (ceil_div(a.seqs.rows, C * sc)) * a.HV;
        const int64_t steps = ceil_div(units * (vs + ks), cus) * sc + ceil_div(units * vs, cus) * sc +
                              ceil_div(longest, sc) + 3;
        if (steps < best) best = steps, chosen = sc * C;
    }
    return (int)chosen;
}

}  // namespace tg
