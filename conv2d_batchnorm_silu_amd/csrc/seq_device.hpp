// seq_device.hpp -- what the sequence operators' kernels share: element types,
// where the sequences of a batch lie, and wave reductions.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tg_device.hpp"
#include "tg_sequence.h"

namespace tg {

typedef __bf16 bf16;

template <typename T, int V>
struct VecOf {
    typedef T type __attribute__((ext_vector_type(V)));
};
template <typename T>
struct VecOf<T, 1> {
    typedef T type;
};

// V consecutive elements at p (aligned to V elements) as fp32, and back with
// one rounding to nearest even.
template <typename T, int V>
__device__ __forceinline__ void load_f32(const T* p, float (&v)[V]) {
    if constexpr (V == 1) {
        v[0] = (float)*p;
    } else {
        const typename VecOf<T, V>::type r = *(const typename VecOf<T, V>::type*)p;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = (float)r[i];
    }
}
// The same in two steps: the load, and the values once they are needed.
template <typename T, int V>
struct Vec {
    typename VecOf<T, V>::type r;
    __device__ __forceinline__ void load(const T* p) { r = *(const typename VecOf<T, V>::type*)p; }
    __device__ __forceinline__ void values(float (&v)[V]) const {
        if constexpr (V == 1) {
            v[0] = (float)r;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = (float)r[i];
        }
    }
};
template <typename T, int V>
__device__ __forceinline__ void store_f32(T* p, const float (&v)[V]) {
    if constexpr (V == 1) {
        *p = (T)v[0];
    } else {
        typename VecOf<T, V>::type r;
#pragma unroll
        for (int i = 0; i < V; ++i) r[i] = (T)v[i];
        *(typename VecOf<T, V>::type*)p = r;
    }
}

// Sum over the 64 lanes, in every lane, in a fixed order.
__device__ __forceinline__ float wave_sum(float v) {
    v = row_sum16(v);
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    return v;
}

// Where the sequences of a batch lie. L: rows of each sequence of a dense
// batch. The packed offsets are cut to 0 .. rows and to a non-negative
// length, so a wrong one cannot lead outside the tensors.
struct SeqMap {
    const int32_t* offsets;
    int seqs, rows, L;
    __host__ __device__ __forceinline__ int start(int s) const {
        if (!offsets) return s * L;
        const int v = offsets[s];
        return v < 0 ? 0 : (v > rows ? rows : v);
    }
    __host__ __device__ __forceinline__ int end(int s) const {
        if (!offsets) return (s + 1) * L;
        const int b = start(s), v = offsets[s + 1];
        return v < b ? b : (v > rows ? rows : v);
    }
    // Pieces of P rows, counted through the batch: sequence s owns the slots
    // from slot0(s) on, one for each P rows of it (the last may be short). In
    // a packed batch slot0 = floor(start/P) + s: floor(a/P) + floor(b/P) <=
    // floor((a+b)/P) keeps the sequences' slots apart, so rows/P + seqs slots
    // serve any lengths, which the host does not know.
    __host__ __device__ __forceinline__ int slot0(int s, int P) const {
        return offsets ? start(s) / P + s : s * ((L + P - 1) / P);
    }
    // The rows lo .. hi-1 of sequence s (len rows) in `slot`, its first slot
    // being first. False for a slot past the sequence's (or, with wrong offsets,
    // before them), which belongs to nobody. An empty sequence has one slot.
    static __host__ __device__ __forceinline__ bool piece(int slot, int first, int len, int P,
                                                          int& lo, int& hi) {
        const int64_t l = ((int64_t)slot - first) * P;
        if (l != 0 && (l < 0 || l >= len)) return false;
        lo = (int)l;
        hi = l + P < len ? (int)l + P : len;
        return true;
    }
    // The last sequence s with at(s) <= key (0 if there is none), by all 64
    // lanes of a wave: each round narrows the range 64 times with one load.
    template <typename At>
    __device__ __forceinline__ int last_at(int key, At at) const {
        const int lane = threadIdx.x & 63;
        int lo = 0, hi = seqs;
        while (hi - lo > 1) {
            const int step = (hi - lo + 63) >> 6, s = lo + lane * step;
            const int n = __popcll(__ballot(s < hi && at(s) <= key));
            if (n > 1) lo += (n - 1) * step;
            hi = imin(lo + step, hi);
        }
        return __builtin_amdgcn_readfirstlane(lo);
    }
    // The sequence that owns `slot`: the last one whose slot0 is not past it.
    // By whole waves, like holder().
    __device__ __forceinline__ int owner(int slot, int P) const {
        if (!offsets) return slot / ((L + P - 1) / P);
        return last_at(slot, [&](int s) { return slot0(s, P); });
    }
    // The sequence that holds row t < rows, past any empty ones: the last one that
    // starts at or before t. Rows that wrong offsets leave uncovered belong to a
    // sequence that ended before them.
    __device__ __forceinline__ int holder(int t) const {
        if (!offsets) return t / L;
        return last_at(t, [&](int s) { return start(s); });
    }
};

// Rows of a tensor in element strides; row l (packed: row start+l) of
// sequence s.
template <typename P>
struct Rows {
    P* p;
    int64_t seq, row;
};
template <typename T, typename P>
__device__ __forceinline__ T* row_of(const Rows<P>& r, const SeqMap& m, int s, int start, int l) {
    return (T*)r.p + (m.offsets ? ((int64_t)start + l) * r.row
                                : (int64_t)s * r.seq + (int64_t)l * r.row);
}

inline SeqMap map_of(const tg_seqs& s) {
    return {s.offsets, (int)s.seqs, (int)s.rows, (int)(s.rows / s.seqs)};
}
template <typename P>
Rows<P> rows_of(const tg_rows& r) {
    return {(P*)r.p, r.seq_stride, r.row_stride};
}

// log(1 + e^v) = max(v, 0) + log(1 + u), u = e^-|v|, to a few units in the last
// place at both ends: small step sizes come from far negative v, where 1 + u would
// drop u's bits. log(1 + u) = 2 atanh(s) with s = u / (2 + u) <= 1/3, and
// atanh(s) / s as a polynomial in s^2 <= 1/9 through the function's values at the
// five Chebyshev points there (off by at most 2^-27).
__device__ __forceinline__ float softplus_from(float v, float u) {
    const float s = u * __builtin_amdgcn_rcpf(2.0f + u), q = s * s;
    float r = __builtin_fmaf(0.14078889f, q, 0.13982579f);
    r = __builtin_fmaf(r, q, 0.20012298f);
    r = __builtin_fmaf(r, q, 0.33333161f);
    r = __builtin_fmaf(r, q, 1.0f);
    return __builtin_fmaf(s + s, r, fmaxf(v, 0.0f));
}
__device__ __forceinline__ float softplus_f32(float v) {
    return softplus_from(v, __builtin_amdgcn_exp2f(-fabsf(v) * kLog2e));
}
// And its slope, the logistic function.
__device__ __forceinline__ void softplus_grad_f32(float v, float& d, float& slope) {
    const float u = __builtin_amdgcn_exp2f(-fabsf(v) * kLog2e);
    d = softplus_from(v, u);
    slope = (v < 0.0f ? u : 1.0f) * __builtin_amdgcn_rcpf(1.0f + u);
}
__device__ __forceinline__ float sigmoid_f32(float v) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-v * kLog2e));
}

}  // namespace tg
