// gmm_softmax.h - device helpers shared by the softmax-over-codes kernels:
// unaligned wide loads, bf16 conversion, online softmax statistics and sorted
// top-m lists.
#pragma once
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

namespace gmm {

constexpr int TOP_MAX = 16;  // GMM_TOP_MAX: alternatives kept per row
// exp(d) for d <= 0 on the hardware's base-2 exponential; results below 2^-126
// come out as 0, which no sum here can tell from themselves.
__device__ __forceinline__ float exp_neg(float d) {
    return __builtin_amdgcn_exp2f(d * 1.44269504088896341f);
}

// A logit l = scale x, rounded to fp32 on its own. Every use of it sees this number: a
// product fused into l - max would leave the maximum's own rounding in the difference,
// 2^-24 of a logit of any size (the contraction is off for that).
__device__ __forceinline__ float scaled(float x, float scale) {
#pragma clang fp contract(off)
    return x * scale;
}

// 16 bytes of a row at any element alignment (the hardware's global accesses
// need no alignment, so rows of any stride take the same path).
struct __attribute__((packed, aligned(2))) Raw16 {
    uint32_t w[4];
};

__device__ __forceinline__ float bf16_to_f32(uint32_t b) { return __uint_as_float(b << 16); }
// round to nearest even; NaN stays a quiet NaN
__device__ __forceinline__ uint32_t f32_to_bf16(float f) {
    const uint32_t u = __float_as_uint(f);
    if (f != f) return (u >> 16) | 0x40u;
    return (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
}

// T = float or uint16_t (bf16 bits): VE values per 16 bytes.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int VE = 4;
    static __device__ __forceinline__ float get(const Raw16& r, int k) {
        return __uint_as_float(r.w[k]);
    }
    static __device__ __forceinline__ float one(const float* p) { return *p; }
    static __device__ __forceinline__ void set(Raw16& r, int k, float v) {
        r.w[k] = __float_as_uint(v);
    }
    static __device__ __forceinline__ void put(Raw16& r, int k, float v) { set(r, k, v); }
    static __device__ __forceinline__ float store(float v) { return v; }
};
template <>
struct Vec<uint16_t> {
    static constexpr int VE = 8;
    static __device__ __forceinline__ float get(const Raw16& r, int k) {
        return __uint_as_float((k & 1) ? (r.w[k >> 1] & 0xffff0000u) : (r.w[k >> 1] << 16));
    }
    static __device__ __forceinline__ float one(const uint16_t* p) { return bf16_to_f32(*p); }
    static __device__ __forceinline__ void set(Raw16& r, int k, float v) {
        const uint32_t b = f32_to_bf16(v);
        r.w[k >> 1] = (k & 1) ? ((r.w[k >> 1] & 0xffffu) | (b << 16)) : b;
    }
    // replaces value k (set() takes the values in order)
    static __device__ __forceinline__ void put(Raw16& r, int k, float v) {
        const uint32_t b = f32_to_bf16(v);
        r.w[k >> 1] = (k & 1) ? ((r.w[k >> 1] & 0xffffu) | (b << 16)) : ((r.w[k >> 1] & 0xffff0000u) | b);
    }
    static __device__ __forceinline__ uint16_t store(float v) { return (uint16_t)f32_to_bf16(v); }
};

// The VE values of p[i .. i+VE), those at or past `end` as -inf.
template <typename T>
__device__ __forceinline__ Raw16 load_vec(const T* p, int64_t i, int64_t end) {
    constexpr int VE = Vec<T>::VE;
    if (i + VE <= end) return *reinterpret_cast<const Raw16*>(p + i);
    Raw16 r = {{0u, 0u, 0u, 0u}};
#pragma unroll
    for (int k = 0; k < VE; ++k)
        Vec<T>::set(r, k, i + k < end ? Vec<T>::one(p + i + k) : -INFINITY);
    return r;
}

// 16 bytes of a row, 0 at or past `end`.
template <typename T>
__device__ __forceinline__ Raw16 load_zero(const T* p, int64_t i, int64_t end) {
    constexpr int VE = Vec<T>::VE;
    if (i + VE <= end) return *reinterpret_cast<const Raw16*>(p + i);
    Raw16 r = {{0u, 0u, 0u, 0u}};
#pragma unroll
    for (int k = 0; k < VE; ++k)
        if (i + k < end) Vec<T>::set(r, k, Vec<T>::one(p + i + k));
    return r;
}

// ---- wave-wide reductions on the data-parallel lanes (no LDS)

// v of another lane: 0x120 + N rotates each group of 16 lanes by N, 0x140 and 0x141 mirror
// groups of 16 and of 8, 0xb1 and 0x4e swap neighbours and pairs within each four.
template <int CTRL>
__device__ __forceinline__ float lane_move(float v) {
    const int u = (int)__float_as_uint(v);
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(u, u, CTRL, 0xf, 0xf, false));
}
template <int CTRL>
__device__ __forceinline__ int lane_move(int v) {
    return __builtin_amdgcn_update_dpp(v, v, CTRL, 0xf, 0xf, false);
}
__device__ __forceinline__ float lane_get(float v, int lane) {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}
// over each group of 16 lanes
__device__ __forceinline__ float max16(float v) {
    v = fmaxf(v, lane_move<0x128>(v));
    v = fmaxf(v, lane_move<0x124>(v));
    v = fmaxf(v, lane_move<0x122>(v));
    return fmaxf(v, lane_move<0x121>(v));
}
__device__ __forceinline__ float sum16(float v) {
    v += lane_move<0x128>(v);
    v += lane_move<0x124>(v);
    v += lane_move<0x122>(v);
    return v + lane_move<0x121>(v);
}
// over the wave, the same in every lane
__device__ __forceinline__ float wave_max(float v) {
    v = max16(v);
    return fmaxf(fmaxf(lane_get(v, 0), lane_get(v, 16)), fmaxf(lane_get(v, 32), lane_get(v, 48)));
}
__device__ __forceinline__ float wave_sum(float v) {
    v = sum16(v);
    return (lane_get(v, 0) + lane_get(v, 16)) + (lane_get(v, 32) + lane_get(v, 48));
}
__device__ __forceinline__ int wave_min(int v) {
    v = min(v, lane_move<0x128>(v));
    v = min(v, lane_move<0x124>(v));
    v = min(v, lane_move<0x122>(v));
    v = min(v, lane_move<0x121>(v));
    return min(min(__builtin_amdgcn_readlane(v, 0), __builtin_amdgcn_readlane(v, 16)),
               min(__builtin_amdgcn_readlane(v, 32), __builtin_amdgcn_readlane(v, 48)));
}

// Online softmax statistics of a set of scaled logits l: m = max l (or
// -FLT_MAX where none is above it), s = sum exp(l - m), a = sum exp(l - m)
// (l - m). An empty set, or one of -inf only, has s = 0. A NaN or +inf leaves
// s = NaN. m starts at the lowest finite value instead of -inf so that l - m
// is never inf - inf for a masked l; differences are cut at -1000, where exp
// is 0 in fp32 already, so that 0 * (l - m) stays 0.
struct Stats {
    float m, s, a;
    __device__ __forceinline__ void clear() {
        m = -3.402823466e38f;
        s = 0.f;
        a = 0.f;
    }
    // restates s and a for the larger maximum mn
    __device__ __forceinline__ void raise(float mn) {
        const float d = fmaxf(m - mn, -1000.f);
        const float e = exp_neg(d);
        a = e * fmaf(s, d, a);
        s *= e;
        m = mn;
    }
    __device__ __forceinline__ void join(float m2, float s2, float a2) {
        const float mn = fmaxf(m, m2);
        Stats o{m2, s2, a2};
        raise(mn);
        o.raise(mn);
        s += o.s;
        a += o.a;
    }
    // over the wave's 64 lanes, in a fixed order, the same in every lane
    __device__ __forceinline__ void wave_join() {
        raise(wave_max(m));
        s = wave_sum(s);
        a = wave_sum(a);
    }
    __device__ __forceinline__ bool empty() const { return s == 0.f; }
};

// (v, i) before (v2, i2): larger value first, ties to the smaller index.
__device__ __forceinline__ bool top_before(float v, int i, float v2, int i2) {
    return v > v2 || (v == v2 && i < i2);
}

// A wave's sorted list of m (value, index) pairs: entry j in lane j, the empty entry
// is (-inf, INT_MAX).
struct TopList {
    float v;
    int i;
    __device__ __forceinline__ void clear() {
        v = -INFINITY;
        i = 0x7fffffff;
    }
};

// Whole number in the order of the float (NaN apart).
__device__ __forceinline__ uint32_t order_of(float v) {
    const uint32_t u = __float_as_uint(v + 0.f);  // -0 counts as 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// A bound that at least m of the wave's 64 values reach: the m-th largest, cut
// to its upper 20 bits, found bit by bit by counting.
__device__ __forceinline__ uint32_t order_bound(float v, int m) {
    const uint32_t key = order_of(v);
    uint32_t t = 0;
#pragma unroll
    for (int bit = 31; bit >= 12; --bit) {
        const uint32_t c = t | (1u << bit);
        if (__popcll(__builtin_amdgcn_ballot_w64(key >= c)) >= m) t = c;
    }
    return t;
}

// The m best of C * 64 candidates, C per lane, as a sorted list: m rounds of the
// best value and, among its equals, the smallest index. -inf is the empty entry.
template <int C>
__device__ __forceinline__ TopList top_pick(float* cv, int* ci, int m, int lane) {
    TopList out;
    out.clear();
    for (int j = 0; j < m; ++j) {
        float v = cv[0];
#pragma unroll
        for (int c = 1; c < C; ++c) v = fmaxf(v, cv[c]);
        const float best = wave_max(v);
        if (best == -INFINITY) break;
        int i = 0x7fffffff;
#pragma unroll
        for (int c = 0; c < C; ++c) i = cv[c] == best ? min(i, ci[c]) : i;
        const int at = wave_min(i);
        if (lane == j) {
            out.v = best;
            out.i = at;
        }
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (ci[c] == at) cv[c] = -INFINITY;
    }
    return out;
}

// cnt sorted-or-not candidates (cv, ci) in LDS; the thread holding candidate c
// writes it to rank's place in (ov, oi) when its rank is below m. Distinct
// candidates have distinct ranks (indices differ); places that no candidate
// takes must hold the empty entry before.
__device__ __forceinline__ void top_rank(const float* cv, const int* ci, int cnt, int m, float* ov,
                                         int* oi, int tid, int nt) {
    for (int c = tid; c < cnt; c += nt) {
        const float v = cv[c];
        const int i = ci[c];
        if (v == -INFINITY) continue;
        int rank = 0;
        for (int q = 0; q < cnt; ++q) rank += top_before(cv[q], ci[q], v, i);
        if (rank < m) {
            ov[rank] = v;
            oi[rank] = i;
        }
    }
}

}  // namespace gmm
