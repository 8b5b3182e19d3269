// gmm_score.hip - scores of given codes under a softmax over v codes, from its
// logits, and their gradient (gmm_logits_score, gmm_logits_score_backward,
// declared in include/gmm_em.h).
//
// Scores: with l = scale * x (rounded once, see scaled()), one pass over a row keeps, per thread, the maximum m,
// s = sum exp(l - m) and a = sum exp(l - m)(l - m) (restated when m rises), so that
//   log p_t = (l_t - m) - log s      entropy = log s - a / s
// with nothing of the row stored; the threads' sums are joined over the lanes and
// the waves in a fixed order.
// Alternatives: the threads form 64 groups; the m-th largest of the groups' maxima is a
// bound that m values of the row reach and hardly more than m do (about
// 64 ln(64 / (64 - m))). The values of the few threads whose maximum reaches it are
// read again by all threads (they are in the caches), those at the bound are gathered
// in LDS, and one wave picks the m best. Where ties or a mask put more values at the bound than LDS holds, the m
// best are found one by one over the whole row.
// Gradient: dx = scale (g_lp ([v = t] - p) - g_H p (log p + H)) with p from the
// stored m and log s: each logit is read once and its gradient written once.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "gmm_em.h"
#include "gmm_nn.h"
#include "gmm_softmax.h"

namespace gmm {

constexpr int SC_U = 4;       // vectors of 16 bytes in flight per thread
constexpr int SC_CAND = 256;  // gathered values

// The logit of the row's target (thread 0; where there is none, unused).
template <typename T>
__device__ __forceinline__ float target_logit(const ScoreArgs& p, int64_t row, int tid) {
    if (tid != 0 || !p.targets) return 0.f;
    const int t = p.targets[row];
    return t >= 0 && t < p.v ? Vec<T>::one((const T*)p.x + row * p.ldl + t) : 0.f;
}

// The largest value of each group of G = NT / 64 neighbouring lanes.
template <int G>
__device__ __forceinline__ float group_max(float v) {
    if (G > 1) v = fmaxf(v, lane_move<0xb1>(v));   // the lane next to it
    if (G > 2) v = fmaxf(v, lane_move<0x4e>(v));   // the other two of four
    if (G > 4) v = fmaxf(v, lane_move<0x141>(v));  // the other four of eight
    if (G > 8) v = fmaxf(v, lane_move<0x140>(v));  // the other eight of sixteen
    return v;
}

// A part of a row, read in vectors: vector j of NT * SC_U threads' worth starts at value
// j VE; one that would pass the end is the last whole one instead, and the
// values that belong to others are -inf in it.
template <typename T>
struct RowPart {
    static constexpr int VE = Vec<T>::VE;
    const T* x;
    int len;
    __device__ __forceinline__ int first(int at) const { return len < VE ? 0 : min(at, len - VE); }
    __device__ __forceinline__ Raw16 get(int at) const {
        if (len < VE) return load_vec(x, (int64_t)at, (int64_t)len);
        return *reinterpret_cast<const Raw16*>((const char*)x + (uint32_t)first(at) * sizeof(T));
    }
    __device__ __forceinline__ void mask(Raw16& r, int at) const {
        if (at + VE > len && len >= VE) {
#pragma unroll
            for (int k = 0; k < VE; ++k)
                if (k < at - first(at)) Vec<T>::put(r, k, -INFINITY);
        }
    }
};

// NT threads per (row, part). parts == 1: writes the results; else the part's
// statistics and list go to the workspace for k_score_join.
// Bound by its reads: 4096 rows of 32768 bf16 values in 51 us without alternatives
// (5.3 TB/s), 58 us with 4; the insertion of every value above a wave's own m-th best
// into its sorted list took 73.
template <typename T, int NT, bool TOP>
__global__ __launch_bounds__(NT) void k_score(ScoreArgs p) {
    constexpr int VE = Vec<T>::VE, NW = NT / 64, G = NT / 64, CHUNK = NT * VE * SC_U;
    __shared__ float sst[NW][3], gmax[64], cv[SC_CAND], best_v;
    __shared__ int ci[SC_CAND], hot[NT], hots, count, best_i;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int64_t item = blockIdx.x; item < p.n * p.parts; item += gridDim.x) {
        const int64_t row = item / p.parts;
        const int part = (int)(item - row * p.parts);
        const int64_t i0 = (int64_t)part * p.part_len;
        const RowPart<T> x{(const T*)p.x + row * p.ldl + i0,
                           (int)(p.v - i0 < p.part_len ? p.v - i0 : p.part_len)};
        Stats st;
        st.clear();
        float cm = -INFINITY;  // largest l of this thread
        for (int b = 0; b < x.len; b += CHUNK) {
            Raw16 raw[SC_U];
#pragma unroll
            for (int u = 0; u < SC_U; ++u) raw[u] = x.get(b + (u * NT + tid) * VE);
            if (b + CHUNK > x.len) {
#pragma unroll
                for (int u = 0; u < SC_U; ++u) x.mask(raw[u], b + (u * NT + tid) * VE);
            }
            float xm = -INFINITY;
#pragma unroll
            for (int u = 0; u < SC_U; ++u)
#pragma unroll
                for (int k = 0; k < VE; ++k) xm = fmaxf(xm, Vec<T>::get(raw[u], k));
            const float lm = scaled(xm, p.scale);
            cm = fmaxf(cm, lm);
            st.raise(fmaxf(st.m, lm));
            // l - m before the exponential's factor log2 e: the rounding of m log2 e would
            // stay in every term
            float s = 0.f, a = 0.f;
#pragma unroll
            for (int u = 0; u < SC_U; ++u)
#pragma unroll
                for (int k = 0; k < VE; ++k) {
                    const float d = scaled(Vec<T>::get(raw[u], k), p.scale) - st.m;
                    const float e = exp_neg(d);
                    s += e;
                    a = fmaf(e, fmaxf(d, -1000.f), a);
                }
            st.s += s;
            st.a += a;
        }
        st.wave_join();
        float gm = TOP ? group_max<G>(cm) : 0.f;
        if constexpr (NW > 1) {
            if (lane == 0) {
                sst[wave][0] = st.m;
                sst[wave][1] = st.s;
                sst[wave][2] = st.a;
            }
            if (TOP && lane % G == 0) gmax[tid / G] = gm;
        }
        if (TOP && tid == 0) hots = count = 0;
        __syncthreads();
        if constexpr (NW > 1) {
            if (wave == 0) {
                st.clear();
                if (lane < NW) st = Stats{sst[lane][0], sst[lane][1], sst[lane][2]};
                st.wave_join();
            }
            if (TOP) gm = gmax[lane];
        }
        TopList top;
        top.clear();
        if constexpr (TOP) {
            const uint32_t bound = order_bound(gm, p.m);
            auto in = [&](float l) { return l > -INFINITY && order_of(l) >= bound; };
            if (in(cm)) hot[atomicAdd(&hots, 1)] = tid;
            __syncthreads();
            // the hot threads' values, a value per thread at a time
            const uint32_t mine = (x.len + CHUNK - 1) / CHUNK * SC_U * VE;  // values of a thread
            const uint32_t total = (uint32_t)hots * mine;  // at most the row, rounded up
            for (uint32_t e = tid; e < total; e += NT) {
                const int h = (int)(e / mine), j = (int)(e - h * mine);
                const int u = j / VE, k = j % VE;
                const int at = u / SC_U * CHUNK + (u % SC_U * NT + hot[h]) * VE + k;
                if (at < x.len) {
                    const float l = scaled(Vec<T>::one(x.x + at), p.scale);
                    if (in(l)) {
                        const int to = atomicAdd(&count, 1);
                        if (to < SC_CAND) {
                            cv[to] = l;
                            ci[to] = (int)i0 + at;
                        }
                    }
                }
            }
            __syncthreads();
            int cnt = count;
            if (cnt > SC_CAND) {
                // one by one: the best that comes after the one before
                float lv = INFINITY;
                int li = -1;
                for (int j = 0; j < p.m; ++j) {
                    float bv = -INFINITY;
                    int bi = 0x7fffffff;
                    for (int at = tid * VE; at < x.len; at += NT * VE) {
                        const Raw16 r = load_vec(x.x, (int64_t)at, (int64_t)x.len);
#pragma unroll
                        for (int k = 0; k < VE; ++k) {
                            const float l = scaled(Vec<T>::get(r, k), p.scale);
                            const int i = (int)i0 + at + k;
                            if (top_before(lv, li, l, i) && top_before(l, i, bv, bi)) {
                                bv = l;
                                bi = i;
                            }
                        }
                    }
                    float* rv = cv + TOP_MAX;  // the waves' best, after the results
                    int* ri = ci + TOP_MAX;
                    const float wv = wave_max(bv);
                    const int wi = wave_min(bv == wv ? bi : 0x7fffffff);
                    if (lane == 0) {
                        rv[wave] = wv;
                        ri[wave] = wi;
                    }
                    __syncthreads();
                    if (wave == 0) {
                        const float v = lane < NW ? rv[lane] : -INFINITY;
                        const float mv = wave_max(v);
                        const int mi = wave_min(lane < NW && v == mv ? ri[lane] : 0x7fffffff);
                        if (lane == 0) {
                            best_v = cv[j] = mv;
                            best_i = ci[j] = mi;
                        }
                    }
                    __syncthreads();
                    lv = best_v;
                    li = lv > -INFINITY ? best_i : 0x7fffffff;  // nothing comes after the last
                }
                cnt = p.m;
            }
            if (wave == 0) {
                auto pick = [&](auto per) {
                    constexpr int C = decltype(per)::value;
                    float v[C];
                    int i[C];
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        const int e = c * 64 + lane;
                        v[c] = e < cnt ? cv[e] : -INFINITY;
                        i[c] = e < cnt ? ci[e] : 0x7fffffff;
                    }
                    return top_pick<C>(v, i, p.m, lane);
                };
                top = cnt <= 64 ? pick(std::integral_constant<int, 1>())
                                : pick(std::integral_constant<int, SC_CAND / 64>());
            }
        }
        if (wave == 0) {
            if (p.parts == 1) {
                score_out(p, row, st, target_logit<T>(p, row, lane), top.v, top.i, lane);
            } else {
                if (lane == 0) p.part[item] = ScorePart{st.m, st.s, st.a};
                if (TOP && lane < p.m) {
                    p.part_v[item * p.m + lane] = top.v;
                    p.part_i[item * p.m + lane] = top.i;
                }
            }
        }
        __syncthreads();  // LDS is free for the next item
    }
}

// One wave per row joins its parts' statistics and lists.
template <typename T>
__global__ __launch_bounds__(64) void k_score_join(ScoreArgs p) {
    constexpr int C = SC_MAX_PARTS * TOP_MAX / 64;
    const int lane = threadIdx.x;
    for (int64_t row = blockIdx.x; row < p.n; row += gridDim.x) {
        Stats st;
        st.clear();
        if (lane < p.parts) {
            const ScorePart q = p.part[row * p.parts + lane];
            st = Stats{q.m, q.s, q.a};
        }
        st.wave_join();
        const int cnt = p.parts * p.m;
        float cv[C];
        int ci[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int at = c * 64 + lane;
            cv[c] = at < cnt ? p.part_v[row * cnt + at] : -INFINITY;
            ci[c] = at < cnt ? p.part_i[row * cnt + at] : 0x7fffffff;
        }
        const TopList top = top_pick<C>(cv, ci, p.m, lane);
        score_out(p, row, st, target_logit<T>(p, row, lane), top.v, top.i, lane);
    }
}

// One block per (row, segment). Bound by its traffic: 4096 x 32768 bf16 (537 MB) in
// 101 us, 5.3 TB/s.
constexpr int SG_NT = 256, SG_U = 4;
template <typename T>
__global__ __launch_bounds__(SG_NT) void k_score_grad(ScoreGradArgs p) {
    constexpr int VE = Vec<T>::VE;
    constexpr int SEG = SG_NT * SG_U * VE;
    const int segs = (p.v + SEG - 1) / SEG;
    for (int64_t item = blockIdx.x; item < p.n * segs; item += gridDim.x) {
        const int64_t row = item / segs;
        const int64_t b = (item - row * segs) * SEG;
        const T* x = (const T*)p.x + row * p.ldl;
        T* dx = (T*)p.dx + row * p.lddl;
        const GradRow g = grad_row(p, row);
#pragma unroll
        for (int u = 0; u < SG_U; ++u) {
            const int64_t i = b + ((int64_t)u * SG_NT + threadIdx.x) * VE;
            if (i >= p.v) continue;
            const Raw16 raw = load_vec(x, i, (int64_t)p.v);
            Raw16 out = {{0u, 0u, 0u, 0u}};
#pragma unroll
            for (int k = 0; k < VE; ++k)
                Vec<T>::set(out, k, g.at(Vec<T>::get(raw, k), (int)(i + k)));
            if (i + VE <= p.v) {
                *reinterpret_cast<Raw16*>(dx + i) = out;
            } else {
#pragma unroll
                for (int k = 0; k < VE; ++k)
                    if (i + k < p.v) dx[i + k] = Vec<T>::store(Vec<T>::get(out, k));
            }
        }
    }
}

// Parts per row and threads per (row, part).
ScorePlan score_plan(int64_t n, int32_t v, int32_t m) {
    ScorePlan q;
    q.parts = 1;
    // few long rows: parts of at least 32768 values until 256 workgroups run, where that makes
    // three or more. fp32, m = 4, cut against whole rows: 1 x 131072 12.1 us (14.7), 1 x 524288
    // 12.3 (43.3), 64 x 262144 20.7 (26.5), 80 x 180000 18.7 (20.8); two parts lose to the join's
    // launch: 1 x 80000 13.4 us (11.0), 100 x 131072 18.0 (16.2), 127 x 262144 29.9 (27.6).
    int64_t want = n > 0 ? 256 / n : 1;
    const int64_t most = v / 32768;
    if (want > most) want = most;
    if (want > SC_MAX_PARTS) want = SC_MAX_PARTS;
    if (want > 2) q.parts = (int)want;
    q.part_len = ((v + q.parts - 1) / q.parts + 7) / 8 * 8;
    q.parts = (v + q.part_len - 1) / q.part_len;
    if (q.parts < 1) q.parts = 1;
    auto align = [](size_t b) { return (b + 255) & ~(size_t)255; };
    const size_t items = q.parts > 1 ? (size_t)n * q.parts : 0;
    q.o_v = align(items * sizeof(ScorePart));
    q.o_i = q.o_v + align(items * m * sizeof(float));
    q.bytes = q.o_i + align(items * m * sizeof(int32_t));
    if (q.bytes < 256) q.bytes = 256;
    return q;
}

template <typename T, int NT>
static void launch_score_nt(const ScoreArgs& a, hipStream_t st) {
    const int64_t items = a.n * a.parts;
    const int64_t most = (int64_t)1 << 20;  // grid threads stay below 2^32
    const dim3 grid((unsigned)(items < most ? items : most));
    if (a.m > 0)
        hipLaunchKernelGGL((k_score<T, NT, true>), grid, dim3(NT), 0, st, a);
    else
        hipLaunchKernelGGL((k_score<T, NT, false>), grid, dim3(NT), 0, st, a);
}

// Threads per (row, part): one wave where it has at most 8 chunks to go through (8192
// rows of 5000 bf16 values, m = 8: 37 us, with 256 threads 47), else 256; 1024 while every
// workgroup has a CU of its own (fp32, m = 4: 256 rows of 40000 11.7 us, with 256 threads 13.8;
// 257 rows 18.5 against 14.1).
template <typename T>
static void launch_score_t(const ScoreArgs& a, hipStream_t st) {
    constexpr int64_t PER = SC_U * Vec<T>::VE;
    const bool few = a.n * a.parts <= 256;
    if (a.part_len <= 64 * PER || (!few && a.part_len <= 8 * 64 * PER))
        launch_score_nt<T, 64>(a, st);
    else if (!few)
        launch_score_nt<T, 256>(a, st);
    else
        launch_score_nt<T, 1024>(a, st);
    if (a.parts > 1) {
        const int64_t most = (int64_t)1 << 20;
        hipLaunchKernelGGL((k_score_join<T>), dim3((unsigned)(a.n < most ? a.n : most)), dim3(64), 0,
                           st, a);
    }
}

hipError_t launch_score(ScoreArgs a, int dtype, void* ws, hipStream_t st) {
    const ScorePlan q = score_plan(a.n, a.v, a.m);
    a.parts = q.parts;
    a.part_len = q.part_len;
    a.part = (ScorePart*)ws;
    a.part_v = (float*)((char*)ws + q.o_v);
    a.part_i = (int32_t*)((char*)ws + q.o_i);
    if (dtype == GMM_F32)
        launch_score_t<float>(a, st);
    else
        launch_score_t<uint16_t>(a, st);
    return hipGetLastError();
}

template <typename T>
static void launch_grad_t(const ScoreGradArgs& a, hipStream_t st) {
    const int64_t seg = (int64_t)SG_NT * SG_U * Vec<T>::VE;
    const int64_t items = a.n * ((a.v + seg - 1) / seg);
    const int64_t most = (int64_t)1 << 22;
    hipLaunchKernelGGL((k_score_grad<T>), dim3((unsigned)(items < most ? items : most)), dim3(SG_NT),
                       0, st, a);
}

}  // namespace gmm

using namespace gmm;

extern "C" {

size_t gmm_logits_score_workspace_bytes(int64_t n, int32_t v, int32_t m) {
    if (!score_shape_ok(n, v) || m < 0 || m > TOP_MAX || m > v) return 0;
    return score_plan(n, v, m).bytes;
}

int gmm_logits_score(const void* logits, int64_t n, int32_t v, int64_t ldl, int32_t dtype,
                     const int32_t* targets, int32_t m, float scale, float* logprob,
                     float* entropy, float* norm, int32_t* top_idx, float* top_logprob,
                     void* workspace, size_t workspace_bytes, void* stream) {
    if (dtype != GMM_F32 && dtype != GMM_BF16) return GMM_E_DTYPE;
    const size_t need = gmm_logits_score_workspace_bytes(n, v, m);
    if (need == 0 || ldl < v || !scale_ok(scale)) return GMM_E_INVALID;
    if (n > 0 && (!logits || (targets && !logprob) || (m > 0 && (!top_idx || !top_logprob))))
        return GMM_E_INVALID;
    if (!workspace || workspace_bytes < need || (uintptr_t)workspace % 256 != 0)
        return GMM_E_WORKSPACE;
    if (n == 0) return GMM_OK;
    ScoreArgs a{};
    a.x = logits;
    a.n = n;
    a.ldl = ldl;
    a.v = v;
    a.m = m;
    a.scale = scale;
    a.targets = targets;
    a.logprob = logprob;
    a.entropy = entropy;
    a.norm = norm;
    a.top_idx = top_idx;
    a.top_logprob = top_logprob;
    return launch_score(a, dtype, workspace, (hipStream_t)stream) == hipSuccess ? GMM_OK : GMM_E_HIP;
}

int gmm_logits_score_backward(const void* logits, int64_t n, int32_t v, int64_t ldl, int32_t dtype,
                              const int32_t* targets, const float* norm, const float* entropy,
                              const float* g_logprob, const float* g_entropy, float scale,
                              void* dlogits, int64_t lddl, void* stream) {
    if (dtype != GMM_F32 && dtype != GMM_BF16) return GMM_E_DTYPE;
    if (!score_shape_ok(n, v) || ldl < v || lddl < v || !scale_ok(scale)) return GMM_E_INVALID;
    if (n > 0 && (!logits || !dlogits || !norm)) return GMM_E_INVALID;
    if (n > 0 && ((g_logprob && !targets) || (g_entropy && !entropy))) return GMM_E_INVALID;
    if (n == 0) return GMM_OK;
    ScoreGradArgs a{};
    a.x = logits;
    a.dx = dlogits;
    a.n = n;
    a.ldl = ldl;
    a.lddl = lddl;
    a.v = v;
    a.scale = scale;
    a.targets = targets;
    a.norm = norm;
    a.entropy = entropy;
    a.g_logprob = g_logprob;
    a.g_entropy = g_entropy;
    if (dtype == GMM_F32)
        launch_grad_t<float>(a, (hipStream_t)stream);
    else
        launch_grad_t<uint16_t>(a, (hipStream_t)stream);
    return hipGetLastError() == hipSuccess ? GMM_OK : GMM_E_HIP;
}

}  // extern "C"
