// gmm_score.hip - scores of given codes under a softmax over v codes, from its
// logits, and their gradient (gmm_logits_score, gmm_logits_score_backward,
// declared in include/gmm_em.h).
//
// Scores: with l = scale * x, one pass over a row keeps the running maximum
// m, s = sum exp(l - m) and a = sum exp(l - m)(l - m) (restated when m
// rises), so that
//   log p_t = (l_t - m) - log s      entropy = log s - a / s
// with nothing of the row stored. Sums run per thread, then over the lanes and
// the waves in a fixed order.
// Alternatives: each wave keeps its m best so far in its lanes. Values that
// cannot enter are dismissed by one comparison per lane and chunk (the
// lane's maximum, needed anyway, against the list's last entry); otherwise the
// m-th largest of the lane maxima bounds the list's last entry from below, and
// only the few values at or above it are inserted one by one.
// Gradient: dx = scale (g_lp ([v = t] - p) - g_H p (log p + H)) with p from the
// stored m and log s: each logit is read once and its gradient written once.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "gmm_em.h"
#include "gmm_internal.h"
#include "gmm_nn.h"
#include "gmm_softmax.h"

namespace gmm {

// Threads per row; vectors of 16 bytes in flight per thread.
constexpr int SC_U = 4;

// The logit of the row's target (thread 0; where there is none, unused).
template <typename T>
__device__ __forceinline__ float target_logit(const ScoreArgs& p, int64_t row, int tid) {
    if (tid != 0 || !p.targets) return 0.f;
    const int t = p.targets[row];
    return t >= 0 && t < p.v ? Vec<T>::one((const T*)p.x + row * p.ldl + t) : 0.f;
}

// NT threads per (row, part). parts == 1: writes the results; else the part's
// statistics and list go to the workspace for k_score_join.
template <typename T, int NT, bool TOP>
__global__ __launch_bounds__(NT) void k_score(ScoreArgs p) {
    constexpr int VE = Vec<T>::VE, NW = NT / 64;
    __shared__ float sst[NW][3];
    __shared__ float sv[NW * TOP_MAX];
    __shared__ int si[NW * TOP_MAX];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int64_t item = blockIdx.x; item < p.n * p.parts; item += gridDim.x) {
        const int64_t row = item / p.parts;
        const int part = (int)(item - row * p.parts);
        const int64_t i0 = (int64_t)part * p.part_len;
        const int64_t i1 = i0 + p.part_len < p.v ? i0 + p.part_len : p.v;
        const T* x = (const T*)p.x + row * p.ldl;
        Stats st;
        st.clear();
        TopList top;
        top.clear();
        for (int64_t b = i0; b < i1; b += (int64_t)NT * VE * SC_U) {
            Raw16 raw[SC_U];
#pragma unroll
            for (int u = 0; u < SC_U; ++u)
                raw[u] = load_vec(x, b + ((int64_t)u * NT + tid) * VE, i1);
            float cm = -INFINITY;
#pragma unroll
            for (int u = 0; u < SC_U; ++u)
#pragma unroll
                for (int k = 0; k < VE; ++k) cm = fmaxf(cm, Vec<T>::get(raw[u], k));
            cm *= p.scale;
            st.raise(fmaxf(st.m, cm));
#pragma unroll
            for (int u = 0; u < SC_U; ++u)
#pragma unroll
                for (int k = 0; k < VE; ++k) st.add(fmaf(Vec<T>::get(raw[u], k), p.scale, -st.m));
            if constexpr (TOP) {
                const float least = top.least(p.m);
                if (__builtin_amdgcn_ballot_w64(cm > least)) {
                    // the m-th largest lane maximum: at least m values reach it
                    float cur = cm, bound = -INFINITY;
                    for (int j = 0; j < p.m; ++j) {
                        bound = wave_max(cur);
                        const uint64_t at = __builtin_amdgcn_ballot_w64(cur == bound);
                        if (at && lane == __builtin_ctzll(at)) cur = -INFINITY;
                    }
#pragma unroll
                    for (int u = 0; u < SC_U; ++u)
#pragma unroll
                        for (int k = 0; k < VE; ++k) {
                            const float l = Vec<T>::get(raw[u], k) * p.scale;
                            uint64_t in = __builtin_amdgcn_ballot_w64(l >= bound && l > least);
                            while (in) {
                                const int from = __builtin_ctzll(in);
                                in &= in - 1;
                                const int64_t i =
                                    b + ((int64_t)u * NT + wave * 64 + from) * VE + k;
                                top.insert(lane_get(l, from), (int)i, p.m, lane);
                            }
                        }
                }
            }
        }
        st.wave_join();
        if constexpr (NW > 1) {
            if (lane == 0) {
                sst[wave][0] = st.m;
                sst[wave][1] = st.s;
                sst[wave][2] = st.a;
            }
            if constexpr (TOP) {
                if (lane < p.m) {
                    sv[wave * p.m + lane] = top.v;
                    si[wave * p.m + lane] = top.i;
                }
            }
            __syncthreads();
            // wave 0 joins the waves' statistics and lists
            if (wave == 0) {
                st.clear();
                if (lane < NW) st = Stats{sst[lane][0], sst[lane][1], sst[lane][2]};
                st.wave_join();
                if constexpr (TOP) {
                    constexpr int C = (NW * TOP_MAX + 63) / 64;
                    float cv[C];
                    int ci[C];
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        const int at = c * 64 + lane;
                        cv[c] = at < NW * p.m ? sv[at] : -INFINITY;
                        ci[c] = at < NW * p.m ? si[at] : 0x7fffffff;
                    }
                    top = top_pick<C>(cv, ci, p.m, lane);
                }
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
        if constexpr (NW > 1) __syncthreads();  // LDS is free for the next item
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

// One block per (row, segment of NT * SC_U vectors).
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
    // few long rows: parts of at least 16384 values until 512 blocks run
    if (n < 256) {
        const int64_t most = v / 16384;
        int64_t want = n > 0 ? 512 / n : 1;
        if (want > most) want = most;
        if (want > SC_MAX_PARTS) want = SC_MAX_PARTS;
        if (want > 1) q.parts = (int)want;
    }
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

template <typename T>
static void launch_score_t(const ScoreArgs& a, hipStream_t st) {
    if (a.part_len <= 2048)
        launch_score_nt<T, 64>(a, st);
    else if (a.n * a.parts >= 512)
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
