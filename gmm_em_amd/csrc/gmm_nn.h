// gmm_nn.h - arguments and launchers shared by the softmax-over-codes
// operators (gmm_score.hip, gmm_head.hip, gmm_moe.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "gmm_softmax.h"

namespace gmm {

constexpr int SC_MAX_PARTS = 64;  // parts of a row (one lane each when joined)
// Rows and codes per call: keeps (row, segment) counts within 64 bits and code
// indices, rounded up to whole tiles, within 32.
constexpr int64_t SC_MAX_ROWS = (int64_t)1 << 40;
constexpr int32_t SC_MAX_CODES = (int32_t)1 << 30;
inline bool score_shape_ok(int64_t n, int32_t v) {
    return n >= 0 && n <= SC_MAX_ROWS && v >= 1 && v <= SC_MAX_CODES;
}

// Softmax statistics of a part of a row, handed from one kernel to the next.
struct ScorePart {
    float m, s, a;
};

struct ScoreArgs {
    const void* x;
    int64_t n, ldl;
    int32_t v, m, parts, part_len;
    float scale;
    const int32_t* targets;
    float *logprob, *entropy, *norm;
    int32_t* top_idx;
    float* top_logprob;
    ScorePart* part;
    float* part_v;
    int32_t* part_i;
};

// Writes a row's results from its statistics and its target's logit xt
// (thread 0) and its sorted alternatives (thread j < m holds entry j).
__device__ __forceinline__ void score_out(const ScoreArgs& p, int64_t row, const Stats& st, float xt,
                                          float tv, int ti, int tid) {
    const bool none = st.empty();
    const float logs = none ? 0.f : logf(st.s);
    if (tid == 0) {
        if (p.norm) {
            p.norm[2 * row] = none ? -INFINITY : (st.s == st.s ? st.m : NAN);
            p.norm[2 * row + 1] = logs;
        }
        if (p.entropy) p.entropy[row] = none ? 0.f : logs - st.a / st.s;
        if (p.targets) {
            const int t = p.targets[row];
            float lp = 0.f;  // no code given
            if (t >= p.v)
                lp = NAN;
            else if (t >= 0)
                lp = none ? -INFINITY : (scaled(xt, p.scale) - st.m) - logs;
            p.logprob[row] = lp;
        }
    }
    if (tid < p.m) {
        const bool there = tv > -INFINITY;
        p.top_idx[row * p.m + tid] = there ? ti : -1;
        p.top_logprob[row * p.m + tid] = there ? (tv - st.m) - logs : -INFINITY;
    }
}

struct ScorePlan {
    int32_t parts, part_len;
    size_t o_v, o_i, bytes;
};
ScorePlan score_plan(int64_t n, int32_t v, int32_t m);
// a.parts, a.part_len and the part pointers are filled in from the workspace.
hipError_t launch_score(ScoreArgs a, int dtype, void* ws, hipStream_t st);

struct ScoreGradArgs {
    const void* x;
    void* dx;
    int64_t n, ldl, lddl;
    int32_t v;
    float scale;
    const int32_t* targets;
    const float *norm, *entropy, *g_logprob, *g_entropy;
};

inline bool scale_ok(float s) { return s > 0.f && s < INFINITY; }

// What the gradient of one row's scores with respect to its logits needs.
struct GradRow {
    float scale, m, logs, glp, gh, h;
    int t;
    // dl of logit x at code i; a code of probability 0 has no entropy term
    __device__ __forceinline__ float at(float x, int i) const {
        const float lp = (scaled(x, scale) - m) - logs;
        const float p = exp_neg(lp);
        const float hot = i == t ? glp : 0.f;
        // lp is cut at -1000, where p is 0: 0 * lp stays 0 for a masked logit
        const float d = fmaf(-p, fmaf(gh, fmaxf(lp, -1000.f) + h, glp), hot);
        return scale * d;
    }
};

template <typename A>
__device__ __forceinline__ GradRow grad_row(const A& a, int64_t row) {
    GradRow g;
    g.scale = a.scale;
    g.m = a.norm[2 * row];
    g.logs = a.norm[2 * row + 1];
    g.t = a.targets ? a.targets[row] : -1;
    g.glp = a.g_logprob && g.t >= 0 ? (g.t < a.v ? a.g_logprob[row] : NAN) : 0.f;
    g.gh = a.g_entropy ? a.g_entropy[row] : 0.f;
    g.h = a.g_entropy ? a.entropy[row] : 0.f;
    if (g.m == -INFINITY) {  // nothing left in the row: p = 0, and no gradient
        g.m = INFINITY;
        g.logs = 0.f;
        g.glp = g.glp == g.glp ? 0.f : g.glp;
        g.gh = 0.f;
        g.t = -1;
    }
    return g;
}

}  // namespace gmm
