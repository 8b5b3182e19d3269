// gmm_beam.hip - a step of beam search (gmm_beam_step, gmm_beam_reorder, declared in
// include/gmm_em.h): the m best of a search's w x v continuations
//   score[w] + (l_v - max l) - log sum exp(l - max l)
// and the move of the states that go with the beams.
//
// A beam's m best codes are those of its row of logits (gmm_score.hip: one pass, the rows of dead
// and ended beams are not read); within a beam the order of the scores is that of the
// logits, so the m best of all are a merge of w sorted lists, where each entry counts those before it.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "gmm_em.h"
#include "gmm_nn.h"
#include "gmm_softmax.h"

namespace gmm {

struct BeamArgs {
    const float* scores;
    const int32_t* last;
    const int32_t* top_idx;      // [b w][per], -1 where there is none
    const float* top_logprob;
    int64_t b;
    int32_t w, m, per, end;
    int32_t *parent, *code;
    float* score;
};

// A thread per continuation of the search's w lists finds its place: the entries before it in its
// own list, and in each other list those that are larger (or equal, in an earlier beam's).
constexpr int BJ_NT = TOP_MAX * TOP_MAX;
__global__ __launch_bounds__(BJ_NT) void k_beam_join(BeamArgs p) {
    __shared__ __align__(16) uint32_t key[TOP_MAX][TOP_MAX];  // 0: none
    __shared__ int parent[TOP_MAX], codes[TOP_MAX];
    __shared__ float scores[TOP_MAX];
    const int tid = threadIdx.x, w = tid / TOP_MAX, j = tid % TOP_MAX;
    const bool in = w < p.w && j < p.per;
    for (int64_t b = blockIdx.x; b < p.b; b += gridDim.x) {
        float score = -INFINITY;
        int code = -1;
        if (in) {
            const int64_t row = b * p.w + w, e = row * p.per + j;
            // unwritten for beams that are dead or have ended
            const int i = p.top_idx[e];
            const float lp = p.top_logprob[e], s = p.scores[row];
            const bool ended = beam_ended(p.last, p.end, row);
            if (fabsf(s) < INFINITY && (ended ? j == 0 : i >= 0)) {
                score = ended ? s : s + lp;
                code = ended ? p.end : i;
            }
        }
        const uint32_t mine = score > -INFINITY ? order_of(score) : 0;  // NaN is no continuation
        key[w][j] = mine;
        if (tid < TOP_MAX) {
            parent[tid] = codes[tid] = -1;
            scores[tid] = -INFINITY;
        }
        __syncthreads();
        int rank = j;
#pragma unroll 4
        for (int q = 0; q < p.w; ++q) {
            const uint32_t least = q < w ? mine - 1 : mine;  // mine > 0 where it counts
            int more = 0;
#pragma unroll
            for (int k = 0; k < TOP_MAX; k += 4) {
                const uint4 o = *(const uint4*)&key[q][k];
                more += (o.x > least) + (o.y > least) + (o.z > least) + (o.w > least);
            }
            rank += q == w ? 0 : more;
        }
        if (mine > 0 && rank < p.m) {
            parent[rank] = w;
            codes[rank] = code;
            scores[rank] = score;
        }
        __syncthreads();
        if (tid < p.m) {
            p.parent[b * p.m + tid] = parent[tid];
            p.code[b * p.m + tid] = codes[tid];
            p.score[b * p.m + tid] = scores[tid];
        }
        __syncthreads();
    }
}

// ---- states

struct ReorderArgs {
    const char* in;
    char* out;
    const int32_t* parent;
    int64_t outer, in_outer, out_outer, b, in_row, out_row, bytes;
    int32_t w, m;
};

// A wave per row of the result, or part of a long one.
constexpr int BR_U = 4;
__global__ __launch_bounds__(256) void k_beam_copy(ReorderArgs p) {
    constexpr int64_t SEG = 64 * 16 * BR_U;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t segs = (p.bytes + SEG - 1) / SEG, rows = p.b * p.m, items = p.outer * rows * segs;
    for (int64_t item = (int64_t)blockIdx.x * 4 + wave; item < items; item += (int64_t)gridDim.x * 4) {
        const int64_t all = segs == 1 ? item : item / segs, o = all / rows, r = all - o * rows;
        const int64_t k0 = (item - all * segs) * SEG + lane * 16;
        const int from = p.parent[r];
        const bool there = from >= 0 && from < p.w;
        const char* x = p.in + o * p.in_outer + (r / p.m * p.w + (there ? from : 0)) * p.in_row;
        char* y = p.out + o * p.out_outer + r * p.out_row;
        Any16 v[BR_U];
#pragma unroll
        for (int u = 0; u < BR_U; ++u) {
            const int64_t k = k0 + u * 1024;
            v[u] = Any16{{0u, 0u, 0u, 0u}};
            if (k + 16 <= p.bytes && there) v[u] = *(const Any16*)(x + k);
        }
#pragma unroll
        for (int u = 0; u < BR_U; ++u) {
            const int64_t k = k0 + u * 1024;
            if (k + 16 <= p.bytes)
                *(Any16*)(y + k) = v[u];
            else
                for (int64_t q = k; q < p.bytes; ++q) y[q] = there ? x[q] : 0;
        }
    }
}

// In place: a thread holds its 16 bytes of all the search's rows before it writes them where they go.
__global__ __launch_bounds__(256) void k_beam_swap(ReorderArgs p) {
    const int64_t segs = (p.bytes + 4095) / 4096, items = p.outer * p.b * segs;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t all = item / segs, o = all / p.b, b = all - o * p.b;
        const int64_t k = (item - all * segs) * 4096 + threadIdx.x * 16;
        if (k >= p.bytes) continue;
        const int32_t* parent = p.parent + b * p.m;
        char* x = p.out + o * p.out_outer + b * p.m * p.out_row + k;
        const int n = p.bytes - k < 16 ? (int)(p.bytes - k) : 16;
        Any16 v[TOP_MAX];
#pragma unroll
        for (int j = 0; j < TOP_MAX; ++j) {
            v[j] = Any16{{0u, 0u, 0u, 0u}};
            if (j >= p.m) continue;
            const int from = parent[j];
            if (from < 0 || from >= p.w || from == j) continue;
            const char* s = x + from * p.out_row;
            if (n == 16) {
                v[j] = *(const Any16*)s;
            } else {
#pragma unroll
                for (int q = 0; q < 15; ++q)
                    if (q < n) v[j].w[q >> 2] |= (uint32_t)(uint8_t)s[q] << (8 * (q & 3));
            }
        }
#pragma unroll
        for (int j = 0; j < TOP_MAX; ++j) {
            if (j >= p.m || parent[j] == j) continue;
            char* y = x + j * p.out_row;
            if (n == 16) {
                *(Any16*)y = v[j];
            } else {
#pragma unroll
                for (int q = 0; q < 15; ++q)
                    if (q < n) y[q] = (char)(v[j].w[q >> 2] >> (8 * (q & 3)));
            }
        }
    }
}

struct BeamPlan {
    int32_t per;
    size_t o_idx, o_lp, o_score, bytes;
};
static BeamPlan beam_plan(int64_t b, int32_t w, int32_t v, int32_t m) {
    BeamPlan q{};
    auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
    q.per = m < v ? m : v;
    const size_t list = up((size_t)(b * w) * q.per * 4);
    q.o_idx = 0;
    q.o_lp = list;
    q.o_score = 2 * list;
    q.bytes = 2 * list + up(score_plan(b * w, v, q.per).bytes);
    return q;
}
static bool beam_ok(int64_t b, int32_t w, int32_t v, int32_t m) {
    return b >= 0 && w >= 1 && w <= TOP_MAX && m >= 1 && m <= TOP_MAX && v >= 1 && b <= SC_MAX_ROWS / TOP_MAX &&
           score_shape_ok(b * w, v);
}

}  // namespace gmm

using namespace gmm;

extern "C" {

size_t gmm_beam_step_workspace_bytes(int64_t b, int32_t w, int32_t v, int32_t m) {
    return beam_ok(b, w, v, m) ? beam_plan(b, w, v, m).bytes : 0;
}

int gmm_beam_step(const void* logits, int64_t b, int32_t w, int32_t v, int64_t ldl, int32_t dtype,
                  const float* scores, const int32_t* last, int32_t end, int32_t m, float scale,
                  int32_t* parent, int32_t* code, float* score, void* workspace,
                  size_t workspace_bytes, void* stream) {
    if (dtype != GMM_F32 && dtype != GMM_BF16) return GMM_E_DTYPE;
    if (!beam_ok(b, w, v, m) || ldl < v || !scale_ok(scale)) return GMM_E_INVALID;
    if (b > 0 && (!logits || !scores || !parent || !code || !score)) return GMM_E_INVALID;
    const BeamPlan q = beam_plan(b, w, v, m);
    if (!workspace || workspace_bytes < q.bytes || (uintptr_t)workspace % 256 != 0)
        return GMM_E_WORKSPACE;
    if (b == 0) return GMM_OK;
    hipStream_t st = (hipStream_t)stream;
    char* ws = (char*)workspace;
    ScoreArgs s{};
    s.x = logits;
    s.n = b * w;
    s.ldl = ldl;
    s.v = v;
    s.m = q.per;
    s.scale = scale;
    s.top_idx = (int32_t*)(ws + q.o_idx);
    s.top_logprob = (float*)(ws + q.o_lp);
    s.beam_score = scores;
    s.beam_last = last;
    s.beam_end = end;
    if (w == 1 && score_plan(b, v, q.per).parts == 1) {
        // one beam: its list is the result (8 codes of 4 x 16384 fp32: 13.7 us a call, with the merge 15.7)
        s.top_logprob = score;
        s.beam_parent = parent;
        s.beam_code = code;
        s.beam_m = m;
        return launch_score(s, dtype, ws + q.o_score, st) == hipSuccess ? GMM_OK : GMM_E_HIP;
    }
    if (launch_score(s, dtype, ws + q.o_score, st) != hipSuccess) return GMM_E_HIP;
    const BeamArgs a{scores, last, s.top_idx, s.top_logprob, b, w, m, q.per, end, parent, code, score};
    const int64_t most = (int64_t)1 << 20;
    hipLaunchKernelGGL(k_beam_join, dim3((unsigned)(b < most ? b : most)), dim3(BJ_NT), 0, st, a);
    return hipGetLastError() == hipSuccess ? GMM_OK : GMM_E_HIP;
}

int gmm_beam_reorder(const void* state, int64_t outer, int64_t stride_outer, int64_t b, int32_t w,
                     int64_t stride_row, int64_t row_bytes, const int32_t* parent, int32_t m,
                     void* out, int64_t out_stride_outer, int64_t out_stride_row, void* stream) {
    if (outer < 0 || b < 0 || w < 1 || w > TOP_MAX || m < 1 || m > TOP_MAX || row_bytes < 1) return GMM_E_INVALID;
    // sizes whose byte offsets stay within 64 bits
    const int64_t big = (int64_t)1 << 60;
    if ((double)outer * (double)b * TOP_MAX * (double)row_bytes > (double)big || outer > big || b > big / TOP_MAX)
        return GMM_E_INVALID;
    for (const int64_t s : {stride_row, out_stride_row})
        if (s < 0 || (double)s * (double)b * TOP_MAX > (double)big) return GMM_E_INVALID;
    for (const int64_t s : {stride_outer, out_stride_outer})
        if (s < 0 || (double)s * (double)outer > (double)big) return GMM_E_INVALID;
    // rows of the result must not overlap
    const bool rows = b * m > 1, many = outer > 1;
    if ((rows && out_stride_row < row_bytes) || (many && out_stride_outer < row_bytes)) return GMM_E_INVALID;
    if (rows && many && out_stride_outer < (b * m - 1) * out_stride_row + row_bytes &&
        out_stride_row < (outer - 1) * out_stride_outer + row_bytes)
        return GMM_E_INVALID;
    if (outer > 0 && b > 0 && (!state || !parent || !out)) return GMM_E_INVALID;
    const bool swap = state == out;
    if (swap && (w != m || stride_row != out_stride_row || stride_outer != out_stride_outer)) return GMM_E_INVALID;
    if (outer == 0 || b == 0) return GMM_OK;
    const ReorderArgs a{(const char*)state, (char*)out, parent, outer, stride_outer, out_stride_outer, b,
                        stride_row, out_stride_row, row_bytes, w, m};
    auto grid = [](int64_t blocks) {
        const int64_t most = (int64_t)1 << 20;
        return dim3((unsigned)(blocks < most ? blocks : most));
    };
    if (swap) {
        hipLaunchKernelGGL(k_beam_swap, grid(outer * b * ((row_bytes + 4095) / 4096)), dim3(256), 0,
                           (hipStream_t)stream, a);
    } else {
        const int64_t segs = (row_bytes + 64 * 16 * BR_U - 1) / (64 * 16 * BR_U);
        hipLaunchKernelGGL(k_beam_copy, grid((outer * b * m * segs + 3) / 4), dim3(256), 0, (hipStream_t)stream, a);
    }
    return hipGetLastError() == hipSuccess ? GMM_OK : GMM_E_HIP;
}

}  // extern "C"
