// gmm_moe.hip - a mixture-of-experts layer for a few rows (gmm_moe_layer,
// declared in include/gmm_em.h):
//   z = x G^T; the m experts of largest z (ties: smaller index) with their
//   softmax shares r_j;  y = sum_j r_j W_out[e_j] (silu(a_j) * b_j),
//   [a_j; b_j] = W_in[e_j] x.
//
// With few rows the layer is the reading of the weights of the experts that
// some row picked: every weight is read once per 64 rows that need it, straight
// into registers in the operand order of the matrix units (16 weight rows by
// 16 rows of x), which then cost nothing beside the reads, also for one row.
//   k_moe_route: a workgroup per row: z, the choice, the shares.
//   k_moe_in:    (expert, 16 features of a and of b): the contracted axis is
//                split over the waves and joined in LDS; silu(a) b goes to the
//                workspace, as two bf16 parts for bf16 data (16 bits of it).
//   k_moe_out:   (expert, 32 or 16 features of y): as before; r_j times it goes to
//                the workspace. One or two rows: k_moe_out_row instead of both.
//   k_moe_join:  y = the sum over j in order, rounded once.
// Every sum is fp32 in a fixed order.
// Measured, bf16: 64 rows of 2048, f = 1408, 4 of 64 experts (1.09 GB of weights):
// k_moe_in 145 us (5.0 TB/s), k_moe_out 88 us (4.2 TB/s), route 9, join 5; one row of 768,
// f = 2048, 2 of 64: 5 + 5 + 9 us, bound by latency and the three launches.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "gmm_em.h"
#include "gmm_gemm.h"
#include "gmm_nn.h"
#include "gmm_softmax.h"

namespace gmm {

constexpr int MOE_MAX_EXPERTS = 4096;    // gate logits of a row in LDS
constexpr int64_t MOE_MAX_PAIRS = 1 << 20;  // (row, pick) pairs per call
constexpr int32_t MOE_MAX_DIM = 1 << 20;
constexpr int MOE_FEW_ROWS = 2;          // rows whose second product is made row by row
constexpr int MOE_WIN = 2048;            // pairs looked through at a time

struct MoeArgs {
    const void *x, *gate, *w_in, *w_out;
    int64_t ldx, ldy;
    int32_t n, d, f, e, m, pairs;
    int32_t slots;     // workgroups' second index: an expert, or a pair where those are fewer
    int32_t by_pair;
    int32_t all;       // shares over all experts instead of the picked ones
    int32_t fp;        // row stride of act: f padded
    int32_t* idx;
    float* resp;
    void* act;         // [parts][pairs][fp]
    int64_t act_plane;
    float* part;       // [pairs][d]
    void* y;
};

// c += the 16 x 16 product of 4 VE contracted values: lane 16 h + i holds
// values VE h .. VE h + VE of row i of both operands.
__device__ __forceinline__ f32x4 mfma_raw(const Raw16& a, const Raw16& b, f32x4 c, uint16_t) {
    return mfma32(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c);
}
__device__ __forceinline__ f32x4 mfma_raw(const Raw16& a, const Raw16& b, f32x4 c, float) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.w[k]), __uint_as_float(b.w[k]), c,
                                                 0, 0, 0);
    return c;
}

// ---- the choice of experts

// Dot products of one row of x with RT_U gates at a time (all their loads in
// flight), a wave for each group. Up to RT_PICK experts are ranked in one wave's
// registers, more by counting in LDS.
constexpr int RT_NT = 1024, RT_U = 4, RT_PICK = 512;
template <typename T>
__global__ __launch_bounds__(RT_NT) void k_moe_route(MoeArgs p) {
    constexpr int VE = Vec<T>::VE;
    __shared__ float z[MOE_MAX_EXPERTS], key[MOE_MAX_EXPERTS];
    __shared__ int id[MOE_MAX_EXPERTS];
    __shared__ float ov[TOP_MAX], part[RT_NT / 64];
    __shared__ int oi[TOP_MAX];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t row = blockIdx.x;
    const T* x = (const T*)p.x + row * p.ldx;
    for (int e0 = wave * RT_U; e0 < p.e; e0 += RT_NT / 64 * RT_U) {
        float s[RT_U];
        const T* g[RT_U];
#pragma unroll
        for (int j = 0; j < RT_U; ++j) {
            s[j] = 0.f;
            g[j] = (const T*)p.gate + (int64_t)(e0 + j < p.e ? e0 + j : p.e - 1) * p.d;
        }
#pragma unroll 2
        for (int k = lane * VE; k < p.d; k += 64 * VE) {
            const Raw16 a = load_zero(x, k, (int64_t)p.d);
            Raw16 b[RT_U];
#pragma unroll
            for (int j = 0; j < RT_U; ++j) b[j] = load_zero(g[j], k, (int64_t)p.d);
#pragma unroll
            for (int j = 0; j < RT_U; ++j)
#pragma unroll
                for (int u = 0; u < VE; ++u)
                    s[j] = fmaf(Vec<T>::get(a, u), Vec<T>::get(b[j], u), s[j]);
        }
#pragma unroll
        for (int j = 0; j < RT_U; ++j) {
            const float t = wave_sum(s[j]);
            if (lane == 0 && e0 + j < p.e) {
                // -inf and NaN have the lowest number's key and rank after it by their ids
                z[e0 + j] = t;
                key[e0 + j] = t > -3.402823466e38f ? t : -3.402823466e38f;
                id[e0 + j] = e0 + j + (t != t ? 2 : t == -INFINITY ? 1 : 0) * MOE_MAX_EXPERTS;
            }
        }
    }
    __syncthreads();
    if (p.e <= RT_PICK) {
        if (wave == 0) {
            constexpr int C = RT_PICK / 64;
            float cv[C];
            int ci[C];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int i = c * 64 + lane;
                ci[c] = i < p.e ? id[i] : i;
                cv[c] = i < p.e ? key[i] : -INFINITY;
            }
            const TopList t = top_pick<C>(cv, ci, p.m, lane);
            if (lane < p.m) {
                ov[lane] = t.v;
                oi[lane] = t.i % MOE_MAX_EXPERTS;
            }
        }
    } else {
        top_rank(key, id, p.e, p.m, ov, oi, tid, RT_NT);
        __syncthreads();
        if (tid < p.m) oi[tid] %= MOE_MAX_EXPERTS;
    }
    __syncthreads();
    const float top = ov[0];
    float sum = 0.f;
    if (p.all) {
        for (int e = tid; e < p.e; e += RT_NT) sum += exp_neg(z[e] - top);
        sum = wave_sum(sum);
        if (lane == 0) part[wave] = sum;
        __syncthreads();
        sum = 0.f;
        for (int w = 0; w < RT_NT / 64; ++w) sum += part[w];
    } else if (wave == 0) {
        sum = wave_sum(lane < p.m ? exp_neg(z[oi[lane]] - top) : 0.f);
    }
    if (tid < p.m) {
        p.idx[row * p.m + tid] = oi[tid];
        p.resp[row * p.m + tid] = exp_neg(z[oi[tid]] - top) / sum;
    }
}

// The pairs of window [w0, w0 + MOE_WIN) that picked expert e, in order.
// Returns their count; all W waves call it. Where the picks of one call fit a wave
// (pairs <= 64), every wave finds them from one load and a ballot, here and in moe_expert.
template <int W>
__device__ __forceinline__ int moe_list(const MoeArgs& p, int e, int w0, int* list, int* cnt) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const uint64_t below = (uint64_t(1) << lane) - 1;
    if (p.pairs <= 64) {  // every wave writes the same list
        const bool in = lane < p.pairs && p.idx[lane] == e;
        const uint64_t mask = __builtin_amdgcn_ballot_w64(in);
        if (in) list[__popcll(mask & below)] = lane;
        __builtin_amdgcn_wave_barrier();
        return __popcll(mask);
    }
    int base = 0;
    for (int b = 0; b < MOE_WIN && w0 + b < p.pairs; b += 64 * W) {
        const int i = w0 + b + tid;
        const bool in = i < p.pairs && p.idx[i] == e;
        const uint64_t mask = __builtin_amdgcn_ballot_w64(in);
        if (lane == 0) cnt[wave] = __popcll(mask);
        __syncthreads();
        int at = base;
        for (int w = 0; w < W; ++w) {
            if (w < wave) at += cnt[w];
            base += cnt[w];
        }
        if (in) list[at + __popcll(mask & below)] = i;
        __syncthreads();
    }
    return base;
}

// The expert of this workgroup, or -1: by pair, the first pair that picked an
// expert does its work. All threads call it.
template <int W>
__device__ __forceinline__ int moe_expert(const MoeArgs& p) {
    const int slot = blockIdx.y;
    if (!p.by_pair) return slot;
    if (p.pairs <= 64) {
        const int lane = threadIdx.x & 63;
        const int mine = lane < p.pairs ? p.idx[lane] : -1;
        const int e = __builtin_amdgcn_readlane(mine, slot);
        const uint64_t same = __builtin_amdgcn_ballot_w64(mine == e);
        return e < 0 || e >= p.e || __builtin_ctzll(same) != slot ? -1 : e;
    }
    const int e = p.idx[slot];
    int before = 0;
    for (int i = threadIdx.x; i < slot; i += 64 * W) before |= p.idx[i] == e;
    before = __syncthreads_or(before);
    return before || e < 0 || e >= p.e ? -1 : e;
}

// ---- products

// One group of U steps of the contracted axis, W apart, from step s.
// FULL: the steps lie within k_end.
template <typename T, int R, int TT, int PB, int W, int U, bool FULL>
__device__ __forceinline__ void moe_steps(const T* const* rows, const T* const* col, int64_t plane,
                                          int s, int k_end, f32x4 (*acc)[TT]) {
    constexpr int VE = Vec<T>::VE, STEP = 4 * VE;
    const int h = (threadIdx.x & 63) >> 4;
    Raw16 a[R][U], b[TT][PB][U];
    auto get = [&](const T* q, int k) {
        if constexpr (FULL)
            return *reinterpret_cast<const Raw16*>(q + k);
        else
            return load_zero(q, k, (int64_t)k_end);
    };
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int k = (s + u * W) * STEP + h * VE;
#pragma unroll
        for (int r = 0; r < R; ++r) a[r][u] = get(rows[r], k);
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int q = 0; q < PB; ++q) b[t][q][u] = get(col[t] + q * plane, k);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int q = PB - 1; q >= 0; --q)
                    acc[r][t] = mfma_raw(a[r][u], b[t][q][u], acc[r][t], T());
}

// acc[r][t] += W_r B_t over this wave's steps of the contracted axis (step s
// belongs to wave s % W): R sets of 16 weight rows, of which rows[r] is
// this lane's, TT sets of 16 columns (col[t]), each in PB planes. Groups of
// 8 steps in flight, then 4, 2 and 1.
template <typename T, int R, int TT, int PB, int W>
__device__ __forceinline__ void moe_dot(const T* const* rows, const T* const* col, int64_t plane,
                                        int k_end, f32x4 (*acc)[TT]) {
    constexpr int STEP = 4 * Vec<T>::VE;
    const int full = k_end / STEP;
    int s = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if constexpr (TT == 1 && R <= 2)
        for (; s + 7 * W < full; s += 8 * W)
            moe_steps<T, R, TT, PB, W, 8, true>(rows, col, plane, s, k_end, acc);
    for (; s + 3 * W < full; s += 4 * W)
        moe_steps<T, R, TT, PB, W, 4, true>(rows, col, plane, s, k_end, acc);
    for (; s + W < full; s += 2 * W)
        moe_steps<T, R, TT, PB, W, 2, true>(rows, col, plane, s, k_end, acc);
    for (; s < full; s += W)
        moe_steps<T, R, TT, PB, W, 1, true>(rows, col, plane, s, k_end, acc);
    if (s * STEP < k_end) moe_steps<T, R, TT, PB, W, 1, false>(rows, col, plane, s, k_end, acc);
}

// Sums the waves' blocks: afterwards sh[b][lane][q] of wave 0's place holds the sum.
template <int NB, int W>
__device__ __forceinline__ void moe_join_waves(const f32x4* acc, f32x4* sh) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
#pragma unroll
    for (int b = 0; b < NB; ++b) sh[(wave * NB + b) * 64 + lane] = acc[b];
    __syncthreads();
    for (int j = tid; j < NB * 64; j += 64 * W) {
        f32x4 s = sh[j];
#pragma unroll
        for (int w = 1; w < W; ++w) s += sh[w * NB * 64 + j];
        sh[j] = s;
    }
    __syncthreads();
}

__device__ __forceinline__ void store_act(const MoeArgs& p, int64_t at, float v, float) {
    ((float*)p.act)[at] = v;
}
// two bf16 parts: together 16 bits of v
__device__ __forceinline__ void store_act(const MoeArgs& p, int64_t at, float v, uint16_t) {
    uint16_t* a = (uint16_t*)p.act;
    const uint32_t hi = f32_to_bf16(v);
    const float rest = v - bf16_to_f32(hi);
    a[at] = (uint16_t)hi;
    a[p.act_plane + at] = rest == rest ? (uint16_t)f32_to_bf16(rest) : (uint16_t)0;
}

template <typename T, int TT, int W>
__device__ __forceinline__ void moe_in_tile(const MoeArgs& p, int e, int f0, const int* list, int cnt,
                                            f32x4* sh) {
    const int tid = threadIdx.x, lane = tid & 63, i = lane & 15;
    const int row = f0 + i < p.f ? f0 + i : p.f - 1;
    const T* w = (const T*)p.w_in + (int64_t)e * 2 * p.f * p.d;
    const T* rows[2] = {w + (int64_t)row * p.d, w + ((int64_t)p.f + row) * p.d};
    const T* col[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const int c = t * 16 + i < cnt ? t * 16 + i : cnt - 1;
        col[t] = (const T*)p.x + (int64_t)(list[c] / p.m) * p.ldx;
    }
    f32x4 acc[2][TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[0][t] = acc[1][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    moe_dot<T, 2, TT, 1, W>(rows, col, 0, p.d, acc);
    moe_join_waves<2 * TT, W>(&acc[0][0], sh);
    // block t: gate part, block TT + t: the other; C[4 h + q][i] at lane 16 h + i
    for (int j = tid; j < TT * 64; j += 64 * W) {
        const int t = j >> 6, c = t * 16 + (j & 15), fq = f0 + 4 * ((j >> 4) & 3);
        if (c >= cnt) continue;
        const f32x4 a = sh[j], b = sh[TT * 64 + j];
        const int64_t at = (int64_t)list[c] * p.fp;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (fq + q < p.f) store_act(p, at + fq + q, a[q] / (1.f + __expf(-a[q])) * b[q], T());
    }
    __syncthreads();
}

// Runs tile<TT>(list, count) over the expert's rows: 64 at a time while more than
// 16 are left, then 16.
template <int W, typename F>
__device__ __forceinline__ void moe_each(const MoeArgs& p, int e, int* list, int* cnt, F tile) {
    for (int w0 = 0; w0 < p.pairs; w0 += MOE_WIN) {
        const int c = moe_list<W>(p, e, w0, list, cnt);
        int at = 0;
        for (; c - at > 16; at += 64)
            tile(std::integral_constant<int, 4>(), list + at, c - at < 64 ? c - at : 64);
        if (at < c) tile(std::integral_constant<int, 1>(), list + at, c - at);
        __syncthreads();
    }
}

template <typename T, int W>
__global__ __launch_bounds__(64 * W) void k_moe_in(MoeArgs p) {
    __shared__ f32x4 sh[W * 8 * 64];
    __shared__ int list[MOE_WIN], cnt[W];
    const int e = moe_expert<W>(p);
    if (e < 0) return;
    const int f0 = blockIdx.x * 16;
    moe_each<W>(p, e, list, cnt, [&](auto tt, const int* l, int c) {
        moe_in_tile<T, decltype(tt)::value, W>(p, e, f0, l, c, sh);
    });
}

template <typename T, int TT, int R, int W>
__device__ __forceinline__ void moe_out_tile(const MoeArgs& p, int e, int d0, const int* list, int cnt,
                                             f32x4* sh) {
    constexpr int PB = std::is_same<T, uint16_t>::value ? 2 : 1;
    const int tid = threadIdx.x, lane = tid & 63, i = lane & 15;
    const T* rows[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = d0 + r * 16 + i < p.d ? d0 + r * 16 + i : p.d - 1;
        rows[r] = (const T*)p.w_out + ((int64_t)e * p.d + row) * p.f;
    }
    const T* col[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const int c = t * 16 + i < cnt ? t * 16 + i : cnt - 1;
        col[t] = (const T*)p.act + (int64_t)list[c] * p.fp;
    }
    f32x4 acc[R][TT];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    moe_dot<T, R, TT, PB, W>(rows, col, p.act_plane, p.f, acc);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        moe_join_waves<TT, W>(acc[r], sh);
        for (int j = tid; j < TT * 64; j += 64 * W) {
            const int t = j >> 6, c = t * 16 + (j & 15), dq = d0 + r * 16 + 4 * ((j >> 4) & 3);
            if (c >= cnt) continue;
            const f32x4 a = sh[j];
            const int pair = list[c];
            const float w = p.resp[pair];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (dq + q < p.d) p.part[(int64_t)pair * p.d + dq + q] = w * a[q];
        }
        __syncthreads();
    }
}

template <typename T, int R, int W>
__global__ __launch_bounds__(64 * W) void k_moe_out(MoeArgs p) {
    __shared__ f32x4 sh[W * 4 * 64];
    __shared__ int list[MOE_WIN], cnt[W];
    const int e = moe_expert<W>(p);
    if (e < 0) return;
    const int d0 = blockIdx.x * 16 * R;
    moe_each<W>(p, e, list, cnt, [&](auto tt, const int* l, int c) {
        moe_out_tile<T, decltype(tt)::value, R, W>(p, e, d0, l, c, sh);
    });
}

// Few rows: one workgroup makes 16 features of one row from all its experts and
// writes y itself (experts that rows share are read again, from the caches).
// 16 waves split the contracted axis; a wave's sums over the experts stay in its
// accumulators, scaled by the shares, in the picks' order.
constexpr int MOE_ROW_W = 16;
template <typename T>
__global__ __launch_bounds__(64 * MOE_ROW_W) void k_moe_out_row(MoeArgs p) {
    constexpr int PB = std::is_same<T, uint16_t>::value ? 2 : 1;
    __shared__ f32x4 sh[MOE_ROW_W * 64];
    const int tid = threadIdx.x, lane = tid & 63, i = lane & 15;
    const int t = blockIdx.y, d0 = blockIdx.x * 16;
    const int row = d0 + i < p.d ? d0 + i : p.d - 1;
    f32x4 y{0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < p.m; ++j) {
        const int pair = t * p.m + j;
        const int e = p.idx[pair];
        if (e < 0 || e >= p.e) continue;
        const T* rows[1] = {(const T*)p.w_out + ((int64_t)e * p.d + row) * p.f};
        const T* col[1] = {(const T*)p.act + (int64_t)pair * p.fp};
        f32x4 acc[1][1] = {{f32x4{0.f, 0.f, 0.f, 0.f}}};
        moe_dot<T, 1, 1, PB, MOE_ROW_W>(rows, col, p.act_plane, p.f, acc);
        y += p.resp[pair] * acc[0][0];
    }
    moe_join_waves<1, MOE_ROW_W>(&y, sh);
    // all 16 columns are this row: column 0's four features per lane 16 h
    if (tid < 64 && i == 0) {
        const f32x4 v = sh[lane];
        const int c = d0 + 4 * (lane >> 4);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (c + q < p.d) ((T*)p.y)[(int64_t)t * p.ldy + c + q] = Vec<T>::store(v[q]);
    }
}

template <typename T>
__global__ __launch_bounds__(256) void k_moe_join(MoeArgs p) {
    const int64_t total = (int64_t)p.n * p.d;
    for (int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x; j < total;
         j += (int64_t)gridDim.x * 256) {
        const int64_t row = j / p.d;
        const int c = (int)(j - row * p.d);
        float y = 0.f;
        for (int k = 0; k < p.m; ++k) {
            const int64_t pair = row * p.m + k;
            const int e = p.idx[pair];
            if (e >= 0 && e < p.e) y += p.part[pair * p.d + c];
        }
        ((T*)p.y)[row * p.ldy + c] = Vec<T>::store(y);
    }
}

struct MoePlan {
    int fp;
    size_t o_act, o_part, bytes;
};

static MoePlan moe_plan(int64_t n, int32_t d, int32_t f, int32_t m) {
    auto align = [](size_t b) { return (b + 255) & ~(size_t)255; };
    const size_t pairs = (size_t)n * m;
    MoePlan q;
    q.fp = (f + 15) / 16 * 16;
    q.o_act = 0;
    // fp32, or two parts of bf16
    q.o_part = align(pairs * q.fp * 4);
    q.bytes = q.o_part + align(pairs * d * 4);
    if (q.bytes < 256) q.bytes = 256;
    return q;
}

static int moe_check(int64_t n, int32_t d, int32_t f, int32_t e, int32_t dtype, int32_t m) {
    if (dtype != GMM_F32 && dtype != GMM_BF16) return GMM_E_DTYPE;
    if (n < 0 || d < 1 || f < 1 || e < 1 || m < 1 || m > TOP_MAX || m > e) return GMM_E_INVALID;
    if (d > MOE_MAX_DIM || f > MOE_MAX_DIM || e > MOE_MAX_EXPERTS || n > MOE_MAX_PAIRS / m)
        return GMM_E_UNSUPPORTED;
    return GMM_OK;
}

template <typename T>
static hipError_t launch_moe(const MoeArgs& a, hipStream_t st) {
    if (a.gate) hipLaunchKernelGGL((k_moe_route<T>), dim3(a.n), dim3(RT_NT), 0, st, a);
    const int ft = (a.f + 15) / 16, dt = (a.d + 15) / 16;
    hipLaunchKernelGGL((k_moe_in<T, 4>), dim3(ft, a.slots), dim3(256), 0, st, a);
    if (a.n <= MOE_FEW_ROWS) {
        hipLaunchKernelGGL((k_moe_out_row<T>), dim3(dt, a.n), dim3(64 * MOE_ROW_W), 0, st, a);
        return hipGetLastError();
    }
    // bf16, the layer with 32 features sharing the loads of act / 16 features in 4 waves / in 16:
    // 8192 tiles of 16 (64 rows of 2048 x 1408, 4 of 64 experts) 248 / 271 / 344 us, 4096 (8
    // rows) 122 / 132 / 156, 1024 (64 rows of 2048 x 1408, 4 of 8) 61 / 73 / 83, 1024 (64 rows of
    // 1024 x 1024, 2 of 16) 35.2 / 34.7 / 43.3; 768 (64 rows of 768 x 1024, 2 of 16) 32.6 / 30.8 /
    // 36.8, 512 (12 rows of 1024 x 2048, 2 of 8) 36.9 / 35.8 / 36.1; 256 (300 rows of 512 x 512, 2 of
    // 8) 37.8 / 39.6 / 34.6
    if ((int64_t)dt * a.slots >= 1024)
        hipLaunchKernelGGL((k_moe_out<T, 2, 4>), dim3((dt + 1) / 2, a.slots), dim3(256), 0, st, a);
    else if ((int64_t)dt * a.slots >= 512)
        hipLaunchKernelGGL((k_moe_out<T, 1, 4>), dim3(dt, a.slots), dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((k_moe_out<T, 1, 16>), dim3(dt, a.slots), dim3(1024), 0, st, a);
    const int64_t work = ((int64_t)a.n * a.d + 255) / 256;
    hipLaunchKernelGGL((k_moe_join<T>), dim3((unsigned)(work < 16384 ? work : 16384)), dim3(256), 0, st,
                       a);
    return hipGetLastError();
}

}  // namespace gmm

using namespace gmm;

extern "C" {

size_t gmm_moe_layer_workspace_bytes(int64_t n, int32_t d, int32_t f, int32_t e, int32_t dtype,
                                     int32_t m) {
    return moe_check(n, d, f, e, dtype, m) == GMM_OK ? moe_plan(n, d, f, m).bytes : 0;
}

int gmm_moe_layer(const void* x, int64_t n, int32_t d, int64_t ldx, const void* gate, int32_t e,
                  const void* w_in, const void* w_out, int32_t f, int32_t dtype, int32_t m,
                  int32_t share_all, int32_t* idx, float* resp, void* y, int64_t ldy,
                  void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = moe_check(n, d, f, e, dtype, m);
    if (rc != GMM_OK) return rc;
    if (ldx < d || ldy < d) return GMM_E_INVALID;
    if (n > 0 && (!x || !w_in || !w_out || !idx || !resp || !y)) return GMM_E_INVALID;
    const MoePlan q = moe_plan(n, d, f, m);
    if (!workspace || workspace_bytes < q.bytes || (uintptr_t)workspace % 256 != 0)
        return GMM_E_WORKSPACE;
    if (n == 0) return GMM_OK;
    MoeArgs a{};
    a.x = x;
    a.gate = gate;
    a.w_in = w_in;
    a.w_out = w_out;
    a.ldx = ldx;
    a.ldy = ldy;
    a.n = (int32_t)n;
    a.d = d;
    a.f = f;
    a.e = e;
    a.m = m;
    a.pairs = (int32_t)(n * m);
    a.by_pair = a.pairs < e;
    a.slots = a.by_pair ? a.pairs : e;
    a.all = share_all != 0;
    a.fp = q.fp;
    a.idx = idx;
    a.resp = resp;
    a.act = (char*)workspace + q.o_act;
    a.act_plane = (int64_t)a.pairs * q.fp;
    a.part = (float*)((char*)workspace + q.o_part);
    a.y = y;
    const hipError_t err = dtype == GMM_F32 ? launch_moe<float>(a, (hipStream_t)stream)
                                            : launch_moe<uint16_t>(a, (hipStream_t)stream);
    return err == hipSuccess ? GMM_OK : GMM_E_HIP;
}

}  // extern "C"
