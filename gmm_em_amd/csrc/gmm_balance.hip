// gmm_balance.hip - the balance loss of a router and its gradient (gmm_balance_loss,
// gmm_balance_loss_backward, declared in include/gmm_em.h). With p = softmax(z) of a row's
// gate logits, f_c = picks of expert c / all picks, P_c = the rows' mean of p_c:
//   loss = E sum_c f_c P_c        dz_c = g E / rows p_c (f_c - sum_c' f_c' p_c')
// (f is constant for the gradient: picks have none).
//
// One pass over the logits: 8, 16, 32 or 64 lanes hold a row, so that a wave has up to eight
// rows at once and a lane always the same experts: their sums of p stay in its registers. A
// workgroup leaves its sums and counts in the workspace and k_balance_join adds them in order.
// 1 / s and log s are the hardware's, off by one unit in the last place (2^-23): no more than the fp32 sums of
// many rows leave in the means and the loss. 65536 x 128 bf16: rows 9, join 5, gradient 12 us.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "gmm_em.h"
#include "gmm_nn.h"
#include "gmm_softmax.h"

namespace gmm {

constexpr int BAL_MAX_EXPERTS = 4096;  // as the layer's
constexpr int BAL_PARTS = 256;         // workgroups of the pass over the rows, at most

struct BalancePart {
    float mass;     // sum of p
    int32_t picks;
};

// A join workgroup's share of the loss.
struct BalanceSum {
    float dot;      // sum of picks * mass over its experts
    int32_t picks;
};

struct BalanceArgs {
    const void* z;
    void* dz;
    const int32_t* idx;
    int64_t n, ldz, lddz;
    int32_t e, m, parts;
    float *norm, *loss, *prob;
    int32_t* counts;
    int64_t* totals;
    const float* g_loss;
    BalancePart* part;   // [parts][e]
    int32_t* part_rows;  // [parts]
    BalanceSum* sum;     // [join workgroups]
    int32_t* done;       // join workgroups that have written theirs
};

// over groups of LPR lanes
template <int LPR>
__device__ __forceinline__ float group_reduce_max(float v) {
    if constexpr (LPR == 8) {
        v = fmaxf(v, lane_move<0xb1>(v));
        v = fmaxf(v, lane_move<0x4e>(v));
        return fmaxf(v, lane_move<0x141>(v));
    }
    v = max16(v);
    if (LPR > 16) v = fmaxf(v, __shfl_xor(v, 16));
    if (LPR > 32) v = fmaxf(v, __shfl_xor(v, 32));
    return v;
}
template <int LPR>
__device__ __forceinline__ float group_reduce_sum(float v) {
    if constexpr (LPR == 8) {
        v += lane_move<0xb1>(v);
        v += lane_move<0x4e>(v);
        return v + lane_move<0x141>(v);
    }
    v = sum16(v);
    if (LPR > 16) v += __shfl_xor(v, 16);
    if (LPR > 32) v += __shfl_xor(v, 32);
    return v;
}

// The values of a row that a lane holds: vectors at gl VE, gl VE + LPR VE, ...
template <typename T, int LPR, int CV>
struct RouterRow {
    static constexpr int VE = Vec<T>::VE, C = CV * VE;
    static __device__ __forceinline__ int at(int gl, int j) { return (j / VE * LPR + gl) * VE + j % VE; }
    float v[C];
    static __device__ __forceinline__ void fetch(const T* z, int e, int gl, Raw16* r) {
#pragma unroll
        for (int q = 0; q < CV; ++q) r[q] = load_vec(z, (int64_t)(q * LPR + gl) * VE, (int64_t)e);
    }
    __device__ __forceinline__ void take(const Raw16* r) {
#pragma unroll
        for (int q = 0; q < CV; ++q)
#pragma unroll
            for (int k = 0; k < VE; ++k) v[q * VE + k] = Vec<T>::get(r[q], k);
    }
};

// A wave takes 64 / LPR rows at once and U such groups in one go (their loads, and the next
// go's, are in flight together).
template <typename T, int LPR, int CV, int NT, int U>
__global__ __launch_bounds__(NT) void k_balance_rows(BalanceArgs p) {
    using Row = RouterRow<T, LPR, CV>;
    constexpr int C = Row::C, RPW = 64 / LPR, W = NT / 64;
    // the waves' sums [SLABS][e], then counts [e] and each wave's rows
    constexpr int SLABS = CV == 1 ? W : 1;
    extern __shared__ float sums[];
    int* cnt = (int*)(sums + SLABS * p.e);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int gl = lane % LPR, grp = lane / LPR;
    if (blockIdx.x == 0 && tid == 0) *p.done = 0;  // for the kernel after this one
    for (int c = tid; c < p.e; c += NT) cnt[c] = 0;
    __syncthreads();
    int rows = 0;  // of this wave, with a pick
    float acc[C];
#pragma unroll
    for (int j = 0; j < C; ++j) acc[j] = 0.f;
    const int64_t step = (int64_t)p.parts * W * RPW * U;
    const uint64_t mine = (LPR == 64 ? ~uint64_t(0) : (uint64_t(1) << (LPR & 63)) - 1) << (grp * LPR);
    struct Next {
        Raw16 z[CV];
        int pick;
    } next[U];
    auto fetch = [&](int64_t r0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            int64_t row = r0 + u * RPW + grp;
            row = row < p.n ? row : p.n - 1;
            next[u].pick = gl < p.m ? p.idx[row * p.m + gl] : -1;
            Row::fetch((const T*)p.z + row * p.ldz, p.e, gl, next[u].z);
        }
    };
    int64_t r0 = ((int64_t)blockIdx.x * W + wave) * RPW * U;
    if (r0 < p.n) fetch(r0);
    for (; r0 < p.n; r0 += step) {
        Row x[U];
        int pick[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u].take(next[u].z);
            pick[u] = r0 + u * RPW + grp < p.n ? next[u].pick : -1;
        }
        if (r0 + step < p.n) fetch(r0 + step);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = r0 + u * RPW + grp;
            const bool picked = pick[u] >= 0 && pick[u] < p.e;
            const bool live = (__builtin_amdgcn_ballot_w64(picked) & mine) != 0;
            if (picked) atomicAdd(&cnt[pick[u]], 1);
            rows += __popcll(__builtin_amdgcn_ballot_w64(gl == 0 && live));
            float m = -3.402823466e38f, s = 0.f;
#pragma unroll
            for (int j = 0; j < C; ++j) m = fmaxf(m, x[u].v[j]);
            m = group_reduce_max<LPR>(m);
#pragma unroll
            for (int j = 0; j < C; ++j) {
                x[u].v[j] = exp_neg(x[u].v[j] - m);
                s += x[u].v[j];
            }
            s = group_reduce_sum<LPR>(s);
            const bool none = s == 0.f;  // every logit -inf
            if (live) {
                const float inv = none ? 0.f : __builtin_amdgcn_rcpf(s);
#pragma unroll
                for (int j = 0; j < C; ++j) acc[j] = fmaf(x[u].v[j], inv, acc[j]);
            }
            if (gl == 0 && row < p.n) {
                p.norm[2 * row] = !live ? INFINITY : none ? -INFINITY : (s == s ? m : NAN);
                p.norm[2 * row + 1] = !live || none ? 0.f : __builtin_amdgcn_logf(s) * 0.693147180559945309f;
            }
        }
    }
    // the rows of a wave, then its workgroup's waves in order
#pragma unroll
    for (int j = 0; j < C; ++j) {
        if (LPR < 16) acc[j] += __shfl_xor(acc[j], 8);
        if (LPR < 32) acc[j] += __shfl_xor(acc[j], 16);
        if (LPR < 64) acc[j] += __shfl_xor(acc[j], 32);
    }
    if (lane == 0) cnt[p.e + wave] = rows;
    if constexpr (SLABS > 1) {
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c = Row::at(gl, j);
            if (grp == 0 && c < p.e) sums[wave * p.e + c] = acc[j];
        }
        __syncthreads();
        for (int c = tid; c < p.e; c += NT) {
            float s = sums[c];
#pragma unroll
            for (int w = 1; w < SLABS; ++w) s += sums[w * p.e + c];
            sums[c] = s;  // (read and written by this thread alone)
        }
    } else {
        for (int w = 0; w < W; ++w) {
            if (w == wave && grp == 0) {
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    const int c = Row::at(gl, j);
                    if (c < p.e) sums[c] = w == 0 ? acc[j] : sums[c] + acc[j];
                }
            }
            __syncthreads();
        }
    }
    for (int c = tid; c < p.e; c += NT)
        p.part[(int64_t)blockIdx.x * p.e + c] = BalancePart{sums[c], cnt[c]};
    if (tid == 0) {
        for (int w = 1; w < W; ++w) rows += cnt[p.e + w];
        p.part_rows[blockIdx.x] = rows;
    }
}

// A workgroup adds the parts of 64 experts, 16 groups of parts side by side, then the groups in
// order. The one that comes last adds the workgroups' shares of the loss, in their order.
constexpr int BJ_G = 16, BJ_NT = 64 * BJ_G;
__global__ __launch_bounds__(BJ_NT) void k_balance_join(BalanceArgs p) {
    __shared__ BalancePart sh[BJ_G][64];
    const int lane = threadIdx.x & 63, g = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane;
    const int a = p.parts * g / BJ_G, z = p.parts * (g + 1) / BJ_G;
    float s = 0.f;
    int n = 0, rows = 0;
    if (c < p.e) {
#pragma unroll 16
        for (int t = a; t < z; ++t) {
            const BalancePart q = p.part[(int64_t)t * p.e + c];
            s += q.mass;
            n += q.picks;
        }
    }
    if (g == 0) {
#pragma unroll
        for (int t = lane; t < BAL_PARTS; t += 64) rows += t < p.parts ? p.part_rows[t] : 0;
    }
    sh[g][lane] = BalancePart{s, n};
    __syncthreads();
    if (g != 0) return;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) rows += __shfl_xor(rows, o);
#pragma unroll
    for (int q = 1; q < BJ_G; ++q) {
        s += sh[q][lane].mass;
        n += sh[q][lane].picks;
    }
    if (c < p.e) {
        p.counts[c] = n;
        p.prob[c] = s / (float)(rows > 0 ? rows : 1);
    }
    float dot = wave_sum(c < p.e ? (float)n * s : 0.f);
    int total = n;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) total += __shfl_xor(total, o);
    if (gridDim.x > 1) {
        int before = 0;
        if (lane == 0) {
            BalanceSum* mine = p.sum + blockIdx.x;
            __hip_atomic_store(&mine->dot, dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __hip_atomic_store(&mine->picks, total, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            before = __hip_atomic_fetch_add(p.done, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
        }
        if (__builtin_amdgcn_readfirstlane(before) + 1 != (int)gridDim.x) return;
        dot = 0.f;
        total = 0;
        if (lane < (int)gridDim.x) {  // at most 64 workgroups
            BalanceSum* theirs = p.sum + lane;
            dot = __hip_atomic_load(&theirs->dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            total = __hip_atomic_load(&theirs->picks, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        dot = wave_sum(dot);
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) total += __shfl_xor(total, o);
    }
    if (lane == 0) {
        p.totals[0] = rows;
        p.totals[1] = total;  // below 2^31, as n m is
        p.loss[0] = rows > 0 ? (float)p.e * (dot / (float)total / (float)rows) : 0.f;
    }
}

constexpr int BG_W = 4;
// Workgroups, at most: the preparation of f is paid by several rows.
constexpr int64_t bg_most(int cv) { return cv == 1 ? 1024 : cv <= 4 ? 512 : 256; }
template <typename T, int LPR, int CV, int U>
__global__ __launch_bounds__(64 * BG_W) void k_balance_grad(BalanceArgs p) {
    using Row = RouterRow<T, LPR, CV>;
    constexpr int C = Row::C, RPW = 64 / LPR, VE = Vec<T>::VE;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int gl = lane % LPR, grp = lane / LPR;
    const float rows = (float)p.totals[0], inv = 1.f / fmaxf((float)p.totals[1], 1.f);
    const float by = (p.g_loss ? p.g_loss[0] : 1.f) * ((float)p.e / fmaxf(rows, 1.f));
    float f[C];
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const int c = Row::at(gl, j);
        f[j] = c < p.e ? (float)p.counts[c] * inv : 0.f;
    }
    struct Next {
        Raw16 z[CV];
        float m, logs;
    } next[U];
    auto fetch = [&](int64_t r0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            int64_t row = r0 + u * RPW + grp;
            row = row < p.n ? row : p.n - 1;
            next[u].m = p.norm[2 * row];
            next[u].logs = p.norm[2 * row + 1];
            Row::fetch((const T*)p.z + row * p.ldz, p.e, gl, next[u].z);
        }
    };
    // p.dz may be p.z: the rows fetched ahead are other ones than those written
    const int64_t step = (int64_t)gridDim.x * BG_W * RPW * U;
    int64_t r0 = ((int64_t)blockIdx.x * BG_W + wave) * RPW * U;
    if (r0 < p.n) fetch(r0);
    for (; r0 < p.n; r0 += step) {
        Row x[U];
        float m[U], logs[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u].take(next[u].z);
            m[u] = next[u].m;
            logs[u] = next[u].logs;
        }
        if (r0 + step < p.n) fetch(r0 + step);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = r0 + u * RPW + grp;
            const bool off = m[u] == INFINITY || m[u] == -INFINITY;  // left out, or no logit above -inf
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < C; ++j) {
                x[u].v[j] = off ? 0.f : exp_neg((x[u].v[j] - m[u]) - logs[u]);
                s = fmaf(f[j], x[u].v[j], s);
            }
            s = group_reduce_sum<LPR>(s);
            if (row >= p.n) continue;
            T* out = (T*)p.dz + row * p.lddz;
#pragma unroll
            for (int q = 0; q < CV; ++q) {
                const int64_t i = (int64_t)(q * LPR + gl) * VE;
                float w[VE];
#pragma unroll
                for (int k = 0; k < VE; ++k) {
                    const int j = q * VE + k;
                    w[k] = off ? 0.f : by * (x[u].v[j] * (f[j] - s));
                }
                const Raw16 o = pack16<T>(w);
                if (i + VE <= p.e) {
                    *reinterpret_cast<Raw16*>(out + i) = o;
                } else {
#pragma unroll
                    for (int k = 0; k < VE; ++k)
                        if (i + k < p.e) out[i + k] = Vec<T>::store(Vec<T>::get(o, k));
                }
            }
        }
    }
}

static size_t bal_up(size_t b) { return (b + 255) & ~(size_t)255; }
static int balance_parts(int64_t n) {
    const int64_t want = (n + 15) / 16;
    return (int)(want < 1 ? 1 : want < BAL_PARTS ? want : BAL_PARTS);
}
static bool balance_ok(int64_t n, int32_t e, int32_t m) {
    return n >= 0 && e >= 1 && m >= 1 && m <= TOP_MAX;
}
static bool balance_fits(int64_t n, int32_t e, int32_t m) {
    return e <= BAL_MAX_EXPERTS && n <= 0x7fffffff / m;  // counts are 32-bit
}

// Lanes of a row and vectors of a lane: as few lanes as hold the row in one vector each (and its
// m picks, one each).
template <typename T, typename F>
static void with_row(int e, int m, F f) {
    constexpr int VE = Vec<T>::VE;
    using std::integral_constant;
    if (e <= 8 * VE && m <= 8) f(integral_constant<int, 8>(), integral_constant<int, 1>());
    else if (e <= 16 * VE) f(integral_constant<int, 16>(), integral_constant<int, 1>());
    else if (e <= 32 * VE) f(integral_constant<int, 32>(), integral_constant<int, 1>());
    else if (e <= 64 * VE) f(integral_constant<int, 64>(), integral_constant<int, 1>());
    else if (e <= 256 * VE) f(integral_constant<int, 64>(), integral_constant<int, 4>());
    else f(integral_constant<int, 64>(), integral_constant<int, BAL_MAX_EXPERTS / 64 / VE>());
}

template <typename T>
static hipError_t balance(const BalanceArgs& a, hipStream_t st) {
    with_row<T>(a.e, a.m, [&](auto l, auto c) {
        constexpr int LPR = decltype(l)::value, CV = decltype(c)::value;
        auto launch = [&](auto nt, auto groups) {
            constexpr int NT = decltype(nt)::value, U = decltype(groups)::value, SLABS = CV == 1 ? NT / 64 : 1;
            const size_t lds = ((size_t)(SLABS + 1) * a.e + NT / 64) * 4;
            hipLaunchKernelGGL((k_balance_rows<T, LPR, CV, NT, U>), dim3(a.parts), dim3(NT), lds, st, a);
        };
        using std::integral_constant;
        // sixteen waves and several groups where there are rows and registers for them
        constexpr int MOST = CV == 1 ? 1024 : CV <= 4 ? 512 : 256;
        if (a.n <= 32 * a.parts)
            launch(integral_constant<int, 256>(), integral_constant<int, 1>());
        else
            launch(integral_constant<int, MOST>(), integral_constant<int, CV == 1 ? 4 : 1>());
    });
    hipLaunchKernelGGL(k_balance_join, dim3((a.e + 63) / 64), dim3(BJ_NT), 0, st, a);
    return hipGetLastError();
}

template <typename T>
static hipError_t balance_grad(const BalanceArgs& a, hipStream_t st) {
    with_row<T>(a.e, 1, [&](auto l, auto c) {
        constexpr int LPR = decltype(l)::value, CV = decltype(c)::value;
        auto launch = [&](auto groups) {
            constexpr int U = decltype(groups)::value;
            const int64_t per = BG_W * (64 / LPR) * U, blocks = (a.n + per - 1) / per;
            hipLaunchKernelGGL((k_balance_grad<T, LPR, CV, U>), dim3((unsigned)(blocks < bg_most(CV) ? blocks : bg_most(CV))),
                               dim3(64 * BG_W), 0, st, a);
        };
        using std::integral_constant;
        if (CV > 1 || a.n <= 256 * BG_W * (64 / LPR))
            launch(integral_constant<int, 1>());
        else
            launch(integral_constant<int, CV == 1 ? 4 : 1>());
    });
    return hipGetLastError();
}

}  // namespace gmm

using namespace gmm;

extern "C" {

size_t gmm_balance_loss_workspace_bytes(int64_t n, int32_t e, int32_t m) {
    if (!balance_ok(n, e, m) || !balance_fits(n, e, m)) return 0;
    const size_t parts = balance_parts(n);
    return bal_up(parts * e * sizeof(BalancePart)) + bal_up(parts * 4) + bal_up(64 * sizeof(BalanceSum)) + 256;
}

int gmm_balance_loss(const void* logits, int64_t n, int32_t e, int64_t ldz, int32_t dtype,
                     const int32_t* idx, int32_t m, float* loss, int32_t* counts, int64_t* totals,
                     float* prob, float* norm, void* workspace, size_t workspace_bytes, void* stream) {
    if (dtype != GMM_F32 && dtype != GMM_BF16) return GMM_E_DTYPE;
    if (!balance_ok(n, e, m) || ldz < e || !loss || !counts || !totals || !prob) return GMM_E_INVALID;
    if (n > 0 && (!logits || !idx || !norm)) return GMM_E_INVALID;
    if (!balance_fits(n, e, m)) return GMM_E_UNSUPPORTED;
    if (!workspace || workspace_bytes < gmm_balance_loss_workspace_bytes(n, e, m) ||
        (uintptr_t)workspace % 256 != 0)
        return GMM_E_WORKSPACE;
    BalanceArgs a{};
    a.z = logits;
    a.idx = idx;
    a.n = n;
    a.ldz = ldz;
    a.e = e;
    a.m = m;
    a.parts = balance_parts(n);
    a.norm = norm;
    a.loss = loss;
    a.prob = prob;
    a.counts = counts;
    a.totals = totals;
    char* ws = (char*)workspace;
    a.part = (BalancePart*)ws;
    ws += bal_up((size_t)a.parts * e * sizeof(BalancePart));
    a.part_rows = (int32_t*)ws;
    ws += bal_up((size_t)a.parts * 4);
    a.sum = (BalanceSum*)ws;
    a.done = (int32_t*)(ws + bal_up(64 * sizeof(BalanceSum)));
    const hipError_t err = dtype == GMM_F32 ? balance<float>(a, (hipStream_t)stream)
                                            : balance<uint16_t>(a, (hipStream_t)stream);
    return err == hipSuccess ? GMM_OK : GMM_E_HIP;
}

int gmm_balance_loss_backward(const void* logits, int64_t n, int32_t e, int64_t ldz, int32_t dtype,
                              const int32_t* counts, const int64_t* totals, const float* norm,
                              const float* g_loss, void* dlogits, int64_t lddz, void* stream) {
    if (dtype != GMM_F32 && dtype != GMM_BF16) return GMM_E_DTYPE;
    if (!balance_ok(n, e, 1) || ldz < e || lddz < e) return GMM_E_INVALID;
    if (!balance_fits(n, e, 1)) return GMM_E_UNSUPPORTED;
    if (n > 0 && (!logits || !counts || !totals || !norm || !dlogits)) return GMM_E_INVALID;
    if (n == 0) return GMM_OK;
    BalanceArgs a{};
    a.z = logits;
    a.dz = dlogits;
    a.n = n;
    a.ldz = ldz;
    a.lddz = lddz;
    a.e = e;
    a.counts = (int32_t*)counts;
    a.totals = (int64_t*)totals;
    a.norm = (float*)norm;
    a.g_loss = g_loss;
    const hipError_t err = dtype == GMM_F32 ? balance_grad<float>(a, (hipStream_t)stream)
                                            : balance_grad<uint16_t>(a, (hipStream_t)stream);
    return err == hipSuccess ? GMM_OK : GMM_E_HIP;
}

}  // extern "C"
