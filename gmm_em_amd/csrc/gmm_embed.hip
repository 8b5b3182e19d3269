// gmm_embed.hip - the embedding of codes and its gradient (gmm_embed,
// gmm_embed_backward, declared in include/gmm_em.h):
//   out[r] = scale table[c_r]          dT[c] = scale sum over r with c_r = c of g[r]
//
// The forward call is a gather of whole rows: a wave per row (or part of a long one).
//
// Gradient: the rows are sorted by code (stable, so that every sum has one order), cut
// into segments of 64 and summed segment by segment: the work of a segment does not depend
// on how often its codes occur. A run of one code that lies inside a segment is written
// from there; what a run leaves in each of several segments goes to the workspace and is
// added in order by k_embed_join. The sort is by digits of the code, lowest first:
//   k_embed_count: per tile of rows, how often each digit occurs
//   k_embed_place: the place of a tile's digits from everyone's counts, then its rows in
//                  order (one ballot per bit ranks 64 rows among those of the same digit)
// Codes that no row has are told by a bitmap and set to 0 by waves of the summing kernel.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "gmm_em.h"
#include "gmm_nn.h"
#include "gmm_softmax.h"

namespace gmm {

constexpr int32_t EMB_MAX_DIM = 1 << 20;
constexpr int32_t EMB_MAX_CODES = 1 << 22;   // as the head's
constexpr int64_t EMB_MAX_ROWS = 0x7fffffff;  // of a gradient: row numbers are 32-bit

// ---- forward

struct EmbedArgs {
    const void* table;
    const int32_t* codes;
    void* out;
    int64_t n, ldt, ldo;
    int32_t v, d;
    float scale;
};

// A vector's first value: one that would pass the row's end is the last whole one instead
// (the values that it shares with its neighbour are written twice, the same).
template <int VE>
__device__ __forceinline__ int whole(int k, int d) {
    return k + VE <= d || d < VE ? k : d - VE;
}

// VE values of a row from k = whole(k), or the fewer that a short row has.
template <typename T>
__device__ __forceinline__ Raw16 row_get(const T* x, int k, int d) {
    return d < Vec<T>::VE ? load_zero(x, k, (int64_t)d) : *reinterpret_cast<const Raw16*>(x + k);
}
template <typename T>
__device__ __forceinline__ void row_put(T* x, int k, int d, const Raw16& r) {
    if (d >= Vec<T>::VE) {
        *reinterpret_cast<Raw16*>(x + k) = r;
    } else {
#pragma unroll
        for (int u = 0; u < Vec<T>::VE; ++u)
            if (u < d) x[u] = Vec<T>::store(Vec<T>::get(r, u));
    }
}

constexpr int EMB_U = 4;  // vectors in flight per lane
template <typename T>
__global__ __launch_bounds__(256) void k_embed(EmbedArgs p) {
    constexpr int VE = Vec<T>::VE, SEG = 64 * VE * EMB_U;
    const int lane = threadIdx.x & 63;
    const int segs = (p.d + SEG - 1) / SEG;
    const int64_t items = p.n * segs;
    for (int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); item < items;
         item += (int64_t)gridDim.x * 4) {
        const int64_t row = segs == 1 ? item : item / segs;
        const int k0 = (int)(item - row * segs) * SEG + lane * VE;
        const int c = p.codes[row];
        const float none = c < 0 ? 0.f : NAN;  // what a row without a code holds
        const bool there = c >= 0 && c < p.v;
        const T* x = (const T*)p.table + (int64_t)(there ? c : 0) * p.ldt;
        T* y = (T*)p.out + row * p.ldo;
        Raw16 r[EMB_U];
#pragma unroll
        for (int u = 0; u < EMB_U; ++u) {
            const int k = k0 + u * 64 * VE;
            r[u] = Raw16{{0u, 0u, 0u, 0u}};
            if (k < p.d && there) r[u] = row_get(x, whole<VE>(k, p.d), p.d);
        }
#pragma unroll
        for (int u = 0; u < EMB_U; ++u) {
            const int k = k0 + u * 64 * VE;
            if (k >= p.d) continue;
            Raw16 o = {{0u, 0u, 0u, 0u}};
#pragma unroll
            for (int j = 0; j < VE; ++j)
                Vec<T>::set(o, j, there ? Vec<T>::get(r[u], j) * p.scale : none);
            row_put(y, whole<VE>(k, p.d), p.d, o);
        }
    }
}

// ---- the sort of the rows by code

constexpr int ES_BITS = 9, ES_BINS = 1 << ES_BITS;  // a digit
constexpr int ES_NT = 1024, ES_W = ES_NT / 64;
constexpr int ES_MAX_TILES = 256;

struct SortArgs {
    const int32_t* codes;            // of the caller (first digit), else keys
    const uint32_t *key_in, *row_in;
    uint32_t *key, *row;             // sorted by this digit and the ones before
    uint32_t* mat;                   // [tiles][ES_BINS]
    uint32_t* present;               // a bit for each code that occurs
    int64_t n, tile;                 // tile: rows per workgroup, a multiple of ES_NT
    int32_t v, tiles, shift, words;
};

// Sort key of row i: its code, or v where that is none (those rows come last).
__device__ __forceinline__ uint32_t sort_key(const SortArgs& p, int64_t i) {
    if (!p.codes) return p.key_in[i];
    const int c = p.codes[i];
    return c >= 0 && c < p.v ? (uint32_t)c : (uint32_t)p.v;
}

__global__ __launch_bounds__(ES_NT) void k_embed_count(SortArgs p) {
    __shared__ uint32_t h[ES_BINS];
    const int tid = threadIdx.x;
    if (p.codes)
        for (int64_t j = (int64_t)blockIdx.x * ES_NT + tid; j < p.words; j += (int64_t)gridDim.x * ES_NT)
            p.present[j] = 0;
    if (tid < ES_BINS) h[tid] = 0;
    __syncthreads();
    const int64_t b = blockIdx.x * p.tile, e = b + p.tile < p.n ? b + p.tile : p.n;
    for (int64_t i = b + tid; i < e; i += ES_NT)
        atomicAdd(&h[(sort_key(p, i) >> p.shift) & (ES_BINS - 1)], 1u);
    __syncthreads();
    if (tid < ES_BINS) p.mat[(int64_t)blockIdx.x * ES_BINS + tid] = h[tid];
}

__global__ __launch_bounds__(ES_NT) void k_embed_place(SortArgs p) {
    __shared__ uint32_t at[ES_W][ES_BINS];  // each wave's next place for a digit
    __shared__ uint32_t tot[2][ES_BINS], bef[2][ES_BINS], sums[ES_BINS / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int t0 = blockIdx.x;
    // how many rows of each digit there are, and how many in the tiles before
    {
        const int bin = tid & (ES_BINS - 1), half = tid >> ES_BITS;
        uint32_t all = 0, before = 0;
#pragma unroll 8
        for (int t = half; t < p.tiles; t += ES_NT / ES_BINS) {
            const uint32_t c = p.mat[(int64_t)t * ES_BINS + bin];
            all += c;
            before += t < t0 ? c : 0;
        }
        tot[half][bin] = all;
        bef[half][bin] = before;
    }
    for (int j = tid; j < ES_W * ES_BINS; j += ES_NT) (&at[0][0])[j] = 0;
    __syncthreads();
    // each wave counts its own stretch of the tile
    const int64_t per = p.tile / ES_W;
    const int64_t b = blockIdx.x * p.tile + wave * per;
    const int64_t e = b + per < p.n ? b + per : p.n;
    for (int64_t i = b + lane; i < e; i += 64)
        atomicAdd(&at[wave][(sort_key(p, i) >> p.shift) & (ES_BINS - 1)], 1u);
    uint32_t mine = 0, scan = 0;
    if (tid < ES_BINS) {
        mine = tot[0][tid] + tot[1][tid];
        scan = mine;  // prefix over the wave's 64 digits
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t up = __shfl_up(scan, o);
            scan += lane >= o ? up : 0;
        }
        if (lane == 63) sums[wave] = scan;
    }
    __syncthreads();
    if (tid < ES_BINS) {
        uint32_t run = scan - mine + bef[0][tid] + bef[1][tid];
        for (int w = 0; w < wave; ++w) run += sums[w];
        for (int w = 0; w < ES_W; ++w) {
            const uint32_t c = at[w][tid];
            at[w][tid] = run;
            run += c;
        }
    }
    __syncthreads();
    const uint64_t below = (uint64_t(1) << lane) - 1;
    for (int64_t i0 = b; i0 < e; i0 += 64) {
        const int64_t i = i0 + lane;
        const bool in = i < e;
        const uint32_t key = in ? sort_key(p, i) : 0;
        const uint32_t row = in ? (p.codes ? (uint32_t)i : p.row_in[i]) : 0;
        const uint32_t dig = (key >> p.shift) & (ES_BINS - 1);
        uint64_t same = __builtin_amdgcn_ballot_w64(in);
#pragma unroll
        for (int bit = 0; bit < ES_BITS; ++bit) {
            const bool set = (dig >> bit) & 1;
            const uint64_t m = __builtin_amdgcn_ballot_w64(set);
            same &= set ? m : ~m;
        }
        if (in) {
            const uint32_t first = at[wave][dig];
            const uint32_t to = first + __popcll(same & below);
            p.key[to] = key;
            p.row[to] = row;
            // one wave: its LDS accesses complete in order, so the reads above come first
            if ((same & below) == 0) at[wave][dig] = first + __popcll(same);
            if (p.codes && key < (uint32_t)p.v) {
                const uint32_t bit = 1u << (key & 31);
                uint32_t* word = p.present + (key >> 5);
                if (!(__hip_atomic_load(word, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) & bit))
                    atomicOr(word, bit);
            }
        }
    }
}

// ---- the sums

constexpr int EG_SEG = 64;  // sorted rows of a segment: one per lane
constexpr int EG_U = 8;     // rows in flight

struct EmbedGradArgs {
    const void* g;
    void* out;
    const uint32_t *key, *row, *present;
    float* part;  // [segments][2][dp]: the segment's share of a run from before, and of one that goes on
    int64_t n, ldg, ldt, segs;
    int32_t v, d, dp, cols;  // cols: blocks of 64 VE dims
    float scale;
};

template <typename T>
__device__ __forceinline__ void embed_out(const EmbedGradArgs& p, uint32_t code, int k, const float* acc) {
    constexpr int VE = Vec<T>::VE;
    Raw16 o = {{0u, 0u, 0u, 0u}};
#pragma unroll
    for (int j = 0; j < VE; ++j) Vec<T>::set(o, j, acc[j] * p.scale);
    row_put((T*)p.out + code * p.ldt, k, p.d, o);
}

template <typename T>
__global__ __launch_bounds__(256) void k_embed_sum(EmbedGradArgs p) {
    constexpr int VE = Vec<T>::VE;
    const int lane = threadIdx.x & 63;
    const int64_t work = p.segs * p.cols, zero = (p.v + 63) / 64;
    for (int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); item < work + zero;
         item += (int64_t)gridDim.x * 4) {
        if (item >= work) {
            // 64 codes: those that no row has
            const int c0 = (int)(item - work) * 64;
            const int c = c0 + lane;
            const bool none = c < p.v && !((p.present[c >> 5] >> (c & 31)) & 1);
            uint64_t left = __builtin_amdgcn_ballot_w64(none);
            const Raw16 zeros = {{0u, 0u, 0u, 0u}};
            while (left) {
                const int j = __builtin_ctzll(left);
                left &= left - 1;
                T* y = (T*)p.out + (int64_t)(c0 + j) * p.ldt;
                for (int k = lane * VE; k < p.d; k += 64 * VE) row_put(y, whole<VE>(k, p.d), p.d, zeros);
            }
            continue;
        }
        const int64_t seg = item / p.cols;
        const int kc = (int)(item - seg * p.cols) * 64 * VE + lane * VE;
        const bool has = kc < p.d;
        const int k = whole<VE>(kc, p.d);
        const int64_t i0 = seg * EG_SEG;
        const bool in = i0 + lane < p.n;
        const uint32_t key = in ? p.key[i0 + lane] : (uint32_t)p.v;
        const uint32_t row = in ? p.row[i0 + lane] : 0;
        const uint32_t before = i0 > 0 ? p.key[i0 - 1] : 0xffffffffu;
        const uint32_t after = i0 + EG_SEG < p.n ? p.key[i0 + EG_SEG] : 0xffffffffu;
        const int cnt = __popcll(__builtin_amdgcn_ballot_w64(key < (uint32_t)p.v));
        float acc[VE];
#pragma unroll
        for (int j = 0; j < VE; ++j) acc[j] = 0.f;
        bool whole_run = true;  // the run began in this segment
        for (int j0 = 0; j0 < cnt; j0 += EG_U) {
            Raw16 r[EG_U];
#pragma unroll
            for (int u = 0; u < EG_U; ++u) {
                const uint32_t at = (uint32_t)__builtin_amdgcn_readlane((int)row, j0 + u < cnt ? j0 + u : cnt - 1);
                r[u] = Raw16{{0u, 0u, 0u, 0u}};
                if (has) r[u] = row_get((const T*)p.g + (int64_t)at * p.ldg, k, p.d);
            }
#pragma unroll
            for (int u = 0; u < EG_U; ++u) {
                const int j = j0 + u;
                if (j >= cnt) break;
                const uint32_t code = (uint32_t)__builtin_amdgcn_readlane((int)key, j);
                const uint32_t next = j + 1 < EG_SEG
                                          ? (uint32_t)__builtin_amdgcn_readlane((int)key, j + 1 < 64 ? j + 1 : 63)
                                          : after;
                if (j == 0) whole_run = code != before;
#pragma unroll
                for (int q = 0; q < VE; ++q) acc[q] += Vec<T>::get(r[u], q);
                if (next == code && j + 1 < EG_SEG) continue;
                if (has) {
                    if (whole_run && next != code) {
                        embed_out<T>(p, code, k, acc);
                    } else {
                        float* to = p.part + (seg * 2 + (whole_run ? 1 : 0)) * p.dp + kc;
#pragma unroll
                        for (int q = 0; q < VE; ++q) to[q] = acc[q];
                    }
                }
#pragma unroll
                for (int q = 0; q < VE; ++q) acc[q] = 0.f;
                whole_run = true;
            }
        }
    }
}

// Adds what a run left in its segments, in their order: a workgroup per segment (and 64 VE
// dims) in which a run begins that goes on; its waves share the run's segments.
constexpr int EJ_W = 4;
template <typename T>
__global__ __launch_bounds__(64 * EJ_W) void k_embed_join(EmbedGradArgs p) {
    constexpr int VE = Vec<T>::VE;
    __shared__ float sh[EJ_W][64][VE + 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int kc = blockIdx.y * 64 * VE + lane * VE;
    const bool has = kc < p.d;
    for (int64_t seg = blockIdx.x; seg + 1 < p.segs; seg += gridDim.x) {
        const int64_t i0 = seg * EG_SEG, last = i0 + EG_SEG - 1;
        const uint32_t code = p.key[last];
        if (code >= (uint32_t)p.v || p.key[last + 1] != code) continue;
        if (p.key[i0] == code && i0 > 0 && p.key[i0 - 1] == code) continue;  // began before
        int64_t end = seg + 1;  // first segment that does not begin with this code
        for (;;) {
            const int64_t t = end + lane;
            const bool on = t < p.segs && p.key[t * EG_SEG] == code;
            const uint64_t m = __builtin_amdgcn_ballot_w64(on);
            end += __popcll(m);
            if (m != ~uint64_t(0)) break;
        }
        // shares of segments seg (its second) and seg + 1 .. end - 1 (their first)
        const int64_t count = end - seg;
        const int64_t a = count * wave / EJ_W, z = count * (wave + 1) / EJ_W;
        float acc[VE];
#pragma unroll
        for (int q = 0; q < VE; ++q) acc[q] = 0.f;
        if (has) {
#pragma unroll 4
            for (int64_t t = a; t < z; ++t) {
                const float* from = p.part + ((seg + t) * 2 + (t == 0 ? 1 : 0)) * p.dp + kc;
#pragma unroll
                for (int q = 0; q < VE; ++q) acc[q] += from[q];
            }
        }
#pragma unroll
        for (int q = 0; q < VE; ++q) sh[wave][lane][q] = acc[q];
        __syncthreads();
        if (wave == 0 && has) {
#pragma unroll
            for (int q = 0; q < VE; ++q) {
                float s = sh[0][lane][q];
#pragma unroll
                for (int w = 1; w < EJ_W; ++w) s += sh[w][lane][q];
                acc[q] = s;
            }
            embed_out<T>(p, code, whole<VE>(kc, p.d), acc);
        }
        __syncthreads();
    }
}

struct EmbedPlan {
    int32_t passes, tiles, words, dp;
    int64_t tile, segs;
    size_t o_key[2], o_row[2], o_mat, o_present, o_part, bytes;
};
static EmbedPlan embed_plan(int64_t n, int32_t d, int32_t v) {
    EmbedPlan q{};
    const int bits = 32 - __builtin_clz((unsigned)v);  // of keys 0 .. v
    q.passes = (bits + ES_BITS - 1) / ES_BITS;
    q.tile = ES_NT;
    while ((n + q.tile - 1) / q.tile > ES_MAX_TILES) q.tile *= 2;
    q.tiles = (int32_t)((n + q.tile - 1) / q.tile);
    q.segs = (n + EG_SEG - 1) / EG_SEG;
    q.words = (v + 31) / 32 + 1;  // 64 codes are looked at at a time
    q.dp = (d + 7) / 8 * 8;
    size_t off = 0;
    auto take = [&](size_t b) {
        const size_t o = off;
        off += (b + 255) & ~(size_t)255;
        return o;
    };
    for (int i = 0; i < 2; ++i) {
        q.o_key[i] = take((size_t)n * 4);
        q.o_row[i] = take((size_t)n * 4);
    }
    q.o_mat = take((size_t)q.tiles * ES_BINS * 4);
    q.o_present = take((size_t)q.words * 4);
    q.o_part = take((size_t)q.segs * 2 * q.dp * 4);
    q.bytes = off < 256 ? 256 : off;
    return q;
}

static unsigned grid_of(int64_t blocks) {
    const int64_t most = (int64_t)1 << 20;
    return (unsigned)(blocks < most ? blocks : most);
}

template <typename T>
static hipError_t embed_grad(EmbedGradArgs a, const EmbedPlan& q, const int32_t* codes, char* ws, hipStream_t st) {
    SortArgs s{};
    s.mat = (uint32_t*)(ws + q.o_mat);
    s.present = (uint32_t*)(ws + q.o_present);
    s.n = a.n;
    s.tile = q.tile;
    s.v = a.v;
    s.tiles = q.tiles;
    s.words = q.words;
    for (int i = 0; i < q.passes; ++i) {
        s.codes = i == 0 ? codes : nullptr;
        s.key_in = s.key;
        s.row_in = s.row;
        s.key = (uint32_t*)(ws + q.o_key[i & 1]);
        s.row = (uint32_t*)(ws + q.o_row[i & 1]);
        s.shift = i * ES_BITS;
        hipLaunchKernelGGL(k_embed_count, dim3(q.tiles), dim3(ES_NT), 0, st, s);
        hipLaunchKernelGGL(k_embed_place, dim3(q.tiles), dim3(ES_NT), 0, st, s);
    }
    a.key = s.key;
    a.row = s.row;
    a.present = s.present;
    a.part = (float*)(ws + q.o_part);
    a.segs = q.segs;
    a.dp = q.dp;
    const int block = 64 * Vec<T>::VE;
    a.cols = (a.d + block - 1) / block;
    const int64_t waves = a.segs * a.cols + (a.v + 63) / 64;
    hipLaunchKernelGGL((k_embed_sum<T>), dim3(grid_of((waves + 3) / 4)), dim3(256), 0, st, a);
    if (a.segs > 1)
        hipLaunchKernelGGL((k_embed_join<T>), dim3(grid_of(a.segs - 1), a.cols), dim3(64 * EJ_W), 0, st, a);
    return hipGetLastError();
}

// the gradient of no rows
template <typename T>
__global__ __launch_bounds__(256) void k_embed_zero(T* out, int64_t rows, int d, int64_t ld) {
    for (int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x; j < rows * d; j += (int64_t)gridDim.x * 256)
        out[j / d * ld + j % d] = 0;
}

}  // namespace gmm

using namespace gmm;

extern "C" {

int gmm_embed(const void* table, int32_t v, int32_t d, int64_t ldt, int32_t dtype,
              const int32_t* codes, int64_t n, float scale, void* out, int64_t ldo, void* stream) {
    if (dtype != GMM_F32 && dtype != GMM_BF16) return GMM_E_DTYPE;
    if (n < 0 || n > SC_MAX_ROWS || v < 1 || d < 1 || ldt < d || ldo < d || !isfinite(scale))
        return GMM_E_INVALID;
    if (d > EMB_MAX_DIM || v > EMB_MAX_CODES) return GMM_E_UNSUPPORTED;
    if (n > 0 && (!table || !codes || !out)) return GMM_E_INVALID;
    if (n == 0) return GMM_OK;
    const EmbedArgs a{table, codes, out, n, ldt, ldo, v, d, scale};
    const int seg = 64 * EMB_U * (dtype == GMM_F32 ? 4 : 8);
    const dim3 grid(grid_of((n * ((d + seg - 1) / seg) + 3) / 4));
    if (dtype == GMM_F32)
        hipLaunchKernelGGL((k_embed<float>), grid, dim3(256), 0, (hipStream_t)stream, a);
    else
        hipLaunchKernelGGL((k_embed<uint16_t>), grid, dim3(256), 0, (hipStream_t)stream, a);
    return hipGetLastError() == hipSuccess ? GMM_OK : GMM_E_HIP;
}

size_t gmm_embed_backward_workspace_bytes(int64_t n, int32_t d, int32_t v) {
    if (n < 0 || n > EMB_MAX_ROWS || d < 1 || d > EMB_MAX_DIM || v < 1 || v > EMB_MAX_CODES) return 0;
    return embed_plan(n, d, v).bytes;
}

int gmm_embed_backward(const void* grad, int64_t n, int32_t d, int64_t ldg, int32_t dtype,
                       const int32_t* codes, int32_t v, float scale, void* d_table, int64_t ldt,
                       void* workspace, size_t workspace_bytes, void* stream) {
    if (dtype != GMM_F32 && dtype != GMM_BF16) return GMM_E_DTYPE;
    if (n < 0 || v < 1 || d < 1 || ldg < d || ldt < d || !isfinite(scale) || !d_table)
        return GMM_E_INVALID;
    if (n > EMB_MAX_ROWS || d > EMB_MAX_DIM || v > EMB_MAX_CODES) return GMM_E_UNSUPPORTED;
    if (n > 0 && (!grad || !codes)) return GMM_E_INVALID;
    const EmbedPlan q = embed_plan(n, d, v);
    if (!workspace || workspace_bytes < q.bytes || (uintptr_t)workspace % 256 != 0)
        return GMM_E_WORKSPACE;
    hipStream_t st = (hipStream_t)stream;
    if (n == 0) {
        const dim3 grid(grid_of(((int64_t)v * d + 1023) / 1024));
        if (dtype == GMM_F32)
            hipLaunchKernelGGL((k_embed_zero<float>), grid, dim3(256), 0, st, (float*)d_table, (int64_t)v, d, ldt);
        else
            hipLaunchKernelGGL((k_embed_zero<uint16_t>), grid, dim3(256), 0, st, (uint16_t*)d_table, (int64_t)v, d, ldt);
        return hipGetLastError() == hipSuccess ? GMM_OK : GMM_E_HIP;
    }
    EmbedGradArgs a{};
    a.g = grad;
    a.out = d_table;
    a.n = n;
    a.ldg = ldg;
    a.ldt = ldt;
    a.v = v;
    a.d = d;
    a.scale = scale;
    const hipError_t e = dtype == GMM_F32 ? embed_grad<float>(a, q, codes, (char*)workspace, st)
                                          : embed_grad<uint16_t>(a, q, codes, (char*)workspace, st);
    return e == hipSuccess ? GMM_OK : GMM_E_HIP;
}

}  // extern "C"
