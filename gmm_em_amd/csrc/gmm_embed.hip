// gmm_embed.hip - the embedding of codes and its gradient (gmm_embed,
// gmm_embed_backward, declared in include/gmm_em.h):
//   out[r] = scale table[c_r]          dT[c] = scale sum over r with c_r = c of g[r]
//
// The forward call is a gather of whole rows: a wave per row (or part of a long one).
//
// Gradient: the rows are sorted by code (stable, so that every sum has one order), cut
// into segments of 8 to 64 and summed segment by segment: the work of a segment does not depend
// on how often its codes occur. A run of one code that lies inside a segment is written
// from there; what a run leaves in each of several segments goes to the workspace and is
// added in order by k_embed_join. The sort is by digits of the code, lowest first:
//   k_embed_count: per tile of rows, how often each digit occurs
//   k_embed_place: the place of a tile's digits from everyone's counts, then its rows in
//                  order (one ballot per bit ranks 64 rows among those of the same digit)
// Codes that no row has are found in the sorted keys and set to 0 by waves of the summing
// kernel. Up to 4096 rows are sorted by one workgroup (k_embed_sort); up to 1024 take one launch
// instead of all this (k_embed_few): the first row of a code adds the others.
// The sum is bound by reading the rows and writing the table, everything else by the latency of
// short kernels. 65536 x 768 bf16 against 16384 codes of uneven frequency, 57 us a call (52 where the caches
// still hold part of the rows): counts 2 x 3, places 2 x 6.5, sums 25 (126 MB, 5.0 TB/s), join 9.5. 4096 rows 27
// (sorted by four launches and their codes without rows found by the sum, 34), 2048 rows 27 (sort 13 beside the
// zeros, sums 6, join 8), 1024 rows 10.5.
// Not kept: a bitmap of the codes that occur (its atomics took 65 us), segments joined by a
// workgroup each (19 us).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "gmm_em.h"
#include "gmm_nn.h"
#include "gmm_search.h"
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
            float o[VE];
#pragma unroll
            for (int j = 0; j < VE; ++j) o[j] = there ? Vec<T>::get(r[u], j) * p.scale : none;
            row_put(y, whole<VE>(k, p.d), p.d, pack16<T>(o));
        }
    }
}

// ---- the sort of the rows by code

constexpr int ES_BITS = 10, ES_BINS = 1 << ES_BITS;  // a digit, at most
constexpr int ES_NT = 1024, ES_W = ES_NT / 64;
constexpr int ES_MAX_TILES = 256;

struct SortArgs {
    const int32_t* codes;            // of the caller (first digit), else keys
    const uint32_t *key_in, *row_in;
    uint32_t *key, *row;             // sorted by this digit and the ones before
    uint32_t* mat;                   // [tiles][2^bits]
    int64_t n, tile;                 // tile: rows per workgroup, a multiple of ES_NT
    int32_t v, tiles, shift;
    int32_t bits;                    // of a digit (k_embed_sort: of a key)
};

// Sort key of row i: its code, or v where that is none (those rows come last).
__device__ __forceinline__ uint32_t sort_key(const SortArgs& p, int64_t i) {
    if (!p.codes) return p.key_in[i];
    const int c = p.codes[i];
    return c >= 0 && c < p.v ? (uint32_t)c : (uint32_t)p.v;
}

__global__ __launch_bounds__(ES_NT) void k_embed_count(SortArgs p) {
    __shared__ uint32_t h[ES_BINS];
    const int tid = threadIdx.x, bins = 1 << p.bits;
    h[tid] = 0;
    __syncthreads();
    const int64_t b = blockIdx.x * p.tile, e = b + p.tile < p.n ? b + p.tile : p.n;
    for (int64_t i = b + tid; i < e; i += ES_NT) atomicAdd(&h[(sort_key(p, i) >> p.shift) & (bins - 1)], 1u);
    __syncthreads();
    if (tid < bins) p.mat[(int64_t)blockIdx.x * bins + tid] = h[tid];
}

__global__ __launch_bounds__(ES_NT) void k_embed_place(SortArgs p) {
    __shared__ uint32_t at[ES_W][ES_BINS];  // each wave's next place for a digit
    __shared__ uint32_t tot[ES_NT], bef[ES_NT], sums[ES_BINS / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int t0 = blockIdx.x, bins = 1 << p.bits, per_bin = ES_NT >> p.bits;
    // how many rows of each digit there are, and how many in the tiles before
    {
        const int bin = tid & (bins - 1);
        uint32_t all = 0, before = 0;
#pragma unroll 8
        for (int t = tid >> p.bits; t < p.tiles; t += per_bin) {
            const uint32_t c = p.mat[(int64_t)t * bins + bin];
            all += c;
            before += t < t0 ? c : 0;
        }
        tot[tid] = all;
        bef[tid] = before;
    }
    // each wave counts its own stretch of the tile
    for (int j = lane; j < bins; j += 64) at[wave][j] = 0;
    const int64_t per = p.tile / ES_W;
    const int64_t b = blockIdx.x * p.tile + wave * per;
    const int64_t e = b + per < p.n ? b + per : p.n;
    for (int64_t i = b + lane; i < e; i += 64) atomicAdd(&at[wave][(sort_key(p, i) >> p.shift) & (bins - 1)], 1u);
    __syncthreads();
    uint32_t mine = 0, scan = 0;
    if (tid < bins) {
        for (int q = 0; q < per_bin; ++q) mine += tot[q * bins + tid];
        scan = mine;  // prefix over the wave's 64 digits
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t up = __shfl_up(scan, o);
            scan += lane >= o ? up : 0;
        }
        if (lane == 63) sums[wave] = scan;
    }
    __syncthreads();
    if (tid < bins) {
        uint32_t run = scan - mine;
        for (int q = 0; q < per_bin; ++q) run += bef[q * bins + tid];
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
        const uint32_t dig = (key >> p.shift) & (bins - 1);
        uint64_t same = __builtin_amdgcn_ballot_w64(in);
        for (int bit = 0; bit < p.bits; ++bit) {
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
        }
    }
}

// ---- the sums

constexpr int EG_U = 8;     // rows in flight
// Waves below which the segments get shorter. 65536 x 768 against 16384 codes: bf16 51 us with
// segments of 32 (57 with 64, 62 with 16), fp32 66 with 64 (73 with 32).
constexpr int EG_WAVES = 2400;

struct EmbedGradArgs {
    const void* g;
    void* out;
    const int32_t* codes;
    const uint32_t *key, *row;
    float* part;  // [segments][2][dp]: the segment's share of a run from before, and of one that goes on
    int64_t n, ldg, ldt, segs;
    int32_t seg;          // sorted rows of a segment, at most one per lane
    int32_t v, d, dp;
    int32_t cols, width;  // a row's blocks of `width` vectors, one per lane
    int32_t zero;         // k_embed_sum: waves that look for codes without rows
    float scale;
};

template <typename T>
__device__ __forceinline__ void embed_out(const EmbedGradArgs& p, uint32_t code, int k, const float* acc) {
    constexpr int VE = Vec<T>::VE;
    float o[VE];
#pragma unroll
    for (int j = 0; j < VE; ++j) o[j] = acc[j] * p.scale;
    row_put((T*)p.out + code * p.ldt, k, p.d, pack16<T>(o));
}

// A row of zeros, by a wave.
template <typename T>
__device__ __forceinline__ void embed_zero_row(const EmbedGradArgs& p, int64_t code, int lane) {
    constexpr int VE = Vec<T>::VE;
    T* y = (T*)p.out + code * p.ldt;
    for (int k = lane * VE; k < p.d; k += 64 * VE) row_put(y, whole<VE>(k, p.d), p.d, Raw16{{0u, 0u, 0u, 0u}});
}

// Sets those of the codes [c0, c0 + EF_ZERO) to 0 that none of n rows has; W waves, `seen`: EF_ZERO
// words of LDS.
constexpr int EF_ZERO = 64;
template <typename T, int W>
__device__ __forceinline__ void embed_zero_absent(const EmbedGradArgs& p, int n, int64_t c0, uint32_t* seen, int tid) {
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    if (tid < EF_ZERO) seen[tid] = 0;
    __syncthreads();
#pragma unroll 4
    for (int i = tid; i < n; i += 64 * W) {
        const int64_t c = (int64_t)p.codes[i] - c0;
        if (c >= 0 && c < EF_ZERO) seen[c] = 1;
    }
    __syncthreads();
    uint64_t left = __builtin_amdgcn_ballot_w64(c0 + lane < p.v && seen[lane] == 0);
    for (int k = 0; left; left &= left - 1, ++k)
        if (k % W == wave) embed_zero_row<T>(p, c0 + __builtin_ctzll(left), lane);
}

// All rows in one workgroup, in LDS, for up to EO_ROWS of them: each wave has its own stretch of the
// rows, as in k_embed_place, and the digits are short. The other workgroups set codes without rows
// to 0 meanwhile.
constexpr int EO_ROWS = 4096, EO_PER = EO_ROWS / ES_NT, EO_BITS = 8, EO_BINS = 1 << EO_BITS;
template <typename T>
__global__ __launch_bounds__(ES_NT) void k_embed_sort(SortArgs p, EmbedGradArgs g) {
    __shared__ uint2 buf[EO_ROWS];               // key, row
    __shared__ uint32_t at[ES_W][EO_BINS], sums[EO_BINS / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = (int)p.n;
    if (blockIdx.x > 0) {
        embed_zero_absent<T, ES_W>(g, n, (int64_t)(blockIdx.x - 1) * EF_ZERO, &at[0][0], tid);
        return;
    }
    const int chunks = (n + ES_NT - 1) / ES_NT;  // of 64 rows, for each wave
    const int b = wave * chunks * 64;
    const uint64_t below = (uint64_t(1) << lane) - 1;
    uint2 e[EO_PER];
#pragma unroll
    for (int j = 0; j < EO_PER; ++j) {
        const int i = b + j * 64 + lane;
        e[j] = j < chunks && i < n ? uint2{sort_key(p, i), (uint32_t)i} : uint2{0, 0};
    }
    for (int shift = 0; shift < p.bits; shift += EO_BITS) {
        for (int k = lane; k < EO_BINS; k += 64) at[wave][k] = 0;
#pragma unroll
        for (int j = 0; j < EO_PER; ++j)
            if (j < chunks && b + j * 64 + lane < n) atomicAdd(&at[wave][(e[j].x >> shift) & (EO_BINS - 1)], 1u);
        __syncthreads();
        uint32_t mine = 0, scan = 0;
        if (tid < EO_BINS) {
#pragma unroll
            for (int w = 0; w < ES_W; ++w) mine += at[w][tid];
            scan = mine;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const uint32_t up = __shfl_up(scan, o);
                scan += lane >= o ? up : 0;
            }
            if (lane == 63) sums[wave] = scan;
        }
        __syncthreads();
        if (tid < EO_BINS) {
            uint32_t run = scan - mine;
            for (int w = 0; w < wave; ++w) run += sums[w];
#pragma unroll
            for (int w = 0; w < ES_W; ++w) {
                const uint32_t c = at[w][tid];
                at[w][tid] = run;
                run += c;
            }
        }
        __syncthreads();
        for (int j = 0; j < chunks; ++j) {
            const bool in = b + j * 64 + lane < n;
            uint2 mineof = e[0];
#pragma unroll
            for (int k = 1; k < EO_PER; ++k) mineof = k == j ? e[k] : mineof;
            const uint32_t dig = (mineof.x >> shift) & (EO_BINS - 1);
            uint64_t same = __builtin_amdgcn_ballot_w64(in);
#pragma unroll
            for (int bit = 0; bit < EO_BITS; ++bit) {
                const bool set = (dig >> bit) & 1;
                const uint64_t m = __builtin_amdgcn_ballot_w64(set);
                same &= set ? m : ~m;
            }
            if (in) {
                const uint32_t first = at[wave][dig];
                buf[first + __popcll(same & below)] = mineof;
                if ((same & below) == 0) at[wave][dig] = first + __popcll(same);
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < EO_PER; ++j) {
            const int i = b + j * 64 + lane;
            if (j < chunks && i < n) e[j] = buf[i];
        }
    }
#pragma unroll
    for (int j = 0; j < EO_PER; ++j) {
        const int i = b + j * 64 + lane;
        if (j < chunks && i < n) {
            p.key[i] = e[j].x;
            p.row[i] = e[j].y;
        }
    }
}

// Loads rows j0 .. j0 + EG_U - 1 of a list of cnt > j0, this lane's VE dims of each. Places from cnt on hold the
// list's last row once more (no branch around a load): the caller leaves them out.
template <typename T, typename F>
__device__ __forceinline__ void embed_rows(const EmbedGradArgs& p, bool has, int k, int j0, int cnt, F row_of,
                                           Raw16* r) {
#pragma unroll
    for (int u = 0; u < EG_U; ++u) {
        const uint32_t at = row_of(j0 + u < cnt ? j0 + u : cnt - 1);
        r[u] = Raw16{{0u, 0u, 0u, 0u}};
        if (has) r[u] = row_get((const T*)p.g + (int64_t)at * p.ldg, k, p.d);
    }
}

// Of the codes [c0, c0 + EZ_CODES), a bit for each that the sorted keys do not hold. Four lanes look
// for a code's first place, at four places at a time: 7 steps for 65536 keys.
constexpr int EZ_CODES = 16;
__device__ __forceinline__ uint32_t absent_codes(const EmbedGradArgs& p, uint32_t c0, int lane) {
    const uint32_t c = c0 + (lane >> 2);
    Search at{0, p.n};
    while (__builtin_amdgcn_ballot_w64(at.lo < at.hi)) {
        const int64_t probe = at.place(lane & 3);
        const bool below = at.inside(probe) && p.key[probe] < c;
        at.narrow(__popc((uint32_t)(__builtin_amdgcn_ballot_w64(below) >> (lane & ~3)) & 15u));
    }
    const uint64_t none = __builtin_amdgcn_ballot_w64(at.lo >= p.n || p.key[at.lo] != c);
    uint32_t absent = 0;
#pragma unroll
    for (int j = 0; j < EZ_CODES; ++j) absent |= (uint32_t)(none >> (4 * j) & 1) << j;
    return absent;
}

template <typename T>
__global__ __launch_bounds__(256) void k_embed_sum(EmbedGradArgs p) {
    constexpr int VE = Vec<T>::VE;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // the codes without rows come first: their search takes longest
    const int64_t zero = p.zero, items = p.segs * p.cols + zero;
    for (int64_t item = (int64_t)blockIdx.x * 4 + wave - zero; item < items - zero; item += (int64_t)gridDim.x * 4) {
        if (item < 0) {
            const uint32_t c0 = (uint32_t)((item + zero) * EZ_CODES);
            const uint32_t absent = absent_codes(p, c0, lane);
#pragma unroll 1
            for (int j = 0; j < EZ_CODES; ++j)
                if ((absent >> j & 1) && c0 + j < (uint32_t)p.v) embed_zero_row<T>(p, c0 + j, lane);
            continue;
        }
        const int64_t seg = item / p.cols;
        const int kc = ((int)(item - seg * p.cols) * p.width + lane) * VE;
        const bool has = lane < p.width && kc < p.d;
        const int k = whole<VE>(kc, p.d);
        const int64_t i0 = seg * p.seg;
        const bool in = lane < p.seg && i0 + lane < p.n;
        const uint32_t key = in ? p.key[i0 + lane] : (uint32_t)p.v;
        const uint32_t row = in ? p.row[i0 + lane] : 0;
        const uint32_t before = i0 > 0 ? p.key[i0 - 1] : 0xffffffffu;
        const uint32_t after = i0 + p.seg < p.n ? p.key[i0 + p.seg] : 0xffffffffu;
        const int cnt = __popcll(__builtin_amdgcn_ballot_w64(key < (uint32_t)p.v));
        auto key_at = [&](int j) { return (uint32_t)__builtin_amdgcn_readlane((int)key, j); };
        auto row_at = [&](int j) { return (uint32_t)__builtin_amdgcn_readlane((int)row, j); };
        float acc[VE];
#pragma unroll
        for (int j = 0; j < VE; ++j) acc[j] = 0.f;
        bool began = key_at(0) != before;  // the run began in this segment
        for (int j0 = 0; j0 < cnt; j0 += EG_U) {
            Raw16 r[EG_U];
            embed_rows<T>(p, has, k, j0, cnt, row_at, r);
#pragma unroll
            for (int u = 0; u < EG_U; ++u) {
                const int j = j0 + u;
                if (j >= cnt) break;
#pragma unroll
                for (int q = 0; q < VE; ++q) acc[q] += Vec<T>::get(r[u], q);
                const uint32_t code = key_at(j);
                const bool last = j + 1 == p.seg;
                const uint32_t next = last ? after : key_at(j + 1 < 64 ? j + 1 : 63);
                if (next == code && !last) continue;
                if (has) {
                    if (began && next != code) {
                        embed_out<T>(p, code, k, acc);
                    } else {
                        float* to = p.part + (seg * 2 + (began ? 1 : 0)) * p.dp + kc;
#pragma unroll
                        for (int q = 0; q < VE; ++q) to[q] = acc[q];
                    }
                }
#pragma unroll
                for (int q = 0; q < VE; ++q) acc[q] = 0.f;
                began = true;
            }
        }
    }
}

// The sum of the waves' acc, in their order, in wave 0's. All threads call it.
template <int W, int VE>
__device__ __forceinline__ void join_waves(float (*sh)[64][VE + 1], float* acc, int wave, int lane) {
#pragma unroll
    for (int q = 0; q < VE; ++q) sh[wave][lane][q] = acc[q];
    __syncthreads();
    if (wave == 0) {
#pragma unroll
        for (int w = 1; w < W; ++w)
#pragma unroll
            for (int q = 0; q < VE; ++q) acc[q] += sh[w][lane][q];
    }
}

// acc += shares [a, z) of the run that begins in segment seg, in order: that segment's second
// slot, then the first slots of those that follow.
template <int VE>
__device__ __forceinline__ void embed_shares(const EmbedGradArgs& p, int64_t seg, int64_t a, int64_t z, int kc,
                                             float* acc) {
#pragma unroll 8
    for (int64_t t = a; t < z; ++t) {
        const float* from = p.part + ((seg + t) * 2 + (t == 0 ? 1 : 0)) * p.dp + kc;
#pragma unroll
        for (int q = 0; q < VE; ++q) acc[q] += from[q];
    }
}

// Adds what a run left in its segments, in their order. A wave per segment (and block of dims)
// looks whether a run begins in it that goes on and adds up to EJ_FEW shares itself; the waves of
// its workgroup share longer runs.
constexpr int EJ_W = 16, EJ_FEW = 8;
template <typename T>
__global__ __launch_bounds__(64 * EJ_W) void k_embed_join(EmbedGradArgs p) {
    constexpr int VE = Vec<T>::VE;
    __shared__ float sh[EJ_W][64][VE + 1];
    __shared__ int64_t lengths[EJ_W];
    __shared__ uint32_t codes[EJ_W];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kc = (blockIdx.y * p.width + lane) * VE;
    const bool has = lane < p.width && kc < p.d;
    for (int64_t base = (int64_t)blockIdx.x * EJ_W; base + 1 < p.segs; base += (int64_t)gridDim.x * EJ_W) {
        const int64_t seg = base + wave;
        int64_t count = 0;
        uint32_t code = 0;
        float acc[VE];
#pragma unroll
        for (int q = 0; q < VE; ++q) acc[q] = 0.f;
        if (seg + 1 < p.segs) {
            const int64_t i0 = seg * p.seg, last = i0 + p.seg - 1;
            code = p.key[last];
            const uint32_t next = p.key[last + 1], first = p.key[i0], before = i0 > 0 ? p.key[i0 - 1] : 0xffffffffu;
            auto begins = [&](int64_t t) { return t < p.segs && p.key[t * p.seg] == code; };
            uint64_t on = __builtin_amdgcn_ballot_w64(begins(seg + 1 + lane));
            if (code < (uint32_t)p.v && next == code && !(first == code && before == code)) {
                count = 1 + (on == ~uint64_t(0) ? 64 : __builtin_ctzll(~on));  // segments that the run lies in
                while (on == ~uint64_t(0)) {
                    on = __builtin_amdgcn_ballot_w64(begins(seg + count + lane));
                    count += __popcll(on);
                }
            }
        }
        if (count > 0 && count <= EJ_FEW && has) {
            embed_shares<VE>(p, seg, 0, count, kc, acc);
            embed_out<T>(p, code, whole<VE>(kc, p.d), acc);
        }
        if (lane == 0) {
            lengths[wave] = count > EJ_FEW ? count : 0;
            codes[wave] = code;
        }
        __syncthreads();
        for (int w = 0; w < EJ_W; ++w) {
            const int64_t n = lengths[w];
            if (n == 0) continue;
#pragma unroll
            for (int q = 0; q < VE; ++q) acc[q] = 0.f;
            if (has) embed_shares<VE>(p, base + w, n * wave / EJ_W, n * (wave + 1) / EJ_W, kc, acc);
            join_waves<EJ_W, VE>(sh, acc, wave, lane);
            if (wave == 0 && has) embed_out<T>(p, codes[w], whole<VE>(kc, p.d), acc);
            __syncthreads();
        }
        __syncthreads();
    }
}

// Up to EF_ROWS rows in one launch: a workgroup per row (and block of dims) looks for its code
// among all rows; the code's first row adds them, the waves sharing its list. The first
// workgroups set EF_ZERO codes each to 0 where no row has them.
constexpr int EF_ROWS = 1024, EF_W = 4, EF_NT = 64 * EF_W;
template <typename T>
__global__ __launch_bounds__(EF_NT) void k_embed_few(EmbedGradArgs p) {
    constexpr int VE = Vec<T>::VE, CH = EF_ROWS / EF_NT;
    __shared__ float sh[EF_W][64][VE + 1];
    __shared__ int list[EF_ROWS], cnt[CH][EF_W];
    const int tid = threadIdx.x, lane = tid & 63, n = (int)p.n;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t zero = ((uint32_t)p.v + EF_ZERO - 1) / EF_ZERO;
    if (blockIdx.x < zero) {
        embed_zero_absent<T, EF_W>(p, n, (int64_t)blockIdx.x * EF_ZERO, (uint32_t*)list, tid);
        return;
    }
    const uint32_t item = blockIdx.x - zero;
    const int r = (int)(item / (uint32_t)p.cols);
    const int code = p.codes[r];
    if (code < 0 || code >= p.v) return;
    uint64_t mask[CH];
    int before = 0;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int i = j * EF_NT + tid;
        const bool same = i < n && p.codes[i] == code;
        before |= same && i < r;
        mask[j] = __builtin_amdgcn_ballot_w64(same && i >= r);
        if (lane == 0) cnt[j][wave] = __popcll(mask[j]);
    }
    if (__syncthreads_or(before)) return;
    int total = 0;
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int w = 0; w < EF_W; ++w) {
            if (w == wave && (mask[j] >> lane & 1))
                list[total + __popcll(mask[j] & ((uint64_t(1) << lane) - 1))] = j * EF_NT + tid;
            total += cnt[j][w];
        }
    __syncthreads();
    const int kc = ((int)(item - (uint32_t)r * p.cols) * p.width + lane) * VE;
    const bool has = lane < p.width && kc < p.d;
    const int k = whole<VE>(kc, p.d);
    const int a = total * wave / EF_W, z = total * (wave + 1) / EF_W;
    float acc[VE];
#pragma unroll
    for (int q = 0; q < VE; ++q) acc[q] = 0.f;
    for (int j0 = a; j0 < z; j0 += EG_U) {
        Raw16 x[EG_U];
        embed_rows<T>(p, has, k, j0, z, [&](int j) { return (uint32_t)list[j]; }, x);
#pragma unroll
        for (int u = 0; u < EG_U; ++u)
            if (j0 + u < z) {
#pragma unroll
                for (int q = 0; q < VE; ++q) acc[q] += Vec<T>::get(x[u], q);
            }
    }
    join_waves<EF_W, VE>(sh, acc, wave, lane);
    if (wave == 0 && has) embed_out<T>(p, (uint32_t)code, k, acc);
}

struct EmbedPlan {
    int32_t passes, bits, tiles, dp, cols, width, seg;
    int64_t tile, segs;
    size_t o_key[2], o_row[2], o_mat, o_part, bytes;
};
static EmbedPlan embed_plan(int64_t n, int32_t d, int32_t v, int ve) {
    EmbedPlan q{};
    const int vecs = (d + ve - 1) / ve;
    q.cols = (vecs + 63) / 64;
    q.width = (vecs + q.cols - 1) / q.cols;  // blocks of about one size
    q.dp = (d + 7) / 8 * 8;
    if (n <= EF_ROWS) {
        q.bytes = 256;
        return q;
    }
    const int bits = 32 - __builtin_clz((unsigned)v);  // of keys 0 .. v
    q.passes = (bits + ES_BITS - 1) / ES_BITS;
    q.bits = (bits + q.passes - 1) / q.passes;
    q.tile = ES_NT;
    while ((n + q.tile - 1) / q.tile > ES_MAX_TILES) q.tile *= 2;
    q.tiles = (int32_t)((n + q.tile - 1) / q.tile);
    // shorter segments while the chip has room for more waves
    q.seg = 64;
    while (q.seg > 8 && (n + q.seg - 1) / q.seg * q.cols < EG_WAVES) q.seg /= 2;
    q.segs = (n + q.seg - 1) / q.seg;
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
    q.o_mat = take(((size_t)q.tiles << q.bits) * 4);
    q.o_part = take((size_t)q.segs * 2 * q.dp * 4);
    q.bytes = off;
    return q;
}

static unsigned grid_of(int64_t blocks) {
    const int64_t most = (int64_t)1 << 20;
    return (unsigned)(blocks < most ? blocks : most);
}

template <typename T>
static hipError_t embed_grad(EmbedGradArgs a, const EmbedPlan& q, char* ws, hipStream_t st) {
    a.dp = q.dp;
    a.cols = q.cols;
    a.width = q.width;
    if (a.n <= EF_ROWS) {
        const int64_t zero = (a.v + EF_ZERO - 1) / EF_ZERO;
        hipLaunchKernelGGL((k_embed_few<T>), dim3((unsigned)(a.n * q.cols + zero)), dim3(EF_NT), 0, st, a);
        return hipGetLastError();
    }
    SortArgs s{};
    s.mat = (uint32_t*)(ws + q.o_mat);
    s.n = a.n;
    s.tile = q.tile;
    s.v = a.v;
    s.tiles = q.tiles;
    s.bits = q.bits;
    if (a.n <= EO_ROWS) {
        s.codes = a.codes;
        s.bits = 32 - __builtin_clz((unsigned)a.v);
        s.key = (uint32_t*)(ws + q.o_key[0]);
        s.row = (uint32_t*)(ws + q.o_row[0]);
        hipLaunchKernelGGL((k_embed_sort<T>), dim3((unsigned)(1 + (a.v + EF_ZERO - 1) / EF_ZERO)), dim3(ES_NT), 0, st, s,
                           a);
    } else {
        a.zero = (a.v + EZ_CODES - 1) / EZ_CODES;
    }
    for (int i = 0; a.n > EO_ROWS && i < q.passes; ++i) {
        s.codes = i == 0 ? a.codes : nullptr;
        s.key_in = s.key;
        s.row_in = s.row;
        s.key = (uint32_t*)(ws + q.o_key[i & 1]);
        s.row = (uint32_t*)(ws + q.o_row[i & 1]);
        s.shift = i * q.bits;
        hipLaunchKernelGGL(k_embed_count, dim3(q.tiles), dim3(ES_NT), 0, st, s);
        hipLaunchKernelGGL(k_embed_place, dim3(q.tiles), dim3(ES_NT), 0, st, s);
    }
    a.key = s.key;
    a.row = s.row;
    a.part = (float*)(ws + q.o_part);
    a.seg = q.seg;
    a.segs = q.segs;
    const int64_t waves = a.segs * a.cols + a.zero;
    hipLaunchKernelGGL((k_embed_sum<T>), dim3(grid_of((waves + 3) / 4)), dim3(256), 0, st, a);
    if (a.segs > 1) {
        const int64_t blocks = (a.segs - 2) / EJ_W + 1;
        hipLaunchKernelGGL((k_embed_join<T>), dim3((unsigned)(blocks < 4096 ? blocks : 4096), a.cols), dim3(64 * EJ_W),
                           0, st, a);
    }
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
    const EmbedPlan a = embed_plan(n, d, v, 4), b = embed_plan(n, d, v, 8);  // fp32, bf16
    return a.bytes > b.bytes ? a.bytes : b.bytes;
}

int gmm_embed_backward(const void* grad, int64_t n, int32_t d, int64_t ldg, int32_t dtype,
                       const int32_t* codes, int32_t v, float scale, void* d_table, int64_t ldt,
                       void* workspace, size_t workspace_bytes, void* stream) {
    if (dtype != GMM_F32 && dtype != GMM_BF16) return GMM_E_DTYPE;
    if (n < 0 || v < 1 || d < 1 || ldg < d || ldt < d || !isfinite(scale) || !d_table)
        return GMM_E_INVALID;
    if (n > EMB_MAX_ROWS || d > EMB_MAX_DIM || v > EMB_MAX_CODES) return GMM_E_UNSUPPORTED;
    if (n > 0 && (!grad || !codes)) return GMM_E_INVALID;
    const EmbedPlan q = embed_plan(n, d, v, dtype == GMM_F32 ? 4 : 8);
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
    a.codes = codes;
    a.out = d_table;
    a.n = n;
    a.ldg = ldg;
    a.ldt = ldt;
    a.v = v;
    a.d = d;
    a.scale = scale;
    const hipError_t e = dtype == GMM_F32 ? embed_grad<float>(a, q, (char*)workspace, st)
                                          : embed_grad<uint16_t>(a, q, (char*)workspace, st);
    return e == hipSuccess ? GMM_OK : GMM_E_HIP;
}

}  // extern "C"
