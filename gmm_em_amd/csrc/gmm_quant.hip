// gmm_quant.hip - rows in 8-bit integers and their products (gmm_quantize_rows,
// gmm_quantized_product, declared in include/gmm_em.h):
//   s_r = max |x_r| / 127,  q = x / s_r to the nearest integer;   y = (sum q w) s_q s_w
// Products of 8-bit integers and their sums are exact in 32 bits, so the order of the sum
// and the kernel that makes it leave no trace in y.
//
// k_quant_few: up to 16 rows. The product is the reading of w: 16 weight rows by 16 rows of q
// per matrix instruction, both straight from memory, the contracted axis split over the
// waves and joined in LDS. 16 x 4096 x 16384 in 17.8 to 19.7 us (67 MB of w: 3.4 TB/s and more).
// k_quant_tiles: more rows, by the tiles of gmm_gemm.h (codes are the tile rows, turned so that a
// lane has eight neighbouring codes of a row to write: 16 bytes of bf16). Operands whose rows
// are not 16-byte aligned, or not whole steps of 128 long, are laid out in panels first.
// 8192^3 in 400 us (2750 TOP/s; another card 470), with operands of zeros 330: on other numbers the chip's
// power sets part of the pace. 8192 x 4096 x 16384 in 457 (bf16 results; 427 the kernel by itself), zeros 422.
// Not kept, on the card that took 470: stores of four codes (8192 x 4096 x 16384 500 against 465 and
// 8192 x 768 x 16384 164 against 136), blocks of 32 x 32 (508 at 8192^3), four waves of 128 x 128 (770), stores
// past the caches (607).
// k_quant_odd: tiles of 64 x 64 read as the rows lie, where the layout would cost more than it saves
// (odd rows in few tiles): 20 x 8191 x 32767 in 69 us, laid out 200; 64 x 8191 x 32767 86, 197;
// 64 x 1003 x 32767 16, 26.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "gmm_em.h"
#include "gmm_gemm.h"
#include "gmm_grid.h"
#include "gmm_nn.h"
#include "gmm_softmax.h"
#include "gmm_tiles.h"

namespace gmm {

constexpr int32_t QU_MAX_DIM = (1 << 17) - 1;  // 128 * 128 * d stays below 2^31
constexpr int32_t QU_MAX_CODES = 1 << 22;

// ---- rows to integers

struct QuantArgs {
    const void* x;
    int8_t* q;
    float* scale;
    int64_t n, ldx, ldq;
    int32_t d;
};

// Integers by adding 1.5 2^23, whose last digit is worth 1: the low byte of the sum's bits.
constexpr float QR_ROUND = 12582912.f;

// The bits of 1.5 2^23 + the integer nearest x / s, ties to the even one, within 127. The estimate
// is off by one at most; the remainder of it is exact (|q| s is a few bits longer than s, and
// x - q s shorter than either) and tells.
__device__ __forceinline__ uint32_t quant(float x, float s, float inv) {
    float q = rintf(x * inv);
    const float r = fmaf(-q, s, x), a = fabsf(r), half = 0.5f * s;
    if (a > half || (a == half && ((int)q & 1))) q += r > 0.f ? 1.f : -1.f;
    return __float_as_uint(fminf(fmaxf(q, -127.f), 127.f) + QR_ROUND);
}

// 16 values of a row, as a thread holds them.
template <typename T>
struct QuantRun {
    static constexpr int VE = Vec<T>::VE, NV = 16 / VE;
    Raw16 r[NV];
    __device__ __forceinline__ float get(int j) const { return Vec<T>::get(r[j / VE], j % VE); }
    // from k on; a run that would pass the end is the last whole one (short rows: 0 behind it)
    __device__ __forceinline__ void load(const T* x, int k, int d) {
        if (d >= 16) {
#pragma unroll
            for (int h = 0; h < NV; ++h) r[h] = *reinterpret_cast<const Raw16*>(x + whole<16>(k, d) + h * VE);
        } else {
#pragma unroll
            for (int h = 0; h < NV; ++h) r[h] = load_zero(x, k + h * VE, (int64_t)d);
        }
    }
    // the largest magnitude; infinite for a NaN
    __device__ __forceinline__ float most() const {
        float m = 0.f, sum = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            m = fmaxf(m, fabsf(get(j)));
            sum = fmaf(get(j), 0.f, sum);  // NaN with an infinity or a NaN, else 0
        }
        return sum == 0.f ? m : INFINITY;
    }
    __device__ __forceinline__ void store(int8_t* q, int k, int d, float s, float inv, float up) const {
        uint32_t b[16];
        if (inv > 0.f) {  // the same for the row
            float worst = 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float t = fmaf(get(j), inv, QR_ROUND);
                b[j] = __float_as_uint(t);
                worst = fmaxf(worst, fabsf(fmaf(-(t - QR_ROUND), s, get(j))));
            }
            // a remainder of half a step or more: the estimate may be the other neighbour
            if (worst >= 0.5f * s || up != 1.f) {
#pragma unroll
                for (int j = 0; j < 16; ++j) b[j] = quant(get(j) * up, s, inv);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) b[j] = 0;
        }
        Any16 o;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o.w[j] = (b[4 * j] & 255) | (b[4 * j + 1] & 255) << 8 | (b[4 * j + 2] & 255) << 16 | b[4 * j + 3] << 24;
        if (d >= 16) {
            *reinterpret_cast<Any16*>(q + whole<16>(k, d)) = o;
        } else {
#pragma unroll
            for (int j = 0; j < 15; ++j)
                if (k + j < d) q[k + j] = (int8_t)(o.w[j >> 2] >> (8 * (j & 3)));
        }
    }
};

// The largest of a group of LPR lanes.
template <int LPR>
__device__ __forceinline__ float lanes_max(float v) {
    if constexpr (LPR == 64) return wave_max(v);
    if constexpr (LPR == 16) return max16(v);
    v = fmaxf(v, lane_move<0xb1>(v));
    v = fmaxf(v, lane_move<0x4e>(v));
    return fmaxf(v, lane_move<0x141>(v));
}

// A row's scale, and what its integers are made with: s, 1 / s (0: they are 0), and the power of two
// that rows whose 1 / s would leave fp32 are multiplied by first (nothing is rounded by it).
struct QuantScale {
    float scale, s, inv, up;
    __device__ __forceinline__ QuantScale(float m) {
        scale = m < INFINITY ? m / 127.f : NAN;
        up = scale < 0x1p-100f ? 0x1p100f : 1.f;
        s = scale * up;
        inv = s > 0.f ? 1.f / s : 0.f;
    }
};

// LPR lanes per row, which holds it: at most 16 LPR U values.
// 8192 x 4096 in 31 us (bf16, 3.3 TB/s) and 34 us (fp32, 5.0 TB/s); 28 and 29 where the caches still hold part of
// the rows, and 36 (bf16) for the kernel that follows a product of 450 us.
template <typename T, int LPR, int U>
__global__ __launch_bounds__(256) void k_quant_rows(QuantArgs p) {
    constexpr int RPW = 64 / LPR;
    const int lane = threadIdx.x & 63, gl = lane % LPR, grp = lane / LPR;
    const int64_t wave = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int64_t r0 = wave * RPW; r0 < p.n; r0 += (int64_t)gridDim.x * 4 * RPW) {
        const int64_t row = r0 + grp;
        const bool in = row < p.n;
        const T* x = (const T*)p.x + (in ? row : p.n - 1) * p.ldx;
        QuantRun<T> v[U];
        float m = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (u * LPR + gl) * 16;
            if (k < p.d) v[u].load(x, k, p.d);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if ((u * LPR + gl) * 16 < p.d) m = fmaxf(m, v[u].most());
        const QuantScale c(lanes_max<LPR>(m));
        if (!in) continue;
        if (gl == 0) p.scale[row] = c.scale;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (u * LPR + gl) * 16;
            if (k < p.d) v[u].store(p.q + row * p.ldq, k, p.d, c.s, c.inv, c.up);
        }
    }
}

// A workgroup per longer row. HOLD: its registers hold it, else it is read twice.
template <typename T, int NT, bool HOLD>
__global__ __launch_bounds__(NT) void k_quant_long(QuantArgs p) {
    constexpr int U = HOLD ? 4 : 1;
    __shared__ float part[NT / 64];
    const int tid = threadIdx.x;
    for (int64_t row = blockIdx.x; row < p.n; row += gridDim.x) {
        const T* x = (const T*)p.x + row * p.ldx;
        QuantRun<T> v[U];
        float m = 0.f;
        for (int k0 = tid * 16; k0 < p.d; k0 += U * NT * 16) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (k0 + u * NT * 16 < p.d) v[u].load(x, k0 + u * NT * 16, p.d);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (k0 + u * NT * 16 < p.d) m = fmaxf(m, v[u].most());
        }
        m = wave_max(m);
        if ((tid & 63) == 0) part[tid >> 6] = m;
        __syncthreads();
        m = part[0];
#pragma unroll
        for (int w = 1; w < NT / 64; ++w) m = fmaxf(m, part[w]);
        const QuantScale c(m);
        if (tid == 0) p.scale[row] = c.scale;
        for (int k0 = tid * 16; k0 < p.d; k0 += U * NT * 16)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = k0 + u * NT * 16;
                if (k >= p.d) break;
                if (!HOLD) v[u].load(x, k, p.d);
                v[u].store(p.q + row * p.ldq, k, p.d, c.s, c.inv, c.up);
            }
        __syncthreads();
    }
}

template <typename T>
static void quant_rows(const QuantArgs& a, hipStream_t st) {
    // workgroups of nt threads that take `rows` rows at once
    auto launch = [&](auto kernel, int nt, int64_t rows) {
        hipLaunchKernelGGL(kernel, dim3(grid_for((a.n + rows - 1) / rows, nt)), dim3(nt), 0, st, a);
    };
    if (a.d <= 8 * 16)
        launch(k_quant_rows<T, 8, 1>, 256, 32);
    else if (a.d <= 2 * 16 * 16)
        launch(k_quant_rows<T, 16, 2>, 256, 16);
    else if (a.d <= 4 * 64 * 16)
        launch(k_quant_rows<T, 64, 4>, 256, 4);
    else if (a.d <= 4 * 256 * 16)
        launch(k_quant_long<T, 256, true>, 256, 1);
    else
        launch(k_quant_long<T, 1024, false>, 1024, 1);
}

// ---- products

struct ProductArgs {
    const int8_t *q, *w;
    const float *q_scale, *w_scale;
    void* y;
    int64_t n, ldq, ldw, ldy;
    int32_t d, v;
};

__device__ __forceinline__ i32x4 mfma_i8(const Raw16& a, const Raw16& b, i32x4 c) {
    return mfma32(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c);
}

// 16 bytes of a row, 0 at or past `end`.
__device__ __forceinline__ Raw16 load_bytes(const int8_t* p, int i, int end) {
    if (i + 16 <= end) return __builtin_bit_cast(Raw16, *reinterpret_cast<const Any16*>(p + i));
    Raw16 r = {{0u, 0u, 0u, 0u}};
#pragma unroll
    for (int k = 0; k < 16; ++k)
        if (i + k < end) r.w[k >> 2] |= (uint32_t)(uint8_t)p[i + k] << (8 * (k & 3));
    return r;
}

// 16 bytes of a row at a time where they lie within it. BYTES: rows at any address, read as the
// aligned words that hold their bytes (up to three bytes before a row's first and behind its last
// one come with them, never another word) and shifted into place: pieces of many rows whose words are
// not aligned come at half the rate (1 x 8191 x 32767: 124 us so, 70 shifted; 16 rows 227, 106).
template <bool BYTES>
struct ByteRow {
    const int8_t* row;
    uint32_t shift, more;  // bytes from a word's start; from there to the word of the 16th byte
    __device__ __forceinline__ void set(const int8_t* p) {
        shift = BYTES ? (uint32_t)(uintptr_t)p & 3 : 0;
        more = (shift + 15) & ~3u;
        row = p - shift;
    }
    struct __attribute__((packed, aligned(4))) Words {
        uint32_t w[4];
    };
    struct Piece {
        Words v;
        uint32_t next;
    };
    __device__ __forceinline__ Piece fetch(int k) const {
        Piece r;
        r.v = *reinterpret_cast<const Words*>(row + k);
        r.next = BYTES ? *reinterpret_cast<const uint32_t*>(row + k + more) : 0;
        return r;
    }
    __device__ __forceinline__ Raw16 take(const Piece& p) const {
        Raw16 r;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            r.w[j] = BYTES ? __builtin_amdgcn_alignbyte(j < 3 ? p.v.w[(j + 1) & 3] : p.next, p.v.w[j], shift) : p.v.w[j];
        return r;
    }
    __device__ __forceinline__ Raw16 get(int k) const { return take(fetch(k)); }
    // 0 at or past `end`
    __device__ __forceinline__ Raw16 get(int k, int end) const {
        return k + 16 <= end ? get(k) : load_bytes(row + shift, k, end);
    }
};
// Whether rows do not start at words.
static bool odd_rows(const int8_t* p, int64_t ld) { return ((uintptr_t)p | (uint64_t)ld) % 4 != 0; }

template <typename T>
__device__ __forceinline__ T scaled_sum(int acc, float qs, float ws) {
    return Vec<T>::store((float)acc * qs * ws);
}

// 16 codes by up to 16 rows.
constexpr int QF_W = 4;
template <typename T, bool BYTES>
__global__ __launch_bounds__(64 * QF_W) void k_quant_few(ProductArgs p) {
    __shared__ i32x4 sh[QF_W][64];
    const int lane = threadIdx.x & 63, h = lane >> 4, i = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c0 = blockIdx.x * 16;
    ByteRow<BYTES> w, q;
    w.set(p.w + (int64_t)(c0 + i < p.v ? c0 + i : p.v - 1) * p.ldw);
    q.set(p.q + (i < p.n ? i : p.n - 1) * p.ldq);
    i32x4 acc = {0, 0, 0, 0};
    // steps of 64 integers, step s for wave s % QF_W, in groups whose loads are in flight together
    constexpr int STEP = 64 * QF_W;
    int k = wave * 64 + h * 16;
    auto steps = [&](auto count) {
        constexpr int U = decltype(count)::value;
        for (; k - h * 16 + (U - 1) * STEP + 64 <= p.d; k += U * STEP) {
            Raw16 a[U], b[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                a[u] = w.get(k + u * STEP);
                b[u] = q.get(k + u * STEP);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) acc = mfma_i8(a[u], b[u], acc);
        }
    };
    steps(std::integral_constant<int, 8>());
    steps(std::integral_constant<int, 2>());
    steps(std::integral_constant<int, 1>());
    if (k - h * 16 < p.d) acc = mfma_i8(w.get(k, p.d), q.get(k, p.d), acc);
    sh[wave][lane] = acc;
    __syncthreads();
    // lane (h, i) holds codes 4 h .. 4 h + 3 of row i: one of them for each wave
    const int c = c0 + 4 * h + wave;
    if (i >= p.n || c >= p.v) return;
    int sum = 0;
#pragma unroll
    for (int x = 0; x < QF_W; ++x) sum += ((const int*)&sh[x][lane])[wave];
    ((T*)p.y)[i * p.ldy + c] = scaled_sum<T>(sum, p.q_scale[i], p.w_scale[c]);
}

// ---- tiles

constexpr int QT_STEP = 2 * GK;              // integers of a step
constexpr int64_t QT_MAX_LD = (int64_t)1 << 23;  // 256 rows span at most 2^31 bytes
constexpr size_t QT_PACK_BYTES = (size_t)256 << 20;   // rows of q laid out at a time
constexpr size_t QT_SPLIT_BYTES = (size_t)128 << 20;  // partial sums of a split product
constexpr int QT_MAX_SPLIT = 16;
// Rows for k_quant_few. The tiles take 32 rows of 4096 against 16384 codes in 19 us, 2 or 4 blocks of
// its 16 rows a workgroup took 33.
constexpr int QT_FEW_ROWS = 16;

struct TilesArgs {
    GemmIn in;           // a: codes, b: rows of q
    int32_t mt, nt, split;
    const float *q_scale, *w_scale;
    void* y;
    int64_t ldy;
    int32_t* part;       // [split][rows][codes]
};

// Values of neighbouring codes, at any element's address.
template <typename T, int N>
struct __attribute__((packed, aligned(sizeof(T)))) Run {
    T v[N];
};
constexpr int QT_RUN = 8;  // codes that a lane has of two blocks

// Writes eight sums of row r from code c on: to y, or to their part of a split product.
template <typename T>
__device__ __forceinline__ void run_out(const TilesArgs& p, int r, int c, const Run<float, QT_RUN>& ws, float qs,
                                        const i32x4& lo, const i32x4& hi) {
    constexpr int VE = Vec<T>::VE;
    T* o = (T*)p.y + (int64_t)r * p.ldy + c;
    float v[QT_RUN];
#pragma unroll
    for (int q = 0; q < QT_RUN; ++q) v[q] = (float)(q < 4 ? lo[q & 3] : hi[q & 3]) * qs * ws.v[q];
    if (c + QT_RUN <= p.in.m) {
#pragma unroll
        for (int q = 0; q < QT_RUN; q += VE) *(Raw16*)(o + q) = pack16<T>(v + q);
    } else {
#pragma unroll
        for (int q = 0; q < QT_RUN; ++q)
            if (c + q < p.in.m) o[q] = Vec<T>::store(v[q]);
    }
}
__device__ __forceinline__ void run_part(const TilesArgs& p, int r, int c, const i32x4& lo, const i32x4& hi) {
    int32_t* o = p.part + ((int64_t)blockIdx.y * p.in.n + r) * p.in.m + c;
    Run<int32_t, QT_RUN> v;
#pragma unroll
    for (int q = 0; q < QT_RUN; ++q) v.v[q] = q < 4 ? lo[q & 3] : hi[q & 3];
    if (c + QT_RUN <= p.in.m) {
        *(Run<int32_t, QT_RUN>*)o = v;
    } else {
#pragma unroll
        for (int q = 0; q < QT_RUN; ++q)
            if (c + q < p.in.m) o[q] = v.v[q];
    }
}
// The scales of eight codes.
__device__ __forceinline__ Run<float, QT_RUN> run_scales(const TilesArgs& p, int c) {
    if (c + QT_RUN <= p.in.m) return *(const Run<float, QT_RUN>*)(p.w_scale + c);
    Run<float, QT_RUN> ws;
#pragma unroll
    for (int q = 0; q < QT_RUN; ++q) ws.v[q] = c + q < p.in.m ? p.w_scale[c + q] : 0.f;
    return ws;
}

template <typename T, int BM, int BN, int WM, int WN, bool SPLIT>
__global__ __launch_bounds__(64 * WM * WN) void k_quant_tiles(TilesArgs p) {
    using G = Gemm<BM, BN, WM, WN, true, false, i32x4>;
    __shared__ __align__(16) unsigned char l0[G::STAGE], l1[G::STAGE];
    if constexpr (SPLIT) {
        int tm, tn;
        if (!gemm_tile(blockIdx.x, p.mt, p.nt, &tm, &tn)) return;
        const int m0 = tm * BM, n0 = tn * BN, steps = G::all_steps(p.in);
        G g;
        g.begin(p.in, m0, n0, steps * (int)blockIdx.y / p.split, steps * ((int)blockIdx.y + 1) / p.split, l0, l1);
        g.template finish<i32x4>(p.in, m0, n0, l0, l1);
#pragma unroll
        for (int y = 0; y < G::TN; ++y) {
            const int r = n0 + G::col(y);
            if (r >= p.in.n) continue;
#pragma unroll
            for (int x = 0; x < G::TM; x += 2) run_part(p, r, m0 + G::row(x), g.acc[x][y], g.acc[x + 1][y]);
        }
    } else {
        gemm_walk<i32x4, G, BM, BN>(p.in, p.mt, p.nt, l0, l1, [&](G& g, int m0, int n0) {
            float qs[G::TN];
#pragma unroll
            for (int y = 0; y < G::TN; ++y) {
                const int r = n0 + G::col(y);
                qs[y] = p.q_scale[r < p.in.n ? r : p.in.n - 1];
            }
#pragma unroll
            for (int x = 0; x < G::TM; x += 2) {
                const int c = m0 + G::row(x);
                const Run<float, QT_RUN> ws = run_scales(p, c);
#pragma unroll
                for (int y = 0; y < G::TN; ++y) {
                    const int r = n0 + G::col(y);
                    if (r < p.in.n) run_out<T>(p, r, c, ws, qs[y], g.acc[x][y], g.acc[x + 1][y]);
                }
            }
        });
    }
}

// The same product for operands of any stride and alignment, without laying them out: 64 codes by 64
// rows, steps of 128 integers read into registers, 16 bytes a lane, QO_AHEAD ahead, and put into LDS (rows
// turned and pieces rotated as in gmm_gemm.h) when the step before has been multiplied.
struct OddArgs {
    TilesArgs t;         // in.m codes, in.n rows
    const int8_t *w, *q;
    int64_t ldw, ldq;
    int32_t d, steps;
};
constexpr int QO_TILE = 64, QO_STAGE = 2 * QO_TILE * QT_STEP;
// Steps in flight, an even number (2: 20 x 8191 x 32767 69 us, 8000 x 5001 x 9000 950; 4: 70 and 1049).
constexpr int QO_AHEAD = 2;
template <typename T, bool SPLIT, bool BYTES>
__global__ __launch_bounds__(256) void k_quant_odd(OddArgs p) {
    __shared__ __align__(16) unsigned char lds[2][QO_STAGE];
    int tm, tn;
    if (!gemm_tile(blockIdx.x, p.t.mt, p.t.nt, &tm, &tn)) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h = lane >> 4, i = lane & 15, wm = wave >> 1, wn = wave & 1;
    const int m0 = tm * QO_TILE, n0 = tn * QO_TILE;
    const int first = SPLIT ? p.steps * (int)blockIdx.y / p.t.split : 0;
    const int last = SPLIT ? p.steps * ((int)blockIdx.y + 1) / p.t.split : p.steps;
    const int full = p.d / QT_STEP;  // steps that lie within the rows
    const int r8 = lane >> 3, k0 = (lane & 7) * 16;
    ByteRow<BYTES> src[4];           // this lane's pieces: two groups of 8 rows of w, two of q
    int to[4];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const int row = wave * 16 + g * 8 + r8, in32 = row & 31;
        const int code = m0 + (row & 32) + 8 * (in32 >> 2 & 3) + 4 * (in32 >> 4) + (in32 & 3);
        src[g].set(p.w + (int64_t)(code < p.t.in.m ? code : p.t.in.m - 1) * p.ldw);
        src[2 + g].set(p.q + (int64_t)(n0 + row < p.t.in.n ? n0 + row : p.t.in.n - 1) * p.ldq);
        to[g] = row * QT_STEP + (k0 ^ (r8 << 4));
        to[2 + g] = QO_TILE * QT_STEP + to[g];
    }
    i32x4 acc[2][2];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) acc[x][y] = i32x4{0, 0, 0, 0};
    auto put = [&](unsigned char* l, int g, const Raw16& v) {
        *(uint4*)(l + to[g]) = uint4{v.w[0], v.w[1], v.w[2], v.w[3]};
    };
    auto multiply = [&](const unsigned char* l) {
        // A barrier for LDS alone: the loads in flight go on. The other buffer is free again (every wave
        // has read it).
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            i32x4 a[2], b[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int piece = ((4 * c + h) ^ (i & 7)) << 4;
                a[x] = *(const i32x4*)(l + (wm * 32 + x * 16 + i) * QT_STEP + piece);
                b[x] = *(const i32x4*)(l + (QO_TILE + wn * 32 + x * 16 + i) * QT_STEP + piece);
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y) acc[x][y] = mfma32(a[x], b[y], acc[x][y]);
        }
    };
    const int end = last < full ? last : full;  // whole steps; at most one that is cut follows
    int buf = 0;
    if (first < end) {
        using Piece = typename ByteRow<BYTES>::Piece;
        Piece v[QO_AHEAD][4];
        auto fetch = [&](Piece(&to_v)[4], int s) {
            const int k = (s < end ? s : end - 1) * QT_STEP + k0;  // (no branch around a load)
#pragma unroll
            for (int g = 0; g < 4; ++g) to_v[g] = src[g].fetch(k);
        };
#pragma unroll
        for (int u = 0; u < QO_AHEAD; ++u) {
            fetch(v[u], first + u);
            __builtin_amdgcn_sched_barrier(0);  // loads in the order in which they are waited for
        }
        for (int s0 = first; s0 < end; s0 += QO_AHEAD) {
#pragma unroll
            for (int u = 0; u < QO_AHEAD; ++u) {
                if (s0 + u >= end) break;
                unsigned char* l = lds[u & 1];
#pragma unroll
                for (int g = 0; g < 4; ++g) put(l, g, src[g].take(v[u][g]));
                fetch(v[u], s0 + u + QO_AHEAD);
                __builtin_amdgcn_sched_barrier(0);
                multiply(l);
                buf = (u & 1) ^ 1;
            }
        }
    }
    if (last > full) {
#pragma unroll
        for (int g = 0; g < 4; ++g) put(lds[buf], g, src[g].get(full * QT_STEP + k0, p.d));
        multiply(lds[buf]);
    }
    const int c = m0 + wm * 32 + 8 * h;
    const Run<float, QT_RUN> ws = run_scales(p.t, c);
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const int r = n0 + wn * 32 + y * 16 + i;
        if (r >= p.t.in.n) continue;
        if constexpr (SPLIT)
            run_part(p.t, r, c, acc[0][y], acc[1][y]);
        else
            run_out<T>(p.t, r, c, ws, p.t.q_scale[r], acc[0][y], acc[1][y]);
    }
}

// The sums of a split product, four codes of a row per thread.
template <typename T>
__global__ __launch_bounds__(256) void k_quant_sum(TilesArgs p) {
    const int per = (p.in.m + 3) / 4;
    const int64_t total = (int64_t)p.in.n * per, plane = (int64_t)p.in.n * p.in.m;
    for (int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x; j < total; j += (int64_t)gridDim.x * 256) {
        const int64_t r = j / per;
        const int c = (int)(j - r * per) * 4, left = p.in.m - c < 4 ? p.in.m - c : 4;
        const int32_t* from = p.part + r * p.in.m + c;
        int acc[4] = {0, 0, 0, 0};
        for (int s = 0; s < p.split; ++s)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (q < left) acc[q] += from[s * plane + q];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (q < left)
                ((T*)p.y)[r * p.ldy + c + q] = scaled_sum<T>(acc[q], p.q_scale[r], p.w_scale[c + q]);
    }
}

// Operands in panels of 128 integers, 0 past the d-th (blockIdx.y: w, then q; rows == 0 is none).
struct PackArgs {
    struct {
        const int8_t* x;
        int64_t rows, ld;
        int8_t* out;
    } o[2];
    int32_t d, dp;
};
// Eight lanes copy a row's piece of a panel, a wave eight rows: 1 KB in one piece.
__global__ __launch_bounds__(256) void k_quant_pack(PackArgs p) {
    const auto o = p.o[blockIdx.y];
    const int lane = threadIdx.x & 63;
    const uint32_t panels = (uint32_t)p.dp / QT_STEP, items = (uint32_t)((o.rows + 7) / 8) * panels;
    for (uint32_t i = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); i < items; i += gridDim.x * 4) {
        const uint32_t group = i / panels, panel = i - group * panels;
        const int64_t r = (int64_t)group * 8 + (lane >> 3);
        if (r >= o.rows) continue;
        const int k = (int)panel * QT_STEP + (lane & 7) * 16;
        ByteRow<true> x;
        x.set(o.x + r * o.ld);
        *(Raw16*)(o.out + (panel * o.rows + r) * QT_STEP + (lane & 7) * 16) = x.get(k, p.d);
    }
}

static bool quant_direct(const int8_t* x, int32_t d, int64_t ld) {
    return d % QT_STEP == 0 && ld % 16 == 0 && ld <= QT_MAX_LD && (uintptr_t)x % 16 == 0;
}

// The tile and the split that take least time by a model of it: the chip's workgroups take
// (fixed + steps * per_step) for each full load of the CUs; fewer workgroups per CU take their share of a
// step's time, but not less than `alone`. A split adds the writing and reading of its sums.
// Calls with each tile in their order (us, steps of 128 integers): 8192^3 470, 532, 592, 867; 4096^3
// 58, 84, 72, 102; 2048^3 31, 25, 15, 17; 777 x 1024 x 5001 24, 19.5, 15.5, 13.8; 300 x 4096 x 4096 48,
// 40, 28, 13 (the least is picked in each); 128 x 8192 x 4096 81, 65, 47, 33, as picked, split, 19.
struct QuantCost {
    int bm, bn, per_cu;
    float per_step, fixed, alone;  // microseconds
};
constexpr QuantCost QUANT_COST[4] = {
    {256, 256, 1, 1.75f, 6.f, 1.75f}, {192, 256, 1, 1.35f, 6.f, 1.35f}, {128, 128, 2, 1.13f, 4.f, 0.7f},
    {64, 64, 4, 0.82f, 3.f, 0.4f}};
// Operands as they lie (k_quant_odd), tile QT_ODD, against the tiles and `pack` bytes laid out before
// (us as they lie, laid out): 64 x 1003 x 32767 16, 26; 1000 x 333 x 1111 10.5, 12; 200 x 1003 x 16384 21, 22;
// 200 x 8191 x 32767 231, 222; 777 x 1003 x 5001 27, 20; 500 x 8191 x 16384 203, 135; 3000 x 3001 x 8000 219, 84.
constexpr int QT_ODD = 4;
constexpr QuantCost ODD_COST = {QO_TILE, QO_TILE, 4, 1.6f, 6.f, 0.85f};
static Choice quant_choice(int64_t m, int64_t n, int64_t steps, size_t pack) {
    Choice best{0, 1};
    double least = 1e300;
    for (int t = 0; t < (pack > 0 ? 5 : 4); ++t) {
        const QuantCost& c = t == QT_ODD ? ODD_COST : QUANT_COST[t];
        const int64_t tiles = ((m + c.bm - 1) / c.bm) * ((n + c.bn - 1) / c.bn);
        if (t == QT_ODD && tiles > ((int64_t)1 << 22)) break;  // a workgroup for each: within a grid
        for (int s = 1; s <= QT_MAX_SPLIT && s <= steps; ++s) {
            if (s > 1 && (size_t)s * m * n * 4 > QT_SPLIT_BYTES) break;
            const double load = (double)((tiles * s + 255) / 256) / c.per_cu, each = (double)((steps + s - 1) / s);
            const double part = c.per_step * load > c.alone ? c.per_step * load : c.alone;
            double us = load >= 1.0 ? load * (c.fixed + c.per_step * each) : c.fixed + part * each;
            if (s > 1) us += 4.0 + (double)m * n * 8 * s / 4.0e6;
            if (t != QT_ODD && pack > 0) us += 4.0 + (double)pack * 2 / 4.0e6;
            if (us < least) {
                least = us;
                best = Choice{t, s};
            }
        }
    }
    return best;
}

// What a product lays out and where.
struct QuantPlan {
    int32_t dp;
    int64_t chunk;  // rows at a time
    Choice first;   // of the first chunk
    size_t o_w, o_q, o_part, bytes;
};
static QuantPlan quant_rows_at_once(int64_t n, int32_t d) {
    QuantPlan q{};
    q.dp = (d + QT_STEP - 1) / QT_STEP * QT_STEP;
    q.chunk = (int64_t)(QT_PACK_BYTES / q.dp) / 256 * 256;
    if (q.chunk > n) q.chunk = n;
    return q;
}
// The bytes of a chunk's operands that have to be laid out for the tiles (packed: w has been).
static size_t pack_bytes(const QuantPlan& q, int32_t v, int64_t rows, bool pack_q, bool pack_w, bool packed) {
    return (pack_w && !packed ? (size_t)v * q.dp : 0) + (pack_q ? (size_t)rows * q.dp : 0);
}
// pack_q, pack_w: whether the operands are ones that the tiles cannot read in place. A workspace that is
// used has more than 256 bytes.
static QuantPlan quant_plan(int64_t n, int32_t d, int32_t v, bool pack_q, bool pack_w) {
    if (n <= QT_FEW_ROWS) {
        QuantPlan q{};
        q.bytes = 256;
        return q;
    }
    QuantPlan q = quant_rows_at_once(n, d);
    size_t w = 0, rows_q = 0, part = 0;
    bool packed = false;
    auto visit = [&](int64_t rows) {
        const Choice c = quant_choice(v, rows, q.dp / QT_STEP, pack_bytes(q, v, rows, pack_q, pack_w, packed));
        if (c.tile != QT_ODD) {
            packed = true;
            if (pack_w) w = (size_t)v * q.dp;
            if (pack_q && (size_t)rows * q.dp > rows_q) rows_q = (size_t)rows * q.dp;
        }
        const size_t sums = c.split > 1 ? (size_t)c.split * rows * v * 4 : 0;
        if (sums > part) part = sums;
        return c;
    };
    // the first chunk, those between it and the last, which are alike, and the last
    const int64_t chunks = (n + q.chunk - 1) / q.chunk;
    q.first = visit(q.chunk);
    if (chunks > 2) visit(q.chunk);
    if (chunks > 1) visit(n - (chunks - 1) * q.chunk);
    q.o_q = up256(w);
    q.o_part = q.o_q + up256(rows_q);
    q.bytes = q.o_part + up256(part);
    if (q.bytes < 512) q.bytes = q.bytes == 0 ? 256 : 512;
    return q;
}
// Enough for any operands.
static size_t quant_most_bytes(int64_t n, int32_t d, int32_t v) {
    if (n <= QT_FEW_ROWS) return 256;
    const QuantPlan q = quant_rows_at_once(n, d);
    const size_t sums = (size_t)q.chunk * v * 4 * QT_MAX_SPLIT;
    return up256((size_t)v * q.dp) + up256((size_t)q.chunk * q.dp) + up256(sums < QT_SPLIT_BYTES ? sums : QT_SPLIT_BYTES);
}

template <typename T>
static hipError_t quant_product(const ProductArgs& a, const QuantPlan& q, char* ws, hipStream_t st) {
    if (a.n <= QT_FEW_ROWS) {
        const dim3 grid((unsigned)((a.v + 15) / 16)), block(64 * QF_W);
        if (odd_rows(a.w, a.ldw) || odd_rows(a.q, a.ldq))
            hipLaunchKernelGGL((k_quant_few<T, true>), grid, block, 0, st, a);
        else
            hipLaunchKernelGGL((k_quant_few<T, false>), grid, block, 0, st, a);
        return hipGetLastError();
    }
    const bool pq = !quant_direct(a.q, a.d, a.ldq), pw = !quant_direct(a.w, a.d, a.ldw);
    TilesArgs t{};
    t.w_scale = a.w_scale;
    t.ldy = a.ldy;
    t.part = (int32_t*)(ws + q.o_part);
    t.in.pairs = 1;
    t.in.kp = q.dp / 2;
    t.in.m = a.v;
    t.in.a = (const uint16_t*)(pw ? (const int8_t*)ws + q.o_w : a.w);
    t.in.lda = pw ? GK : a.ldw / 2;
    t.in.step_a = pw ? (int64_t)a.v * GK : GK;
    bool packed = false;  // w
    for (int64_t r0 = 0; r0 < a.n; r0 += q.chunk) {
        const int64_t rows = a.n - r0 < q.chunk ? a.n - r0 : q.chunk;
        t.in.n = (int32_t)rows;
        t.q_scale = a.q_scale + r0;
        t.y = (T*)a.y + r0 * a.ldy;
        const Choice c = r0 == 0 ? q.first
                                 : quant_choice(a.v, rows, q.dp / QT_STEP, pack_bytes(q, a.v, rows, pq, pw, packed));
        t.split = c.split;
        auto sums = [&]() {
            if (c.split < 2) return;
            const int64_t work = (rows * ((a.v + 3) / 4) + 255) / 256;
            hipLaunchKernelGGL((k_quant_sum<T>), dim3((unsigned)(work < 16384 ? work : 16384)), dim3(256), 0, st, t);
        };
        if (c.tile == QT_ODD) {
            t.mt = (a.v + QO_TILE - 1) / QO_TILE;
            t.nt = (int32_t)((rows + QO_TILE - 1) / QO_TILE);
            const OddArgs o{t, a.w, a.q + r0 * a.ldq, a.ldw, a.ldq, a.d, q.dp / QT_STEP};
            const dim3 grid(tile_grid(t.mt, t.nt), c.split);
            auto launch = [&](auto bytes) {
                constexpr bool BYTES = decltype(bytes)::value;
                if (c.split > 1)
                    hipLaunchKernelGGL((k_quant_odd<T, true, BYTES>), grid, dim3(256), 0, st, o);
                else
                    hipLaunchKernelGGL((k_quant_odd<T, false, BYTES>), grid, dim3(256), 0, st, o);
            };
            if (odd_rows(o.w, o.ldw) || odd_rows(o.q, o.ldq))
                launch(std::true_type());
            else
                launch(std::false_type());
            sums();
            continue;
        }
        PackArgs p{};
        p.d = a.d;
        p.dp = q.dp;
        if (pw && !packed) p.o[0] = {a.w, a.v, a.ldw, (int8_t*)ws + q.o_w};
        packed = true;
        if (pq) p.o[1] = {a.q + r0 * a.ldq, rows, a.ldq, (int8_t*)ws + q.o_q};
        const int64_t most = p.o[0].rows > p.o[1].rows ? p.o[0].rows : p.o[1].rows;
        if (most > 0) {
            const int64_t b = ((most + 7) / 8 * (q.dp / QT_STEP) + 3) / 4;
            hipLaunchKernelGGL(k_quant_pack, dim3((unsigned)(b < 65536 ? b : 65536), 2), dim3(256), 0, st, p);
        }
        t.in.b = (const uint16_t*)(pq ? (const int8_t*)ws + q.o_q : a.q + r0 * a.ldq);
        t.in.ldb = pq ? GK : a.ldq / 2;
        t.in.step_b = pq ? rows * GK : GK;
        with_tile(c.tile, [&](auto id) {
            using C = Tile<decltype(id)::value>;
            t.mt = (a.v + C::BM - 1) / C::BM;
            t.nt = (int32_t)((rows + C::BN - 1) / C::BN);
            unsigned grid = tile_grid(t.mt, t.nt);
            const dim3 block(64 * C::WM * C::WN);
            if (c.split > 1) {
                hipLaunchKernelGGL((k_quant_tiles<T, C::BM, C::BN, C::WM, C::WN, true>), dim3(grid, c.split), block, 0,
                                   st, t);
            } else {
                const unsigned most_at_once = 256u * QUANT_COST[decltype(id)::value].per_cu;
                if (grid > most_at_once) grid = most_at_once;
                hipLaunchKernelGGL((k_quant_tiles<T, C::BM, C::BN, C::WM, C::WN, false>), dim3(grid), block, 0, st, t);
            }
        });
        sums();
    }
    return hipGetLastError();
}

}  // namespace gmm

using namespace gmm;

extern "C" {

int gmm_quantize_rows(const void* x, int64_t n, int32_t d, int64_t ldx, int32_t dtype, int8_t* q,
                      int64_t ldq, float* scale, void* stream) {
    if (dtype != GMM_F32 && dtype != GMM_BF16) return GMM_E_DTYPE;
    if (n < 0 || n > SC_MAX_ROWS || d < 1 || ldx < d || ldq < d) return GMM_E_INVALID;
    if (d > QU_MAX_DIM) return GMM_E_UNSUPPORTED;
    if (n > 0 && (!x || !q || !scale)) return GMM_E_INVALID;
    if (n == 0) return GMM_OK;
    const QuantArgs a{x, q, scale, n, ldx, ldq, d};
    if (dtype == GMM_F32)
        quant_rows<float>(a, (hipStream_t)stream);
    else
        quant_rows<uint16_t>(a, (hipStream_t)stream);
    return hipGetLastError() == hipSuccess ? GMM_OK : GMM_E_HIP;
}

static bool product_sizes_ok(int64_t n, int32_t d, int32_t v) {
    return n >= 0 && n <= SC_MAX_ROWS && d >= 1 && v >= 1 && d <= QU_MAX_DIM && v <= QU_MAX_CODES;
}

size_t gmm_quantized_product_workspace_bytes(int64_t n, int32_t d, int32_t v) {
    return product_sizes_ok(n, d, v) ? quant_most_bytes(n, d, v) : 0;
}

size_t gmm_quantized_product_call_workspace_bytes(const int8_t* q, int64_t n, int32_t d, int64_t ldq,
                                                  const int8_t* w, int32_t v, int64_t ldw) {
    if (!product_sizes_ok(n, d, v) || ldq < d || ldw < d) return 0;
    return quant_plan(n, d, v, !quant_direct(q, d, ldq), !quant_direct(w, d, ldw)).bytes;
}

int gmm_quantized_product(const int8_t* q, int64_t n, int32_t d, int64_t ldq, const float* q_scale,
                          const int8_t* w, int32_t v, int64_t ldw, const float* w_scale, void* y,
                          int64_t ldy, int32_t dtype, void* workspace, size_t workspace_bytes,
                          void* stream) {
    if (dtype != GMM_F32 && dtype != GMM_BF16) return GMM_E_DTYPE;
    if (n < 0 || n > SC_MAX_ROWS || d < 1 || v < 1 || ldq < d || ldw < d || ldy < v) return GMM_E_INVALID;
    if (d > QU_MAX_DIM || v > QU_MAX_CODES) return GMM_E_UNSUPPORTED;
    if (n > 0 && (!q || !q_scale || !w || !w_scale || !y)) return GMM_E_INVALID;
    const QuantPlan plan = quant_plan(n, d, v, !quant_direct(q, d, ldq), !quant_direct(w, d, ldw));
    if (!workspace || workspace_bytes < plan.bytes || (uintptr_t)workspace % 256 != 0) return GMM_E_WORKSPACE;
    if (n == 0) return GMM_OK;
    const ProductArgs a{q, w, q_scale, w_scale, y, n, ldq, ldw, ldy, d, v};
    const hipError_t e = dtype == GMM_F32 ? quant_product<float>(a, plan, (char*)workspace, (hipStream_t)stream)
                                          : quant_product<uint16_t>(a, plan, (char*)workspace, (hipStream_t)stream);
    return e == hipSuccess ? GMM_OK : GMM_E_HIP;
}

}  // extern "C"
