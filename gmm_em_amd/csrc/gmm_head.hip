// gmm_head.hip - the scores of a head (logits x = h W^T of rows h under a code
// matrix W) and their gradients, without the n x v matrix of logits
// (gmm_head_score, gmm_head_score_backward, declared in include/gmm_em.h).
//
// Scores without alternatives: each tile of logits stays in the accumulators
// of the product (gmm_gemm.h); its epilogue turns it into one (max, sum exp,
// sum exp (l - max)) per row and tile, and the row's parts are joined by a
// second kernel. With alternatives (m > 0), chunks of rows are written as
// fp32 logits into the workspace and scored from there.
// Gradient: the logits' tiles are computed again, and the epilogue turns them
// into dx = scale (g_lp ([v = t] - p) - g_H p (log p + H)), written for a chunk of
// rows, from which two more products make dh = dx W and dW = dx^T h (the latter
// reads dx across, see gmm_gemm.h). For fp32 data dx is cut into three planes like the
// operands. For bf16 data dx is rounded to fp16, whose 11 bits leave an eighth
// of bf16's error at the same rate; W and h (8 bits each) go into fp16
// unrounded. fp16's short range is met by powers of two taken out of the sums
// again: dx's rows are multiplied by their own bounds' (a row of small gradients keeps its
// digits); W by one for each dim, to a largest value in [2^14, 2^15); h by one for each dim
// too, after its rows are divided by what dx's were multiplied by (so that rows count by
// what they can add to dW, and those without a gradient not at all). What then lies
// below 2^-29 of the largest of its dim or row loses digits, and below 2^-39 is dropped.
// Measured, bf16, 8192 x 768 x 16384 (medians of one trace): scores 197 us: tiles 192 (the
// product without epilogue 148; the softmax of an accumulator is 8 operations and an
// exponential), join 5; gradient 705 us: ranges 14 + 5, dx 233, turned operands 16, dh 208 + 14
// for its split, dW 215. Bound by the matrix products (950 to 1400 TFLOP/s in them).
//
// Orientation: the tiles' rows are the axis that the outputs are contiguous in
// (codes for logits, dims for the gradients), their columns the rows of h (or
// the codes, for dW). A lane then holds four neighbouring values of an output
// row at a time, and of only TN rows: a row's softmax statistics are sums
// within a lane and over four lanes, and its constants stay in registers.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "gmm_em.h"
#include "gmm_gemm.h"
#include "gmm_nn.h"
#include "gmm_softmax.h"
#include "gmm_tiles.h"

namespace gmm {

constexpr int32_t HEAD_MAX_DIM = 1 << 20;
constexpr int32_t HEAD_MAX_CODES = 1 << 22;
constexpr int64_t HEAD_MAX_LD = (int64_t)1 << 22;  // 256 rows span at most 2^31 bytes
constexpr size_t HEAD_LOGIT_BYTES = (size_t)256 << 20;  // fp32 logits of one chunk of rows
constexpr size_t HEAD_PART_BYTES = (size_t)64 << 20;    // tile statistics of one chunk
constexpr size_t HEAD_DX_BYTES = (size_t)512 << 20;       // dx of one chunk
constexpr size_t HEAD_SPLIT_BYTES = (size_t)128 << 20;  // partial sums of a split product
constexpr int HEAD_MAX_SPLIT = 16;

// ---- operand planes

// Cuts a finite fp32 value into three bf16 values that add up to it exactly (where the third
// stays in bf16's range, above 2^-110). The upper two are rounded to nearest, so that the rest
// is at most 2^-8 and 2^-17 of a value in [1, 2), of either sign: cut off instead, 2^-7 and
// 2^-15 of the value's sign, and the products left out add up. An infinity becomes NaN: its
// product with another operand's planes is NaN where one of those is 0, and would be infinite
// elsewhere.
__device__ __forceinline__ void cut3(float x, uint16_t* p) {
    const uint32_t u = __float_as_uint(x);
    p[1] = p[2] = 0;
    if ((u & 0x7f800000u) == 0x7f800000u) {
        p[0] = 0x7fc0;
        return;
    }
    uint32_t hi = (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
    if ((hi & 0x7f80u) == 0x7f80u) hi = u >> 16;  // would round to infinity
    const float r = x - bf16_to_f32(hi);
    const uint32_t mid = f32_to_bf16(r);
    p[0] = (uint16_t)hi;
    p[1] = (uint16_t)mid;
    p[2] = (uint16_t)(__float_as_uint(r - bf16_to_f32(mid)) >> 16);
}

template <typename T>
struct Planes;
template <>
struct Planes<float> {
    static constexpr int P = 3;
    static __device__ __forceinline__ void cut(float x, uint16_t* p) { cut3(x, p); }
};
template <>
struct Planes<uint16_t> {
    static constexpr int P = 1;
    static __device__ __forceinline__ void cut(float x, uint16_t* p) {
        p[0] = (uint16_t)f32_to_bf16(x);
    }
};

// Operands laid out here lie in panels (gmm_gemm.h): [plane][c / 64][r][c % 64].
// Row-major they would be read as 256 pieces of 128 bytes, 32 KB apart, per step.
__device__ __forceinline__ int64_t panel_at(int64_t rows, int64_t r, int64_t c) {
    return ((c / GK) * rows + r) * GK + c % GK;
}

// An operand to be laid out: rows x d values of a caller's matrix.
struct Layout {
    const void* x;
    int64_t rows, ld;
    uint16_t* out;
};
// One launch lays out W and the first rows of h (blockIdx.y): rows == 0 is none.
struct LayoutPair {
    Layout o[2];
    int32_t d;
};

// The planes of x for c < kp, 0 past the d-th value; 8 values per thread.
template <typename T>
__global__ __launch_bounds__(256) void k_planes(LayoutPair p, int kp) {
    constexpr int P = Planes<T>::P;
    const Layout o = p.o[blockIdx.y];
    const int per = kp / 8;
    const int64_t total = o.rows * per, plane = o.rows * kp;
    for (int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x; j < total;
         j += (int64_t)gridDim.x * 256) {
        const int64_t r = j / per;
        const int c = (int)(j - r * per) * 8;
        const T* x = (const T*)o.x + r * o.ld;
        union {
            uint16_t v[8];
            uint4 q;
        } u[P];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            uint16_t cut[P];
            Planes<T>::cut(c + k < p.d ? Vec<T>::one(x + c + k) : 0.f, cut);
#pragma unroll
            for (int q = 0; q < P; ++q) u[q].v[k] = cut[q];
        }
#pragma unroll
        for (int q = 0; q < P; ++q) *(uint4*)(o.out + q * plane + panel_at(o.rows, r, c)) = u[q].q;
    }
}

// ---- fp16's powers of two

// The exponent e for which a value with these magnitude bits, times 2^e, lies in
// [2^14, 2^15); 0 for zero and for what is not finite. 2^e may lie outside fp32's
// range: it is applied with ldexpf.
__device__ __forceinline__ int range_of(uint32_t bits) {
    if (bits == 0 || bits >= 0x7f800000u) return 0;
    int e;
    (void)frexpf(__uint_as_float(bits), &e);  // in [2^(e-1), 2^e)
    return 15 - e;
}

constexpr int ROW_NONE = -(1 << 20);    // power of two of a row whose dx is 0
constexpr int KEY_NONE = -(1 << 30);    // of a dim without a finite value other than 0
constexpr int RANGE_COLS = 2048;        // dims of a workgroup: 8 per thread

// Row parts that the dims' ranges are made in: up to 512 workgroups for each of W and h, with 8
// rows or more of the longer of them.
inline int range_parts(int64_t n, int32_t v, int dp) {
    const int chunks = (dp + RANGE_COLS - 1) / RANGE_COLS;
    const int64_t most = chunks < 512 ? 512 / chunks : 1, rows = (n > v ? n : v) / 8;
    return (int)(rows < 1 ? 1 : rows < most ? rows : most);
}

struct RangeArgs {
    const uint16_t *h, *w;
    int64_t n, ldh, ldw;
    int32_t d, dp, v;
    ScoreGradArgs g;
    int32_t* part;     // [parts][2][dp]: W's and h's largest exponents
    int32_t* row_exp;  // [n]: dx's power of two for each row
};

// What dx's row can reach: |g_lp| + |g_H| max p |log p + H|, with p |log p| < 0.37.
__device__ __forceinline__ float grad_bound(const GradRow& g) {
    const float b = g.scale * (fabsf(g.glp) + fabsf(g.gh) * (0.375f + fabsf(g.h)));
    return fminf(b, 3.402823466e38f);  // NaN: any power of two leaves it so
}

// m[k]: the largest e with a value of the 8 dims below 2^e (row_exp: times 2^-row_exp[r]) over
// rows r, r + step, ... < end.
template <bool H>
__device__ __forceinline__ void dims_range(const uint16_t* x, int64_t ld, int c, int d, int64_t r,
                                           int64_t end, int step, const int32_t* row_exp, int* m) {
    constexpr int U = 4;  // rows in flight
    for (; r < end; r += U * step) {
        Raw16 v[U];
        int e[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t q = r + u * step < end ? r + u * step : r;
            v[u] = load_zero(x + q * ld, c, (int64_t)d);
            e[u] = H ? row_exp[q] : 0;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (H && e[u] == ROW_NONE) continue;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int b = (int)((v[u].w[k >> 1] >> (k & 1 ? 16 : 0)) & 0x7fffu);
                const int key = max(b >> 7, 1) - 126 - e[u];
                if (b != 0 && b < 0x7f80) m[k] = max(m[k], key);
            }
        }
    }
}

// The powers of two of dx's rows, and the largest exponents of W's and h's dims over a part
// of their rows. Reads W and h once: 38 MB (8192 x 768 x 16384) in 19 us.
__global__ __launch_bounds__(256) void k_head_range(RangeArgs p) {
    __shared__ __align__(16) int sh[256][8];
    const int tid = threadIdx.x;
    const int c0 = blockIdx.y * RANGE_COLS;
    const int left = (p.dp - c0) / 8, cols = left < 256 ? left : 256;  // vectors of a row
    const int per = 256 / cols, row = tid / cols, c = c0 + (tid - row * cols) * 8;
    const int64_t parts = gridDim.x, b = blockIdx.x;
    int m[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) m[k] = KEY_NONE;
    if (blockIdx.z == 0) {
        if (row < per)
            dims_range<false>(p.w, p.ldw, c, p.d, p.v * b / parts + row, p.v * (b + 1) / parts, per, nullptr, m);
    } else {
        const int64_t r0 = p.n * b / parts, r1 = p.n * (b + 1) / parts;
        for (int64_t r = r0 + tid; r < r1; r += 256) {
            const float most = grad_bound(grad_row(p.g, r));
            p.row_exp[r] = most == 0.f ? ROW_NONE : range_of(__float_as_uint(most));
        }
        __syncthreads();
        if (row < per) dims_range<true>(p.h, p.ldh, c, p.d, r0 + row, r1, per, p.row_exp, m);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) sh[tid][k] = m[k];
    __syncthreads();
    for (int j = tid; j < cols * 8; j += 256) {
        int o = KEY_NONE;
        for (int q = 0; q < per; ++q) o = max(o, sh[q * cols + j / 8][j % 8]);
        p.part[(b * 2 + blockIdx.z) * p.dp + c0 + j] = o;
    }
}

// The powers of two of W's dims (blockIdx.y 0) and of h's: 15 - the largest exponent.
__global__ __launch_bounds__(1024) void k_head_dims(const int32_t* part, int parts, int dp, int32_t* out) {
    __shared__ int sh[16][64];
    const int tid = threadIdx.x, c = blockIdx.x * 64 + (tid & 63);
    int m = KEY_NONE;
#pragma unroll 8
    for (int b = tid >> 6; b < parts; b += 16)
        m = max(m, part[((int64_t)b * 2 + blockIdx.y) * dp + c]);
    sh[tid >> 6][tid & 63] = m;
    __syncthreads();
    if (tid < 64) {
#pragma unroll
        for (int q = 1; q < 16; ++q) m = max(m, sh[q][tid]);
        out[(int64_t)blockIdx.y * dp + c] = m == KEY_NONE ? 0 : 15 - m;
    }
}

__device__ __forceinline__ uint16_t f32_to_f16(float f) {
    return __builtin_bit_cast(uint16_t, (_Float16)f);
}

// ---- transposed operands

// The planes of x^T: d rows of x's rows, padded with 0 to a multiple of 64: 64 x 64 tiles
// turned through LDS. bf16 values become fp16 times the power of two of their dim
// (dim_exp: W's dims, then h's), h's rows divided by dx's (row_exp).
template <typename T>
__global__ __launch_bounds__(256) void k_planes_t(LayoutPair p, const int32_t* dim_exp,
                                                  const int32_t* row_exp) {
    constexpr int P = Planes<T>::P;
    constexpr bool F16 = std::is_same<T, uint16_t>::value;
    constexpr int VE = Vec<T>::VE, PER_ROW = 64 / VE;  // vectors of a tile's row
    __shared__ __align__(16) uint16_t tile[P][64][72];
    const Layout o = p.o[blockIdx.y];
    const int ct = (p.d + 63) / 64;
    const int64_t rp = (o.rows + 63) / 64 * 64, total = ct * (rp / 64), plane = p.d * rp;
    const int tid = threadIdx.x;
    const int32_t* exps = dim_exp + (int64_t)blockIdx.y * (ct * 64);
    for (int64_t b = blockIdx.x; b < total; b += gridDim.x) {
        const int64_t r0 = b / ct * 64;
        const int c0 = (int)(b % ct) * 64;
        constexpr int N = 64 * PER_ROW / 256;  // vectors per thread
        Raw16 v[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int r = (k * 256 + tid) / PER_ROW, c = (k * 256 + tid) % PER_ROW * VE;
            v[k] = r0 + r < o.rows ? load_zero((const T*)o.x + (r0 + r) * o.ld, c0 + c, (int64_t)p.d)
                                   : Raw16{{0u, 0u, 0u, 0u}};
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int r = (k * 256 + tid) / PER_ROW, c = (k * 256 + tid) % PER_ROW * VE;
            const int down = F16 && blockIdx.y == 1 && r0 + r < o.rows ? row_exp[r0 + r] : 0;
#pragma unroll
            for (int u = 0; u < VE; ++u) {
                uint16_t cut[P];
                float y = Vec<T>::get(v[k], u);
                if constexpr (F16) {
                    // a row without gradient adds 0, whatever finite values it has
                    if (down == ROW_NONE && fabsf(y) < INFINITY) y = 0.f;
                    cut[0] = f32_to_f16(ldexpf(y, exps[c0 + c + u] - down));
                } else {
                    Planes<T>::cut(y, cut);
                }
#pragma unroll
                for (int q = 0; q < P; ++q) tile[q][c + u][r] = cut[q];
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int c = (k * 256 + tid) / 8, r = (k * 256 + tid) % 8 * 8;
            if (c0 + c < p.d)
#pragma unroll
                for (int q = 0; q < P; ++q)
                    *(uint4*)(o.out + q * plane + panel_at(p.d, c0 + c, r0 + r)) =
                        *(const uint4*)&tile[q][c][r];
        }
        __syncthreads();
    }
}

// ---- epilogues

struct HeadArgs {
    GemmIn in;           // a: codes, b: rows of h
    int32_t mt, nt;      // tiles of codes and rows
    int32_t rows;        // rows of this chunk (in.n)
    ScoreArgs s;         // s.v = in.m
    float* x;            // logits or target logits of the chunk
    ScorePart* part;     // [rows][mt]
    const float *norm, *entropy, *g_logprob, *g_entropy;
    uint16_t* dx;        // planes of rows x vp, in panels
    int64_t plane_dx;
    int32_t vp;
    const int32_t* row_exp;  // of dx's rows
};

__host__ __device__ __forceinline__ ScoreGradArgs grad_args(const HeadArgs& p) {
    ScoreGradArgs a{};
    a.v = p.s.v;
    a.scale = p.s.scale;
    a.targets = p.s.targets;
    a.norm = p.norm;
    a.entropy = p.entropy;
    a.g_logprob = p.g_logprob;
    a.g_entropy = p.g_entropy;
    return a;
}

// over the four lanes 16 apart that share a column of the accumulators
__device__ __forceinline__ float max4(float v) {
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float sum4(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// Statistics of each row over the tile's codes, and the targets' logits. Sums
// are of exp(l - max), the maximum subtracted before the exponential's factor log2 e.
template <bool ONE, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void k_head_stats(HeadArgs p) {
    using G = Gemm<BM, BN, WM, WN, ONE>;
    __shared__ __align__(16) unsigned char l0[G::STAGE], l1[G::STAGE];
    __shared__ float sh[WM * BN * 3];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const float scale = p.s.scale;
    gemm_walk<bf16x8, G, BM, BN>(p.in, p.mt, p.nt, l0, l1, [&](G& g, int m0, int n0) {
        const bool edge = m0 + BM > p.in.m;  // some of the tile's codes are not there
        const int code0 = m0 + G::row(0);
#pragma unroll
        for (int y = 0; y < G::TN; ++y) {
            const int r = n0 + G::col(y);
            if (edge) {
#pragma unroll
                for (int x = 0; x < G::TM; ++x)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (code0 + x * 16 + q >= p.in.m) g.acc[x][y][q] = -INFINITY;
            }
            float mx = -3.402823466e38f;
#pragma unroll
            for (int x = 0; x < G::TM; ++x)
#pragma unroll
                for (int q = 0; q < 4; ++q) mx = fmaxf(mx, g.acc[x][y][q]);
            mx = max4(mx);
            const float m = fmaxf(scaled(mx, scale), -3.402823466e38f);  // finite where all are masked
            float s = 0.f, a = 0.f;
#pragma unroll
            for (int x = 0; x < G::TM; ++x)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float d = scaled(g.acc[x][y][q], scale) - m;
                    const float e = exp_neg(d);
                    s += e;
                    a = fmaf(e, d, a);
                }
            if (a != a) {
                // a masked code's 0 * -inf: once more with the difference cut (the cut in
                // every sum costs 4 of 196 us at 8192 x 768 x 16384)
                a = 0.f;
#pragma unroll
                for (int x = 0; x < G::TM; ++x)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float d = scaled(g.acc[x][y][q], scale) - m;
                        a = fmaf(exp_neg(d), fmaxf(d, -1000.f), a);
                    }
            }
            s = sum4(s);
            a = sum4(a);
            if (lane < 16) {
                float* o = sh + (wave / WN * BN + G::col(y)) * 3;
                o[0] = m;
                o[1] = s;
                o[2] = a;
            }
            if (p.s.targets && r < p.in.n) {
                const int t = p.s.targets[r], u = t - code0;
                if (t < p.in.m && u >= 0 && u < 16 * G::TM && (u & 12) == 0) {
                    float v = 0.f;
#pragma unroll
                    for (int x = 0; x < G::TM; ++x)
#pragma unroll
                        for (int q = 0; q < 4; ++q) v = u == x * 16 + q ? g.acc[x][y][q] : v;
                    p.x[r] = v;
                }
            }
        }
        __syncthreads();
        if (tid < BN && n0 + tid < p.in.n) {
            Stats st{sh[tid * 3], sh[tid * 3 + 1], sh[tid * 3 + 2]};
#pragma unroll
            for (int w = 1; w < WM; ++w) {
                const float* o = sh + (w * BN + tid) * 3;
                st.join(o[0], o[1], o[2]);
            }
            p.part[(int64_t)(n0 + tid) * p.mt + m0 / BM] = ScorePart{st.m, st.s, st.a};
        }
    });
}

// One wave per row joins its tiles' statistics.
__global__ __launch_bounds__(256) void k_head_join(HeadArgs p) {
    const int lane = threadIdx.x & 63;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (row >= p.rows) return;
    Stats st;
    st.clear();
    for (int t = lane; t < p.mt; t += 64) {
        const ScorePart q = p.part[row * p.mt + t];
        st.join(q.m, q.s, q.a);
    }
    st.wave_join();
    score_out(p.s, row, st, p.x[row], -INFINITY, -1, lane);
}

// fp32 logits of a chunk of rows, row stride v.
template <bool ONE, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void k_head_logits(HeadArgs p) {
    using G = Gemm<BM, BN, WM, WN, ONE>;
    __shared__ __align__(16) unsigned char l0[G::STAGE], l1[G::STAGE];
    int tm, tn;
    if (!gemm_tile(blockIdx.x, p.mt, p.nt, &tm, &tn)) return;
    const int m0 = tm * BM, n0 = tn * BN;
    G g;
    g.begin(p.in, m0, n0, 0, G::all_steps(p.in), l0, l1);
    g.template finish<bf16x8>(p.in, m0, n0, l0, l1);
    const bool fours = p.in.m % 4 == 0;  // rows start at 16-byte boundaries
#pragma unroll
    for (int y = 0; y < G::TN; ++y) {
        const int r = n0 + G::col(y);
        if (r >= p.in.n) continue;
        float* o = p.x + (int64_t)r * p.in.m;
#pragma unroll
        for (int x = 0; x < G::TM; ++x) {
            const int c = m0 + G::row(x);
            if (fours) {
                if (c < p.in.m) *(f32x4*)(o + c) = g.acc[x][y];
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (c + q < p.in.m) o[c + q] = g.acc[x][y][q];
            }
        }
    }
}

// dx of a chunk of rows; 0 in the padding.
template <typename T, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void k_head_dx(HeadArgs p) {
    using G = Gemm<BM, BN, WM, WN, std::is_same<T, uint16_t>::value>;
    constexpr int P = Planes<T>::P;
    constexpr bool F16 = std::is_same<T, uint16_t>::value;
    __shared__ __align__(16) unsigned char l0[G::STAGE], l1[G::STAGE];
    gemm_walk<bf16x8, G, BM, BN>(p.in, p.mt, p.nt, l0, l1, [&](G& g, int m0, int n0) {
        const bool edge = m0 + BM > p.in.m;  // some of the tile's codes are not there
#pragma unroll
        for (int y = 0; y < G::TN; ++y) {
            const int r = n0 + G::col(y);
            if (r >= p.in.n) continue;
            const GradRow k = grad_row(grad_args(p), r);
            // the scale and the row's power of two go into the gradients
            const int up = F16 ? p.row_exp[r] : 0;
            const float gh = -ldexpf(k.scale * k.gh, up);
            const float base = -ldexpf(k.scale * fmaf(k.gh, k.h, k.glp), up);
            const float hot = ldexpf(k.scale * k.glp, up);
            const int t4 = k.t & ~3;  // the four that the target is among
#pragma unroll
            for (int x = 0; x < G::TM; ++x) {
                const int c = m0 + G::row(x);
                float v[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float lp = (scaled(g.acc[x][y][q], k.scale) - k.m) - k.logs;
                    v[q] = exp_neg(lp) * fmaf(gh, fmaxf(lp, -1000.f), base);  // 0 for a masked code
                }
                if (c == t4) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (c + q == k.t) v[q] += hot;
                }
                if (edge) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (c + q >= p.in.m) v[q] = 0.f;
                }
                uint16_t o[P][4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint16_t cut[P];
                    if (F16)
                        cut[0] = f32_to_f16(v[q]);
                    else
                        Planes<T>::cut(v[q], cut);
#pragma unroll
                    for (int j = 0; j < P; ++j) o[j][q] = cut[j];
                }
                if (c < p.vp)  // vp is a multiple of 64: whole fours
#pragma unroll
                    for (int j = 0; j < P; ++j)
                        *(uint2*)(p.dx + j * p.plane_dx + panel_at(p.in.n, r, c)) =
                            uint2{(uint32_t)o[j][0] | ((uint32_t)o[j][1] << 16),
                                  (uint32_t)o[j][2] | ((uint32_t)o[j][3] << 16)};
            }
        }
    });
}

struct GradOut {
    GemmIn in;         // a: dims, b: rows of the output
    int32_t mt, nt;
    int32_t split;     // parts of the contracted axis: blockIdx.y
    float* part;       // [split][n][m], split > 1
    const float* add;  // sum of the earlier chunks, n x m, or null
    float* sum;        // where the sum so far goes, or null: the result goes to out
    void* out;
    int64_t ldo;
    int32_t fours;     // wide stores: see grad_store
    // fp16 operands: the powers of two of the dims and, where they are given, of the rows
    const int32_t *dim_exp, *row_exp;
};

// The powers of two of four neighbouring dims, c a multiple of 4 (dim_exp is padded to 64).
template <typename T>
__device__ __forceinline__ int4 grad_dims(const GradOut& p, int c) {
    if (std::is_same<T, uint16_t>::value) return *(const int4*)(p.dim_exp + c);
    return int4{0, 0, 0, 0};
}

// Four neighbouring values of row r from dim c on (dim: grad_dims), summed over the split already.
// p.fours: every row starts at a multiple of four values, m is one too.
template <typename T>
__device__ __forceinline__ void grad_store(const GradOut& p, int64_t r, int c, f32x4 v, int4 dim) {
    if (std::is_same<T, uint16_t>::value) {
        const int row = p.row_exp ? p.row_exp[r] : 0;
        const int by[4] = {dim.x + row, dim.y + row, dim.z + row, dim.w + row};
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = ldexpf(v[q], -by[q]);
    }
    const int64_t at = r * p.in.m + c;
    if (p.fours) {
        if (p.add) v += *(const f32x4*)(p.add + at);
        if (p.sum) {
            *(f32x4*)(p.sum + at) = v;
        } else if constexpr (std::is_same<T, uint16_t>::value) {
            *(uint2*)((T*)p.out + r * p.ldo + c) =
                uint2{f32_to_bf16(v[0]) | (f32_to_bf16(v[1]) << 16),
                      f32_to_bf16(v[2]) | (f32_to_bf16(v[3]) << 16)};
        } else {
            *(f32x4*)((T*)p.out + r * p.ldo + c) = v;
        }
        return;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (c + q >= p.in.m) break;
        float y = v[q];
        if (p.add) y += p.add[at + q];
        if (p.sum)
            p.sum[at + q] = y;
        else
            ((T*)p.out)[r * p.ldo + c + q] = Vec<T>::store(y);
    }
}

template <typename T, bool TB, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void k_head_grad(GradOut p) {
    using G = Gemm<BM, BN, WM, WN, std::is_same<T, uint16_t>::value, TB>;
    __shared__ __align__(16) unsigned char l0[G::STAGE], l1[G::STAGE];
    int tm, tn;
    if (!gemm_tile(blockIdx.x, p.mt, p.nt, &tm, &tn)) return;
    const int m0 = tm * BM, n0 = tn * BN;
    constexpr bool F16 = std::is_same<T, uint16_t>::value;
    const int steps = G::all_steps(p.in);
    const int z = blockIdx.y;
    G g;
    g.begin(p.in, m0, n0, (int)((int64_t)steps * z / p.split),
            (int)((int64_t)steps * (z + 1) / p.split), l0, l1);
    g.template finish<std::conditional_t<F16, f16x8, bf16x8>>(p.in, m0, n0, l0, l1);
    int4 dim[G::TM];
#pragma unroll
    for (int x = 0; x < G::TM; ++x) {
        const int c = m0 + G::row(x);
        dim[x] = p.split > 1 || c >= p.in.m ? int4{0, 0, 0, 0} : grad_dims<T>(p, c);
    }
#pragma unroll
    for (int y = 0; y < G::TN; ++y) {
        const int r = n0 + G::col(y);
        if (r >= p.in.n) continue;
#pragma unroll
        for (int x = 0; x < G::TM; ++x) {
            const int c = m0 + G::row(x);
            if (c >= p.in.m) continue;
            if (p.split > 1) {
                float* o = p.part + ((int64_t)z * p.in.n + r) * p.in.m + c;
                if (p.in.m % 4 == 0) {
                    *(f32x4*)o = g.acc[x][y];
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (c + q < p.in.m) o[q] = g.acc[x][y][q];
                }
            } else {
                grad_store<T>(p, r, c, g.acc[x][y], dim[x]);
            }
        }
    }
}

// The sum over a split product's parts, in order.
template <typename T>
__global__ __launch_bounds__(256) void k_head_sum(GradOut p) {
    const int per = (p.in.m + 3) / 4;
    const int64_t total = (int64_t)p.in.n * per;
    for (int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x; j < total;
         j += (int64_t)gridDim.x * 256) {
        const int64_t r = j / per;
        const int c = (int)(j - r * per) * 4;
        f32x4 v{0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
        for (int z = 0; z < p.split; ++z) {
            const float* o = p.part + ((int64_t)z * p.in.n + r) * p.in.m + c;
            if (p.in.m % 4 == 0) {
                v += *(const f32x4*)o;
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (c + q < p.in.m) v[q] += o[q];
            }
        }
        grad_store<T>(p, r, c, v, grad_dims<T>(p, c));
    }
}

// ---- host side

// Costs of the tiles. per_step: measured over long products of bf16 rows read in place, per workgroup with the chip
// full; the gradients' operands take longer (a step of 192 x 256 1.6 us), all tiles alike.
// What it picks against the best of the four tiles with splits of 1, 2, 4, 8 and 16 (microseconds of
// a call for dh, for dW; in those dx has the tile too), bf16: 8192 x 768 x 16384 469 and 461 (469,
// 474), 4096 x 1024 x 8192 179 and 155 (167, 167), 2048 x 512 x 32768 188 and 170 (206, 170), 1024 x
// 768 x 4096 50 and 44 (49, 44), 300 x 256 x 5000 37 and 26 (36, 26); fp32: 2048 x 768 x 8192 315 and
// 309 (323, 326), 777 x 100 x 1001 35 and 34 (34, 32).
constexpr TileCost TILE_COST[4] = {
    {256, 256, 256, 1.42f, 6.f}, {192, 256, 256, 1.12f, 6.f}, {128, 128, 512, 0.92f, 4.f},
    {64, 64, 1024, 0.55f, 3.f}};


// Workspace of a head call: operands that need laying out, then the chunk's
// scratch. Offsets in bytes; a part that is not needed takes none.
struct HeadPlan {
    int planes, pairs, dp, vp, np;
    int64_t chunk;      // rows per chunk, a multiple of 256
    bool pack_h, pack_w;
    size_t o_w, o_h, o_x, o_part, o_wt, o_ht, o_dx, o_sum, o_split, o_score, o_range, o_dims, o_exp, bytes;
};

static bool direct(const void* p, int32_t d, int64_t ld, int dtype) {
    return dtype == GMM_BF16 && d % GK == 0 && ld % 8 == 0 && ld <= HEAD_MAX_LD &&
           (uintptr_t)p % 16 == 0;
}

// pack_h, pack_w: whether hidden and weight have to be laid out (the sizing
// entry point assumes both, so its result serves every alignment).
static HeadPlan head_plan(int64_t n, int32_t d, int32_t v, int dtype, int32_t m, bool grad,
                          bool pack_h, bool pack_w) {
    HeadPlan q{};
    q.planes = dtype == GMM_F32 ? 3 : 1;
    q.pairs = dtype == GMM_F32 ? 6 : 1;
    q.dp = pad(d);
    q.vp = pad(v);
    q.pack_h = pack_h;
    q.pack_w = pack_w;
    const int64_t tiles = (v + 63) / 64;
    size_t row, most;
    if (grad) {
        row = (size_t)q.planes * q.vp * 2;
        most = HEAD_DX_BYTES;
    } else if (m > 0) {
        row = (size_t)v * 4;
        most = HEAD_LOGIT_BYTES;
    } else {
        row = (size_t)tiles * sizeof(ScorePart);
        most = HEAD_PART_BYTES;
    }
    int64_t chunk = (int64_t)(most / row) / 256 * 256;
    if (chunk < 256) chunk = 256;
    if (chunk > ((int64_t)1 << 20)) chunk = (int64_t)1 << 20;
    const int64_t all = (n + 255) / 256 * 256;
    q.chunk = chunk < all ? chunk : (all > 0 ? all : 256);
    q.np = (int)q.chunk;
    size_t off = 0;
    auto take = [&](size_t b) {
        const size_t o = off;
        off += up256(b);
        return o;
    };
    const size_t c = (size_t)q.chunk, ps = (size_t)q.planes * 2;
    q.o_w = take(pack_w ? ps * v * q.dp : 0);
    q.o_h = take(pack_h ? ps * c * q.dp : 0);
    q.o_x = take(grad ? 0 : (m > 0 ? c * v * 4 : c * 4));
    q.o_part = take(!grad && m == 0 ? c * tiles * sizeof(ScorePart) : 0);
    q.o_score = take(!grad && m > 0 ? score_plan(q.chunk, v, m).bytes + score_plan(1, v, m).bytes * 256 : 0);
    q.o_wt = take(grad ? ps * d * q.vp : 0);
    q.o_ht = take(grad ? ps * d * q.np : 0);
    q.o_dx = take(grad ? ps * c * q.vp : 0);
    q.o_sum = take(grad && q.chunk < n ? (size_t)v * d * 4 : 0);
    const size_t most_out = (size_t)(q.chunk > v ? q.chunk : v) * d * 4 * HEAD_MAX_SPLIT;
    q.o_split = take(grad ? (most_out < HEAD_SPLIT_BYTES ? most_out : HEAD_SPLIT_BYTES) : 0);
    const bool f16 = grad && dtype == GMM_BF16;
    q.o_range = take(f16 ? (size_t)range_parts(n, v, q.dp) * 2 * q.dp * sizeof(int32_t) : 0);
    q.o_dims = take(f16 ? (size_t)2 * q.dp * sizeof(int32_t) : 0);
    q.o_exp = take(f16 ? (size_t)n * sizeof(int32_t) : 0);
    q.bytes = off < 256 ? 256 : off;
    return q;
}

static bool head_shape_ok(int64_t n, int32_t d, int32_t v) {
    return n >= 0 && n <= SC_MAX_ROWS && d >= 1 && v >= 1;
}
static bool head_supported(int32_t d, int32_t v) { return d <= HEAD_MAX_DIM && v <= HEAD_MAX_CODES; }

template <typename T>
static void planes(const LayoutPair& p, int kp, hipStream_t st) {
    const int64_t rows = p.o[0].rows > p.o[1].rows ? p.o[0].rows : p.o[1].rows;
    const int64_t work = (rows * (kp / 8) + 255) / 256;
    const unsigned grid = (unsigned)(work < 65536 ? work : 65536);
    if (grid) hipLaunchKernelGGL((k_planes<T>), dim3(grid, 2), dim3(256), 0, st, p, kp);
}
template <typename T>
static void planes_t(const LayoutPair& p, const int32_t* dim_exp, const int32_t* row_exp,
                     hipStream_t st) {
    const int64_t rows = p.o[0].rows > p.o[1].rows ? p.o[0].rows : p.o[1].rows;
    const int64_t work = (int64_t)((p.d + 63) / 64) * ((rows + 63) / 64);
    const unsigned grid = (unsigned)(work < 65536 ? work : 65536);
    if (grid) hipLaunchKernelGGL((k_planes_t<T>), dim3(grid, 2), dim3(256), 0, st, p, dim_exp,
                                 row_exp);
}

// walk: the kernel's workgroups walk over the tiles, as many as the chip holds.
template <int ID, typename K, typename A>
static void launch_tiles(K kernel, A& a, int split, bool walk, hipStream_t st) {
    using C = Tile<ID>;
    a.mt = (a.in.m + C::BM - 1) / C::BM;
    a.nt = (a.in.n + C::BN - 1) / C::BN;
    unsigned grid = tile_grid(a.mt, a.nt);
    if (walk && grid > (unsigned)TILE_COST[ID].at_once) grid = TILE_COST[ID].at_once;
    hipLaunchKernelGGL(kernel, dim3(grid, split), dim3(64 * C::WM * C::WN), 0, st, a);
}

// out = the product of o.in, with the tile and split that suit it.
template <typename T, bool TB>
static void launch_grad(GradOut& o, float* part, hipStream_t st) {
    const Choice c = choose_tile(TILE_COST, o.in.m, o.in.n, (int64_t)o.in.kp / GK * o.in.pairs, HEAD_MAX_SPLIT,
                                 HEAD_SPLIT_BYTES);
    o.split = c.split;
    o.part = part;
    o.fours = o.in.m % 4 == 0 && o.ldo % 4 == 0 && (uintptr_t)o.out % (4 * sizeof(T)) == 0;
    with_tile(c.tile, [&](auto b) {
        constexpr int B = decltype(b)::value;
        using C = Tile<B>;
        launch_tiles<B>(k_head_grad<T, TB, C::BM, C::BN, C::WM, C::WN>, o, c.split, false, st);
    });
    if (c.split > 1) {
        const int64_t work = ((int64_t)o.in.n * ((o.in.m + 3) / 4) + 255) / 256;
        hipLaunchKernelGGL((k_head_sum<T>), dim3((unsigned)(work < 16384 ? work : 16384)), dim3(256), 0,
                           st, o);
    }
}

struct HeadIn {
    const void *h, *w;
    int64_t n, ldh, ldw;
    int32_t d, v, dtype;
};

// The logits' product for `rows` rows from r0 on: lays out what needs it (W with the
// first rows).
template <typename T>
static void head_rows(const HeadIn& x, const HeadPlan& q, char* ws, int64_t r0, int64_t rows, HeadArgs* a,
                      hipStream_t st) {
    const T* h = (const T*)x.h + r0 * x.ldh;
    GemmIn* g = &a->in;
    LayoutPair p{};
    p.d = x.d;
    g->pairs = q.pairs;
    g->kp = q.dp;
    g->m = x.v;
    g->n = a->rows = (int32_t)rows;
    if (q.pack_w) {
        g->a = (const uint16_t*)(ws + q.o_w);
        g->lda = GK;
        g->step_a = (int64_t)x.v * GK;
        g->plane_a = (int64_t)x.v * q.dp;
        if (r0 == 0) p.o[0] = Layout{x.w, x.v, x.ldw, (uint16_t*)(ws + q.o_w)};
    } else {
        g->a = (const uint16_t*)x.w;
        g->lda = x.ldw;
        g->step_a = GK;
    }
    if (q.pack_h) {
        g->b = (const uint16_t*)(ws + q.o_h);
        g->ldb = GK;
        g->step_b = rows * GK;
        g->plane_b = rows * q.dp;
        p.o[1] = Layout{h, rows, x.ldh, (uint16_t*)(ws + q.o_h)};
    } else {
        g->b = (const uint16_t*)h;
        g->ldb = x.ldh;
        g->step_b = GK;
    }
    planes<T>(p, q.dp, st);
}

template <typename T>
static hipError_t head_score(const HeadIn& x, const HeadPlan& q, ScoreArgs s, char* ws,
                             hipStream_t st) {
    HeadArgs a{};
    a.x = (float*)(ws + q.o_x);
    a.part = (ScorePart*)(ws + q.o_part);
    for (int64_t r0 = 0; r0 < x.n; r0 += q.chunk) {
        const int64_t rows = x.n - r0 < q.chunk ? x.n - r0 : q.chunk;
        head_rows<T>(x, q, ws, r0, rows, &a, st);
        a.s = s;
        a.s.n = rows;
        if (s.targets) {
            a.s.targets = s.targets + r0;
            a.s.logprob = s.logprob + r0;
        }
        if (s.entropy) a.s.entropy = s.entropy + r0;
        if (s.norm) a.s.norm = s.norm + 2 * r0;
        if (s.m > 0) {
            a.s.top_idx = s.top_idx + r0 * s.m;
            a.s.top_logprob = s.top_logprob + r0 * s.m;
        }
        const Choice c = choose_tile(TILE_COST, x.v, rows, (int64_t)q.dp / GK * q.pairs, 1, 0);
        with_tile(c.tile, [&](auto b) {
            constexpr int B = decltype(b)::value;
            constexpr bool ONE = Planes<T>::P == 1;
            using C = Tile<B>;
            if (s.m > 0)
                launch_tiles<B>(k_head_logits<ONE, C::BM, C::BN, C::WM, C::WN>, a, 1, false, st);
            else
                launch_tiles<B>(k_head_stats<ONE, C::BM, C::BN, C::WM, C::WN>, a, 1, true, st);
        });
        if (s.m > 0) {
            ScoreArgs l = a.s;
            l.x = a.x;
            l.ldl = x.v;
            const hipError_t e = launch_score(l, GMM_F32, ws + q.o_score, st);
            if (e != hipSuccess) return e;
        } else {
            hipLaunchKernelGGL(k_head_join, dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, st, a);
        }
    }
    return hipGetLastError();
}

template <typename T>
static hipError_t head_grad(const HeadIn& x, const HeadPlan& q, HeadArgs a, void* dh, int64_t lddh,
                            void* dw, int64_t lddw, char* ws, hipStream_t st) {
    uint16_t* wt = (uint16_t*)(ws + q.o_wt);
    uint16_t* ht = (uint16_t*)(ws + q.o_ht);
    int32_t* dim_exp = (int32_t*)(ws + q.o_dims);  // W's, h's
    int32_t* row_exp = (int32_t*)(ws + q.o_exp);
    float* part = (float*)(ws + q.o_split);
    if (std::is_same<T, uint16_t>::value) {
        RangeArgs r{};
        r.h = (const uint16_t*)x.h;
        r.w = (const uint16_t*)x.w;
        r.n = x.n;
        r.ldh = x.ldh;
        r.ldw = x.ldw;
        r.d = x.d;
        r.dp = q.dp;
        r.v = x.v;
        r.g = grad_args(a);
        r.part = (int32_t*)(ws + q.o_range);
        r.row_exp = row_exp;
        const int parts = range_parts(x.n, x.v, q.dp);
        hipLaunchKernelGGL(k_head_range, dim3(parts, (q.dp + RANGE_COLS - 1) / RANGE_COLS, 2), dim3(256),
                           0, st, r);
        hipLaunchKernelGGL(k_head_dims, dim3(q.dp / 64, 2), dim3(1024), 0, st, r.part, parts, q.dp, dim_exp);
    }
    a.dx = (uint16_t*)(ws + q.o_dx);
    a.vp = q.vp;
    const HeadArgs all = a;
    for (int64_t r0 = 0; r0 < x.n; r0 += q.chunk) {
        const int64_t rows = x.n - r0 < q.chunk ? x.n - r0 : q.chunk;
        head_rows<T>(x, q, ws, r0, rows, &a, st);
        a.row_exp = row_exp + r0;
        a.plane_dx = rows * q.vp;
        a.s.targets = all.s.targets ? all.s.targets + r0 : nullptr;
        a.norm = all.norm + 2 * r0;
        a.entropy = all.entropy ? all.entropy + r0 : nullptr;
        a.g_logprob = all.g_logprob ? all.g_logprob + r0 : nullptr;
        a.g_entropy = all.g_entropy ? all.g_entropy + r0 : nullptr;
        const Choice c = choose_tile(TILE_COST, x.v, rows, (int64_t)q.dp / GK * q.pairs, 1, 0);
        with_tile(c.tile, [&](auto b) {
            constexpr int B = decltype(b)::value;
            using C = Tile<B>;
            launch_tiles<B>(k_head_dx<T, C::BM, C::BN, C::WM, C::WN>, a, 1, true, st);
        });
        LayoutPair turned{};
        turned.d = x.d;
        if (dh && r0 == 0) turned.o[0] = Layout{x.w, x.v, x.ldw, wt};
        if (dw) turned.o[1] = Layout{(const T*)x.h + r0 * x.ldh, rows, x.ldh, ht};
        planes_t<T>(turned, dim_exp, a.row_exp, st);
        if (dh) {
            GradOut o{};
            o.in = GemmIn{wt, a.dx, GK, GK, (int64_t)x.d * GK, rows * GK, (int64_t)x.d * q.vp, a.plane_dx,
                          x.d, (int32_t)rows, q.vp, q.pairs};
            o.out = (T*)dh + r0 * lddh;
            o.ldo = lddh;
            o.dim_exp = dim_exp;
            o.row_exp = row_exp + r0;
            launch_grad<T, false>(o, part, st);
        }
        if (dw) {
            GradOut o{};
            // dx read across: panels of 64 codes, rows * 64 values each
            const int np = pad(rows);
            o.in = GemmIn{ht, a.dx, GK, rows, (int64_t)x.d * GK, GK * GK, (int64_t)x.d * np,
                          a.plane_dx, x.d, x.v, np, q.pairs, (int32_t)rows};
            float* sum = (float*)(ws + q.o_sum);
            o.add = r0 > 0 ? sum : nullptr;
            o.sum = r0 + q.chunk < x.n ? sum : nullptr;
            o.out = dw;
            o.ldo = lddw;
            o.dim_exp = dim_exp + q.dp;
            launch_grad<T, true>(o, part, st);
        }
    }
    return hipGetLastError();
}

// dw of no rows is 0
template <typename T>
__global__ __launch_bounds__(256) void k_head_zero(T* out, int64_t rows, int d, int64_t ld) {
    for (int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x; j < rows * d;
         j += (int64_t)gridDim.x * 256)
        out[j / d * ld + j % d] = 0;
}

}  // namespace gmm

using namespace gmm;

extern "C" {

size_t gmm_head_score_workspace_bytes(int64_t n, int32_t d, int32_t v, int32_t dtype, int32_t m) {
    if (!head_shape_ok(n, d, v) || !head_supported(d, v) || m < 0 || m > TOP_MAX || m > v) return 0;
    if (dtype != GMM_F32 && dtype != GMM_BF16) return 0;
    return head_plan(n, d, v, dtype, m, false, true, true).bytes;
}

size_t gmm_head_score_backward_workspace_bytes(int64_t n, int32_t d, int32_t v, int32_t dtype) {
    if (!head_shape_ok(n, d, v) || !head_supported(d, v)) return 0;
    if (dtype != GMM_F32 && dtype != GMM_BF16) return 0;
    return head_plan(n, d, v, dtype, 0, true, true, true).bytes;
}

int gmm_head_score(const void* hidden, int64_t n, int32_t d, int64_t ldh, const void* weight,
                   int32_t v, int64_t ldw, int32_t dtype, const int32_t* targets, int32_t m,
                   float scale, float* logprob, float* entropy, float* norm, int32_t* top_idx,
                   float* top_logprob, void* workspace, size_t workspace_bytes, void* stream) {
    if (dtype != GMM_F32 && dtype != GMM_BF16) return GMM_E_DTYPE;
    if (!head_shape_ok(n, d, v) || ldh < d || ldw < d || m < 0 || m > TOP_MAX || m > v ||
        !scale_ok(scale))
        return GMM_E_INVALID;
    if (!head_supported(d, v)) return GMM_E_UNSUPPORTED;
    if (n > 0 && (!hidden || !weight || (targets && !logprob) ||
                  (m > 0 && (!top_idx || !top_logprob))))
        return GMM_E_INVALID;
    const bool ph = !direct(hidden, d, ldh, dtype), pw = !direct(weight, d, ldw, dtype);
    const HeadPlan q = head_plan(n, d, v, dtype, m, false, ph, pw);
    if (!workspace || workspace_bytes < q.bytes || (uintptr_t)workspace % 256 != 0)
        return GMM_E_WORKSPACE;
    if (n == 0) return GMM_OK;
    const HeadIn x{hidden, weight, n, ldh, ldw, d, v, dtype};
    ScoreArgs s{};
    s.v = v;
    s.m = m;
    s.scale = scale;
    s.targets = targets;
    s.logprob = logprob;
    s.entropy = entropy;
    s.norm = norm;
    s.top_idx = top_idx;
    s.top_logprob = top_logprob;
    const hipError_t e =
        dtype == GMM_F32 ? head_score<float>(x, q, s, (char*)workspace, (hipStream_t)stream)
                         : head_score<uint16_t>(x, q, s, (char*)workspace, (hipStream_t)stream);
    return e == hipSuccess ? GMM_OK : GMM_E_HIP;
}

int gmm_head_score_backward(const void* hidden, int64_t n, int32_t d, int64_t ldh,
                            const void* weight, int32_t v, int64_t ldw, int32_t dtype,
                            const int32_t* targets, const float* norm, const float* entropy,
                            const float* g_logprob, const float* g_entropy, float scale,
                            void* d_hidden, int64_t lddh, void* d_weight, int64_t lddw,
                            void* workspace, size_t workspace_bytes, void* stream) {
    if (dtype != GMM_F32 && dtype != GMM_BF16) return GMM_E_DTYPE;
    if (!head_shape_ok(n, d, v) || ldh < d || ldw < d || !scale_ok(scale)) return GMM_E_INVALID;
    if ((d_hidden && lddh < d) || (d_weight && lddw < d) || (!d_hidden && !d_weight))
        return GMM_E_INVALID;
    if (!head_supported(d, v)) return GMM_E_UNSUPPORTED;
    if (n > 0 && (!hidden || !weight || !norm || (g_logprob && !targets) || (g_entropy && !entropy)))
        return GMM_E_INVALID;
    const bool ph = !direct(hidden, d, ldh, dtype), pw = !direct(weight, d, ldw, dtype);
    const HeadPlan q = head_plan(n, d, v, dtype, 0, true, ph, pw);
    if (!workspace || workspace_bytes < q.bytes || (uintptr_t)workspace % 256 != 0)
        return GMM_E_WORKSPACE;
    hipStream_t st = (hipStream_t)stream;
    if (n == 0) {
        if (d_weight) {
            const int64_t work = ((int64_t)v * d + 255) / 256;
            const dim3 grid((unsigned)(work < 4096 ? work : 4096));
            if (dtype == GMM_F32)
                hipLaunchKernelGGL((k_head_zero<float>), grid, dim3(256), 0, st, (float*)d_weight,
                                   (int64_t)v, d, lddw);
            else
                hipLaunchKernelGGL((k_head_zero<uint16_t>), grid, dim3(256), 0, st,
                                   (uint16_t*)d_weight, (int64_t)v, d, lddw);
        }
        return hipGetLastError() == hipSuccess ? GMM_OK : GMM_E_HIP;
    }
    const HeadIn x{hidden, weight, n, ldh, ldw, d, v, dtype};
    HeadArgs a{};
    a.s.targets = targets;
    a.s.scale = scale;
    a.s.v = v;
    a.norm = norm;
    a.entropy = entropy;
    a.g_logprob = g_logprob;
    a.g_entropy = g_entropy;
    const hipError_t e = dtype == GMM_F32
                             ? head_grad<float>(x, q, a, d_hidden, lddh, d_weight, lddw,
                                                (char*)workspace, st)
                             : head_grad<uint16_t>(x, q, a, d_hidden, lddh, d_weight, lddw,
                                                   (char*)workspace, st);
    return e == hipSuccess ? GMM_OK : GMM_E_HIP;
}

}  // extern "C"
