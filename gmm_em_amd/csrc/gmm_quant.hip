// gmm_quant.hip - rows in 8-bit integers and their products (gmm_quantize_rows,
// gmm_quantized_product, declared in include/gmm_em.h):
//   s_r = max |x_r| / 127,  q = x / s_r to the nearest integer;   y = (sum q w) s_q s_w
// Products of 8-bit integers and their sums are exact in 32 bits, so the order of the sum
// and the kernel that makes it leave no trace in y.
//
// k_quant_few: few rows. The product is the reading of w: 16 weight rows by 16 rows of q
// per matrix instruction, both straight from memory, the contracted axis split over the
// waves and joined in LDS.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "gmm_em.h"
#include "gmm_nn.h"
#include "gmm_softmax.h"

namespace gmm {

constexpr int32_t QU_MAX_DIM = (1 << 17) - 1;  // 128 * 128 * d stays below 2^31
constexpr int32_t QU_MAX_CODES = 1 << 22;

typedef int i32x4 __attribute__((ext_vector_type(4)));

// ---- rows to integers

struct QuantArgs {
    const void* x;
    int8_t* q;
    float* scale;
    int64_t n, ldx, ldq;
    int32_t d;
};

// The integer nearest x / s, ties to the even one, within 127. The quotient's rounding is put
// right by the remainder, which is exact: |q| s is a few bits longer than s, and x - q s
// shorter than either.
__device__ __forceinline__ int quant(float x, float s, float inv) {
    float q = rintf(x * inv);
    const float r = fmaf(-q, s, x), a = fabsf(r), half = 0.5f * s;
    // a tie goes to the even integer; the estimate is off by one at most
    if (a > half || (a == half && (((int)q) & 1))) q += r > 0.f ? 1.f : -1.f;
    return (int)fminf(fmaxf(q, -127.f), 127.f);
}

// A workgroup per row: its largest value, then its integers (the row's second reading comes
// from the caches).
constexpr int QR_NT = 256;
template <typename T>
__global__ __launch_bounds__(QR_NT) void k_quant_rows(QuantArgs p) {
    constexpr int VE = Vec<T>::VE;
    __shared__ float part[QR_NT / 64];
    const int tid = threadIdx.x;
    for (int64_t row = blockIdx.x; row < p.n; row += gridDim.x) {
        const T* x = (const T*)p.x + row * p.ldx;
        int8_t* q = p.q + row * p.ldq;
        float m = 0.f;
        bool bad = false;
        for (int k = tid * VE; k < p.d; k += QR_NT * VE) {
            const Raw16 r = load_zero(x, k, (int64_t)p.d);
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                const float v = fabsf(Vec<T>::get(r, j));
                m = fmaxf(m, v);
                bad |= !(v < INFINITY);
            }
        }
        m = wave_max(bad ? INFINITY : m);
        if ((tid & 63) == 0) part[tid >> 6] = m;
        __syncthreads();
        m = part[0];
#pragma unroll
        for (int w = 1; w < QR_NT / 64; ++w) m = fmaxf(m, part[w]);
        float s = m < INFINITY ? m / 127.f : NAN;
        if (tid == 0) p.scale[row] = s;
        const bool zero = !(s > 0.f);
        // rows whose 1 / s would leave fp32 are divided 2^100 higher up, where nothing is rounded
        const float up = s < 0x1p-100f ? 0x1p100f : 1.f;
        s *= up;
        const float inv = zero ? 0.f : 1.f / s;
        for (int k = tid * VE; k < p.d; k += QR_NT * VE) {
            const Raw16 r = load_zero(x, k, (int64_t)p.d);
#pragma unroll
            for (int j = 0; j < VE; ++j)
                if (k + j < p.d) q[k + j] = zero ? 0 : (int8_t)quant(Vec<T>::get(r, j) * up, s, inv);
        }
        __syncthreads();
    }
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
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c,
                                                 0, 0, 0);
}

// 16 bytes of a row, 0 at or past `end`.
__device__ __forceinline__ Raw16 load_bytes(const int8_t* p, int i, int end) {
    if (i + 16 <= end) return *reinterpret_cast<const Raw16*>(p + i);
    Raw16 r = {{0u, 0u, 0u, 0u}};
#pragma unroll
    for (int k = 0; k < 16; ++k)
        if (i + k < end) r.w[k >> 2] |= (uint32_t)(uint8_t)p[i + k] << (8 * (k & 3));
    return r;
}

template <typename T>
__device__ __forceinline__ T scaled_sum(int acc, float qs, float ws) {
    return Vec<T>::store((float)acc * qs * ws);
}

constexpr int QF_W = 4;
template <typename T, int TT>
__global__ __launch_bounds__(64 * QF_W) void k_quant_few(ProductArgs p) {
    __shared__ int sh[QF_W][TT][64][4];
    const int tid = threadIdx.x, lane = tid & 63, h = lane >> 4, i = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t mt = (p.v + 15) / 16, nt = (p.n + 16 * TT - 1) / (16 * TT);
    for (int64_t item = blockIdx.x; item < mt * nt; item += gridDim.x) {
        const int64_t c0 = item % mt * 16, r0 = item / mt * (16 * TT);
        const int8_t* w = p.w + (c0 + i < p.v ? c0 + i : p.v - 1) * p.ldw;
        const int8_t* q[TT];
        i32x4 acc[TT];
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const int64_t r = r0 + t * 16 + i;
            q[t] = p.q + (r < p.n ? r : p.n - 1) * p.ldq;
            acc[t] = i32x4{0, 0, 0, 0};
        }
        for (int k = wave * 64 + h * 16; k - h * 16 < p.d; k += 64 * QF_W) {
            const Raw16 a = load_bytes(w, k, p.d);
#pragma unroll
            for (int t = 0; t < TT; ++t) acc[t] = mfma_i8(a, load_bytes(q[t], k, p.d), acc[t]);
        }
#pragma unroll
        for (int t = 0; t < TT; ++t) *(i32x4*)sh[wave][t][lane] = acc[t];
        __syncthreads();
        // lane (h, i) of a tile holds codes 4 h .. 4 h + 3 of row i
        for (int t = wave; t < TT; t += QF_W) {
            const int64_t r = r0 + t * 16 + i;
            if (r >= p.n) continue;
            const float qs = p.q_scale[r];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t c = c0 + 4 * h + j;
                if (c >= p.v) continue;
                int s = 0;
#pragma unroll
                for (int x = 0; x < QF_W; ++x) s += sh[x][t][lane][j];
                ((T*)p.y)[r * p.ldy + c] = scaled_sum<T>(s, qs, p.w_scale[c]);
            }
        }
        __syncthreads();
    }
}

template <typename T>
static hipError_t quant_product(const ProductArgs& a, char* ws, hipStream_t st) {
    (void)ws;
    const int64_t mt = (a.v + 15) / 16;
    auto grid = [&](int rows) {
        const int64_t b = mt * ((a.n + rows - 1) / rows), most = (int64_t)1 << 22;
        return dim3((unsigned)(b < most ? b : most));
    };
    if (a.n <= 16)
        hipLaunchKernelGGL((k_quant_few<T, 1>), grid(16), dim3(64 * QF_W), 0, st, a);
    else
        hipLaunchKernelGGL((k_quant_few<T, 4>), grid(64), dim3(64 * QF_W), 0, st, a);
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
    const int64_t most = (int64_t)1 << 22;
    const dim3 grid((unsigned)(n < most ? n : most));
    if (dtype == GMM_F32)
        hipLaunchKernelGGL((k_quant_rows<float>), grid, dim3(QR_NT), 0, (hipStream_t)stream, a);
    else
        hipLaunchKernelGGL((k_quant_rows<uint16_t>), grid, dim3(QR_NT), 0, (hipStream_t)stream, a);
    return hipGetLastError() == hipSuccess ? GMM_OK : GMM_E_HIP;
}

size_t gmm_quantized_product_workspace_bytes(int64_t n, int32_t d, int32_t v) {
    if (n < 0 || n > SC_MAX_ROWS || d < 1 || v < 1 || d > QU_MAX_DIM || v > QU_MAX_CODES) return 0;
    return 256;
}

int gmm_quantized_product(const int8_t* q, int64_t n, int32_t d, int64_t ldq, const float* q_scale,
                          const int8_t* w, int32_t v, int64_t ldw, const float* w_scale, void* y,
                          int64_t ldy, int32_t dtype, void* workspace, size_t workspace_bytes,
                          void* stream) {
    if (dtype != GMM_F32 && dtype != GMM_BF16) return GMM_E_DTYPE;
    if (n < 0 || n > SC_MAX_ROWS || d < 1 || v < 1 || ldq < d || ldw < d || ldy < v) return GMM_E_INVALID;
    if (d > QU_MAX_DIM || v > QU_MAX_CODES) return GMM_E_UNSUPPORTED;
    if (n > 0 && (!q || !q_scale || !w || !w_scale || !y)) return GMM_E_INVALID;
    if (!workspace || workspace_bytes < gmm_quantized_product_workspace_bytes(n, d, v) ||
        (uintptr_t)workspace % 256 != 0)
        return GMM_E_WORKSPACE;
    if (n == 0) return GMM_OK;
    const ProductArgs a{q, w, q_scale, w_scale, y, n, ldq, ldw, ldy, d, v};
    const hipError_t e = dtype == GMM_F32 ? quant_product<float>(a, (char*)workspace, (hipStream_t)stream)
                                          : quant_product<uint16_t>(a, (char*)workspace, (hipStream_t)stream);
    return e == hipSuccess ? GMM_OK : GMM_E_HIP;
}

}  // extern "C"
