// gmm_gemm.h - tiles of C = A B^T on the 16-bit matrix units, the product under
// the head's kernels (gmm_head.hip). A is M x K and B is N x K, both with the
// contracted axis contiguous.
//
// fp32 operands come as three bf16 planes whose sum is the fp32 value bit for
// bit (24 bits in three cuts of 8): the product is then the sum of the six
// plane products that reach 2^-24 of it, smallest first, in the same fp32
// accumulators. bf16 and fp16 operands have one plane.
//
// A workgroup of WM x WN waves computes a BM x BN tile, 64 of the contracted
// axis per step: both operands' steps are copied from memory straight into LDS
// (two buffers; the next step's copies run under this step's products), 128
// bytes a row, its 16-byte pieces rotated by the row (piece p of row r lies at
// p ^ (r & 7)), so that the 16 rows that a wave reads at once lie in different
// banks. Rows past the operand's last read as 0 (the buffer's range check).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gmm_device.h"

namespace gmm {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x4 mfma32(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma32(f16x8 a, f16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

constexpr int GK = 64;  // contracted values per step

struct GemmIn {
    const uint16_t *a, *b;       // planes of M x kp and N x kp values, 16 bits each
    int64_t lda, ldb;            // row strides (values)
    int64_t plane_a, plane_b;    // plane strides (values)
    int32_t m, n, kp;            // kp: contracted length, a multiple of GK
    int32_t pairs;               // plane products: 1 or 6
};

// Plane products, smallest first: (lo,hi) (hi,lo) (mid,mid) (mid,hi) (hi,mid) (hi,hi).
__device__ __forceinline__ void gemm_pair(int pairs, int p, int* pa, int* pb) {
    const int q = pairs == 1 ? 5 : p;
    *pa = (0x052 >> (2 * q)) & 3;  // two bits each from the low end: 2 0 1 1 0 0
    *pb = (0x118 >> (2 * q)) & 3;  // 0 2 1 0 1 0
}

template <int BM, int BN, int WM, int WN>
struct Gemm {
    static constexpr int NT = 64 * WM * WN;
    static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;  // 16 x 16 blocks per wave
    static constexpr int A_BYTES = BM * GK * 2, B_BYTES = BN * GK * 2;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int LDS = 2 * STAGE;
    static constexpr int COPIES = STAGE / 1024 / (NT / 64);  // per wave and step

    f32x4 acc[TM][TN];

    // LDS byte offset of piece p of row r within an operand's step
    static __device__ __forceinline__ int at(int r, int p) { return r * 128 + ((p ^ (r & 7)) << 4); }

    // copies BR rows of one step: wave w takes every NT / 64-th group of 8 rows
    template <int BR>
    static __device__ __forceinline__ void copy(__amdgpu_buffer_rsrc_t rs, uint32_t row_bytes, int k,
                                                unsigned char* dst, int wave, int lane) {
        const int r = lane >> 3, p = lane & 7;
#pragma unroll
        for (int g = 0; g < BR / 8 / (NT / 64); ++g) {
            const int grp = g * (NT / 64) + wave;
            // row (8 grp + r) & 7 == r: the piece that belongs at place p is p ^ r
            const uint32_t off = (uint32_t)(grp * 8 + r) * row_bytes + (uint32_t)((p ^ r) << 4);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rs, (__attribute__((address_space(3))) void*)(dst + grp * 1024), 16, (int)off,
                k * 2, 0, 0);
        }
    }

    static __device__ __forceinline__ __amdgpu_buffer_rsrc_t rows(const uint16_t* base, int64_t ld,
                                                                  int64_t r0, int64_t total, int br,
                                                                  int kp) {
        const int64_t left = total - r0;
        const int64_t cnt = left < br ? left : br;
        // the last row ends at its kp-th value
        const int64_t bytes = cnt > 0 ? ((cnt - 1) * ld + kp) * 2 : 0;
        return __builtin_amdgcn_make_buffer_rsrc((void*)(base + r0 * ld), (short)0, (int)bytes,
                                                 BUF_RSRC_WORD3);
    }

    // Steps [first, last) of the tile at rows m0 and columns n0, into acc (V8: bf16x8 or
    // f16x8, the operands' type; a step is GK values of one plane product).
    // Each step is two halves of 32 values; a half's operands are read from LDS
    // while the half before is multiplied, and a step's copies are issued when
    // its buffer's last half has been read, a full step before they are needed.
    // Measured without epilogue, 256 x 256 tiles: 8192^3 746 us (1474 TFLOP/s),
    // 16384 x 8192 x 768 148 us (1389); with the wait left to the scheduler, which
    // moves it before the products, 164 us; with the copies and reads in front of
    // the products instead of between them 180 us.
    template <typename V8>
    __device__ __forceinline__ void run(const GemmIn& in, int m0, int n0, int first, int last,
                                        unsigned char* lds) {
        const int tid = threadIdx.x, lane = tid & 63;
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int wm = wave / WN, wn = wave % WN;
        const int h = lane >> 4, i = lane & 15;
#pragma unroll
        for (int x = 0; x < TM; ++x)
#pragma unroll
            for (int y = 0; y < TN; ++y) acc[x][y] = f32x4{0.f, 0.f, 0.f, 0.f};
        const int ks = in.kp / GK;
        const uint32_t ra = (uint32_t)in.lda * 2, rb = (uint32_t)in.ldb * 2;
        int pair = first / ks, kk = first - pair * ks;  // of the step to be copied next
        auto issue = [&](int buf) {
            int pa, pb;
            gemm_pair(in.pairs, pair, &pa, &pb);
            const __amdgpu_buffer_rsrc_t sa =
                rows(in.a + pa * in.plane_a, in.lda, m0, in.m, BM, in.kp);
            const __amdgpu_buffer_rsrc_t sb =
                rows(in.b + pb * in.plane_b, in.ldb, n0, in.n, BN, in.kp);
            unsigned char* d = lds + buf * STAGE;
            copy<BM>(sa, ra, kk * GK, d, wave, lane);
            copy<BN>(sb, rb, kk * GK, d + A_BYTES, wave, lane);
            if (++kk == ks) {
                kk = 0;
                ++pair;
            }
        };
        auto read = [&](V8(&fa)[TM], V8(&fb)[TN], int buf, int c) {
            const unsigned char* da = lds + buf * STAGE;
            const unsigned char* db = da + A_BYTES;
#pragma unroll
            for (int x = 0; x < TM; ++x)
                fa[x] = *(const V8*)(da + at((wm * TM + x) * 16 + i, 4 * c + h));
#pragma unroll
            for (int y = 0; y < TN; ++y)
                fb[y] = *(const V8*)(db + at((wn * TN + y) * 16 + i, 4 * c + h));
        };
        auto multiply = [&](const V8(&fa)[TM], const V8(&fb)[TN]) {
#pragma unroll
            for (int x = 0; x < TM; ++x)
#pragma unroll
                for (int y = 0; y < TN; ++y) acc[x][y] = mfma32(fa[x], fb[y], acc[x][y]);
        };
        // the order of a half: its copies and LDS reads one by one between the products
        auto spread = [&](const int copies) {
#pragma unroll
            for (int g = 0; g < copies; ++g) {
                __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);   // matrix product
                __builtin_amdgcn_sched_group_barrier(0x20, 1, 0);  // memory read
            }
#pragma unroll
            for (int g = 0; g < TM + TN; ++g) {
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // LDS read
                __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
            }
            __builtin_amdgcn_sched_group_barrier(0x8, TM * TN, 0);
        };
        const int steps = last - first;
        issue(0);
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        if (steps > 1) issue(1);
        V8 fa[2][TM], fb[2][TN];
        read(fa[0], fb[0], 0, 0);
        // one step; ahead: steps that follow it (2: at least two)
        auto step = [&](int buf, auto ahead) {
            constexpr int AHEAD = decltype(ahead)::value;
            read(fa[1], fb[1], buf, 1);
            multiply(fa[0], fb[0]);
            spread(0);
            // the wait stays behind the products: the copies of step s + 1 have
            // had a whole step to land
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (AHEAD > 0) {
                // this wave's copies of step s + 1 have landed, its reads of step s are done
                __builtin_amdgcn_s_waitcnt(0);
                __syncthreads();  // ... and every wave's
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (AHEAD > 1) issue(buf);
                read(fa[0], fb[0], buf ^ 1, 0);
            }
            multiply(fa[1], fb[1]);
            if constexpr (AHEAD > 0) spread(AHEAD > 1 ? COPIES : 0);
            __builtin_amdgcn_sched_barrier(0);
        };
        int s = 0;
        for (; s + 2 < steps; ++s) step(s & 1, std::integral_constant<int, 2>());
        if (s + 1 < steps) {
            step(s & 1, std::integral_constant<int, 1>());
            ++s;
        }
        step(s & 1, std::integral_constant<int, 0>());
        __syncthreads();  // LDS is free for the epilogue
    }
    template <typename V8>
    __device__ __forceinline__ void run(const GemmIn& in, int m0, int n0, unsigned char* lds) {
        run<V8>(in, m0, n0, 0, in.kp / GK * in.pairs, lds);
    }

    // row of this lane's first of four rows of blocks x, its column in blocks y
    static __device__ __forceinline__ int row(int x) {
        return ((threadIdx.x >> 6) / WN * TM + x) * 16 + 4 * ((threadIdx.x & 63) >> 4);
    }
    static __device__ __forceinline__ int col(int y) {
        return ((threadIdx.x >> 6) % WN * TN + y) * 16 + (threadIdx.x & 15);
    }
};

// Tile of workgroup b among mt x nt: the workgroups that one XCD receives
// (every eighth) take neighbouring tiles, walked in bands of 8 tile rows, so
// that its L2 serves their shared rows of A and B. The grid has 8 ceil(mt nt / 8)
// workgroups; false: none.
__device__ __forceinline__ bool gemm_tile(int64_t b, int mt, int nt, int* tm, int* tn) {
    const int64_t total = (int64_t)mt * nt, per = (total + 7) / 8;
    const int64_t id = (b & 7) * per + (b >> 3);
    if ((b >> 3) >= per || id >= total) return false;
    const int64_t band = (int64_t)8 * nt;
    const int b0 = (int)(id / band) * 8;
    const int rows = mt - b0 < 8 ? mt - b0 : 8;
    const int64_t in = id - (int64_t)b0 * nt;
    *tm = b0 + (int)(in % rows);
    *tn = (int)(in / rows);
    return true;
}

}  // namespace gmm
