// gmm_gemm.h - tiles of C = A B^T on the 16-bit matrix units, the product under
// the head's kernels (gmm_head.hip). A is M x K and B is N x K, both with the
// contracted axis contiguous.
//
// fp32 operands come as three bf16 planes whose sum is the fp32 value bit for
// bit (24 bits in three parts of 8, rounded to nearest): the product is then the sum
// of six plane products, smallest first, in the same fp32 accumulators; the three that are
// left out are below 2^-24 of it together, of either sign. bf16 and fp16 operands have one plane.
//
// B may also lie with the contracted axis across (TB): panels of 64 of its rows,
// [n / 64][k][64], as the product before wrote them with those rows contiguous. Its
// fragments are then read with the LDS's transposing load (16 lanes read four
// k of 16 rows and get four k of one row each), and k past the operand's end
// reads as 0.
//
// A workgroup of WM x WN waves computes a BM x BN tile, 64 of the contracted
// axis per step: both operands' steps are copied from memory straight into LDS
// (two buffers; the next step's copies run under this step's products; the
// buffers are variables of their own, so that the compiler sees that a read of one does
// not wait for the copies into the other), 128
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

// An operand is either rows as a caller has them (row stride ld, GK values from one
// step to the next) or panels: the GK values of a step of all rows lie together
// (row stride GK), so that a tile's step is one piece of memory.
struct GemmIn {
    const uint16_t *a, *b;       // M x kp and N x kp values, 16 bits each
    int64_t lda, ldb;            // row strides (values)
    int64_t step_a, step_b;      // from one step to the next (values)
    int64_t plane_a, plane_b;    // plane strides (values)
    int32_t m, n, kp;            // kp: contracted length, a multiple of GK
    int32_t pairs;               // plane products: 1 or 6
    int32_t kb;                  // TB: values of the contracted axis that b has
};

// Plane products, smallest first: (lo,hi) (hi,lo) (mid,mid) (mid,hi) (hi,mid) (hi,hi).
__device__ __forceinline__ void gemm_pair(int pairs, int p, int* pa, int* pb) {
    const int q = pairs == 1 ? 5 : p;
    *pa = (0x052 >> (2 * q)) & 3;  // two bits each from the low end: 2 0 1 1 0 0
    *pb = (0x118 >> (2 * q)) & 3;  // 0 2 1 0 1 0
}

// ONE: operands of one plane. TB: b lies with the contracted axis across.
template <int BM, int BN, int WM, int WN, bool ONE, bool TB = false>
struct Gemm {
    static constexpr int NT = 64 * WM * WN;
    static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;  // 16 x 16 blocks per wave
    static constexpr int A_BYTES = BM * GK * 2, B_BYTES = BN * GK * 2;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int COPIES = STAGE / 1024 / (NT / 64);  // per wave and step

    f32x4 acc[TM][TN];

    // LDS byte offset of piece p of row r within an operand's step
    static __device__ __forceinline__ int at(int r, int p) { return r * 128 + ((p ^ (r & 7)) << 4); }

    // copies BR rows of one step: wave w takes every NT / 64-th group of 8 rows
    template <int BR>
    static __device__ __forceinline__ void copy(__amdgpu_buffer_rsrc_t rs, uint32_t row_bytes,
                                                unsigned char* dst, int wave, int lane) {
        // row (8 grp + r) & 7 == r: the piece that belongs at place p is p ^ r
        const int r = lane >> 3, p = lane & 7;
        const uint32_t off = (uint32_t)(wave * 8 + r) * row_bytes + (uint32_t)((p ^ r) << 4);
#pragma unroll
        for (int g = 0; g < BR / 8 / (NT / 64); ++g)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rs, (__attribute__((address_space(3))) void*)(dst + (g * (NT / 64) + wave) * 1024), 16,
                (int)(off + g * (NT / 8) * row_bytes), 0, 0, 0);
    }

    // TB: this wave's 8-row groups of a step are neighbours, in one panel
    static constexpr int PER = BN / 8 / (NT / 64);
    static __device__ __forceinline__ int turn_key(int k) {
        return (((k >> 3) & 3) ^ ((k >> 1) & 1)) << 1;
    }
    static __device__ __forceinline__ void copy_across(__amdgpu_buffer_rsrc_t rs, unsigned char* dst,
                                                       int wave, int lane) {
        const int r = lane >> 3, p = lane & 7;
#pragma unroll
        for (int g = 0; g < PER; ++g) {
            const int grp = wave * PER + g;
            const int k = grp % 8 * 8 + r;  // of the panel's 64
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rs, (__attribute__((address_space(3))) void*)(dst + grp * 1024), 16,
                k * 128 + ((p ^ turn_key(k)) << 4), 0, 0, 0);
        }
    }
    // rows 16 b .. 16 b + 15 of the tile, half c of a step: lane 16 h + i gets 8 k of row i
    template <typename V8>
    static __device__ __forceinline__ V8 read_across(const unsigned char* d, int b, int c, int h, int i) {
        typedef short s4 __attribute__((ext_vector_type(4)));
        union {
            s4 part[2];
            V8 v;
        } u;
        const int chunk = b % 4 * 2 + ((i & 3) >> 1);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int k = 32 * c + 8 * h + 4 * t + (i >> 2);
            const unsigned char* at =
                d + b / 4 * 8192 + k * 128 + ((chunk ^ turn_key(k)) << 4) + (i & 1) * 8;
            u.part[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4*)at);
        }
        return u.v;
    }

    const uint16_t *next_a, *next_b;  // the step to be copied next, from the tile's first row
    int bytes_a, bytes_b;             // from there to the end of the step's last row (TB: of the panel)
    int steps;                        // of the tile
    int left, pair;                   // steps left in the plane product, its number

    static __device__ __forceinline__ int span(int64_t ld, int r0, int total, int br) {
        const int cnt = total - r0 < br ? total - r0 : br;
        return cnt > 0 ? (int)(((int64_t)(cnt - 1) * ld + GK) * 2) : 0;
    }

    // copies the next step into the buffer at d; m, n: the tile; real: there is a next
    // step (else nothing is read: every place is past the end)
    __device__ __forceinline__ void issue(const GemmIn& in, int m, int n, bool real, unsigned char* d) {
        const int lane = threadIdx.x & 63;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        copy<BM>(__builtin_amdgcn_make_buffer_rsrc((void*)next_a, (short)0, real ? bytes_a : 0, BUF_RSRC_WORD3),
                 (uint32_t)in.lda * 2, d, wave, lane);
        const uint16_t* pb = next_b;
        if constexpr (TB) {  // a wave's own panel: uniform, but not to the compiler
            const uint64_t u = (uint64_t)next_b;
            pb = (const uint16_t*)(((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(u >> 32)) << 32) |
                                   (uint32_t)__builtin_amdgcn_readfirstlane((int)u));
            bytes_b = __builtin_amdgcn_readfirstlane(bytes_b);
        }
        const __amdgpu_buffer_rsrc_t sb = __builtin_amdgcn_make_buffer_rsrc(
            (void*)pb, (short)0, real ? bytes_b : 0, BUF_RSRC_WORD3);
        if constexpr (TB) {
            copy_across(sb, d + A_BYTES, wave, lane);
            bytes_b = bytes_b > GK * 128 ? bytes_b - GK * 128 : 0;
        } else {
            copy<BN>(sb, (uint32_t)in.ldb * 2, d + A_BYTES, wave, lane);
        }
        next_a += in.step_a;
        next_b += in.step_b;
        if constexpr (!ONE)
            if (--left == 0) seek(in, m, n, pair + 1, 0);
    }
    __device__ __forceinline__ void seek(const GemmIn& in, int m, int n, int p, int kk) {
        int pa, pb;
        gemm_pair(ONE ? 1 : in.pairs, p, &pa, &pb);
        next_a = in.a + pa * in.plane_a + kk * in.step_a + m * in.lda;
        next_b = in.b + pb * in.plane_b + kk * in.step_b + n * in.ldb;
        if constexpr (TB) {
            const int row = n + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * PER / 8 * 64;
            next_b += (int64_t)(row - n) * in.ldb;
            bytes_b = row < in.n && in.kb > kk * GK ? (in.kb - kk * GK) * 128 : 0;
        }
        pair = p;
        left = in.kp / GK - kk;
    }

    // Starts steps [first, last) of the tile at rows m and columns n: their first two
    // are copied into l0 and l1, STAGE bytes each (free, by the caller's barrier). A
    // step is GK values of one plane product.
    __device__ __forceinline__ void begin(const GemmIn& in, int m, int n, int first, int last,
                                          unsigned char* l0, unsigned char* l1) {
        const int ks = in.kp / GK;
        steps = last - first;
        bytes_a = span(in.lda, m, in.m, BM);
        if constexpr (!TB) bytes_b = span(in.ldb, n, in.n, BN);
        seek(in, m, n, first / ks, first % ks);
        issue(in, m, n, true, l0);
        issue(in, m, n, steps > 1, l1);
    }

    // The products of the steps begun, into acc (V8: bf16x8 or f16x8, the operands'
    // type); LDS is free afterwards.
    // Each step is two halves of 32 values; a half's operands are read from LDS
    // while the half before is multiplied, and a step's copies are issued when
    // its buffer's last half has been read, a full step before they are needed.
    // Measured without epilogue, 256 x 256 tiles: 8192^3 746 us (1474 TFLOP/s),
    // 16384 x 8192 x 768 148 us (1389); with the wait left to the scheduler, which
    // moves it before the products, 164 us; with the copies and reads in front of
    // the products instead of between them 180 us.
    template <typename V8>
    __device__ __forceinline__ void finish(const GemmIn& in, int m, int n, unsigned char* l0,
                                           unsigned char* l1) {
        const int tid = threadIdx.x, lane = tid & 63;
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int wm = wave / WN, wn = wave % WN;
        const int h = lane >> 4, i = lane & 15;
#pragma unroll
        for (int x = 0; x < TM; ++x)
#pragma unroll
            for (int y = 0; y < TN; ++y) acc[x][y] = f32x4{0.f, 0.f, 0.f, 0.f};
        auto read = [&](V8(&fa)[TM], V8(&fb)[TN], const unsigned char* da, int c) {
            const unsigned char* db = da + A_BYTES;
#pragma unroll
            for (int x = 0; x < TM; ++x)
                fa[x] = *(const V8*)(da + at((wm * TM + x) * 16 + i, 4 * c + h));
#pragma unroll
            for (int y = 0; y < TN; ++y)
                if constexpr (TB)
                    fb[y] = read_across<V8>(db, wn * TN + y, c, h, i);
                else
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
            auto put_copies = [&]() {
#pragma unroll
                for (int g = 0; g < copies; ++g) {
                    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);   // matrix product
                    __builtin_amdgcn_sched_group_barrier(0x20, 1, 0);  // memory read
                }
            };
            if constexpr (!TB) put_copies();
#pragma unroll
            for (int g = 0; g < TM + (TB ? 2 : 1) * TN; ++g) {
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // LDS read
                __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
            }
            if constexpr (TB) put_copies();
            __builtin_amdgcn_sched_group_barrier(0x8, TM * TN, 0);
        };
        // the first step's copies have landed; the second's may be in flight
        __builtin_amdgcn_s_waitcnt((COPIES & 15) | (7 << 4) | (15 << 8) | ((COPIES >> 4) << 14));
        __syncthreads();
        V8 fa[2][TM], fb[2][TN];
        read(fa[0], fb[0], l0, 0);
        int togo = steps;
        // one step, in buffer cur. The last steps copy nothing and read a buffer that
        // is not multiplied: one body for all.
        auto step = [&](unsigned char* cur, unsigned char* other) {
            read(fa[1], fb[1], cur, 1);
            multiply(fa[0], fb[0]);
            spread(0);
            // the wait stays behind the products: the copies of step s + 1 have
            // had a whole step to land
            __builtin_amdgcn_sched_barrier(0);
            // this wave's copies of step s + 1 have landed, its reads of step s are done
            __builtin_amdgcn_s_waitcnt(0);
            __syncthreads();  // ... and every wave's
            __builtin_amdgcn_sched_barrier(0);
            // the transposing loads wait for every copy in flight (the compiler does
            // not tell their buffers apart): they go first
            if constexpr (!TB) issue(in, m, n, togo > 2, cur);
            read(fa[0], fb[0], other, 0);
            if constexpr (TB) issue(in, m, n, togo > 2, cur);
            multiply(fa[1], fb[1]);
            spread(COPIES);
            __builtin_amdgcn_sched_barrier(0);
            return --togo > 0;
        };
        while (step(l0, l1) && step(l1, l0)) {
        }
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();  // LDS is free for the epilogue
    }
    static __device__ __forceinline__ int all_steps(const GemmIn& in) { return in.kp / GK * in.pairs; }

    // row of this lane's first of four rows of blocks x, its column in blocks y
    static __device__ __forceinline__ int row(int x) {
        return ((threadIdx.x >> 6) / WN * TM + x) * 16 + 4 * ((threadIdx.x & 63) >> 4);
    }
    static __device__ __forceinline__ int col(int y) {
        return ((threadIdx.x >> 6) % WN * TN + y) * 16 + (threadIdx.x & 15);
    }
};

// Tile b of a walk over mt x nt tiles: the tiles that one XCD receives (every
// eighth b) are neighbours, walked in bands of 8 tile rows, so that its L2 serves their
// shared rows of A and B. b runs over 8 ceil(mt nt / 8) values; false: no tile.
__device__ __forceinline__ bool gemm_tile(uint32_t b, uint32_t mt, uint32_t nt, int* tm, int* tn) {
    const uint32_t total = mt * nt, per = (total + 7) / 8;
    const uint32_t id = (b & 7) * per + (b >> 3);
    if ((b >> 3) >= per || id >= total) return false;
    const uint32_t band = id / (8 * nt), in = id - band * 8 * nt;
    const uint32_t rows = mt - band * 8 < 8 ? mt - band * 8 : 8;
    *tm = (int)(band * 8 + in % rows);
    *tn = (int)(in / rows);
    return true;
}

// Runs epilogue(g, m0, n0) for this workgroup's tiles (workgroup, + grid, + 2 grids, ...;
// the grid is a multiple of 8); the next tile's first copies run under a tile's
// epilogue, which therefore has LDS of its own. m0, n0: the epilogue's tile.
template <typename V8, typename G, int BM, int BN, typename F>
__device__ __forceinline__ void gemm_walk(const GemmIn& in, int mt, int nt, unsigned char* l0,
                                          unsigned char* l1, F epilogue) {
    const uint32_t end = ((uint32_t)mt * nt + 7) / 8 * 8;
    uint32_t b = blockIdx.x;
    int tm = 0, tn = 0;
    auto next = [&]() {
        for (; b < end; b += gridDim.x)
            if (gemm_tile(b, mt, nt, &tm, &tn)) return true;
        return false;
    };
    if (!next()) return;
    G g;
    g.begin(in, tm * BM, tn * BN, 0, G::all_steps(in), l0, l1);
    for (bool more = true; more;) {
        const int m0 = tm * BM, n0 = tn * BN;
        g.template finish<V8>(in, m0, n0, l0, l1);
        b += gridDim.x;
        more = next();
        if (more) g.begin(in, tm * BM, tn * BN, 0, G::all_steps(in), l0, l1);
        epilogue(g, m0, n0);
    }
}

}  // namespace gmm
