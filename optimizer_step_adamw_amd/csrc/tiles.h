// tiles.h -- matrix products on the matrix cores (MFMA 16x16x32, fp16 or
// bf16 operands, fp32 sums) for the kernels that orthogonalise momenta and
// that take experts' weight gradients: operand tiles staged through LDS, and
// the values of a product held as sums of two fp16 numbers.
//
// A workgroup of 4 wavefronts computes a 128 x 128 tile of P Q^T, 64 x 64 per
// wavefront.  An operand's 128 rows (of P: output rows; of Q: output columns)
// times 64 numbers per row and step lie in 16 KB of LDS:
//   split operands: 32 values along k, each value's two parts;
//   plain operands: 64 values along k.
// Two steps' tiles are held: the next step's loads go straight from global
// memory into LDS while the current one is multiplied.
//
// An operand comes in one of two orders:
//   KC  k runs along a row in memory (X in X X^T): fragments are 16-byte LDS
//       reads;
//   KR  k runs down the rows (X in X^T X): fragments go through the LDS
//       read that transposes 16-bit numbers within groups of 16 lanes.
// Within LDS the 16-byte chunks of a row are permuted (chunk ^ a function of
// the row) so that the lanes of one read meet different banks; a load into
// LDS fills consecutive chunks, so the permutation is made on the global side.
#pragma once

#include "device_common.h"

namespace optim {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
#define LMEM __attribute__((address_space(3)))

constexpr int kTile = 128;                       // output tile side
constexpr int kOperandBytes = kTile * 64 * 2;    // one operand, one step
constexpr int kStageBytes = 2 * kOperandBytes;
enum Order { KC = 0, KR = 1 };

// Split arrays: element (r, c) of a matrix of ld columns (a multiple of 32)
// has its high part at r * 2 ld + (c / 32) * 64 + c % 32 and its low part 32
// numbers behind, so a 128-byte line holds 32 values of a row whole.
__device__ __forceinline__ int64_t split_at(int64_t r, int64_t c, int64_t ld) {
    return r * 2 * ld + (c >> 5) * 64 + (c & 31);
}

// x as hi + lo, both fp16 rounded to nearest even: 22 significant bits where
// lo is a normal number, an absolute error of 2^-25 below that.
__device__ __forceinline__ void split2(float x, _Float16 &hi, _Float16 &lo) {
    hi = (_Float16)x;
    lo = (_Float16)(x - (float)hi);
}

// Permutation of the 16-byte chunks of row k of a KR tile: within a read,
// groups of 16 lanes take 4 rows each, k = 8 g + (0..3) (+ 4).
__device__ __forceinline__ int kr_swizzle(int k) { return 2 * ((k & 3) | ((k >> 3) & 1) << 2); }

// One operand's loads into LDS: 16 of 1 KB per step, 4 per wavefront, each
// lane 16 bytes from `base` + at[t].  base (the same in every lane) moves on
// from step to step.
struct Feed {
    const char *base;
    uint32_t at[4];
};
// Row (KC: of the operand; KR: along k) and 16-byte chunk of load t.
template <Order O, bool SPLIT>
__device__ __forceinline__ void feed_slot(int t, int &row, int &chunk) {
    const int lane = threadIdx.x & 63, i = (threadIdx.x >> 6) * 4 + t;
    if constexpr (O == KC) {        // 8 chunks a row
        row = i * 8 + (lane >> 3);
        chunk = (lane & 7) ^ (row & 7);
    } else if constexpr (SPLIT) {   // 32 chunks a row, 32 rows
        row = i * 2 + (lane >> 5);
        chunk = (lane & 31) ^ kr_swizzle(row);
    } else {                        // 16 chunks a row, 64 rows
        row = i * 4 + (lane >> 4);
        chunk = (lane & 15) ^ kr_swizzle(row);
    }
}
// src: the operand's first byte (KC: row 0 of the tile; KR: column 0 of the
// tile in the first row); ld: bytes between rows (128 rows stay below 2^32);
// chunks: 16-byte chunks of a row that exist (KR plain: the last one stands in for those
// behind it, whose columns are not stored).
template <Order O, bool SPLIT>
__device__ __forceinline__ Feed feed(const char *src, int64_t ld, int chunks = 32) {
    Feed f;
    f.base = uniform_ptr(src);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        int row, chunk;
        feed_slot<O, SPLIT>(t, row, chunk);
        if (O == KR && !SPLIT && chunk >= chunks) chunk = chunks - 1;
        f.at[t] = (uint32_t)(row * ld + chunk * 16);
    }
    return f;
}
__device__ __forceinline__ void stage(const Feed &f, char *lds) {
    const int w = threadIdx.x >> 6;
#pragma unroll
    for (int t = 0; t < 4; ++t)
        __builtin_amdgcn_global_load_lds((const GMEM uint32_t *)gp(f.base + f.at[t]),
                                         (LMEM uint32_t *)(lds + (w * 4 + t) * 1024), 16, 0, 0);
}

// The 16 x 32 fragment of rows (KC) or columns (KR) 16 b .. 16 b + 15; part:
// high or low (split), or which 32 of the step's 64 values along k (plain).
template <Order O, bool SPLIT>
__device__ __forceinline__ s16x8 fragment(const char *lds, int b, int part) {
    const int l = threadIdx.x & 63;
    if constexpr (O == KC) {
        const int row = b * 16 + (l & 15);
        return *(const LMEM s16x8 *)(lds + row * 128 + (((part * 4 + (l >> 4)) ^ (l & 7)) << 4));
    } else {
        const int k = (l >> 4) * 8 + ((l & 15) >> 2) + (SPLIT ? 0 : part * 32);
        const int c = SPLIT ? (b >> 1) * 8 + part * 4 + (b & 1) * 2 : b * 2;
        const int at = k * (SPLIT ? 512 : 256) + (((c | ((l & 3) >> 1)) ^ kr_swizzle(k)) << 4) + (l & 1) * 8;
        const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LMEM s16x4 *)(lds + at));
        const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LMEM s16x4 *)(lds + at + 4 * (SPLIT ? 512 : 256)));
        return s16x8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
    }
}

template <bool BF16>
__device__ __forceinline__ f32x4 mfma(s16x8 a, s16x8 b, f32x4 c) {
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
}

// A wavefront's sums: sum[i][j][e] belongs to output row row0() + 16 j + lane
// % 16, column col0() + 16 i + 4 (lane / 16) + e: four neighbouring columns of
// one row.
struct Sums {
    f32x4 v[4][4];
};
__device__ __forceinline__ int row0() { return ((threadIdx.x >> 6) >> 1) * 64 + (threadIdx.x & 15); }
__device__ __forceinline__ int col0() { return ((threadIdx.x >> 6) & 1) * 64 + ((threadIdx.x & 63) >> 4) * 4; }

// A step's fragments of this wavefront.
struct Fragments {
    s16x8 p[4][2], q[4][2];
};
template <Order OP, Order OQ, bool SPLIT>
__device__ __forceinline__ void fragments(const char *lds, Fragments &f) {
    const int w = threadIdx.x >> 6;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f.p[i][h] = fragment<OP, SPLIT>(lds, (w >> 1) * 4 + i, h);
            f.q[i][h] = fragment<OQ, SPLIT>(lds + kOperandBytes, (w & 1) * 4 + i, h);
        }
}

// One step: the products of the high parts, and of each high part with the
// other operand's low part (the product of both low parts, 2^-22 of the
// whole, is left out), or two plain products.
template <bool SPLIT, bool BF16>
__device__ __forceinline__ void multiply(const Fragments &f, Sums &s) {
#pragma unroll
    for (int h = 0; h < (SPLIT ? 3 : 2); ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s.v[i][j] = mfma<BF16>(f.q[i][SPLIT ? h == 1 : h], f.p[j][SPLIT ? h == 2 : h], s.v[i][j]);
}

// Every load into LDS of this wavefront has landed, and every wavefront's.
__device__ __forceinline__ void staged() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
}

// Sum over `steps` steps; an operand moves on by kp / kq bytes from step to
// step.  A step's fragments are read before the next step's loads into LDS
// are issued: the compiler cannot tell the two halves of the buffer apart and
// would wait for those loads before the first read behind them.
template <Order OP, Order OQ, bool SPLIT, bool BF16>
__device__ __forceinline__ void product(Feed p, int64_t kp, Feed q, int64_t kq, int steps, char *lds, Sums &s) {
    if (steps > 0) {
        stage(p, lds);
        stage(q, lds + kOperandBytes);
    }
    for (int t = 0; t < steps; ++t) {
        char *now = lds + (t & 1) * kStageBytes, *next = lds + (~t & 1) * kStageBytes;
        staged();
        Fragments f;
        fragments<OP, OQ, SPLIT>(now, f);
        p.base += kp;
        q.base += kq;
        if (t + 1 < steps) {
            stage(p, next);
            stage(q, next + kOperandBytes);
        }
        multiply<SPLIT, BF16>(f, s);
    }
}

}  // namespace
}  // namespace optim
