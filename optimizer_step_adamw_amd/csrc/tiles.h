// tiles.h -- matrix products on the matrix cores (MFMA 16x16x32, fp16 or
// bf16 operands, fp32 sums) for the kernels that orthogonalise momenta and
// that take experts' weight gradients: operand tiles staged through LDS, and
// the values of a product held as sums of two fp16 numbers.
//
// A workgroup computes a tile of P Q^T: 128 x 128 by 4 wavefronts of 64 x 64
// (two workgroups a compute unit), or 256 x 256 by 8 wavefronts of 128 rows x
// 64 columns (one), which reads LDS three quarters and global memory half as
// much per product.  Per step an operand's rows (of P: output rows; of Q:
// output columns) hold 64 numbers each in LDS:
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

enum Order { KC = 0, KR = 1 };
// Tiles of side 128 W.  PAIR (W = 1): two groups of 4 wavefronts share a tile,
// each summing every other step, for launches with fewer tiles than compute
// units, where a lone group would wait most of the time.
template <int W, bool PAIR = false>
struct Tile {
    static constexpr int kSide = 128 * W;
    static constexpr int kWaves = W == 1 ? 4 : 8;             // of a group
    static constexpr int kLanes = 64 * kWaves * (PAIR ? 2 : 1);
    static constexpr int kWavesPerSimd = 2;                   // two workgroups a compute unit, or one of 8 wavefronts
    static constexpr int kWaveCols = kSide / 64;              // wavefronts side by side
    static constexpr int kRows = kSide * kWaveCols / kWaves;  // rows of a wavefront: 64 or 128
    static constexpr int kJ = kRows / 16;                     // fragments of 16 rows
    static constexpr int kOutJ = PAIR ? kJ / 2 : kJ;          // of which it stores
    static constexpr int kOperand = kSide * 64 * 2;           // bytes of one operand, one step
    static constexpr int kStage = 2 * kOperand;
    static constexpr int kLds = 2 * kStage * (PAIR ? 2 : 1);
};

// Split arrays lie in blocks of 32 rows x 32 columns, 4 KB each, block rows
// one after another; a block's row is a 128-byte line, 32 high parts, then 32
// low parts.  A step of either order then reads whole blocks, and no two
// lines of a step are a power of two far apart.  ld: columns, a multiple of
// 32.  Place of the high part of element (r, c); its low part is 32 behind.
__device__ __forceinline__ int64_t split_at(int64_t r, int64_t c, int64_t ld) {
    return ((r >> 5) * (ld >> 5) + (c >> 5)) * 2048 + (r & 31) * 64 + (c & 31);
}
// Bytes of a row of blocks: 32 rows.
__device__ __forceinline__ int64_t split_rows32(int64_t ld) { return ld * 128; }
constexpr int kSplitBlock = 4096;

// x as hi + lo, both fp16 rounded to nearest even: 22 significant bits where
// lo is a normal number, an absolute error of 2^-25 below that.
__device__ __forceinline__ void split2(float x, _Float16 &hi, _Float16 &lo) {
    hi = (_Float16)x;
    lo = (_Float16)(x - (float)hi);
}

// Permutation of the 16-byte chunks of row k of a KR tile: within a read,
// groups of 16 lanes take 4 rows each, k = 8 g + (0..3) (+ 4).
__device__ __forceinline__ int kr_swizzle(int k) { return 2 * ((k & 3) | ((k >> 3) & 1) << 2); }

__device__ __forceinline__ int64_t uniform64(int64_t x) { return (int64_t)uniform_ptr((char *)x); }

// A wavefront's group (of a pair) and its place in it.
template <int W>
__device__ __forceinline__ int pair_half() { return (threadIdx.x >> 6) / Tile<W>::kWaves; }
template <int W>
__device__ __forceinline__ int wave() { return (threadIdx.x >> 6) % Tile<W>::kWaves; }

// One operand's loads into LDS: one KB each, 4 per wavefront and step, each
// lane 16 bytes from `base` + at[t].  base (the same in every lane) moves on
// from step to step.
struct Feed {
    const char *base;
    uint32_t at[4];
};
// Row (KC: of the operand; KR: along k) and 16-byte chunk of load t.
template <int W, Order O, bool SPLIT>
__device__ __forceinline__ void feed_slot(int t, int &row, int &chunk) {
    constexpr int kChunks = O == KC ? 8 : (SPLIT ? 32 : 16) * W;  // of a row in LDS
    const int at = (wave<W>() * 4 + t) * 64 + (threadIdx.x & 63);
    row = at / kChunks;
    chunk = at % kChunks ^ (O == KC ? row & 7 : kr_swizzle(row));
}
// src: the operand's first byte (KC: row 0 of the tile; KR: column 0 of the
// tile in the first row).  Split: ld is split_rows32(), and left the rows (KC)
// or columns (KR) from there on that exist, a multiple of 32; plain (KR): ld is
// the bytes between rows, left the columns, a multiple of 8.  The last one
// stands in for those behind it, whose sums are not stored.  (Offsets within a
// step stay below 2^32.)
template <int W, Order O, bool SPLIT>
__device__ __forceinline__ Feed feed(const char *src, int64_t ld, int left) {
    Feed f;
    f.base = uniform_ptr(src);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        int row, chunk;
        feed_slot<W, O, SPLIT>(t, row, chunk);
        if constexpr (SPLIT && O == KC) {
            if (row >= left) row = left - 1;
            f.at[t] = (uint32_t)((row >> 5) * ld + (row & 31) * 128 + chunk * 16);
        } else if constexpr (SPLIT) {
            if ((chunk >> 3) * 32 >= left) chunk = (left / 32 - 1) * 8 + (chunk & 7);
            f.at[t] = (uint32_t)((chunk >> 3) * kSplitBlock + row * 128 + (chunk & 7) * 16);
        } else {
            if (chunk * 8 >= left) chunk = left / 8 - 1;
            f.at[t] = (uint32_t)(row * ld + chunk * 16);
        }
    }
    return f;
}
// Places in LDS are byte offsets held in scalar registers (`lds` below): as
// generic pointers every use of one would be checked and converted again.
__device__ __forceinline__ uint32_t lds_at(const char *lds) {
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)(const LMEM char *)lds);
}
template <class T>
__device__ __forceinline__ LMEM T *lds_ptr(uint32_t at) { return (LMEM T *)(uintptr_t)at; }

// Issues an operand's loads into LDS.  They have no register output; as
// builtins the compiler would wait for them before any LDS read behind them
// that it cannot prove to be elsewhere.  landed() waits for them.  (m0, where
// a wavefront's KB goes, is the compiler's own register for such loads: it
// warns of any mention.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// Load t of the wavefront, whose 4 KB of the operand begin at `to`,
// where `go` (the same in every lane) is above 0.  The branch is part of the
// asm: around it, the registers of two paths would not fit.
__device__ __forceinline__ void stage1_if(int go, const Feed &f, int t, uint32_t to) {
    asm volatile("s_cmp_lt_i32 %3, 1\n\ts_cbranch_scc1 .Lnoload%=\n\ts_mov_b32 m0, %0\n\ts_nop 0\n\t"
                 "global_load_lds_dwordx4 %1, %2\n.Lnoload%=:"
                 :: "s"(to + t * 1024), "v"(f.at[t]), "s"(f.base), "s"(go)
                 : "memory", "m0", "scc");
}
#pragma clang diagnostic pop

// The 16 x 32 fragment of rows (KC) or columns (KR) 16 b .. 16 b + 15; part:
// high or low (split), or which 32 of the step's 64 values along k (plain).
template <int W, Order O, bool SPLIT>
__device__ __forceinline__ s16x8 fragment(uint32_t lds, int b, int part) {
    const int l = threadIdx.x & 63;
    if constexpr (O == KC) {
        const int row = b * 16 + (l & 15);
        return *lds_ptr<const s16x8>(lds + row * 128 + (((part * 4 + (l >> 4)) ^ (l & 7)) << 4));
    } else {
        constexpr int kRowBytes = (SPLIT ? 512 : 256) * W;
        const int k = (l >> 4) * 8 + ((l & 15) >> 2) + (SPLIT ? 0 : part * 32);
        const int c = SPLIT ? (b >> 1) * 8 + part * 4 + (b & 1) * 2 : b * 2;
        const uint32_t at = lds + k * kRowBytes + (((c | ((l & 3) >> 1)) ^ kr_swizzle(k)) << 4) + (l & 1) * 8;
        const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(lds_ptr<s16x4>(at));
        const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(lds_ptr<s16x4>(at + 4 * kRowBytes));
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

// A wavefront's sums: v[i][j][e] belongs to row row0() + 16 j and column
// col0() + 16 i + e of the tile: four neighbouring columns of one row.
template <int W>
struct Sums {
    f32x4 v[4][Tile<W>::kJ];
};
template <int W>
__device__ __forceinline__ int wave_row() { return wave<W>() / Tile<W>::kWaveCols; }
template <int W>
__device__ __forceinline__ int wave_col() { return wave<W>() % Tile<W>::kWaveCols; }
// (of a pair, each group stores half of its rows)
template <int W, bool PAIR = false>
__device__ __forceinline__ int row0() {
    return wave_row<W>() * Tile<W>::kRows + (PAIR ? pair_half<W>() * Tile<W>::kRows / 2 : 0) + (threadIdx.x & 15);
}
template <int W>
__device__ __forceinline__ int col0() { return wave_col<W>() * 64 + ((threadIdx.x & 63) >> 4) * 4; }

// Product k of those of fragment j of the wavefront's rows: of the high parts
// (0-3), of each high part with the other operand's low part (4-11; the
// product of both low parts, 2^-22 of the whole, is left out), or of the two
// halves of a plain step (0-7).
template <bool SPLIT, bool BF16, int W>
__device__ __forceinline__ void multiply1(const s16x8 (&q)[4][2], const s16x8 (&p)[2], Sums<W> &s, int j, int k) {
    const int h = k / 4, i = k % 4;
    s.v[i][j] = mfma<BF16>(q[i][SPLIT ? h == 1 : h], p[SPLIT ? h == 2 : h], s.v[i][j]);
}
template <bool SPLIT, bool BF16, int W>
__device__ __forceinline__ void multiply(const s16x8 (&q)[4][2], const s16x8 (&p)[2], Sums<W> &s, int j) {
#pragma unroll
    for (int k = 0; k < (SPLIT ? 12 : 8); ++k) multiply1<SPLIT, BF16, W>(q, p, s, j, k);
}

// This wavefront's loads into LDS have landed and its LDS reads are done, and
// so are every wavefront's.
__device__ __forceinline__ void landed() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <int W, Order O, bool SPLIT>
__device__ __forceinline__ void read_p(uint32_t now, int j, s16x8 (&p)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) p[h] = fragment<W, O, SPLIT>(now, wave_row<W>() * Tile<W>::kJ + j, h);
}
template <int W, Order O, bool SPLIT>
__device__ __forceinline__ void read_q(uint32_t now, s16x8 (&q)[4][2]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) q[i][h] = fragment<W, O, SPLIT>(now + Tile<W>::kOperand, wave_col<W>() * 4 + i, h);
}

// Sum over `steps` steps; an operand moves on by kp / kq bytes from step to
// step.  All loads into LDS have landed at the end, and of a pair each group
// holds the sums of the rows it stores in v[.][0 .. kOutJ).
//
// 128-tiles: a wavefront holds two steps' fragments.  While one step's are
// multiplied, the next one's are read, and the loads of the step after that go
// to the place of the step being multiplied, whose fragments have all been
// read.  256-tiles have no registers for that: a wavefront goes through its
// rows' fragments, each read while the one before it is multiplied; once the
// last two have been read, the step's place in LDS is free and (after the
// barrier) the next step's is full: the loads of the step after that go out,
// the next step's first fragments are read, and the last two are multiplied
// meanwhile.  Either way the matrix cores have work at the barrier and during a
// step's first reads, and loads and reads are dealt out between the products,
// for a wavefront issues in order: in one piece they would hold them up.
// (The last step reads fragments of a step that is not there, whatever LDS
// holds, and does not use them.)
//
// Measured on MI355X, split operands from L2, random values: 256-tiles on every
// compute unit 2.2 us a step (1450 TFLOP/s of fp16 products at the clock that
// the power limit leaves; the products alone 1.6 us), a lone 128-tile group
// 0.66 us a step, two on one compute unit 0.8 us for both.
template <int W, bool PAIR, Order OP, Order OQ, bool SPLIT, bool BF16>
__device__ __forceinline__ void product(Feed fp, int64_t kp, Feed fq, int64_t kq, int steps, uint32_t lds, Sums<W> &s) {
    using T = Tile<W>;
    constexpr int J = T::kJ;
    static_assert(!PAIR || W == 1, "pairs share 128-tiles");
    int rounds = __builtin_amdgcn_readfirstlane(steps);  // the same for both groups: they share the barriers
    if (rounds <= 0) return;
    kp = uniform64(kp);
    kq = uniform64(kq);
    steps = rounds;
    if constexpr (PAIR) {
        const int g = __builtin_amdgcn_readfirstlane(pair_half<W>());
        fp.base += g * kp;
        fq.base += g * kq;
        kp *= 2;
        kq *= 2;
        steps = (rounds + 1 - g) / 2;
        rounds = (rounds + 1) / 2;
        lds += g * 2 * T::kStage;
    }
    const uint32_t mine = (uint32_t)__builtin_amdgcn_readfirstlane(wave<W>()) * 4096;
    auto load = [&](int go, uint32_t to) {
#pragma unroll
        for (int t = 0; t < 4; ++t) stage1_if(go, fp, t, to + mine);
#pragma unroll
        for (int t = 0; t < 4; ++t) stage1_if(go, fq, t, to + mine + T::kOperand);
        fp.base += kp;
        fq.base += kq;
    };
    load(steps, lds);
    landed();
    load(steps - 1, lds + T::kStage);
    uint32_t now = lds, next = lds + T::kStage;
    if constexpr (W == 1) {
        s16x8 p[2][4][2], q[2][4][2];
        read_q<W, OQ, SPLIT>(now, q[0]);
#pragma unroll
        for (int j = 0; j < 4; ++j) read_p<W, OP, SPLIT>(now, j, p[0][j]);
        auto one = [&](int t, int a, int b) {
            landed();
            const int more = steps - 2 - t;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
#pragma unroll
                for (int l = 2 * c; l < 2 * c + 2; ++l)
                    stage1_if(more, l < 4 ? fp : fq, l % 4, now + mine + (l < 4 ? 0 : T::kOperand));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    q[b][c][h] = fragment<W, OQ, SPLIT>(next + T::kOperand, wave_col<W>() * 4 + c, h);
                    p[b][c][h] = fragment<W, OP, SPLIT>(next, wave_row<W>() * 4 + c, h);
                }
                __builtin_amdgcn_sched_barrier(0);
                if (!PAIR || t < steps) multiply<SPLIT, BF16, W>(q[a], p[a][c], s, c);
                __builtin_amdgcn_sched_barrier(0);
            }
            fp.base += kp;
            fq.base += kq;
            const uint32_t swap = now;
            now = next;
            next = swap;
        };
        for (int t = 0; t < rounds; t += 2) {
            one(t, 0, 1);
            if (t + 1 < rounds) one(t + 1, 1, 0);
        }
    } else {
        s16x8 q[4][2], p[J][2];
        read_q<W, OQ, SPLIT>(now, q);
        read_p<W, OP, SPLIT>(now, 0, p[0]);
        for (int t = 0; t < rounds; ++t) {
#pragma unroll
            for (int j = 0; j + 2 < J; ++j) {
                read_p<W, OP, SPLIT>(now, j + 1, p[j + 1]);
                if (j + 3 == J) read_p<W, OP, SPLIT>(now, j + 2, p[j + 2]);
                __builtin_amdgcn_sched_barrier(0);  // the reads first
                multiply<SPLIT, BF16, W>(q, p[j], s, j);
                __builtin_amdgcn_sched_barrier(0);  // hold no more than the next fragment
            }
            landed();
            // the last two fragments' products by columns, so that the next step's
            // fragments of Q take the registers of this one's
            const int more = steps - 2 - t;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int l = 2 * i; l < 2 * i + 2; ++l)
                    stage1_if(more, l < 4 ? fp : fq, l % 4, now + mine + (l < 4 ? 0 : T::kOperand));
                if (i == 0) read_p<W, OP, SPLIT>(next, 0, p[0]);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int h = 0; h < (SPLIT ? 3 : 2); ++h) {
                    multiply1<SPLIT, BF16, W>(q, p[J - 2], s, J - 2, h * 4 + i);
                    multiply1<SPLIT, BF16, W>(q, p[J - 1], s, J - 1, h * 4 + i);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    q[i][h] = fragment<W, OQ, SPLIT>(next + T::kOperand, wave_col<W>() * 4 + i, h);
                __builtin_amdgcn_sched_barrier(0);
            }
            fp.base += kp;
            fq.base += kq;
            const uint32_t swap = now;
            now = next;
            next = swap;
        }
    }
    landed();
}

// Of a pair, after product(): each group hands the sums of the rows it does
// not store to the other; first group's + second group's.
template <int W, bool PAIR>
__device__ __forceinline__ void join_pair(uint32_t lds, Sums<W> &s) {
    if constexpr (PAIR) {
        constexpr int H = Tile<W>::kJ / 2;
        const int g = __builtin_amdgcn_readfirstlane(pair_half<W>());
        const uint32_t lane = (threadIdx.x & 63) * 16, of = (uint32_t)wave<W>() * (4 * H * 1024);
        const uint32_t give = lds + (g ? 0 : 65536) + of + lane, take = lds + (g ? 65536 : 0) + of + lane;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < H; ++j)
                *lds_ptr<f32x4>(give + (i * H + j) * 1024) = g ? s.v[i][j] : s.v[i][H + j];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < H; ++j) {
                const f32x4 x = *lds_ptr<const f32x4>(take + (i * H + j) * 1024);
                s.v[i][j] = g ? x + s.v[i][H + j] : s.v[i][j] + x;
            }
    }
}

}  // namespace
}  // namespace optim
