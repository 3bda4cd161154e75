// kernels_expert.hip -- the weight gradients of a mixture of experts
// (optim_expert_grad): dW_e (+)= s X_e^T dY_e, one product per expert over
// its own run of rows.
//
// A workgroup computes a 128 x 128 tile of one expert's dW, or a 256 x 256 one,
// with the product of tiles.h, both operands' k (the rows) running down memory.  Whole steps of 64
// rows go straight from global memory into LDS; the rows left over, and every
// step where a row is not a whole number of aligned 16-byte chunks, pass
// through registers, where what lies outside the run or the matrix becomes
// zero.
//
// Bound by the matrix cores where runs are long, by writing dW where they are
// short.  Measured on MI355X: 8 experts 2048 x 8192 over 16384 rows,
// accumulated in fp32, 616-624 us (550 GFLOP, 881-893 TFLOP/s, and 1.4 GB of
// rows and gradients; the matrix cores busy 42%; up to 760 in the first 15 calls
// after a pause), 64 experts 2048 x 1024 over 65536 rows in bf16 367-373 us (275
// GFLOP, 737-749 TFLOP/s, 0.67 GB), 4 experts 256 x 172 over 300 rows 11.8 us.
#include "optim_grads.h"

#include "expert_rows.h"
#include "tiles.h"

#include <algorithm>

namespace optim {
namespace {

// Tiles are taken in blocks of kBand x kBand of one expert, each block by
// one XCD (workgroup b runs on XCD b mod 8), whose L2 then holds the
// block's operands, and consecutive blocks by different XCDs, so that an
// expert with many rows is spread over all of them.
constexpr int kXcds = 8, kBand = 4, kGroup = kBand * kBand;

// One operand's 64 x 128 tile from row k0 on, through registers: 4 chunks of
// 8 values per lane.  With 8 rows of the run and more behind the step, 16 bytes
// from any of its elements are the run's, and all chunks are loaded at once;
// what of them lies past the columns becomes zero on the way to LDS.  Bounded
// one by one, as in a run's last rows, the loads wait for each other: 2 experts
// of 3055 x 1157 over 7334 rows took 407 us instead of 208, 8 of 1001 x 999 over
// 8192 98 instead of 48.
struct Chunks {
    s16x8 v[4];
};
typedef s16x8 __attribute__((aligned(2))) s16x8_any;
template <int W>
__device__ __forceinline__ Chunks load_chunks(const char *src, int64_t ld, int32_t rows, int32_t cols) {
    Chunks r;
    if (rows >= kStepRows + 8) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            int row, chunk;
            feed_slot<W, KR, false>(t, row, chunk);
            r.v[t] = *(const GMEM s16x8_any *)gp(src + row * ld + (chunk * 8 < cols ? chunk * 16 : 0));
        }
        return r;
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        int row, chunk;
        feed_slot<W, KR, false>(t, row, chunk);
        const int32_t left = cols - chunk * 8;
        s16x8 v = {0, 0, 0, 0, 0, 0, 0, 0};
        if (row < rows && left > 0) {
            const char *p = src + row * ld + chunk * 16;
            if (left >= 8) {
                v = *(const GMEM s16x8_any *)gp(p);
            } else {
#pragma unroll
                for (int i = 0; i < 7; ++i)
                    if (i < left) v[i] = ((const GMEM short *)gp(p))[i];
            }
        }
        r.v[t] = v;
    }
    return r;
}
template <int W>
__device__ __forceinline__ void write_chunks(const Chunks &r, char *lds, int32_t cols) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        s16x8 v = r.v[t];
        if (cols < Tile<W>::kSide) {
            int row, chunk;
            feed_slot<W, KR, false>(t, row, chunk);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = chunk * 8 + i < cols ? v[i] : (short)0;
        }
        *(LMEM s16x8 *)(lds + (wave<W>() * 4 + t) * 1024 + (threadIdx.x & 63) * 16) = v;
    }
}

// Four neighbouring elements of dW, n of which exist; `vec`: they are one access.
template <bool F32>
__device__ __forceinline__ f32x4 dw_get(const char *dw, int64_t e, int n, bool vec) {
    f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (F32) {
        if (vec) return *(const GMEM f32x4 *)gp(dw + e * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) x[i] = gp(reinterpret_cast<const float *>(dw))[e + i];
    } else {
        if (vec) {
            const u32x2 u = *(const GMEM u32x2 *)gp(dw + e * 2);
            return f32x4{bf16_to_f32(u.x & 0xFFFFu), bf16_to_f32(u.x >> 16), bf16_to_f32(u.y & 0xFFFFu),
                         bf16_to_f32(u.y >> 16)};
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) x[i] = bf16_to_f32(gp(reinterpret_cast<const uint16_t *>(dw))[e + i]);
    }
    return x;
}
template <bool F32>
__device__ __forceinline__ void dw_put(char *dw, int64_t e, int n, bool vec, f32x4 x) {
    if constexpr (F32) {
        if (vec) {
            *(GMEM f32x4 *)gp(dw + e * 4) = x;
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) gp(reinterpret_cast<float *>(dw))[e + i] = x[i];
    } else {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = f32_to_bf16_rne(x[i]);
        if (vec) {
            *(GMEM u32x2 *)gp(dw + e * 2) = u32x2{u[0] | u[1] << 16, u[2] | u[3] << 16};
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) gp(reinterpret_cast<uint16_t *>(dw))[e + i] = (uint16_t)u[i];
    }
}

template <int W, bool BF16, bool F32, bool DIRECT>
__global__ __launch_bounds__(Tile<W>::kLanes, Tile<W>::kWavesPerSimd) void expert_grad_kernel(ExpertArgs a) {
    __shared__ __align__(1024) char lds[Tile<W>::kLds];
    // workgroup -> piece, expert, tile
    const uint32_t b = blockIdx.x, slot = b / kXcds;
    const uint32_t group = slot / kGroup * kXcds + b % kXcds, in = slot % kGroup;
    const uint32_t gm = (a.mt + kBand - 1) / kBand, gn = (a.nt + kBand - 1) / kBand;
    const uint32_t per = gm * gn, whole = group / per;
    if (whole >= (uint32_t)a.experts * (uint32_t)a.pieces) return;
    const int32_t e = (int32_t)(whole % (uint32_t)a.experts), piece = (int32_t)(whole / (uint32_t)a.experts);
    const int32_t ti = (int32_t)(group % per / gn * kBand + in / kBand), tj = (int32_t)(group % per % gn * kBand + in % kBand);
    if (ti >= a.mt || tj >= a.nt) return;
    const Rows run = expert_piece(expert_run(a.offsets[e], a.offsets[e + 1], a.tokens), a.pieces, piece);
    const int32_t k0 = run.first, k1 = run.end;
    if (k0 >= k1 && a.accumulate && !a.parts) return;
    const int32_t mleft = a.m - ti * Tile<W>::kSide, nleft = a.n - tj * Tile<W>::kSide;
    const char *x = a.x + k0 * a.ldx + (int64_t)ti * Tile<W>::kSide * 2, *y = a.dy + k0 * a.ldy + (int64_t)tj * Tile<W>::kSide * 2;
    const int32_t rows = k1 - k0;
    Sums<W> s{};
    int32_t done = 0;
    if constexpr (DIRECT) {
        const int steps = rows / kStepRows;
        product<W, false, KR, KR, false, BF16>(feed<W, KR, false>(x, a.ldx, mleft), kStepRows * a.ldx,
                                     feed<W, KR, false>(y, a.ldy, nleft), kStepRows * a.ldy, steps, lds_at(lds), s);
        done = steps * kStepRows;
    }
    if (done < rows) {
        Chunks cx = load_chunks<W>(x + done * a.ldx, a.ldx, rows - done, mleft);
        Chunks cy = load_chunks<W>(y + done * a.ldy, a.ldy, rows - done, nleft);
        write_chunks<W>(cx, lds, mleft);
        write_chunks<W>(cy, lds + Tile<W>::kOperand, nleft);
        for (int32_t half = 0;; half ^= 1) {
            char *next = lds + (half ^ 1) * Tile<W>::kStage;
            const uint32_t now = lds_at(lds) + half * Tile<W>::kStage;
            __syncthreads();
            const bool more = next_step(done, rows);
            if (more) {
                cx = load_chunks<W>(x + done * a.ldx, a.ldx, rows - done, mleft);
                cy = load_chunks<W>(y + done * a.ldy, a.ldy, rows - done, nleft);
            }
            s16x8 q[4][2], p[2];
            read_q<W, KR, false>(now, q);
#pragma unroll
            for (int j = 0; j < Tile<W>::kJ; ++j) {
                read_p<W, KR, false>(now, j, p);
                multiply<false, BF16, W>(q, p, s, j);
            }
            if (!more) break;
            write_chunks<W>(cx, next, mleft);
            write_chunks<W>(cy, next + Tile<W>::kOperand, nleft);
        }
    }
    const float sc = rows > 0 && a.scale ? *a.scale : 1.0f;  // zeros whatever the scale
    // (a row's accesses before those of the row ahead of it: the compiler keeps
    // loads and stores of dW in order, and one at a time they would take a
    // memory latency each)
    const int32_t c0 = tj * Tile<W>::kSide + col0<W>();
    auto place = [&](int i, int j, int64_t &at) {  // elements that exist
        const int32_t r = ti * Tile<W>::kSide + row0<W>() + 16 * j, c = c0 + 16 * i;
        at = ((int64_t)e * a.m + r) * a.n + c;
        return r < a.m && c < a.n ? (a.n - c < 4 ? a.n - c : 4) : 0;
    };
    if (a.parts) {
        float *parts = a.parts + ((int64_t)piece * a.experts * a.m) * a.n;
#pragma unroll
        for (int j = 0; j < Tile<W>::kJ; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                int64_t at;
                if (const int n = place(i, j, at))
                    dw_put<true>(reinterpret_cast<char *>(parts), at, n, (a.n & 3) == 0, s.v[i][j]);
            }
        return;
    }
    f32x4 old[2][4];
    auto get = [&](int j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            int64_t at;
            if (const int n = place(i, j, at)) old[j & 1][i] = dw_get<F32>(a.dw, at, n, a.out_vec);
        }
    };
    if (a.accumulate) get(0);
#pragma unroll
    for (int j = 0; j < Tile<W>::kJ; ++j) {
        if (a.accumulate && j + 1 < Tile<W>::kJ) get(j + 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            int64_t at;
            if (const int n = place(i, j, at)) {
                f32x4 x = s.v[i][j] * sc;
                if (a.accumulate) x = old[j & 1][i] + x;
                dw_put<F32>(a.dw, at, n, a.out_vec, x);
            }
        }
    }
}

// The pieces' sums in their order.  Experts without rows get zeros, or keep their
// dW bit for bit, as they do in one piece.  (dW has at most 512 tiles here: its
// elements count in 32 bits.)
template <bool F32>
__global__ __launch_bounds__(kThreads) void expert_join_kernel(ExpertArgs a) {
    const int64_t total = (int64_t)a.experts * a.m * a.n;
    const uint32_t of = (uint32_t)a.m * (uint32_t)a.n;  // elements of an expert
    const float sc = a.scale ? *a.scale : 1.0f;
    auto empty = [&](uint32_t x) {
        const Rows run = expert_run(a.offsets[x], a.offsets[x + 1], a.tokens);
        return run.first == run.end;
    };
    for (int64_t e = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4; e < total; e += (int64_t)gridDim.x * kThreads * 4) {
        const int n = total - e < 4 ? (int)(total - e) : 4;
        f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int32_t p = 0; p < a.pieces; ++p) {
            const float *q = a.parts + (int64_t)p * total + e;
            if ((total & 3) == 0) {
                x = x + *(const GMEM f32x4 *)gp(q);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < n) x[i] += gp(q)[i];
            }
        }
        x = x * sc;
        const bool vec = a.out_vec;
        const uint32_t first = (uint32_t)e / of, last = (uint32_t)(e + n - 1) / of;
        if (first == last && !empty(first)) {
            if (a.accumulate) x = dw_get<F32>(a.dw, e, n, vec) + x;
            dw_put<F32>(a.dw, e, n, vec, x);
            continue;
        }
        // an expert without rows, or elements of several experts: one by one
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i >= n) break;
            const bool none = empty((uint32_t)(e + i) / of);
            if (none && a.accumulate) continue;
            f32x4 y = {none ? 0.0f : x[i], 0.0f, 0.0f, 0.0f};
            if (a.accumulate) y[0] = dw_get<F32>(a.dw, e + i, 1, false)[0] + y[0];
            dw_put<F32>(a.dw, e + i, 1, false, y);
        }
    }
}

template <int W>
int32_t tiles_of(int64_t n) { return (int32_t)((n + Tile<W>::kSide - 1) / Tile<W>::kSide); }

template <int W>
bool set_tiles(ExpertArgs &a, unsigned &grid) {
    a.mt = tiles_of<W>(a.m);
    a.nt = tiles_of<W>(a.n);
    const int64_t per = (int64_t)((a.mt + kBand - 1) / kBand) * ((a.nt + kBand - 1) / kBand);
    const int64_t groups = per * a.experts * a.pieces;
    const int64_t g = (groups + kXcds - 1) / kXcds * kXcds * kGroup;
    grid = (unsigned)g;
    return g <= INT32_MAX;
}

template <int W, bool BF16, bool F32>
hipError_t launch_expert_t(const ExpertArgs &args, bool direct, hipStream_t s) {
    ExpertArgs a = args;
    unsigned grid;
    if (!set_tiles<W>(a, grid)) return hipErrorInvalidValue;
    if (W == 2 || direct)  // wide tiles are for whole chunks
        hipLaunchKernelGGL((expert_grad_kernel<W, BF16, F32, true>), dim3(grid), dim3(Tile<W>::kLanes), 0, s, a);
    else
        hipLaunchKernelGGL((expert_grad_kernel<1, BF16, F32, false>), dim3(grid), dim3(Tile<1>::kLanes), 0, s, a);
    if (a.parts) {
        const int64_t quads = ((int64_t)a.experts * a.m * a.n + 3) / 4;
        const int64_t g = (quads + kThreads - 1) / kThreads;
        hipLaunchKernelGGL((expert_join_kernel<F32>), dim3((unsigned)(g < 4096 ? g : 4096)), dim3(kThreads), 0, s, a);
    }
    return hipGetLastError();
}

template <int W>
hipError_t launch_expert_w(const ExpertArgs &a, bool bf16, bool out_f32, bool direct, hipStream_t s) {
    if (bf16 && out_f32) return launch_expert_t<W, true, true>(a, direct, s);
    if (bf16) return launch_expert_t<W, true, false>(a, direct, s);
    if (out_f32) return launch_expert_t<W, false, true>(a, direct, s);
    return launch_expert_t<W, false, false>(a, direct, s);
}

}  // namespace

// Two workgroups fit a compute unit, 512 the GPU.  Fewer tiles than that with
// runs of many steps are summed in pieces of at least 8 steps (an even share
// of the rows) until about 512 workgroups have work, where that saves more than
// 16 steps, for joining the pieces takes 8 us and more.  Measured, in one piece
// and in several: 2 experts 512x512 over 16384 rows (128 steps, 16 pieces) 91 and
// 25 us, 1 of 1024x1024 over 8192 (128, 8) 93 and 33, 2 of 256x256 over 3584 (28,
// 3) 19 and 15, 4 of 512x512 over 6144 (24, 3) 18.5 and 18.4, 8 of 512x512 over
// 12288 (24, 3) 20 and 24, over 8192 (16, 2) 15 and 23.
int32_t expert_pieces(int32_t experts, int64_t tokens, int64_t m, int64_t n) {
    if (experts <= 0 || m <= 0 || n <= 0) return 1;
    const int64_t tiles = (int64_t)experts * tiles_of<1>(m) * tiles_of<1>(n);
    const int64_t steps = tokens / experts / kStepRows;
    const int64_t p = std::min<int64_t>(512 / tiles, steps / 8);
    return (int32_t)(p > 1 && steps - steps / p > 16 ? p : 1);
}

// Wide tiles where they fill the GPU (one workgroup a compute unit): measured
// on MI355X, 8 experts 2048x8192 over 16384 rows, accumulated in fp32, 616 us
// against 733 with narrow ones, 64 experts 2048x1024 over 65536 rows in bf16
// 310 (runs of equal length) against 388; 8 experts 512x2048 over 8192 rows, 128
// wide tiles, 44 against 31.  Only whole 16-byte chunks go that way.  The rule
// counts tiles, not how much of them is dW or how many steps a run has, and loses
// where sides are just past a tile or runs short: over 65536 rows, wide and
// narrow, 256 experts 128x128 60 and 23 us, 64 of 64x1040 57 and 41, of 264x264 58
// and 37, of 512x512 64 and 48, 128 of 384x384 81 and 42; 64 of 640x640 103 and
// 153.
hipError_t launch_expert_grad(const ExpertArgs &a, bool bf16, bool out_f32, bool direct, hipStream_t s) {
    const int64_t wide = (int64_t)a.experts * tiles_of<2>(a.m) * tiles_of<2>(a.n);
    return direct && wide >= 256 ? launch_expert_w<2>(a, bf16, out_f32, direct, s)
                                 : launch_expert_w<1>(a, bf16, out_f32, direct, s);
}

}  // namespace optim
