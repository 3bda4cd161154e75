// kernels_muon.hip -- the Muon step (include/optim_muon.h): momentum, then
// the orthogonalised direction of every matrix, then the update.
//
// The momentum pass is elementwise and bound by HBM; the iteration is matrix
// products and bound by the matrix cores.  A matrix X (scaled by kMuonScale, so
// that fp16's exponents reach what matters) is kept as a split array (tiles.h),
// rows and columns padded to multiples of 32 with zeros, which the products
// keep zero.  Nothing is ever transposed in memory: where rows <= cols ("wide")
// A = X X^T and X <- aX + B X, else A = X^T X and X <- aX + X B; the operand
// whose k runs down its rows goes through the LDS's transposing read.
// A and B are symmetric: only tiles on and above the diagonal are computed
// and each is stored on both sides.
// One launch of a kernel covers the tiles of every matrix of a run, from a
// table of (matrix, tile row, tile column).  Matrices with a side of at most
// 128 go another way (kernels_muon_slab.hip).
//
// Measured on MI355X, a step of five iterations: the seven matrices of a
// 4096-wide layer (202M elements, 14.8 TFLOP with symmetric products counted
// once, three times that on the matrix cores) 36.2 ms, of it products 35.1 ms at
// 1260 TFLOP/s of fp16 products, the matrix cores busy 68-75% of the time at the
// clock that the power limit leaves (1.83 GHz); momentum 0.38 ms (2.4 GB, 6.4
// TB/s), first split 0.46 ms (2.4 GB).  48 matrices of 1000 x 408: 1.06-1.09 ms,
// the matrix cores busy 25-52%: X passes through the Infinity Cache in
// every product (79 MB read and 79 MB written in 93 us), and 13 to 32 steps a
// tile do not hide a tile's beginning and end.
#include "muon_common.h"

namespace optim {
namespace {

// ---------------------------------------------------------------- momentum
// m <- mu m + g and each unit's sum of u^2 (fp64: a square overflows fp32
// long before a momentum does).
template <int GK>
__global__ __launch_bounds__(kThreads) void muon_momentum_kernel(StepArgs a, int32_t nesterov) {
    __shared__ Scalars S;
    __shared__ double red[kThreads / 64];
    step_begin(a, S);
    const StepCommit commit{a, S};
    if (S.skip) return;
    const float mu = uniform(S.b1), s = uniform(S.inv_scale);
    for_units(a, [&](int64_t u, const SpanDesc &sp, int64_t start, int64_t len) {
        const TensorDesc T = uniform_desc(a.tensors[sp.tensor]);
        double acc = 0.0;
        lane_walk<kAdamGroups>(start, len, T.vec_ok, [&](auto n, int64_t e) {
            constexpr int N = decltype(n)::value;
            float g[N], m[N], x[N];
            load_g<GK, N>(T.g, e, s, g);
            ldf<N>(T.m, e, m);
#pragma unroll
            for (int i = 0; i < N; ++i) m[i] = mu * m[i] + g[i];
            muon_u<N>(g, m, mu, nesterov, x);
#pragma unroll
            for (int i = 0; i < N; ++i) acc = __builtin_fma((double)x[i], (double)x[i], acc);
            stf<N>(T.m, e, m);
        });
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) acc += __shfl_xor(acc, o);
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = acc;
        __syncthreads();
        if (threadIdx.x == 0) a.partials[u] = (red[0] + red[1]) + (red[2] + red[3]);
        __syncthreads();
    });
}

// Per matrix, the factor that normalises it.
__global__ __launch_bounds__(kThreads) void muon_norm_kernel(StepArgs a, int32_t mats) {
    if (skipped(a)) return;
    __shared__ double red[kThreads];
    for (int b = blockIdx.x; b < mats; b += gridDim.x) {
        const int si = a.blockspan[b];
        red[threadIdx.x] = lane_sum(a.partials, 1, a.spans[si].unit_begin, a.spans[si + 1].unit_begin);
        __syncthreads();
        for (int st = kThreads / 2; st > 0; st >>= 1) {
            if ((int)threadIdx.x < st) red[threadIdx.x] += red[threadIdx.x + st];
            __syncthreads();
        }
        if (threadIdx.x == 0) {
            reinterpret_cast<double *>(a.blockfac)[b] = muon_factor(red[0], a.prep.eps);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- X0
__device__ __forceinline__ int muon_find(const MuonArgs &a, int64_t u) {
    int lo = a.mat0, hi = a.mat1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.mats[mid].unit0 <= u) lo = mid; else hi = mid;
    }
    return lo;
}

// Four values of a split array as two 8-byte stores.
__device__ __forceinline__ void put_split4(char *base, int64_t at, uint2 hi, uint2 lo) {
    GMEM u32x2 *q = (GMEM u32x2 *)gp(base + at * 2);
    q[0] = u32x2{hi.x, hi.y};
    q[8] = u32x2{lo.x, lo.y};
}
__device__ __forceinline__ void store_split4(char *base, int64_t at, const float (&x)[4]) {
    uint2 hi, lo;
    split4(x, hi, lo);
    put_split4(base, at, hi, lo);
}
// The normalised direction of a run's matrices as split arrays, padding as
// zeros: kMuonUnit elements of the padded matrix per workgroup.
template <int GK>
__global__ __launch_bounds__(kThreads) void muon_split_kernel(StepArgs a, MuonArgs ma, int32_t nesterov) {
    if (skipped(a)) return;
    const int mi = muon_find(ma, blockIdx.x);
    const MuonMat M = ma.mats[mi];
    const TensorDesc T = uniform_desc(a.tensors[M.tensor]);
    const float mu = (float)a.prep.beta1, s = a.prep.inv_scale ? *a.prep.inv_scale : 1.0f;
    const double f = reinterpret_cast<const double *>(a.blockfac)[mi];
    const bool vec = T.vec_ok && (M.cols & 3) == 0 && (M.elem0 & 3) == 0;
    int64_t at = ((int64_t)blockIdx.x - M.unit0) * kMuonUnit + threadIdx.x * 4;
#pragma unroll
    for (int k = 0; k < (int)(kMuonUnit / kSub); ++k, at += kSub) {
        if (at >= (int64_t)M.rp * M.ld) break;
        const int32_t r = (int32_t)(at / M.ld), c = (int32_t)(at % M.ld);
        float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (r < M.rows && c < M.cols) {
            const int64_t e = M.elem0 + (int64_t)r * M.cols + c;
            if (vec && c + 4 <= M.cols) {
                float g[4], m[4];
                load_g<GK, 4>(T.g, e, s, g);
                ldf<4>(T.m, e, m);
                muon_u<4>(g, m, mu, nesterov, x);
            } else {
                const int n = M.cols - c < 4 ? M.cols - c : 4;
                for (int i = 0; i < n; ++i) {
                    float g[1], m[1], y[1];
                    load_g<GK, 1>(T.g, e + i, s, g);
                    ldf<1>(T.m, e + i, m);
                    muon_u<1>(g, m, mu, nesterov, y);
                    x[i] = y[0];
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = (float)((double)x[i] * f);
        }
        store_split4(ma.ws + M.x[0], split_at(r, c, M.ld), x);
    }
}

// ---------------------------------------------------------------- products
// The operand whose rows (columns) are those of tile row (column) t of an
// array of `rows` (`cols`).
template <int W>
__device__ __forceinline__ Feed row_feed(const char *base, int t, int64_t rows32, int rows) {
    return feed<W, KC, true>(base + (int64_t)t * (Tile<W>::kSide / 32) * rows32, rows32, rows - t * Tile<W>::kSide);
}
template <int W>
__device__ __forceinline__ Feed column_feed(const char *base, int t, int64_t rows32, int cols) {
    return feed<W, KR, true>(base + (int64_t)t * (Tile<W>::kSide / 32) * kSplitBlock, rows32, cols - t * Tile<W>::kSide);
}

// Transposes a 4 x 4 block of 16-bit numbers held by 4 neighbouring lanes:
// lane q's four (element e in half e % 2 of word e / 2) become element q of
// the four lanes.
__device__ __forceinline__ uint2 transpose4(uint2 d) {
    const int q = threadIdx.x & 3;
    // neighbours: halves of both words
    const uint32_t x = (uint32_t)__builtin_amdgcn_mov_dpp((int)d.x, 0xB1, 0xF, 0xF, true);  // lane ^ 1
    const uint32_t y = (uint32_t)__builtin_amdgcn_mov_dpp((int)d.y, 0xB1, 0xF, 0xF, true);
    const uint32_t a = q & 1 ? (d.x & 0xFFFF0000u) | x >> 16 : (d.x & 0xFFFFu) | x << 16;
    const uint32_t b = q & 1 ? (d.y & 0xFFFF0000u) | y >> 16 : (d.y & 0xFFFFu) | y << 16;
    // pairs: whole words
    const uint32_t give = q & 2 ? a : b, keep = q & 2 ? b : a;
    const uint32_t take = (uint32_t)__builtin_amdgcn_mov_dpp((int)give, 0x4E, 0xF, 0xF, true);  // lane ^ 2
    return q & 2 ? make_uint2(take, keep) : make_uint2(keep, take);
}

// Up to four neighbouring split values of a row, as they lie in memory.
struct Split4 {
    u32x2 hi, lo;
};
__device__ __forceinline__ Split4 get_split4(const char *base, int64_t at) {
    const GMEM u32x2 *q = (const GMEM u32x2 *)gp(base + at * 2);
    return Split4{q[0], q[8]};
}
__device__ __forceinline__ void values(const Split4 &s, float (&x)[4]) {
    const f16x4 hi = __builtin_bit_cast(f16x4, s.hi), lo = __builtin_bit_cast(f16x4, s.lo);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (float)hi[i] + (float)lo[i];
}

// A wavefront's sums row by row (of 16): get(j, b) loads what use(j, b) needs
// of row j into b, a row ahead.  The compiler keeps a kernel's loads and stores
// in order, so loaded one by one they would take a memory latency each.
template <int W, bool PAIR, class Buffer, class Get, class Use>
__device__ __forceinline__ void rows_ahead(Get &&get, Use &&use) {
    constexpr int J = Tile<W, PAIR>::kOutJ;
    Buffer b[2];
    get(0, b[0]);
#pragma unroll
    for (int j = 0; j < J; ++j) {
        if (j + 1 < J) get(j + 1, b[(j + 1) & 1]);
        use(j, b[j & 1]);
    }
}

// Stores the values x of row r from column c on, of the symmetric n x n array
// at `base`; four neighbouring lanes hold the rows of a 4 x 4 block.  Above the
// diagonal blocks of 128 they are stored transposed too, below not at all: the
// same in wide and narrow tiles, whose (r, c) and (c, r), off by a rounding,
// would otherwise make a result depend on how the tiles were shared out.
__device__ __forceinline__ void store_symmetric(char *base, int n, int r, int c, const float (&x)[4]) {
    uint2 hi, lo;
    split4(x, hi, lo);
    const uint2 th = transpose4(hi), tl = transpose4(lo);
    // (the same in the four lanes of a block: n is a multiple of 32)
    if (r >= n || c >= n || r / kMuonTile > c / kMuonTile) return;
    put_split4(base, split_at(r, c, n), hi, lo);
    if (r / kMuonTile != c / kMuonTile) put_split4(base, split_at(c + (threadIdx.x & 3), r & ~3, n), th, tl);
}

// Partial sums of piece `part` of tile (i, j) of A or A A, row-major.
__device__ __forceinline__ float *piece_sums(const MuonArgs &ma, const MuonMat &M, const MuonTile &t, int part) {
    const int nt = (M.sp + kMuonTile - 1) / kMuonTile;
    return reinterpret_cast<float *>(ma.ws + M.part) + (((int64_t)part * nt + t.i) * nt + t.j) * kMuonTile * kMuonTile;
}
template <bool PAIR>
__device__ __forceinline__ void store_piece(float *at, const Sums<1> &s) {
    GMEM float *q = gp(at) + row0<1, PAIR>() * kMuonTile + col0<1>();
#pragma unroll
    for (int j = 0; j < Tile<1, PAIR>::kOutJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) *(GMEM f32x4 *)(q + 16 * j * kMuonTile + 16 * i) = s.v[i][j];
}
// Steps of piece `part` of `parts` of a sum of `all`, and where it begins.
__device__ __forceinline__ int piece_steps(int all, int parts, int part, int &first) {
    const int each = (all + parts - 1) / parts;
    first = part * each;
    return all - first < each ? all - first : each;
}

// A = X X^T or X^T X, or the sums over a piece of the longer side
template <int W, bool PAIR>
__global__ __launch_bounds__((Tile<W, PAIR>::kLanes), (Tile<W, PAIR>::kWavesPerSimd)) void muon_gram_kernel(StepArgs a, MuonArgs ma, int32_t from) {
    __shared__ __align__(1024) char lds[Tile<W, PAIR>::kLds];
    if (skipped(a)) return;
    const MuonTile t = ma.sym[blockIdx.x % ma.tiles];
    if (t.mat < 0) return;
    const MuonMat M = ma.mats[t.mat];
    const int part = blockIdx.x / ma.tiles;
    if (part >= M.parts[0]) return;
    const char *X = ma.ws + (from ? M.x[1] : M.x[0]);
    const int64_t rows32 = split_rows32(M.ld), step = M.tall ? rows32 : kSplitBlock;
    int first;
    const int steps = piece_steps(((M.tall ? M.rows : M.cols) + 31) / 32, M.parts[0], part, first);
    X += first * step;
    Sums<W> s{};
    if (M.tall)
        product<W, PAIR, KR, KR, true, false>(column_feed<W>(X, t.i, rows32, M.ld), step,
                                              column_feed<W>(X, t.j, rows32, M.ld), step, steps, lds_at(lds), s);
    else
        product<W, PAIR, KC, KC, true, false>(row_feed<W>(X, t.i, rows32, M.rp), step, row_feed<W>(X, t.j, rows32, M.rp),
                                              step, steps, lds_at(lds), s);
    join_pair<W, PAIR>(lds_at(lds), s);
    const int r0 = row0<W, PAIR>(), c0 = col0<W>();
    if constexpr (W == 1)
        if (M.parts[0] > 1) return store_piece<PAIR>(piece_sums(ma, M, t, part), s);
#pragma unroll
    for (int j = 0; j < Tile<W, PAIR>::kOutJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = s.v[i][j][e] * kMuonUnscale;
            store_symmetric(ma.ws + M.a, M.sp, t.i * Tile<W>::kSide + r0 + 16 * j, t.j * Tile<W>::kSide + c0 + 16 * i, x);
        }
}

// B = b A + c A A, or the sums over a piece of A A
template <int W, bool PAIR>
__global__ __launch_bounds__((Tile<W, PAIR>::kLanes), (Tile<W, PAIR>::kWavesPerSimd)) void muon_square_kernel(StepArgs a, MuonArgs ma) {
    __shared__ __align__(1024) char lds[Tile<W, PAIR>::kLds];
    if (skipped(a)) return;
    const MuonTile t = ma.sym[blockIdx.x % ma.tiles];
    if (t.mat < 0) return;
    const MuonMat M = ma.mats[t.mat];
    const int part = blockIdx.x / ma.tiles;
    if (part >= M.parts[1]) return;
    const char *A = ma.ws + M.a;
    const int64_t rows32 = split_rows32(M.sp);
    int first;
    const int steps = piece_steps(((M.tall ? M.cols : M.rows) + 31) / 32, M.parts[1], part, first);
    const char *P = A + first * kSplitBlock;
    Sums<W> s{};
    product<W, PAIR, KC, KC, true, false>(row_feed<W>(P, t.i, rows32, M.sp), kSplitBlock,
                                          row_feed<W>(P, t.j, rows32, M.sp), kSplitBlock, steps, lds_at(lds), s);
    join_pair<W, PAIR>(lds_at(lds), s);
    if constexpr (W == 1)
        if (M.parts[1] > 1) return store_piece<PAIR>(piece_sums(ma, M, t, part), s);
    struct Row {
        Split4 v[4];
    };
    const int r0 = t.i * Tile<W>::kSide + row0<W, PAIR>(), c0 = t.j * Tile<W>::kSide + col0<W>();
    rows_ahead<W, PAIR, Row>(
        [&](int j, Row &b) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (r0 + 16 * j < M.sp && c0 + 16 * i < M.sp) b.v[i] = get_split4(A, split_at(r0 + 16 * j, c0 + 16 * i, M.sp));
        },
        [&](int j, const Row &b) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x[4];
                values(b.v[i], x);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = ma.qb * x[e] + ma.qc * (s.v[i][j][e] * kMuonUnscale);
                store_symmetric(ma.ws + M.b, M.sp, r0 + 16 * j, c0 + 16 * i, x);
            }
        });
}

// Joins the pieces of tiles of A or A A, in their order: a quarter of a tile's
// rows per workgroup.
template <bool SQUARE>
__global__ __launch_bounds__(kThreads) void muon_join_kernel(StepArgs a, MuonArgs ma) {
    if (skipped(a)) return;
    const MuonTile t = ma.sym[blockIdx.x % ma.tiles];
    if (t.mat < 0) return;
    const MuonMat M = ma.mats[t.mat];
    const int parts = M.parts[SQUARE];
    if (parts <= 1) return;
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int r = (int)(blockIdx.x / ma.tiles) * 32 + (w & 1) * 16 + (lane & 15), c = (w >> 1) * 64 + (lane >> 4) * 4;
    const int64_t apart = piece_sums(ma, M, MuonTile{}, 1) - piece_sums(ma, M, MuonTile{}, 0);
    const GMEM float *q = gp(piece_sums(ma, M, t, 0)) + r * kMuonTile + c;
    f32x4 sum[4] = {};
    constexpr int U = 4;  // pieces under way
    for (int p = 0; p < parts; p += U) {
        f32x4 v[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (p + u < parts) v[u][i] = *(const GMEM f32x4 *)(q + (p + u) * apart + 16 * i);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (p + u < parts) sum[i] += v[u][i];
    }
    const int rt = t.i * kMuonTile + r, ct = t.j * kMuonTile + c;
    Split4 A[4];
    if constexpr (SQUARE)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (rt < M.sp && ct + 16 * i < M.sp) A[i] = get_split4(ma.ws + M.a, split_at(rt, ct + 16 * i, M.sp));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float x[4];
        if constexpr (SQUARE) values(A[i], x);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float y = sum[i][e] * kMuonUnscale;
            x[e] = SQUARE ? ma.qb * x[e] + ma.qc * y : y;
        }
        store_symmetric(ma.ws + (SQUARE ? M.b : M.a), M.sp, rt, ct + 16 * i, x);
    }
}

// X <- a X + B X or a X + X B
template <int W, bool PAIR>
__device__ __forceinline__ void apply_product(const MuonArgs &ma, const MuonTile &t, const MuonMat &M, const char *X,
                                              uint32_t lds, Sums<W> &s) {
    const int64_t x32 = split_rows32(M.ld), b32 = split_rows32(M.sp);
    const char *B = ma.ws + M.b;
    if (M.tall)
        product<W, PAIR, KC, KC, true, false>(row_feed<W>(X, t.i, x32, M.rp), kSplitBlock,
                                              row_feed<W>(B, t.j, b32, M.sp), kSplitBlock,
                                           (M.cols + 31) / 32, lds, s);
    else
        product<W, PAIR, KC, KR, true, false>(row_feed<W>(B, t.i, b32, M.sp), kSplitBlock,
                                              column_feed<W>(X, t.j, x32, M.ld), x32,
                                           (M.rows + 31) / 32, lds, s);
    join_pair<W, PAIR>(lds, s);
}

template <int W, bool PAIR>
__global__ __launch_bounds__((Tile<W, PAIR>::kLanes), (Tile<W, PAIR>::kWavesPerSimd)) void muon_apply_kernel(StepArgs a, MuonArgs ma, int32_t from) {
    __shared__ __align__(1024) char lds[Tile<W, PAIR>::kLds];
    if (skipped(a)) return;
    const MuonTile t = ma.full[blockIdx.x];
    if (t.mat < 0) return;
    const MuonMat M = ma.mats[t.mat];
    const char *X = ma.ws + (from ? M.x[1] : M.x[0]);
    char *Y = ma.ws + (from ? M.x[0] : M.x[1]);
    Sums<W> s{};
    apply_product<W, PAIR>(ma, t, M, X, lds_at(lds), s);
    struct Row {
        Split4 v[4];
    };
    const int r0 = t.i * Tile<W>::kSide + row0<W, PAIR>(), c0 = t.j * Tile<W>::kSide + col0<W>();
    rows_ahead<W, PAIR, Row>(
        [&](int j, Row &b) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (r0 + 16 * j < M.rp && c0 + 16 * i < M.ld) b.v[i] = get_split4(X, split_at(r0 + 16 * j, c0 + 16 * i, M.ld));
        },
        [&](int j, const Row &b) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x[4];
                values(b.v[i], x);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = ma.qa * x[e] + s.v[i][j][e] * kMuonUnscale;
                if (r0 + 16 * j < M.rp && c0 + 16 * i < M.ld) store_split4(Y, split_at(r0 + 16 * j, c0 + 16 * i, M.ld), x);
            }
        });
}

template <int W, bool PAIR, int PK>
__global__ __launch_bounds__((Tile<W, PAIR>::kLanes), (Tile<W, PAIR>::kWavesPerSimd)) void muon_update_kernel(StepArgs a, MuonArgs ma, int32_t from) {
    __shared__ __align__(1024) char lds[Tile<W, PAIR>::kLds];
    __shared__ Scalars sc;
    step_begin(a, sc);
    const StepCommit commit{a, sc};
    if (sc.skip) return;
    const MuonTile t = ma.full[blockIdx.x];
    if (t.mat < 0) return;
    const MuonMat M = ma.mats[t.mat];
    const char *X = ma.ws + (from ? M.x[1] : M.x[0]);
    Sums<W> s{};
    apply_product<W, PAIR>(ma, t, M, X, lds_at(lds), s);
    const TensorDesc T = uniform_desc(a.tensors[M.tensor]);
    const double scale = muon_scale(ma.scale_kind, M.rows, M.cols);
    const float f = (float)(sc.lr64 * scale), lw = sc.lrwd[T.group];
    const bool vec = T.vec_ok && (M.cols & 3) == 0 && (M.elem0 & 3) == 0;
    struct Row {
        Split4 v[4];
        float p[4][4];
    };
    const int r0 = t.i * Tile<W>::kSide + row0<W, PAIR>(), c0 = t.j * Tile<W>::kSide + col0<W>();
    auto at = [&](int i, int j) { return M.elem0 + (int64_t)(r0 + 16 * j) * M.cols + c0 + 16 * i; };
    auto left = [&](int i, int j) { return r0 + 16 * j < M.rows ? M.cols - c0 - 16 * i : 0; };  // elements of the row
    rows_ahead<W, PAIR, Row>(
        [&](int j, Row &b) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (left(i, j) <= 0) continue;
                b.v[i] = get_split4(X, split_at(r0 + 16 * j, c0 + 16 * i, M.ld));
                if (vec && left(i, j) >= 4) {
                    load_p<PK, 4, kStridedKeep>(T, at(i, j), b.p[i]);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < left(i, j)) {
                            float p[1];
                            load_p<PK, 1>(T, at(i, j) + k, p);
                            b.p[i][k] = p[0];
                        }
                }
            }
        },
        [&](int j, const Row &b) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (left(i, j) <= 0) continue;
                float x[4], p[4];
                values(b.v[i], x);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = (ma.qa * x[e] + s.v[i][j][e] * kMuonUnscale) * kMuonUnscale;
                    p[e] = decayed(b.p[i][e], lw, f * x[e]);
                }
                if (vec && left(i, j) >= 4) {
                    store_p_keep<PK, 4>(T, at(i, j), p);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < left(i, j)) {
                            const float y[1] = {p[k]};
                            store_p<PK, 1>(T, at(i, j) + k, y);
                        }
                }
            }
        });
}

}  // namespace

template <int W, bool PAIR>
static void launch_gram(const StepArgs &a, const MuonArgs &ma, int64_t tiles, int32_t parts, int32_t from, hipStream_t s) {
    LAUNCH_TRACED((muon_gram_kernel<W, PAIR>), (unsigned)(tiles * parts), (Tile<W, PAIR>::kLanes), s, a, ma, from);
}
template <int W, bool PAIR>
static void launch_square(const StepArgs &a, const MuonArgs &ma, int64_t tiles, int32_t parts, hipStream_t s) {
    LAUNCH_TRACED((muon_square_kernel<W, PAIR>), (unsigned)(tiles * parts), (Tile<W, PAIR>::kLanes), s, a, ma);
}

template <int W, bool PAIR, int PK>
static void launch_update(const StepArgs &a, const MuonArgs &ma, int64_t tiles, int32_t from, hipStream_t s) {
    LAUNCH_TRACED((muon_update_kernel<W, PAIR, PK>), (unsigned)tiles, (Tile<W, PAIR>::kLanes), s, a, ma, from);
}
// pk < 0: another iteration follows
template <int W, bool PAIR>
static void launch_apply(const StepArgs &a, const MuonArgs &ma, int64_t tiles, int32_t from, int pk, hipStream_t s) {
    if (pk < 0)
        LAUNCH_TRACED((muon_apply_kernel<W, PAIR>), (unsigned)tiles, (Tile<W, PAIR>::kLanes), s, a, ma, from);
    else if (pk == P_F32)
        launch_update<W, PAIR, P_F32>(a, ma, tiles, from, s);
    else if (pk == P_BF16R)
        launch_update<W, PAIR, P_BF16R>(a, ma, tiles, from, s);
    else if (pk == P_MBF16)
        launch_update<W, PAIR, P_MBF16>(a, ma, tiles, from, s);
    else
        launch_update<W, PAIR, P_MF16>(a, ma, tiles, from, s);
}

// One iteration over the tiles of a run: the wide ones, then the others.
static void launch_iteration(const StepArgs &a, const MuonArgs &args, const MuonRun &R, int32_t from, int pk,
                             bool commit, hipStream_t s) {
    MuonArgs ma = args, rest = args;
    ma.sym += R.sym0;
    ma.full += R.full0;
    rest.sym = ma.sym + R.wide_sym;
    rest.full = ma.full + R.wide_full;
    ma.tiles = (int32_t)R.wide_sym;
    rest.tiles = (int32_t)R.nsym;
    if (R.wide_sym) launch_gram<2, false>(a, ma, R.wide_sym, 1, from, s);
    if (R.nsym && R.pair_sym) launch_gram<1, true>(a, rest, R.nsym, R.most_parts[0], from, s);
    else if (R.nsym) launch_gram<1, false>(a, rest, R.nsym, R.most_parts[0], from, s);
    const unsigned quarters = (unsigned)R.nsym * 4;
    if (R.most_parts[0] > 1) LAUNCH_TRACED((muon_join_kernel<false>), quarters, kThreads, s, a, rest);
    if (R.wide_sym) launch_square<2, false>(a, ma, R.wide_sym, 1, s);
    if (R.nsym && R.pair_sym) launch_square<1, true>(a, rest, R.nsym, R.most_parts[1], s);
    else if (R.nsym) launch_square<1, false>(a, rest, R.nsym, R.most_parts[1], s);
    if (R.most_parts[1] > 1) LAUNCH_TRACED((muon_join_kernel<true>), quarters, kThreads, s, a, rest);
    StepArgs b = a;
    b.commit = commit && !R.nfull;  // the last launch publishes the step
    if (R.wide_full) launch_apply<2, false>(b, ma, R.wide_full, from, pk, s);
    b.commit = commit;
    if (R.nfull && R.pair_full) launch_apply<1, true>(b, rest, R.nfull, from, pk, s);
    else if (R.nfull) launch_apply<1, false>(b, rest, R.nfull, from, pk, s);
}

hipError_t launch_muon(const StepArgs &args, const MuonArgs &margs, int pk, int gk, int32_t steps, int32_t nesterov,
                       const MuonRun *runs, int32_t nruns, hipStream_t s) {
    // matrices that one workgroup each takes through the whole step
    const int64_t lone = margs.nmats - margs.lone0;
    StepArgs a = args;
    a.commit = nruns == 0 && lone == 0;  // else the last launch publishes the step
    a.nunits = margs.lone_unit0;
    if (nruns > 0 || lone == 0) {
        if (gk == G_F32)
            LAUNCH_TRACED((muon_momentum_kernel<G_F32>), persistent_grid(0, a), kThreads, s, a, nesterov);
        else
            LAUNCH_TRACED((muon_momentum_kernel<G_BF16>), persistent_grid(0, a), kThreads, s, a, nesterov);
    }
    if (nruns > 0)
        LAUNCH_TRACED(muon_norm_kernel, (unsigned)(margs.lone0 < 2048 ? margs.lone0 : 2048), kThreads, s, a, margs.lone0);
    hipError_t e = hipGetLastError();
    for (int32_t k = 0; k < nruns && e == hipSuccess; ++k) {
        const MuonRun &R = runs[k];
        MuonArgs ma = margs;
        ma.mat0 = R.mat0;
        ma.mat1 = R.mat1;
        if (R.slabs > 0) {
            e = launch_muon_slabs(a, ma, R, pk, gk, steps, nesterov, lone == 0 && k + 1 == nruns, s);
            continue;
        }
        if (gk == G_F32)
            LAUNCH_TRACED((muon_split_kernel<G_F32>), (unsigned)R.units, kThreads, s, a, ma, nesterov);
        else
            LAUNCH_TRACED((muon_split_kernel<G_BF16>), (unsigned)R.units, kThreads, s, a, ma, nesterov);
        for (int32_t i = 0; i < steps; ++i) {
            const bool last = i + 1 == steps;
            launch_iteration(a, ma, R, i & 1, last ? pk : -1, last && lone == 0 && k + 1 == nruns, s);
        }
        e = hipGetLastError();
    }
    if (e == hipSuccess && lone > 0) e = launch_muon_lone(args, margs, pk, gk, steps, nesterov, s);
    return e;
}

}  // namespace optim
