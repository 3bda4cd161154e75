// kernels_muon.hip -- the Muon step (include/optim_muon.h): momentum, then
// the orthogonalised direction of every matrix, then the update.
//
// The momentum pass is elementwise and bound by HBM; the iteration is matrix
// products and bound by the matrix cores.  A matrix X (scaled by kMuonScale, so
// that fp16's exponents reach what matters) is kept as a split array (tiles.h),
// rows and columns padded to whole tiles with zeros, which the products keep
// zero.  Nothing is ever transposed in memory: where rows <= cols ("wide")
// A = X X^T and X <- aX + B X, else A = X^T X and X <- aX + X B; the operand
// whose k runs down its rows goes through the LDS's transposing read.
// A and B are symmetric: only tiles on and above the diagonal are computed
// and each is stored on both sides.
// One launch of a kernel covers the tiles of every matrix of a run, from a
// table of (matrix, tile row, tile column).
#include "optim_muon.h"

#include "tiles.h"

namespace optim {
namespace {

// X, A and B are stored times 2^12: bounded by 15 (checked on the host) they
// stay below fp16's 65504, and a typical element of a 4096 x 4096 X, 2^-12 at
// the start and 2^-6 at the end, has both its parts well above fp16's
// smallest subnormal, 2^-24.
constexpr float kMuonScale = 4096.0f, kMuonUnscale = 1.0f / 4096.0f;

__device__ __forceinline__ bool skipped(const StepArgs &a) {
    return a.prep.found_inf && *a.prep.found_inf != 0.0f;
}

template <int N>
__device__ __forceinline__ void muon_u(const float (&g)[N], float (&m)[N], float mu, bool nesterov, float (&u)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) u[i] = nesterov ? g[i] + mu * m[i] : m[i];
}

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

// Per matrix, the factor kMuonScale / (||u|| + eps), in fp64 (with eps 0 and
// a small u it may leave fp32's range; the scaled u does not).
__global__ __launch_bounds__(kThreads) void muon_norm_kernel(StepArgs a) {
    if (skipped(a)) return;
    __shared__ double red[kThreads];
    for (int b = blockIdx.x; b < a.nblocks; b += gridDim.x) {
        const int si = a.blockspan[b];
        red[threadIdx.x] = lane_sum(a.partials, 1, a.spans[si].unit_begin, a.spans[si + 1].unit_begin);
        __syncthreads();
        for (int st = kThreads / 2; st > 0; st >>= 1) {
            if ((int)threadIdx.x < st) red[threadIdx.x] += red[threadIdx.x + st];
            __syncthreads();
        }
        if (threadIdx.x == 0) {
            const double n = sqrt(red[0]) + a.prep.eps;
            reinterpret_cast<double *>(a.blockfac)[b] = n == 0.0 ? 0.0 : (double)kMuonScale / n;
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
__device__ __forceinline__ void store_split4(char *base, int64_t at, const float (&x)[4]) {
    f16x4 hi, lo;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        _Float16 h, l;
        split2(x[i], h, l);
        hi[i] = h;
        lo[i] = l;
    }
    GMEM f16x4 *q = (GMEM f16x4 *)gp(base + at * 2);
    q[0] = hi;
    q[8] = lo;
}
__device__ __forceinline__ void load_split4(const char *base, int64_t at, float (&x)[4]) {
    const GMEM f16x4 *q = (const GMEM f16x4 *)gp(base + at * 2);
    const f16x4 hi = q[0], lo = q[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (float)hi[i] + (float)lo[i];
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
// Stores this wavefront's 64 x 64 sums times f as part of tile (ti, tj) of
// the symmetric array at `base`, and of tile (tj, ti).
template <class F>
__device__ __forceinline__ void store_symmetric(char *base, int64_t ld, int ti, int tj, F &&value) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t r = (int64_t)ti * kTile + row0() + 16 * j, c = (int64_t)tj * kTile + col0() + 16 * i;
            float x[4];
            value(i, j, r, c, x);
            store_split4(base, split_at(r, c, ld), x);
            if (ti != tj) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    _Float16 hi, lo;
                    split2(x[e], hi, lo);
                    GMEM _Float16 *q = (GMEM _Float16 *)gp(base + split_at(c + e, r, ld) * 2);
                    q[0] = hi;
                    q[32] = lo;
                }
            }
        }
}

// A = X X^T or X^T X
__global__ __launch_bounds__(kThreads, 2) void muon_gram_kernel(StepArgs a, MuonArgs ma, int32_t from) {
    __shared__ __align__(1024) char lds[2 * kStageBytes];
    if (skipped(a)) return;
    const MuonTile t = ma.sym[blockIdx.x];
    const MuonMat M = ma.mats[t.mat];
    const char *X = ma.ws + M.x[from];
    const int64_t row = 4 * (int64_t)M.ld;  // bytes
    Sums s{};
    if (M.tall)
        product<KR, KR, true, false>(feed<KR, true>(X + (int64_t)t.i * kTile * 4, row), 32 * row,
                                     feed<KR, true>(X + (int64_t)t.j * kTile * 4, row), 32 * row, (M.rows + 31) / 32,
                                     lds, s);
    else
        product<KC, KC, true, false>(feed<KC, true>(X + (int64_t)t.i * kTile * row, row), 128,
                                     feed<KC, true>(X + (int64_t)t.j * kTile * row, row), 128, (M.cols + 31) / 32, lds,
                                     s);
    store_symmetric(ma.ws + M.a, M.sp, t.i, t.j, [&](int i, int j, int64_t, int64_t, float(&x)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = s.v[i][j][e] * kMuonUnscale;
    });
}

// B = b A + c A A
__global__ __launch_bounds__(kThreads, 2) void muon_square_kernel(StepArgs a, MuonArgs ma) {
    __shared__ __align__(1024) char lds[2 * kStageBytes];
    if (skipped(a)) return;
    const MuonTile t = ma.sym[blockIdx.x];
    const MuonMat M = ma.mats[t.mat];
    const char *A = ma.ws + M.a;
    const int64_t row = 4 * (int64_t)M.sp;
    Sums s{};
    product<KC, KC, true, false>(feed<KC, true>(A + (int64_t)t.i * kTile * row, row), 128,
                                 feed<KC, true>(A + (int64_t)t.j * kTile * row, row), 128,
                                 ((M.tall ? M.cols : M.rows) + 31) / 32, lds, s);
    store_symmetric(ma.ws + M.b, M.sp, t.i, t.j, [&](int i, int j, int64_t r, int64_t c, float(&x)[4]) {
        load_split4(A, split_at(r, c, M.sp), x);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = ma.qb * x[e] + ma.qc * (s.v[i][j][e] * kMuonUnscale);
    });
}

// X <- a X + B X or a X + X B
__device__ __forceinline__ void apply_product(const MuonArgs &ma, const MuonTile &t, const MuonMat &M, const char *X,
                                              char *lds, Sums &s) {
    const int64_t xrow = 4 * (int64_t)M.ld, brow = 4 * (int64_t)M.sp;
    const char *B = ma.ws + M.b;
    if (M.tall)
        product<KC, KC, true, false>(feed<KC, true>(X + (int64_t)t.i * kTile * xrow, xrow), 128,
                                     feed<KC, true>(B + (int64_t)t.j * kTile * brow, brow), 128, (M.cols + 31) / 32, lds,
                                     s);
    else
        product<KC, KR, true, false>(feed<KC, true>(B + (int64_t)t.i * kTile * brow, brow), 128,
                                     feed<KR, true>(X + (int64_t)t.j * kTile * 4, xrow), 32 * xrow, (M.rows + 31) / 32,
                                     lds, s);
}

__global__ __launch_bounds__(kThreads, 2) void muon_apply_kernel(StepArgs a, MuonArgs ma, int32_t from) {
    __shared__ __align__(1024) char lds[2 * kStageBytes];
    if (skipped(a)) return;
    const MuonTile t = ma.full[blockIdx.x];
    const MuonMat M = ma.mats[t.mat];
    const char *X = ma.ws + M.x[from];
    char *Y = ma.ws + M.x[from ^ 1];
    Sums s{};
    apply_product(ma, t, M, X, lds, s);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t at = split_at((int64_t)t.i * kTile + row0() + 16 * j, (int64_t)t.j * kTile + col0() + 16 * i, M.ld);
            float x[4];
            load_split4(X, at, x);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = ma.qa * x[e] + s.v[i][j][e] * kMuonUnscale;
            store_split4(Y, at, x);
        }
}

// The last application and the update.
template <int PK, int N>
__device__ __forceinline__ void muon_update(const TensorDesc &T, int64_t e, const float *x, float lw, float f) {
    float p[N];
    load_p<PK, N>(T, e, p);
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = decayed(p[i], lw, f * x[i]);
    store_p<PK, N>(T, e, p);
}

template <int PK>
__global__ __launch_bounds__(kThreads, 2) void muon_update_kernel(StepArgs a, MuonArgs ma, int32_t from) {
    __shared__ __align__(1024) char lds[2 * kStageBytes];
    __shared__ Scalars S;
    step_begin(a, S);
    const StepCommit commit{a, S};
    if (S.skip) return;
    const MuonTile t = ma.full[blockIdx.x];
    const MuonMat M = ma.mats[t.mat];
    const char *X = ma.ws + M.x[from];
    Sums s{};
    apply_product(ma, t, M, X, lds, s);
    const TensorDesc T = uniform_desc(a.tensors[M.tensor]);
    const double r = M.rows, c = M.cols;
    const double scale = ma.scale_kind == OPTIM_MUON_SCALE_RMS      ? 0.2 * sqrt(r > c ? r : c)
                         : ma.scale_kind == OPTIM_MUON_SCALE_ASPECT ? sqrt(r > c ? r / c : 1.0)
                                                                    : 1.0;
    const float f = (float)(S.lr64 * scale), lw = S.lrwd[T.group];
    const bool vec = T.vec_ok && (M.cols & 3) == 0 && (M.elem0 & 3) == 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int32_t rr = t.i * kTile + row0() + 16 * j, cc = t.j * kTile + col0() + 16 * i;
            if (rr >= M.rows || cc >= M.cols) continue;
            float x[4];
            load_split4(X, split_at(rr, cc, M.ld), x);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = (ma.qa * x[e] + s.v[i][j][e] * kMuonUnscale) * kMuonUnscale;
            const int64_t e = M.elem0 + (int64_t)rr * M.cols + cc;
            if (vec && cc + 4 <= M.cols)
                muon_update<PK, 4>(T, e, x, lw, f);
            else
                for (int k = 0; k < 4 && cc + k < M.cols; ++k) muon_update<PK, 1>(T, e + k, x + k, lw, f);
        }
}

}  // namespace

template <int PK>
static void launch_update(const StepArgs &a, const MuonArgs &ma, int64_t grid, int32_t from, hipStream_t s) {
    LAUNCH_TRACED((muon_update_kernel<PK>), (unsigned)grid, kThreads, s, a, ma, from);
}

hipError_t launch_muon(const StepArgs &args, const MuonArgs &margs, int pk, int gk, int32_t steps, int32_t nesterov,
                       const MuonRun *runs, int32_t nruns, hipStream_t s) {
    StepArgs a = args;
    a.commit = nruns == 0;  // else the last update publishes the step
    if (gk == G_F32)
        LAUNCH_TRACED((muon_momentum_kernel<G_F32>), persistent_grid(0, a), kThreads, s, a, nesterov);
    else
        LAUNCH_TRACED((muon_momentum_kernel<G_BF16>), persistent_grid(0, a), kThreads, s, a, nesterov);
    if (nruns > 0)
        LAUNCH_TRACED(muon_norm_kernel, (unsigned)(a.nblocks < 2048 ? a.nblocks : 2048), kThreads, s, a);
    hipError_t e = hipGetLastError();
    for (int32_t k = 0; k < nruns && e == hipSuccess; ++k) {
        const MuonRun &R = runs[k];
        MuonArgs ma = margs;
        ma.mat0 = R.mat0;
        ma.mat1 = R.mat1;
        ma.sym += R.sym0;
        ma.full += R.full0;
        if (gk == G_F32)
            LAUNCH_TRACED((muon_split_kernel<G_F32>), (unsigned)R.units, kThreads, s, a, ma, nesterov);
        else
            LAUNCH_TRACED((muon_split_kernel<G_BF16>), (unsigned)R.units, kThreads, s, a, ma, nesterov);
        for (int32_t i = 0; i < steps; ++i) {
            const int32_t from = i & 1;
            LAUNCH_TRACED(muon_gram_kernel, (unsigned)R.nsym, kThreads, s, a, ma, from);
            LAUNCH_TRACED(muon_square_kernel, (unsigned)R.nsym, kThreads, s, a, ma);
            if (i + 1 < steps) {
                LAUNCH_TRACED(muon_apply_kernel, (unsigned)R.nfull, kThreads, s, a, ma, from);
                continue;
            }
            StepArgs b = a;
            b.commit = k + 1 == nruns;
            if (pk == P_F32) launch_update<P_F32>(b, ma, R.nfull, from, s);
            else if (pk == P_BF16R) launch_update<P_BF16R>(b, ma, R.nfull, from, s);
            else if (pk == P_MBF16) launch_update<P_MBF16>(b, ma, R.nfull, from, s);
            else launch_update<P_MF16>(b, ma, R.nfull, from, s);
        }
        e = hipGetLastError();
    }
    return e;
}

}  // namespace optim
