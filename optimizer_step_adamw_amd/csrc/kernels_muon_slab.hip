// kernels_muon_slab.hip -- the Muon step of matrices with a side of at most
// 128 (include/optim_muon.h): heads, adapters, routers, small models.
//
// With the short side s padded to SP = 64 or 128, A and B are one small square
// that a workgroup holds in LDS beside a slab of X: kMuonSlab / SP positions
// along the long side.  Between the slabs of a matrix only their parts of A
// pass: an iteration is one launch in which every slab sums all parts, squares
// A, makes B, applies it to its own X and forms its part of the next A.  A
// matrix of one slab needs no passing at all: momentum, norm, all iterations
// and the update are one launch.
//
// What bounds it is latency (an iteration is a few microseconds of dependent
// LDS reads, products and barriers).  Measured on MI355X: see the table of the
// launches at their kernels.
//
// X lies in LDS as rows of positions along the long side, 32 values along the
// short side to a 128-byte row (32 high parts, 32 low parts; chunks of 16
// bytes permuted by the row), so it is the KC operand of X B and the KR operand
// of X^T X whether the matrix is tall or wide; only the loads of the first and
// the update of the last iteration know the difference.
#include "muon_common.h"

namespace optim {
namespace {

template <int SP>
struct Slab {
    static constexpr int kLong = kMuonSlab / SP;      // positions
    static constexpr int kBlocks = SP / 32;           // 32-value blocks of the short side
    static constexpr int kXBytes = kMuonSlab * 4;     // X in LDS and in the workspace
    static constexpr int kABytes = SP * SP * 4;       // A or B in LDS, or a part of A
    static constexpr int kRowFrags = SP / 64;         // 16-row fragments of A of a wavefront
    static constexpr int kColFrags = SP / 16;
    static constexpr int kLongFrags = kLong / 64;     // 16-position fragments of X of a wavefront
    static constexpr int kPerLane = kMuonSlab / kThreads;
};

// Byte of the 16-byte chunk holding value c (of 8) of row r, in an LDS array
// of `rows` rows.
__device__ __forceinline__ uint32_t slab_chunk(int rows, int r, int c, int part) {
    return (uint32_t)((c >> 5) * rows * 128 + r * 128 + (((part * 4 + ((c & 31) >> 3)) ^ (r & 7)) << 4));
}
// 16 rows x 32 values along the short side
__device__ __forceinline__ s16x8 slab_kc(uint32_t base, int rows, int block, int b, int part) {
    const int l = threadIdx.x & 63;
    return *lds_ptr<const s16x8>(base + slab_chunk(rows, b * 16 + (l & 15), block * 32 + (l >> 4) * 8, part));
}
// 16 columns of the short side x 32 rows from k0
__device__ __forceinline__ s16x8 slab_kr(uint32_t base, int rows, int b, int k0, int part) {
    const int l = threadIdx.x & 63, k = k0 + (l >> 4) * 8 + ((l & 15) >> 2), c = b * 16 + ((l & 3) >> 1) * 8;
    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(lds_ptr<s16x4>(base + slab_chunk(rows, k, c, part) + (l & 1) * 8));
    const s16x4 y =
        __builtin_amdgcn_ds_read_tr16_b64_v4i16(lds_ptr<s16x4>(base + slab_chunk(rows, k + 4, c, part) + (l & 1) * 8));
    return s16x8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
}
// Four neighbouring values of a row.
__device__ __forceinline__ void slab_put4(uint32_t base, int rows, int r, int c, const float (&x)[4]) {
    uint2 hi, lo;
    split4(x, hi, lo);
    *lds_ptr<u32x2>(base + slab_chunk(rows, r, c, 0) + (c & 4) * 2) = u32x2{hi.x, hi.y};
    *lds_ptr<u32x2>(base + slab_chunk(rows, r, c, 1) + (c & 4) * 2) = u32x2{lo.x, lo.y};
}
__device__ __forceinline__ void slab_get4(uint32_t base, int rows, int r, int c, float (&x)[4]) {
    const f16x4 hi = *lds_ptr<const f16x4>(base + slab_chunk(rows, r, c, 0) + (c & 4) * 2);
    const f16x4 lo = *lds_ptr<const f16x4>(base + slab_chunk(rows, r, c, 1) + (c & 4) * 2);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (float)hi[i] + (float)lo[i];
}

// This wavefront's rows of A: v[r][i][e] is row 16 (wave kRowFrags + r) + lane
// % 16, column 16 i + 4 (lane / 16) + e.
template <int SP>
struct Square {
    f32x4 v[Slab<SP>::kRowFrags][Slab<SP>::kColFrags];
};
template <int SP>
__device__ __forceinline__ int square_row(int r) {
    return ((threadIdx.x >> 6) * Slab<SP>::kRowFrags + r) * 16 + (threadIdx.x & 15);
}
__device__ __forceinline__ int square_col(int i) { return i * 16 + ((threadIdx.x & 63) >> 4) * 4; }

template <int SP, class P, class Q>
__device__ __forceinline__ void square_step(Square<SP> &s, P &&rows, Q &&cols) {
    using T = Slab<SP>;
    s16x8 p[T::kRowFrags][2];
#pragma unroll
    for (int r = 0; r < T::kRowFrags; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) p[r][h] = rows((threadIdx.x >> 6) * T::kRowFrags + r, h);
#pragma unroll
    for (int i = 0; i < T::kColFrags; ++i) {
        const s16x8 q0 = cols(i, 0), q1 = cols(i, 1);
#pragma unroll
        for (int r = 0; r < T::kRowFrags; ++r) {
            s.v[r][i] = mfma<false>(q0, p[r][0], s.v[r][i]);
            s.v[r][i] = mfma<false>(q1, p[r][0], s.v[r][i]);
            s.v[r][i] = mfma<false>(q0, p[r][1], s.v[r][i]);
        }
    }
}

// The slab's part of A (times kMuonScale), over `len` positions.
template <int SP>
__device__ __forceinline__ void slab_gram(uint32_t xs, int len, Square<SP> &s) {
    using T = Slab<SP>;
    s = Square<SP>{};
    for (int k = 0; k < len; k += 32)
        square_step<SP>(
            s, [&](int b, int h) { return slab_kr(xs, T::kLong, b, k, h); },
            [&](int b, int h) { return slab_kr(xs, T::kLong, b, k, h); });
#pragma unroll
    for (int r = 0; r < T::kRowFrags; ++r)
#pragma unroll
        for (int i = 0; i < T::kColFrags; ++i) s.v[r][i] = s.v[r][i] * kMuonUnscale;
}

template <int SP>
__device__ __forceinline__ void square_put(uint32_t as, const Square<SP> &s) {
#pragma unroll
    for (int r = 0; r < Slab<SP>::kRowFrags; ++r)
#pragma unroll
        for (int i = 0; i < Slab<SP>::kColFrags; ++i) {
            const float x[4] = {s.v[r][i][0], s.v[r][i][1], s.v[r][i][2], s.v[r][i][3]};
            slab_put4(as, SP, square_row<SP>(r), square_col(i), x);
        }
}

// B = b A + c A A into LDS, from A in registers; `side`: the short side.  X is
// complete in LDS on return.
template <int SP>
__device__ __forceinline__ void slab_polynomial(const MuonArgs &ma, uint32_t as, const Square<SP> &A, int side) {
    square_put<SP>(as, A);
    __syncthreads();
    Square<SP> s{};
    for (int block = 0; block * 32 < side; ++block)
        square_step<SP>(
            s, [&](int b, int h) { return slab_kc(as, SP, block, b, h); },
            [&](int b, int h) { return slab_kc(as, SP, block, b, h); });
    __syncthreads();  // A has been read
#pragma unroll
    for (int r = 0; r < Slab<SP>::kRowFrags; ++r)
#pragma unroll
        for (int i = 0; i < Slab<SP>::kColFrags; ++i)
            s.v[r][i] = ma.qb * A.v[r][i] + ma.qc * (s.v[r][i] * kMuonUnscale);
    square_put<SP>(as, s);
    __syncthreads();
}

// X <- a X + X B: a wavefront's own rows.  put(row, column, four values) takes them.
template <int SP, class F>
__device__ __forceinline__ void slab_apply(const MuonArgs &ma, uint32_t xs, uint32_t as, int side, int len, F &&put) {
    using T = Slab<SP>;
#pragma unroll
    for (int x = 0; x < T::kLongFrags; ++x) {
        const int b = (threadIdx.x >> 6) * T::kLongFrags + x;
        if (b * 16 >= len) break;
        f32x4 acc[T::kColFrags] = {};
        for (int block = 0; block * 32 < side; ++block) {
            const s16x8 p0 = slab_kc(xs, T::kLong, block, b, 0), p1 = slab_kc(xs, T::kLong, block, b, 1);
#pragma unroll
            for (int i = 0; i < T::kColFrags; ++i) {
                const s16x8 q0 = slab_kc(as, SP, block, i, 0), q1 = slab_kc(as, SP, block, i, 1);
                acc[i] = mfma<false>(q0, p0, acc[i]);
                acc[i] = mfma<false>(q1, p0, acc[i]);
                acc[i] = mfma<false>(q0, p1, acc[i]);
            }
        }
        const int row = b * 16 + (threadIdx.x & 15);
#pragma unroll
        for (int i = 0; i < T::kColFrags; ++i) {
            float y[4];
            slab_get4(xs, T::kLong, row, square_col(i), y);
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = ma.qa * y[e] + acc[i][e] * kMuonUnscale;
            put(row, square_col(i), y);
        }
    }
}

// A matrix's shape as its slabs see it.
struct Shape {
    int64_t e0;     // element of the slab's first position, first value
    int32_t cols;   // elements between the matrix's rows
    int32_t side;   // the short side
    int32_t len;    // positions of this slab
    int32_t tall;
};
template <int SP>
__device__ __forceinline__ Shape slab_shape(const MuonMat &M, int32_t slab) {
    Shape h;
    h.tall = M.tall;
    h.cols = M.cols;
    h.side = M.tall ? M.cols : M.rows;
    const int32_t left = (M.tall ? M.rows : M.cols) - slab * Slab<SP>::kLong;
    h.len = left < Slab<SP>::kLong ? left : Slab<SP>::kLong;
    h.e0 = M.elem0 + (int64_t)slab * Slab<SP>::kLong * (M.tall ? M.cols : 1);
    return h;
}
// Position and value of the slab's element k in memory order, and its place.
__device__ __forceinline__ int64_t slab_element(const Shape &h, int32_t k, int32_t &row, int32_t &c) {
    if (h.tall) {
        row = k / h.side;
        c = k - row * h.side;
        return h.e0 + k;
    }
    c = k / h.len;
    row = k - c * h.len;
    return h.e0 + (int64_t)c * h.cols + row;
}

__device__ __forceinline__ void slab_zero(uint32_t xs) {
    for (int k = threadIdx.x; k < kMuonSlab / 4; k += kThreads) *lds_ptr<u32x4>(xs + k * 16) = u32x4{0, 0, 0, 0};
}
template <int SP>
__device__ __forceinline__ void slab_put1(uint32_t xs, int32_t row, int32_t c, float x) {
    _Float16 hi, lo;
    split2(x, hi, lo);
    *lds_ptr<_Float16>(xs + slab_chunk(Slab<SP>::kLong, row, c, 0) + (c & 7) * 2) = hi;
    *lds_ptr<_Float16>(xs + slab_chunk(Slab<SP>::kLong, row, c, 1) + (c & 7) * 2) = lo;
}

// The update of four neighbouring values of a position.
template <int PK>
__device__ __forceinline__ void slab_update(const TensorDesc &T, const Shape &h, int row, int c, const float (&y)[4],
                                            float lw, float f, bool vec) {
    if (row >= h.len || c >= h.side) return;
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = y[i] * kMuonUnscale;
    if (h.tall) {
        const int64_t e = h.e0 + (int64_t)row * h.cols + c;
        if (vec && c + 4 <= h.side) {
            muon_update<PK, 4>(T, e, x, lw, f);
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i < h.side) muon_update<PK, 1>(T, e + i, x + i, lw, f);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i < h.side) muon_update<PK, 1>(T, h.e0 + (int64_t)(c + i) * h.cols + row, x + i, lw, f);
    }
}
template <int PK>
struct Update {
    TensorDesc T;
    Shape h;
    float lw, f;
    bool vec;
    __device__ __forceinline__ Update(const StepArgs &a, const MuonArgs &ma, const MuonMat &M, const Shape &shape,
                                      const Scalars &sc)
        : T(uniform_desc(a.tensors[M.tensor])), h(shape) {
        f = (float)(sc.lr64 * muon_scale(ma.scale_kind, M.rows, M.cols));
        lw = sc.lrwd[T.group];
        vec = T.vec_ok && (M.cols & 3) == 0 && (M.elem0 & 3) == 0;
    }
    __device__ __forceinline__ void operator()(int row, int c, const float (&y)[4]) const {
        slab_update<PK>(T, h, row, c, y, lw, f, vec);
    }
};

// ---------------------------------------------------------------- one slab
// The whole step of one matrix.
template <int SP, int GK, int PK>
__global__ __launch_bounds__(kThreads) void muon_lone_kernel(StepArgs a, MuonArgs ma, int32_t steps, int32_t nesterov) {
    using T = Slab<SP>;
    __shared__ __align__(1024) char lds[T::kXBytes + T::kABytes];
    __shared__ Scalars sc;
    __shared__ double red[kThreads / 64];
    const uint32_t xs = lds_at(lds), as = xs + T::kXBytes;
    const MuonMat M = ma.mats[ma.mat0 + blockIdx.x];
    const Shape h = slab_shape<SP>(M, 0);
    step_begin(a, sc);
    const StepCommit commit{a, sc};
    if (sc.skip) return;
    const TensorDesc D = uniform_desc(a.tensors[M.tensor]);
    const float mu = uniform(sc.b1), s = uniform(sc.inv_scale);
    const int32_t n = h.len * h.side;
    float u[T::kPerLane];
    double acc = 0.0;
#pragma unroll
    for (int k0 = 0; k0 < T::kPerLane; k0 += 8) {
        float g[8][1], m[8][1];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int32_t at = (k0 + k) * kThreads + threadIdx.x;
            int32_t row, c;
            g[k][0] = m[k][0] = 0.0f;
            if (at < n) {
                const int64_t e = slab_element(h, at, row, c);
                load_g<GK, 1>(D.g, e, s, g[k]);
                ldf<1>(D.m, e, m[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int32_t at = (k0 + k) * kThreads + threadIdx.x;
            float x[1];
            m[k][0] = mu * m[k][0] + g[k][0];
            muon_u<1>(g[k], m[k], mu, nesterov, x);
            u[k0 + k] = x[0];
            acc = __builtin_fma((double)x[0], (double)x[0], acc);
            if (at < n) {
                int32_t row, c;
                stf<1>(D.m, slab_element(h, at, row, c), m[k]);
            }
        }
    }
    slab_zero(xs);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) acc += __shfl_xor(acc, o);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = acc;
    __syncthreads();
    const double f = muon_factor((red[0] + red[1]) + (red[2] + red[3]), a.prep.eps);
#pragma unroll
    for (int k = 0; k < T::kPerLane; ++k) {
        const int32_t at = k * kThreads + threadIdx.x;
        int32_t row, c;
        if (at < n) {
            slab_element(h, at, row, c);
            slab_put1<SP>(xs, row, c, (float)((double)u[k] * f));
        }
    }
    const Update<PK> update(a, ma, M, h, sc);
    for (int32_t i = 0; i < steps; ++i) {
        __syncthreads();
        Square<SP> A;
        slab_gram<SP>(xs, h.len, A);
        slab_polynomial<SP>(ma, as, A, h.side);
        if (i + 1 < steps)
            slab_apply<SP>(ma, xs, as, h.side, h.len,
                           [&](int row, int c, const float(&y)[4]) { slab_put4(xs, T::kLong, row, c, y); });
        else
            slab_apply<SP>(ma, xs, as, h.side, h.len, update);
    }
}

// ---------------------------------------------------------------- several slabs
// X of a slab in the workspace: its LDS image.
__device__ __forceinline__ char *slab_image(const MuonArgs &ma, const MuonMat &M, int32_t slab) {
    return ma.ws + M.x[0] + (int64_t)slab * (kMuonSlab * 4);
}
__device__ __forceinline__ void slab_save(char *image, uint32_t xs) {
#pragma unroll 4
    for (int k = threadIdx.x; k < kMuonSlab / 4; k += kThreads)
        ((GMEM u32x4 *)gp(image))[k] = *lds_ptr<const u32x4>(xs + k * 16);
}
template <int SP>
__device__ __forceinline__ float *slab_part(const MuonArgs &ma, const MuonMat &M, int32_t set, int32_t slab) {
    return reinterpret_cast<float *>(ma.ws + (set ? M.b : M.a)) + (int64_t)slab * SP * SP;
}
template <int SP>
__device__ __forceinline__ void slab_save_part(float *part, const Square<SP> &s) {
#pragma unroll
    for (int r = 0; r < Slab<SP>::kRowFrags; ++r)
#pragma unroll
        for (int i = 0; i < Slab<SP>::kColFrags; ++i)
            *(GMEM f32x4 *)gp(part + square_row<SP>(r) * SP + square_col(i)) = s.v[r][i];
}

// X0 of a slab and its part of A.
template <int SP, int GK>
__global__ __launch_bounds__(kThreads) void muon_slab_first_kernel(StepArgs a, MuonArgs ma, int32_t nesterov) {
    using T = Slab<SP>;
    __shared__ __align__(1024) char lds[T::kXBytes];
    if (skipped(a)) return;
    const uint32_t xs = lds_at(lds);
    const MuonTile t = ma.full[blockIdx.x];
    const MuonMat M = ma.mats[t.mat];
    const Shape h = slab_shape<SP>(M, t.i);
    const TensorDesc D = uniform_desc(a.tensors[M.tensor]);
    const float mu = (float)a.prep.beta1, s = a.prep.inv_scale ? *a.prep.inv_scale : 1.0f;
    const double f = reinterpret_cast<const double *>(a.blockfac)[t.mat];
    const int32_t n = h.len * h.side;
    slab_zero(xs);
    __syncthreads();
    for (int32_t k0 = 0; k0 < n; k0 += 8 * kThreads) {
        float g[8][1], m[8][1];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int32_t at = k0 + k * kThreads + threadIdx.x;
            int32_t row, c;
            if (at < n) {
                const int64_t e = slab_element(h, at, row, c);
                load_g<GK, 1>(D.g, e, s, g[k]);
                ldf<1>(D.m, e, m[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int32_t at = k0 + k * kThreads + threadIdx.x;
            int32_t row, c;
            if (at < n) {
                float x[1];
                muon_u<1>(g[k], m[k], mu, nesterov, x);
                slab_element(h, at, row, c);
                slab_put1<SP>(xs, row, c, (float)((double)x[0] * f));
            }
        }
    }
    __syncthreads();
    slab_save(slab_image(ma, M, t.i), xs);
    Square<SP> A;
    slab_gram<SP>(xs, h.len, A);
    slab_save_part<SP>(slab_part<SP>(ma, M, 0, t.i), A);
}

// One iteration: X and the parts of A (set `set`) in, X and its part of the
// next A (the other set) out, or the update (PK >= 0).
template <int SP, int PK>
__global__ __launch_bounds__(kThreads) void muon_slab_kernel(StepArgs a, MuonArgs ma, int32_t set) {
    using T = Slab<SP>;
    __shared__ __align__(1024) char lds[T::kXBytes + T::kABytes];
    const uint32_t xs = lds_at(lds), as = xs + T::kXBytes;
    const MuonTile t = ma.full[blockIdx.x];
    const MuonMat M = ma.mats[t.mat];
    const Shape h = slab_shape<SP>(M, t.i);
    auto work = [&](auto &&update) {
        char *image = slab_image(ma, M, t.i);
        u32x4 x[kMuonSlab / 4 / kThreads];
#pragma unroll
        for (int k = 0; k < kMuonSlab / 4 / kThreads; ++k) x[k] = ((const GMEM u32x4 *)gp(image))[k * kThreads + threadIdx.x];
        Square<SP> A{};
        const float *part = slab_part<SP>(ma, M, set, 0);
#pragma unroll 2
        for (int32_t k = 0; k < M.slabs; ++k, part += SP * SP)
#pragma unroll
            for (int r = 0; r < T::kRowFrags; ++r)
#pragma unroll
                for (int i = 0; i < T::kColFrags; ++i)
                    A.v[r][i] = A.v[r][i] + *(const GMEM f32x4 *)gp(part + square_row<SP>(r) * SP + square_col(i));
#pragma unroll
        for (int k = 0; k < kMuonSlab / 4 / kThreads; ++k) *lds_ptr<u32x4>(xs + (k * kThreads + threadIdx.x) * 16) = x[k];
        slab_polynomial<SP>(ma, as, A, h.side);
        if constexpr (PK >= 0) {
            slab_apply<SP>(ma, xs, as, h.side, h.len, update);
        } else {
            slab_apply<SP>(ma, xs, as, h.side, h.len,
                           [&](int row, int c, const float(&y)[4]) { slab_put4(xs, T::kLong, row, c, y); });
            __syncthreads();
            slab_save(image, xs);
            slab_gram<SP>(xs, h.len, A);
            slab_save_part<SP>(slab_part<SP>(ma, M, set ^ 1, t.i), A);
        }
    };
    if constexpr (PK >= 0) {
        __shared__ Scalars sc;
        step_begin(a, sc);
        const StepCommit commit{a, sc};
        if (sc.skip) return;
        work(Update<PK>(a, ma, M, h, sc));
    } else {
        if (skipped(a)) return;
        work(0);
    }
}

template <int SP, int PK>
void launch_slab(const StepArgs &a, const MuonArgs &ma, int64_t n, int32_t set, hipStream_t s) {
    LAUNCH_TRACED((muon_slab_kernel<SP, PK>), (unsigned)n, kThreads, s, a, ma, set);
}

template <int SP>
void launch_slabs_of(const StepArgs &args, const MuonArgs &ma, int64_t n, int pk, int gk, int32_t steps,
                     int32_t nesterov, bool commit, hipStream_t s) {
    if (n == 0) return;
    StepArgs a = args;
    a.commit = 0;
    if (gk == G_F32)
        LAUNCH_TRACED((muon_slab_first_kernel<SP, G_F32>), (unsigned)n, kThreads, s, a, ma, nesterov);
    else
        LAUNCH_TRACED((muon_slab_first_kernel<SP, G_BF16>), (unsigned)n, kThreads, s, a, ma, nesterov);
    for (int32_t i = 0; i + 1 < steps; ++i) launch_slab<SP, -1>(a, ma, n, i & 1, s);
    a.commit = commit;
    const int32_t set = (steps - 1) & 1;
    if (pk == P_F32) launch_slab<SP, P_F32>(a, ma, n, set, s);
    else if (pk == P_BF16R) launch_slab<SP, P_BF16R>(a, ma, n, set, s);
    else if (pk == P_MBF16) launch_slab<SP, P_MBF16>(a, ma, n, set, s);
    else launch_slab<SP, P_MF16>(a, ma, n, set, s);
}

template <int SP, int GK>
void launch_lone_g(const StepArgs &a, const MuonArgs &ma, int64_t n, int pk, int32_t steps, int32_t nesterov,
                   hipStream_t s) {
    if (pk == P_F32)
        LAUNCH_TRACED((muon_lone_kernel<SP, GK, P_F32>), (unsigned)n, kThreads, s, a, ma, steps, nesterov);
    else if (pk == P_BF16R)
        LAUNCH_TRACED((muon_lone_kernel<SP, GK, P_BF16R>), (unsigned)n, kThreads, s, a, ma, steps, nesterov);
    else if (pk == P_MBF16)
        LAUNCH_TRACED((muon_lone_kernel<SP, GK, P_MBF16>), (unsigned)n, kThreads, s, a, ma, steps, nesterov);
    else
        LAUNCH_TRACED((muon_lone_kernel<SP, GK, P_MF16>), (unsigned)n, kThreads, s, a, ma, steps, nesterov);
}
template <int SP>
void launch_lone_of(const StepArgs &args, const MuonArgs &margs, int32_t mat0, int64_t n, bool commit, int pk, int gk,
                    int32_t steps, int32_t nesterov, hipStream_t s) {
    if (n == 0) return;
    StepArgs a = args;
    a.commit = commit;
    MuonArgs ma = margs;
    ma.mat0 = mat0;
    if (gk == G_F32) launch_lone_g<SP, G_F32>(a, ma, n, pk, steps, nesterov, s);
    else launch_lone_g<SP, G_BF16>(a, ma, n, pk, steps, nesterov, s);
}

}  // namespace

hipError_t launch_muon_slabs(const StepArgs &a, const MuonArgs &args, const MuonRun &R, int pk, int gk, int32_t steps,
                             int32_t nesterov, bool commit, hipStream_t s) {
    MuonArgs ma = args;
    ma.full += R.full0;
    const int64_t rest = R.slabs - R.narrow;
    launch_slabs_of<64>(a, ma, R.narrow, pk, gk, steps, nesterov, commit && rest == 0, s);
    ma.full += R.narrow;
    launch_slabs_of<128>(a, ma, rest, pk, gk, steps, nesterov, commit, s);
    return hipGetLastError();
}

hipError_t launch_muon_lone(const StepArgs &a, const MuonArgs &ma, int pk, int gk, int32_t steps, int32_t nesterov,
                            hipStream_t s) {
    const int32_t n = ma.nmats - ma.lone0, rest = n - ma.lone_narrow;
    launch_lone_of<64>(a, ma, ma.lone0, ma.lone_narrow, rest == 0, pk, gk, steps, nesterov, s);
    launch_lone_of<128>(a, ma, ma.lone0 + ma.lone_narrow, rest, true, pk, gk, steps, nesterov, s);
    return hipGetLastError();
}

}  // namespace optim
