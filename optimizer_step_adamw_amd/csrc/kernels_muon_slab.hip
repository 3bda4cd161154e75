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
// What bounds it is latency: an iteration is a chain of LDS reads, products and
// barriers, 5 us for SP 64 and 12 us for SP 128, whatever the number of
// matrices up to one per compute unit.  Measured on MI355X, the whole step of
// five iterations: one 64 x 64 37 us, 14 of 64 x 172 54 us, 500 of 64 x 64
// 80 us, one 128 x 128 91 us (by tiles and launches per product 190 us and
// more); in several slabs 20 of 3591 x 21 151 us (by tiles 542), one
// 128 x 1024 151 us, one of 128 slabs (1 x 16384 x 128) 228 us (1353).
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

// X <- a X + X B in place: a wavefront's rows depend on its own rows alone.
template <int SP>
__device__ __forceinline__ void slab_apply(const MuonArgs &ma, uint32_t xs, uint32_t as, int side, int len) {
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
            slab_put4(xs, T::kLong, row, square_col(i), y);
        }
    }
}

// A matrix's shape as its slabs see it.  In memory the slab is `outer` runs of
// `inner` elements, `cols` apart: a position's values (tall) or a value's
// positions (wide).
struct Shape {
    int64_t e0;     // element of the slab's first position, first value
    int32_t cols;   // elements between the matrix's rows
    int32_t side;   // the short side
    int32_t len;    // positions of this slab
    int32_t tall;
    int32_t inner, outer;
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
    h.inner = M.tall ? h.side : h.len;
    h.outer = M.tall ? h.len : h.side;
    return h;
}
// A lane's way through the slab in memory order, V neighbouring elements at a
// time, every kThreads-th such group: one division at the start (two an element
// took more time than the memory).
template <int V>
struct Walk {
    int32_t o, i;        // run, place in it
    int32_t step_o, step_i, inner, outer, tall, cols;
    int64_t e;
    __device__ __forceinline__ explicit Walk(const Shape &h)
        : inner(h.inner), outer(h.outer), tall(h.tall), cols(h.cols) {
        const int32_t k = (int32_t)threadIdx.x * V;
        o = k / inner;
        i = k - o * inner;
        step_o = kThreads * V / inner;
        step_i = kThreads * V - step_o * inner;
        e = h.e0 + (int64_t)o * cols + i;
    }
    __device__ __forceinline__ bool there() const { return o < outer; }
    __device__ __forceinline__ void next() {
        o += step_o;
        i += step_i;
        e += (int64_t)step_o * cols + step_i;
        if (i >= inner) {
            i -= inner;
            ++o;
            e += cols - inner;
        }
    }
    __device__ __forceinline__ int32_t row(int k) const { return tall ? o : i + k; }  // position of element k of V
    __device__ __forceinline__ int32_t value(int k) const { return tall ? i + k : o; }
};
// Groups of elements that a lane has under way: a batch is a memory latency.
constexpr int kSlabBatch = 8;
// Whether the slab's runs are whole aligned groups of 4.
__device__ __forceinline__ bool slab_vec(const TensorDesc &D, const Shape &h) {
    return D.vec_ok && ((h.inner | h.cols) & 3) == 0 && (h.e0 & 3) == 0;
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

// Calls body(walk, gradients, momenta) for a lane's groups of V.
template <int GK, int V, class F>
__device__ __forceinline__ void slab_walk(const TensorDesc &D, const Shape &h, float s, F &&body) {
    Walk<V> w(h);
    while (w.there()) {
        float g[kSlabBatch][V], m[kSlabBatch][V];
        Walk<V> ahead = w;
#pragma unroll
        for (int k = 0; k < kSlabBatch; ++k) {
            if (ahead.there()) {
                load_g<GK, V>(D.g, ahead.e, s, g[k]);
                ldf<V>(D.m, ahead.e, m[k]);
            }
            ahead.next();
        }
#pragma unroll
        for (int k = 0; k < kSlabBatch; ++k) {
            if (w.there()) body(w, g[k], m[k]);
            w.next();
        }
    }
}

// m <- mu m + g; this lane's sum of u^2.
template <int GK, int V>
__device__ __forceinline__ double slab_momentum(const TensorDesc &D, const Shape &h, float s, float mu, int32_t nesterov) {
    double acc = 0.0;
    slab_walk<GK, V>(D, h, s, [&](const Walk<V> &w, const float(&g)[V], float(&m)[V]) {
        float x[V];
#pragma unroll
        for (int i = 0; i < V; ++i) m[i] = mu * m[i] + g[i];
        muon_u<V>(g, m, mu, nesterov, x);
#pragma unroll
        for (int i = 0; i < V; ++i) acc = __builtin_fma((double)x[i], (double)x[i], acc);
        stf<V>(D.m, w.e, m);
    });
    return acc;
}
// X0 from the new momentum, into zeroed LDS.
template <int SP, int GK, int V>
__device__ __forceinline__ void slab_fill(uint32_t xs, const TensorDesc &D, const Shape &h, float s, float mu,
                                          int32_t nesterov, double f) {
    slab_walk<GK, V>(D, h, s, [&](const Walk<V> &w, const float(&g)[V], float(&m)[V]) {
        float x[V];
        muon_u<V>(g, m, mu, nesterov, x);
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = (float)((double)x[i] * f);
        if constexpr (V == 4) {
            if (w.tall) {
                slab_put4(xs, Slab<SP>::kLong, w.o, w.i, x);
                return;
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) slab_put1<SP>(xs, w.row(i), w.value(i), x[i]);
    });
}

// The update, from the last X in LDS, in memory order and a batch at a time
// (straight from the sums, a position's values would lie a row apart in a wide
// matrix, and each load would wait for the store before it).
template <int SP, int PK, int V>
__device__ __forceinline__ void slab_update(const TensorDesc &D, const Shape &h, uint32_t xs, float lw, float f) {
    Walk<V> w(h);
    while (w.there()) {
        float p[kSlabBatch][V];
        Walk<V> ahead = w;
#pragma unroll
        for (int k = 0; k < kSlabBatch; ++k) {
            if (ahead.there()) load_p<PK, V>(D, ahead.e, p[k]);
            ahead.next();
        }
#pragma unroll
        for (int k = 0; k < kSlabBatch; ++k) {
            if (w.there()) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int32_t r = w.row(i), c = w.value(i);
                    const float hi = (float)*lds_ptr<const _Float16>(xs + slab_chunk(Slab<SP>::kLong, r, c, 0) + (c & 7) * 2);
                    const float lo = (float)*lds_ptr<const _Float16>(xs + slab_chunk(Slab<SP>::kLong, r, c, 1) + (c & 7) * 2);
                    p[k][i] = decayed(p[k][i], lw, f * ((hi + lo) * kMuonUnscale));
                }
                store_p<PK, V>(D, w.e, p[k]);
            }
            w.next();
        }
    }
}
template <int SP, int PK>
__device__ __forceinline__ void slab_update(const StepArgs &a, const MuonArgs &ma, const MuonMat &M, const Shape &h,
                                            const Scalars &sc, uint32_t xs) {
    const TensorDesc D = uniform_desc(a.tensors[M.tensor]);
    const float f = (float)(sc.lr64 * muon_scale(ma.scale_kind, M.rows, M.cols)), lw = sc.lrwd[D.group];
    if (slab_vec(D, h)) slab_update<SP, PK, 4>(D, h, xs, lw, f);
    else slab_update<SP, PK, 1>(D, h, xs, lw, f);
}

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
    slab_zero(xs);
    const bool vec = slab_vec(D, h);
    double acc = vec ? slab_momentum<GK, 4>(D, h, s, mu, nesterov) : slab_momentum<GK, 1>(D, h, s, mu, nesterov);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) acc += __shfl_xor(acc, o);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = acc;
    __syncthreads();
    const double f = muon_factor((red[0] + red[1]) + (red[2] + red[3]), a.prep.eps);
    if (vec) slab_fill<SP, GK, 4>(xs, D, h, s, mu, nesterov, f);
    else slab_fill<SP, GK, 1>(xs, D, h, s, mu, nesterov, f);
    for (int32_t i = 0; i < steps; ++i) {
        __syncthreads();
        Square<SP> A;
        slab_gram<SP>(xs, h.len, A);
        slab_polynomial<SP>(ma, as, A, h.side);
        slab_apply<SP>(ma, xs, as, h.side, h.len);
    }
    __syncthreads();
    slab_update<SP, PK>(a, ma, M, h, sc, xs);
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
    slab_zero(xs);
    __syncthreads();
    if (slab_vec(D, h)) slab_fill<SP, GK, 4>(xs, D, h, s, mu, nesterov, f);
    else slab_fill<SP, GK, 1>(xs, D, h, s, mu, nesterov, f);
    __syncthreads();
    slab_save(slab_image(ma, M, t.i), xs);
    Square<SP> A;
    slab_gram<SP>(xs, h.len, A);
    slab_save_part<SP>(slab_part<SP>(ma, M, 0, t.i), A);
}

// Matrices with more slabs than this have their parts of A summed by a launch of
// their own, into the first part; else every slab sums them itself.  Measured,
// by itself and by a launch: one 128 x 256 (2 slabs) 146 and 162 us, 128 x 512
// (4) 181 and 164, 128 x 1024 (8) 251 and 151; one 64 x 1024 (4) 99 and 109,
// 64 x 2048 (8) 109 and 108.
template <int SP>
constexpr int32_t kSlabJoin = SP == 64 ? 8 : 3;

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
    auto work = [&](auto &&end) {
        char *image = slab_image(ma, M, t.i);
        u32x4 x[kMuonSlab / 4 / kThreads];
#pragma unroll
        for (int k = 0; k < kMuonSlab / 4 / kThreads; ++k) x[k] = ((const GMEM u32x4 *)gp(image))[k * kThreads + threadIdx.x];
        Square<SP> A{};
        const float *part = slab_part<SP>(ma, M, set, 0);
        const int32_t parts = M.slabs > kSlabJoin<SP> ? 1 : M.slabs;
#pragma unroll 2
        for (int32_t k = 0; k < parts; ++k, part += SP * SP)
#pragma unroll
            for (int r = 0; r < T::kRowFrags; ++r)
#pragma unroll
                for (int i = 0; i < T::kColFrags; ++i)
                    A.v[r][i] = A.v[r][i] + *(const GMEM f32x4 *)gp(part + square_row<SP>(r) * SP + square_col(i));
#pragma unroll
        for (int k = 0; k < kMuonSlab / 4 / kThreads; ++k) *lds_ptr<u32x4>(xs + (k * kThreads + threadIdx.x) * 16) = x[k];
        slab_polynomial<SP>(ma, as, A, h.side);
        slab_apply<SP>(ma, xs, as, h.side, h.len);
        __syncthreads();
        end(image, A);
    };
    if constexpr (PK >= 0) {
        __shared__ Scalars sc;
        step_begin(a, sc);
        const StepCommit commit{a, sc};
        if (sc.skip) return;
        work([&](char *, Square<SP> &) { slab_update<SP, PK>(a, ma, M, h, sc, xs); });
    } else {
        if (skipped(a)) return;
        work([&](char *image, Square<SP> &A) {
            slab_save(image, xs);
            slab_gram<SP>(xs, h.len, A);
            slab_save_part<SP>(slab_part<SP>(ma, M, set ^ 1, t.i), A);
        });
    }
}

// The parts of A of the matrices of many slabs: 4 elements a lane, in the
// parts' order, one workgroup for each slab of the table.
template <int SP>
__global__ __launch_bounds__(kThreads) void muon_slab_join_kernel(StepArgs a, MuonArgs ma, int32_t set) {
    if (skipped(a)) return;
    const MuonTile t = ma.full[blockIdx.x];
    const MuonMat M = ma.mats[t.mat];
    if (M.slabs <= kSlabJoin<SP>) return;
    for (int32_t q = t.i * kThreads + threadIdx.x; q < SP * SP / 4; q += M.slabs * kThreads) {
        float *part = slab_part<SP>(ma, M, set, 0) + q * 4;
        f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
        int32_t k = 0;
        for (; k + 8 <= M.slabs; k += 8) {
            f32x4 y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = *(const GMEM f32x4 *)gp(part + (int64_t)(k + i) * SP * SP);
#pragma unroll
            for (int i = 0; i < 8; ++i) x = x + y[i];
        }
        for (; k < M.slabs; ++k) x = x + *(const GMEM f32x4 *)gp(part + (int64_t)k * SP * SP);
        *(GMEM f32x4 *)gp(part) = x;
    }
}

template <int SP, int PK>
void launch_slab(const StepArgs &a, const MuonArgs &ma, int64_t n, int32_t set, hipStream_t s) {
    LAUNCH_TRACED((muon_slab_kernel<SP, PK>), (unsigned)n, kThreads, s, a, ma, set);
}

template <int SP>
void launch_slabs_of(const StepArgs &args, const MuonArgs &ma, int64_t n, bool many, int pk, int gk, int32_t steps,
                     int32_t nesterov, bool commit, hipStream_t s) {
    if (n == 0) return;
    StepArgs a = args;
    a.commit = 0;
    if (gk == G_F32)
        LAUNCH_TRACED((muon_slab_first_kernel<SP, G_F32>), (unsigned)n, kThreads, s, a, ma, nesterov);
    else
        LAUNCH_TRACED((muon_slab_first_kernel<SP, G_BF16>), (unsigned)n, kThreads, s, a, ma, nesterov);
    auto join = [&](int32_t set) {
        if (many) LAUNCH_TRACED(muon_slab_join_kernel<SP>, (unsigned)n, kThreads, s, a, ma, set);
    };
    for (int32_t i = 0; i + 1 < steps; ++i) {
        join(i & 1);
        launch_slab<SP, -1>(a, ma, n, i & 1, s);
    }
    const int32_t set = (steps - 1) & 1;
    join(set);
    a.commit = commit;
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
    launch_slabs_of<64>(a, ma, R.narrow, R.most_slabs > kSlabJoin<64>, pk, gk, steps, nesterov, commit && rest == 0, s);
    ma.full += R.narrow;
    launch_slabs_of<128>(a, ma, rest, R.most_slabs > kSlabJoin<128>, pk, gk, steps, nesterov, commit, s);
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
