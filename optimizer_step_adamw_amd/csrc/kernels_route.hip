// kernels_route.hip -- routing of tokens to experts and its gradient
// (optim_route, optim_route_grad).
//
// The choice is defined on fp64 scores, and only few tokens need them: most are
// chosen on whole numbers made in fp32, sixteen lanes a token, with a bound on what
// that may have moved; the others again by a wavefront in fp64 (route_token).
// Many tokens of few experts are taken by a lane each.  A choice without scores is
// one of logits, exact in either.
//
// Bound by the VALU at 256 experts: four tokens cost a wavefront some 880
// instructions, 24 us of issue for 65536 tokens.  By the assembly, with groups and a
// bias: loads and their checks 50, sigmoids 64, bias 32, the row's range 60, keys 80,
// sorting a lane's 115, groups 160, joining the lanes' lists 130, a lane's own choice
// out of them 105 (the compiler makes comparisons with every index of it), neighbours
// 60, weights 30.  Measured on MI355X, 8 choices of 65536 tokens, us: fp32, sigmoid,
// bias, 4 of 8 groups, 256 experts 33 (71 MB), 512 56, 1024 210-218, 240 experts in
// 12 groups 76-80; softmax without bias, 32 experts 16, 64 14-15, 128 17, 255 37,
// 256 21, 512 35-36, 1024 146, bf16 64 13-14 and 256 20; 16384 x 64 bf16 5.1-6.0, one
// token of 256 3.7-4.1; by wavefronts in fp64 (more than 16 groups, more than 16
// choices) 32768 x 512, 17 choices, 105.  The gradient reads and writes: of the whole
// softmax, 65536 x 256 bf16, 17-18 us (71 MB, 4.2 TB/s, partly from the Infinity
// Cache), 65536 x 1024 fp32 119 (4.5); renormalised sigmoids 65536 x 256 fp32 19.4
// (3.8), x 1024 76 (3.6, the row passes through 64 KB of LDS a workgroup).
#include "elems.h"

#include <cfloat>
#include <type_traits>

namespace optim {
namespace {

constexpr int kWaves = kThreads / 64;
constexpr double kNone = -__builtin_inf();

// What the wavefront's lanes wrote to LDS is there for all of them.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <int DT>
__device__ __forceinline__ float logit_at(const char *row, int32_t e) {
    return element<DT>(row + (int64_t)e * kElem<DT>);
}
// +inf as the largest float, NaN as -inf
__device__ __forceinline__ float tamed(float l) { return l != l ? -INFINITY : (l > FLT_MAX ? FLT_MAX : l); }

__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

__device__ __forceinline__ float wave_max(float x) {
    for (int m = 32; m; m /= 2) x = fmaxf(x, __shfl_xor(x, m));
    return x;
}
__device__ __forceinline__ float wave_sum(float x) {
    for (int m = 32; m; m /= 2) x += __shfl_xor(x, m);
    return x;
}

// (the runtime's own shuffles of doubles go through scratch memory)
template <class F>
__device__ __forceinline__ double halves(double x, F &&f) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)f((int)(uint32_t)u), hi = (uint32_t)f((int)(uint32_t)(u >> 32));
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Within rows of 16 lanes, values pass between lanes without LDS (DPP).  Each of
// these pairs a lane with one of the other half of its 2, 4, 8 or 16.
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140, kBroadcast = 0x150, kNext = 0x101;
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, true);
}
// The larger key and, of equal ones, the lower expert.
__device__ __forceinline__ void better(double k2, int32_t e2, double &k, int32_t &e) {
    const bool it = (k2 > k) | ((k2 == k) & (e2 < e));
    k = it ? k2 : k;
    e = it ? e2 : e;
}
template <int CTRL>
__device__ __forceinline__ void better_lane(double &k, int32_t &e) {
    better(halves(k, [](int x) { return (int)dpp<CTRL>((uint32_t)x); }), (int32_t)dpp<CTRL>((uint32_t)e), k, e);
}
// The best one of the wavefront.
__device__ __forceinline__ void wave_best(double &k, int32_t &e) {
    better_lane<kXor1>(k, e);
    better_lane<kXor2>(k, e);
    better_lane<kMirror8>(k, e);
    better_lane<kMirror16>(k, e);
#pragma unroll
    for (int m = 16; m < 64; m *= 2) better(halves(k, [&](int x) { return __shfl_xor(x, m); }), __shfl_xor(e, m), k, e);
}

// The two largest keys of a group, b0 >= b1.
__device__ __forceinline__ void keep_two(double k, double &b0, double &b1) {
    b1 = fmax(b1, fmin(b0, k));
    b0 = fmax(b0, k);
}

// Lane j (below topk) returns choice j, or -1.  V: experts of a lane, lane l holds
// experts l, l + 64, ...
template <int V, int DT>
__device__ __forceinline__ int32_t choose(const RouteArgs &a, const char *row, double *lds, int lane) {
    double k[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int32_t e = lane + 64 * v;
        k[v] = e < a.experts ? (double)tamed(logit_at<DT>(row, e)) : kNone;
    }
    const bool sums = a.groups > 1 && a.group_best > 1;
    if (a.bias || sums) {
        double most = 0.0, total = 1.0;
        if (a.score == OPTIM_ROUTE_SOFTMAX) {
            float m = -INFINITY;
#pragma unroll
            for (int v = 0; v < V; ++v) m = fmaxf(m, (float)k[v]);
            most = (double)wave_max(m);
            total = 0.0;
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (k[v] > kNone) total += exp(k[v] - most);
            for (int m = 32; m; m /= 2) total += halves(total, [&](int x) { return __shfl_xor(x, m); });
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int32_t e = lane + 64 * v;
            if (!(k[v] > kNone)) continue;
            const double s = a.score == OPTIM_ROUTE_SOFTMAX ? exp(k[v] - most) / total : 1.0 / (1.0 + exp(-k[v]));
            const double b = a.bias ? (double)a.bias[e] : 0.0;
            k[v] = b > kNone ? s + b : kNone;
        }
    }
    if (a.groups > 1) {
        const int32_t per = a.experts / a.groups;
#pragma unroll
        for (int v = 0; v < V; ++v) lds[lane + 64 * v] = k[v];
        wave_sync();
        // `width` lanes a group, a power of two
        const int32_t width = 64 >> (a.groups > 1 ? 32 - __builtin_clz(a.groups - 1) : 0), mine = lane / width;
        double b0 = kNone, b1 = kNone;
        if (mine < a.groups)
            for (int32_t i = lane & (width - 1); i < per; i += width) keep_two(lds[mine * per + i], b0, b1);
        for (int m = 1; m < width; m *= 2) {
            const double o0 = halves(b0, [&](int x) { return __shfl_xor(x, m); });
            const double o1 = halves(b1, [&](int x) { return __shfl_xor(x, m); });
            b1 = fmax(fmin(b0, o0), fmax(b1, o1));
            b0 = fmax(b0, o0);
        }
        const double rank = a.group_best > 1 && b1 > kNone ? b0 + b1 : b0;
        int32_t ahead = 0;
        for (int32_t g = 0; g < a.groups; ++g) {
            const double r = halves(rank, [&](int x) { return __shfl(x, g * width); });
            ahead += (r > rank) | ((r == rank) & (g < mine)) ? 1 : 0;
        }
        const uint64_t kept = __ballot(mine < a.groups && ahead < a.top_groups);  // in all of a group's lanes
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int32_t e = lane + 64 * v;
            if (e < a.experts && !(kept >> (e / per * width) & 1)) k[v] = kNone;
        }
    }
    int32_t mine = -1;
    for (int32_t j = 0; j < a.topk; ++j) {
        double best = kNone;
        int32_t at = INT32_MAX;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (k[v] > best) {
                best = k[v];
                at = lane + 64 * v;
            }
        wave_best(best, at);
        if (!(best > kNone)) break;
        if (lane == j) mine = at;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (at == lane + 64 * v) k[v] = kNone;
    }
    return mine;
}

// Scores of the chosen experts among themselves: lane j's score over the sum of
// the token's, or the score itself.  mine: the lane's logit, -inf beside none;
// most: the largest of them.  Where that is not above 0 sigmoids are taken relative
// to its own, so that they do not vanish: s_j / s_max = e^(l_j - m) (1 + e^m) / (1 + e^l_j).
__device__ __forceinline__ float part_of_score(int32_t score, float mine, float most) {
    if (!(mine > -INFINITY)) return 0.0f;
    if (score == OPTIM_ROUTE_SOFTMAX) return expf(mine - most);
    return most > 0.0f ? sigmoid(mine) : expf(mine - most) * (1.0f + expf(most)) / (1.0f + expf(mine));
}

// One token by a wavefront.
template <int V, int DT>
__device__ __forceinline__ void route_token(const RouteArgs &a, int64_t t, double *lds, int lane) {
    const char *row = a.logits + t * a.ldl;
    const int32_t e = choose<V, DT>(a, row, lds, lane);
    bool nan = false;
    float most = -INFINITY, total = 0.0f;
    float l[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int32_t x = lane + 64 * v;
        const float raw = x < a.experts ? logit_at<DT>(row, x) : -INFINITY;
        nan |= raw != raw;
        l[v] = tamed(raw);
    }
    nan = __any(nan);
    const float mine = e >= 0 ? tamed(logit_at<DT>(row, e)) : -INFINITY;
    float w = 0.0f;
    if (a.renormalise) {
        w = part_of_score(a.score, mine, wave_max(mine));
        total = wave_sum(w);
    } else if (a.score == OPTIM_ROUTE_SOFTMAX) {
#pragma unroll
        for (int v = 0; v < V; ++v) most = fmaxf(most, l[v]);
        most = wave_max(most);
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (l[v] > -INFINITY) total += expf(l[v] - most);
        total = wave_sum(total);
        w = e >= 0 ? expf(mine - most) : 0.0f;
    } else {
        w = e >= 0 ? sigmoid(mine) : 0.0f;
        total = 1.0f;
    }
    if (e >= 0) w = w / total;
    w *= a.scale;
    if (nan) w = __builtin_nanf("");
    if (lane < a.topk) {
        a.idx[t * a.topk + lane] = e;
        a.weights[t * a.topk + lane] = w;
    }
}

template <int V, int DT>
__global__ __launch_bounds__(kThreads) void route_wave_kernel(RouteArgs a) {
    __shared__ double lds[kWaves][64 * V];
    const int64_t t = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
    if (t < a.tokens) route_token<V, DT>(a, t, lds[threadIdx.x >> 6], threadIdx.x & 63);
}

// ---------------------------------------------------------------- four tokens a wavefront
template <int CTRL>
__device__ __forceinline__ float dpp(float x) { return __uint_as_float(dpp<CTRL>(__float_as_uint(x))); }
// The largest and smallest of numbers that are no NaN (fmaxf and fminf quiet
// each argument first).  The wait state is for an argument that a reciprocal or
// an exponential has just made, which the compiler sees to for its own
// instructions only.
__device__ __forceinline__ float most_of(float x, float y, float z) {
    float r;
    asm("s_nop 0\n\tv_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(x), "v"(y), "v"(z));
    return r;
}
__device__ __forceinline__ float least_of(float x, float y, float z) {
    float r;
    asm("s_nop 0\n\tv_min3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(x), "v"(y), "v"(z));
    return r;
}
__device__ __forceinline__ float more_of(float x, float y) {
    float r;
    asm("s_nop 0\n\tv_max_f32 %0, %1, %2" : "=v"(r) : "v"(x), "v"(y));
    return r;
}
__device__ __forceinline__ float less_of(float x, float y) {
    float r;
    asm("s_nop 0\n\tv_min_f32 %0, %1, %2" : "=v"(r) : "v"(x), "v"(y));
    return r;
}

template <class T, class F>
__device__ __forceinline__ T join16(T x, F &&f) {
    x = f(x, dpp<kXor1>(x));
    x = f(x, dpp<kXor2>(x));
    x = f(x, dpp<kMirror8>(x));
    return f(x, dpp<kMirror16>(x));
}
__device__ __forceinline__ float max16(float x) { return join16(x, [](float a, float b) { return more_of(a, b); }); }
__device__ __forceinline__ float min16(float x) { return join16(x, [](float a, float b) { return less_of(a, b); }); }
__device__ __forceinline__ float sum16(float x) { return join16(x, [](float a, float b) { return a + b; }); }

// f(number, value of that lane) for every by-th lane of the 16, by a power of two
template <int I = 0, class F>
__device__ __forceinline__ void each16(int32_t by, float x, F &&f) {
    if constexpr (I < 16) {
        if (!(I & (by - 1))) f(I, dpp<kBroadcast + I>(x));
        each16<I + 1>(by, x, f);
    }
}

// Sorting networks, the largest first.
__device__ __forceinline__ void order(uint32_t &a, uint32_t &b) {
    const uint32_t hi = a > b ? a : b, lo = a > b ? b : a;
    a = hi;
    b = lo;
}
template <int D>
__device__ __forceinline__ void bitonic(uint32_t (&a)[D]) {
#pragma unroll
    for (int s = D / 2; s; s /= 2)
#pragma unroll
        for (int i = 0; i < D; ++i)
            if (!(i & s)) order(a[i], a[i + s]);
}
template <int D>
__device__ __forceinline__ void sort(uint32_t (&a)[D]) {
    if constexpr (D == 8) {
        constexpr int net[19][2] = {{0, 1}, {2, 3}, {4, 5}, {6, 7}, {0, 2}, {1, 3}, {4, 6}, {5, 7}, {1, 2}, {5, 6},
                                    {0, 4}, {1, 5}, {2, 6}, {3, 7}, {2, 4}, {3, 5}, {1, 2}, {3, 4}, {5, 6}};
#pragma unroll
        for (int i = 0; i < 19; ++i) order(a[net[i][0]], a[net[i][1]]);
    } else {
        uint32_t lo[8], hi[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo[i] = a[i];
            hi[i] = a[8 + i];
        }
        sort<8>(lo);
        sort<8>(hi);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            a[i] = lo[i];
            a[8 + i] = hi[7 - i];
        }
        bitonic<16>(a);
    }
}
// The D largest of two sorted lists, sorted.
template <int D>
__device__ __forceinline__ void absorb(uint32_t (&a)[D], const uint32_t (&b)[D]) {
#pragma unroll
    for (int i = 0; i < D; ++i) a[i] = a[i] > b[D - 1 - i] ? a[i] : b[D - 1 - i];
    bitonic<D>(a);
}
template <int D, int CTRL>
__device__ __forceinline__ void absorb_lane(uint32_t (&a)[D]) {
    uint32_t b[D];
#pragma unroll
    for (int i = 0; i < D; ++i) b[i] = dpp<CTRL>(a[i]);
    absorb<D>(a, b);
}

// How a row lies in a token's 16 lanes: `lanes` of them, a power of two, have a
// group of `per` experts, n each but for the last ones.  (Groups are made up to a
// power of two by empty ones; per <= lanes * n, so that an expert's number and the
// V - 1 behind it stay below 16 V.)
struct Lay {
    int32_t lanes, per, n;
    bool quads;  // four neighbours are one access, all there or none
    bool full;   // every one of the V of every lane is there
};
struct Part {
    int32_t first, n;  // a lane's experts
};
__device__ __forceinline__ Part part_of(const RouteArgs &a, const Lay &lay, int l16) {
    const int32_t g = l16 / lay.lanes, at = (l16 & (lay.lanes - 1)) * lay.n, left = lay.per - at;
    if (g >= a.groups || left <= 0) return Part{0, 0};
    return Part{g * lay.per + at, left < lay.n ? left : lay.n};
}
template <int DT>
__device__ __forceinline__ void load4(const char *p, float *x) {
    if constexpr (DT == OPTIM_F32) {
        const u32x4 u = *(const GMEM u32x4_at4 *)gp(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(u[i]);
    } else {
        const u32x2 u = *(const GMEM u32x2_at2 *)gp(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == OPTIM_BF16) x[i] = __uint_as_float(i % 2 ? u[i / 2] & 0xFFFF0000u : u[i / 2] << 16);
            else x[i] = f16_to_f32(u[i / 2] >> (i % 2 * 16) & 0xFFFFu);
        }
    }
}
// Four of this lane's part of a row, from the q-th on; `none` where there is no
// expert.
template <int DT, bool FULL>
__device__ __forceinline__ void load_four(const char *row, Part part, bool quads, int q, float none, float *x) {
    if (FULL || quads) {
        const bool in = FULL || q < part.n;
        load4<DT>(row + (int64_t)(in ? part.first + q : 0) * kElem<DT>, x);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (!FULL) x[i] = in ? x[i] : none;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool in = q + i < part.n;
            x[i] = logit_at<DT>(row, in ? part.first + q + i : 0);
            x[i] = in ? x[i] : none;
        }
    }
}
template <int V, int DT, bool FULL>
__device__ __forceinline__ void load_row(const char *row, Part part, bool quads, float none, float (&x)[V]) {
#pragma unroll
    for (int q = 0; q < V; q += 4) load_four<DT, FULL>(row, part, quads, q, none, x + q);
}

// Whether a sum of the numbers is finite in every lane: then so are they.
template <int V>
__device__ __forceinline__ bool all_finite(const float (&x)[V]) {
    float s = x[0];
#pragma unroll
    for (int v = 1; v < V; ++v) s += x[v];
    return !__any(!(fabsf(s) < INFINITY));
}

// The whole part; 0 of what is negative, -inf or NaN (which the language leaves
// open, and the instruction does not).  x: an fma's result.
__device__ __forceinline__ uint32_t whole_part(float x) {
    uint32_t u;
    asm("v_cvt_u32_f32 %0, %1" : "=v"(u) : "v"(x));
    return u;
}

// x[at], at below N, from registers
template <int N>
__device__ __forceinline__ uint32_t pick(const uint32_t (&x)[N], int at) {
    uint32_t y[N];
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = x[i];
#pragma unroll
    for (int s = 1; s < N; s *= 2) {
        const bool odd = at & s;
#pragma unroll
        for (int i = 0; i < N; i += 2 * s) y[i] = odd ? y[i + s] : y[i];
    }
    return y[0];
}

// Sixteen lanes a token, V experts a lane, the D largest choices (topk <= D).
//
// The choices are ordered as whole numbers: the choice's place in the row's
// range in the upper bits (24 at most), the expert's number, turned round, in
// the lower ones, so that one maximum carries both.  Every lane sorts its own, and
// four steps join the lanes' lists until each holds the row's D largest.  Choices
// of 16-bit logits without scores are exact that way.  Others may have been
// moved: by less than a step where the choice is an fp32 logit, and by the
// rounding of scores, bias and sums otherwise.  Where two neighbours among the
// chosen and the one behind them are no further apart than that, or two groups
// at the border, the wavefront chooses again for that token in fp64.
//
// Error of a choice c = s + b, in units of 2^-24: a sigmoid 1 / (1 + 2^(-l log2 e))
// has s (1 - s) (1.22 |l| + 2) < 0.8 from the exponent and the exponential, 3 s from
// the sum and the reciprocal, below 4; a softmax has its terms' 2.3 |x| + 3, the sum's
// V + 4 roundings one after another (V <= 64) and the terms' mean 2.3 |x| + 3, and 3
// of itself, below V + 32 of the largest score, as e^-|x| (2.3 |x| + 3) <= 3 and the
// mean of |x| over 1024 terms e^-|x| with a 1 among them is below 4.5; the sum with b |c|.
template <int V, int D, int DT, bool FULL>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs a, Lay lay) {
    constexpr int V64 = V < 4 ? 1 : V / 4;
    constexpr int kBits = V == 4 ? 6 : V == 8 ? 7 : V == 16 ? 8 : V == 32 ? 9 : 10;  // of an expert's number
    constexpr uint32_t kNumber = (1u << kBits) - 1;
    constexpr float kSteps = (float)((1 << (kBits < 8 ? 24 : 32 - kBits)) - 8);
    constexpr float kLog2e = 1.44269504f;
    __shared__ double lds[kWaves][64 * V64];
    const int lane = threadIdx.x & 63, l16 = lane & 15, wave = threadIdx.x >> 6;
    const bool sums = a.groups > 1 && a.group_best > 1, scored = a.bias || sums;
    const bool whole = DT != OPTIM_F32 && !scored;  // exact keys
    const Part part = FULL ? Part{l16 * V, V} : part_of(a, lay, l16);
    const int64_t t0 = ((int64_t)blockIdx.x * kWaves + wave) * 4;
    if (t0 >= a.tokens) return;
    uint64_t redo;
    {
        const int64_t t = t0 + (lane >> 4);
        const bool live = t < a.tokens;
        const char *row = a.logits + (live ? t : t0) * a.ldl;
        float c[V], b[V];
        load_row<V, DT, FULL>(row, part, lay.quads, -INFINITY, c);
        if (a.bias) load_row<V, OPTIM_F32, FULL>(reinterpret_cast<const char *>(a.bias), part, lay.quads, -INFINITY, b);
        // (in every lane) some expert may not be available
        bool masked = !FULL || !all_finite(c), nan = false;
        if (masked) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                nan |= c[v] != c[v];
                c[v] = tamed(c[v]);
            }
        }
        // ---- scores, where they count
        const bool soft = a.score == OPTIM_ROUTE_SOFTMAX;
        float most = -INFINITY, total = 1.0f, error = 0.0f;
        if (soft && (scored || !a.renormalise)) {
#pragma unroll
            for (int v = 0; v < V; v += 2) most = most_of(most, c[v], c[v + 1]);
            most = max16(most);
            total = 0.0f;
            const float from = most > -INFINITY ? most : 0.0f;
            if (!scored) {
#pragma unroll
                for (int v = 0; v < V; ++v) total += __builtin_amdgcn_exp2f((c[v] - from) * kLog2e);
                total = sum16(total);
            } else {
                float s[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    s[v] = __builtin_amdgcn_exp2f((c[v] - from) * kLog2e);
                    total += s[v];
                }
                total = sum16(total);
                const float inv = total > 0.0f ? __builtin_amdgcn_rcpf(total) : 0.0f;
                error = (float)(V + 32) * inv;
                if (masked) {
#pragma unroll
                    for (int v = 0; v < V; ++v) c[v] = c[v] > -INFINITY ? s[v] * inv : -INFINITY;
                } else {
#pragma unroll
                    for (int v = 0; v < V; ++v) c[v] = s[v] * inv;
                }
            }
        } else if (scored) {
            error = 4.0f;
            if (masked) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    c[v] = c[v] > -INFINITY ? __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(c[v] * -kLog2e)) : -INFINITY;
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) c[v] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(c[v] * -kLog2e));
            }
        }
        if (a.bias) {
            if (!FULL || !all_finite(b)) {
                masked = true;
#pragma unroll
                for (int v = 0; v < V; ++v) b[v] = tamed(b[v]);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) c[v] += b[v];
        }
        // ---- the row's range
        float hi = -INFINITY, lo = INFINITY;
#pragma unroll
        for (int v = 0; v < V; v += 2) hi = most_of(hi, c[v], c[v + 1]);
        if (masked) {
#pragma unroll
            for (int v = 0; v < V; ++v) lo = fminf(lo, c[v] > -INFINITY ? c[v] : INFINITY);
        } else {
#pragma unroll
            for (int v = 0; v < V; v += 2) lo = least_of(lo, c[v], c[v + 1]);
        }
        hi = max16(hi);
        lo = min16(lo);
        const float rounding = fmaxf(fabsf(hi), fabsf(lo)) * (1.0625f * 0x1p-24f);  // of a sum
        error = scored ? error * (1.0625f * 0x1p-24f) + rounding : 0.0f;
        // choices far below the largest have no place
        const float floor = fmaxf(lo, hi - fmaxf(32.0f, 0.25f * fminf(hi - lo, 4096.0f)));
        const float step = hi > floor ? fminf(kSteps * __builtin_amdgcn_rcpf(hi - floor), FLT_MAX) : 1.0f;
        // ---- keys: place and number, at first the number within the lane; no place
        // (0) for what is not available
        uint32_t key[V];
        const uint32_t number = kNumber - (uint32_t)part.first - (V - 1);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            uint32_t place;
            if (whole) {
                const uint32_t u = __float_as_uint(c[v] + 0.0f);  // (-0 is 0; of -inf below 2^10)
                place = (u ^ (uint32_t)((int32_t)u >> 31 | INT32_MIN)) >> 13;
                place = c[v] > -INFINITY ? place : 0u;
            } else {
                place = whole_part(__builtin_fmaf(c[v] - floor, step, 1.0f));
            }
            key[v] = place << kBits | (uint32_t)(V - 1 - v);
        }
        uint32_t best[D];
#pragma unroll
        for (int q = 0; q < V; q += D) {
            uint32_t more[D];
#pragma unroll
            for (int i = 0; i < D; ++i) more[i] = q + i < V ? key[q + i] : 0u;
            sort<D>(more);
            if (q == 0) {
#pragma unroll
                for (int i = 0; i < D; ++i) best[i] = more[i];
            } else {
                absorb<D>(best, more);
            }
        }
#pragma unroll
        for (int i = 0; i < D; ++i) best[i] += number;
        // ---- groups
        bool again = false, kept = true;
        if (a.groups > 1) {
            float b0 = -INFINITY, b1 = -INFINITY;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                b1 = __builtin_amdgcn_fmed3f(c[v], b0, b1);
                b0 = more_of(b0, c[v]);
            }
            auto with = [&](float o0, float o1) {
                b1 = most_of(less_of(b0, o0), b1, o1);
                b0 = more_of(b0, o0);
            };
            const int32_t lanes = lay.lanes, first = l16 & -lanes;
            if (lanes >= 2) with(dpp<kXor1>(b0), dpp<kXor1>(b1));
            if (lanes >= 4) with(dpp<kXor2>(b0), dpp<kXor2>(b1));
            if (lanes >= 8) with(dpp<kMirror8>(b0), dpp<kMirror8>(b1));
            const float mine = sums && b1 > -INFINITY ? b0 + b1 : b0;
            const float apart = 4.0f * (error + rounding);
            const bool open = b0 > -INFINITY;  // (two biases may add up to less than any float)
            int32_t above = 0, near = 0;  // groups ahead for certain; and those that may be
            if (scored) {
                const float up = mine + apart, down = mine - apart;
                each16(lanes, mine, [&](int, float r) {
                    above += r > up;
                    near += r >= down;
                });
                near -= open ? 1 : 16 / lanes;  // itself
            } else {
                each16(lanes, mine, [&](int i, float r) { near += (r > mine) | ((r == mine) & (i < first)); });
            }
            kept = near < a.top_groups;
            again = scored && !kept && above < a.top_groups && open;
#pragma unroll
            for (int i = 0; i < D; ++i) best[i] = kept ? best[i] : 0u;
        }
        absorb_lane<D, kXor1>(best);
        absorb_lane<D, kXor2>(best);
        absorb_lane<D, kMirror8>(best);
        absorb_lane<D, kMirror16>(best);
        // ---- lane j takes choice j; are neighbours far enough apart?
        const uint32_t taken = pick<D>(best, l16 & (D - 1));
        const bool mine_is = l16 < a.topk, placed = taken >> kBits;
        const int32_t e = mine_is && placed ? (int32_t)(kNumber - (taken & kNumber)) : -1;
        const float mine = e >= 0 ? tamed(logit_at<DT>(row, e)) : -INFINITY;
        if (!whole) {
            const float far = 2.0f * error * step + 3.0f;  // steps, and what placing rounds
            // (places have at most 32 - kBits bits; a bound past them all makes every two near)
            const uint32_t margin = !scored ? 1u << kBits : far < (float)((1u << (32 - kBits)) - 2u) ? ((uint32_t)far + 1u) << kBits : ~0u;
            uint32_t next = dpp<kNext>(taken);
            if (V < 64 && a.topk == D) {
                const uint32_t last = best[D - 1] - 1u - number;
                uint32_t behind = ~0u;
#pragma unroll
                for (int v = 0; v < V; ++v) behind = last - key[v] < behind ? last - key[v] : behind;
                behind = kept ? behind : ~0u;
                behind = join16(behind, [](uint32_t x, uint32_t y) { return x < y ? x : y; });
                next = l16 == D - 1 ? best[D - 1] - 1u - behind : next;
            }
            bool near = mine_is && placed && next >> kBits && taken - next < margin && !(hi == lo && !scored);
            // Equal logits (and bias) are one choice, whose order the numbers give: as
            // often as not where logits have passed through 16 bits.  The chosen ones
            // are compared each with the next; with the last one, all others as near.
            if (__any(near)) {
                const int from = (lane & 48) + a.topk - 1;  // the last one's lane
                const float with = a.bias && e >= 0 ? gp(a.bias)[e] : 0.0f;  // (+inf is not the largest float here)
                const float mine2 = dpp<kNext>(mine), with2 = dpp<kNext>(with);
                const uint32_t least = (uint32_t)__shfl((int)taken, from);
                const float mine_k = __shfl(mine, from), with_k = __shfl(with, from);
                const uint32_t last = least - 1u - number;
                bool other = false;
#pragma unroll
                for (int q = 0; q < V; q += 4) {  // (of the keys behind the last one's)
                    float l[4], b4[4] = {};
                    load_four<DT, FULL>(row, part, lay.quads, q, -INFINITY, l);
                    if (a.bias) load_four<OPTIM_F32, FULL>(reinterpret_cast<const char *>(a.bias), part, lay.quads, q, -INFINITY, b4);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        other |= last - key[q + i] < margin && key[q + i] >> kBits != 0u &&
                                 (tamed(l[i]) != mine_k || (a.bias && b4[i] != with_k));
                    __builtin_amdgcn_sched_barrier(0);  // four at a time: no registers for more
                }
                other &= kept;
                const uint64_t others = __ballot(other);
                near = near && (l16 == a.topk - 1 ? (others >> (lane & 48) & 0xFFFFull) != 0u : mine != mine2 || with != with2);
            }
            again |= near;
            // choices without a place: chosen ones, or as near to one as rounding goes
            again |= mine_is && lo < floor && (!placed || (scored && taken < margin));
        }
        redo = __ballot(again && live);
        const bool sure = !(redo >> (lane & 48) & 0xFFFFull);
        // ---- weights
        float w;
        if (a.renormalise) {
            if (!soft && !__any(mine < -16.0f && e >= 0))  // (off by 28 x 2^-24 at most)
                w = e >= 0 ? __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(mine * -kLog2e)) : 0.0f;
            else
                w = part_of_score(a.score, mine, max16(mine));
            total = sum16(w);
        } else if (soft) {
            w = e >= 0 ? expf(mine - most) : 0.0f;
        } else {
            w = e >= 0 ? sigmoid(mine) : 0.0f;
        }
        if (e >= 0) w = w / total;
        w *= a.scale;
        const uint64_t nans = __ballot(nan);
        if (nans >> (lane & 48) & 0xFFFFull) w = __builtin_nanf("");
        if (live && sure && mine_is) {
            a.idx[t * a.topk + l16] = e;
            a.weights[t * a.topk + l16] = w;
        }
    }
    while (redo) {
        const int of = __builtin_ctzll(redo) >> 4;
        redo &= ~(0xFFFFull << (of * 16));
        route_token<V64, DT>(a, t0 + of, lds[wave], lane);
        wave_sync();
    }
}

// ---------------------------------------------------------------- a token a lane
// Few experts: a lane holds a whole row, and nothing passes between lanes.  The
// choice is made as it is defined, on fp64 keys where there is a bias (BIAS) and on
// the logits otherwise.
constexpr int kLaneTopk = 8;
template <int V, int DT, bool BIAS>
__global__ __launch_bounds__(kThreads) void route_lane_kernel(RouteArgs a) {
    using Key = std::conditional_t<BIAS, double, float>;
    constexpr Key kShut = -(Key)__builtin_inff();
    const int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (t >= a.tokens) return;
    const char *row = a.logits + t * a.ldl;
    float l[V];
    bool nan = false;
#pragma unroll
    for (int q = 0; q < V; q += 8) {
        const int n = a.experts - q;
        float x[8] = {};
        if (n > 0) floats<DT>(get8<DT>(row + q * kElem<DT>, n), x);
#pragma unroll
        for (int v = 0; v < 8; ++v) {
            l[q + v] = v < n ? x[v] : -INFINITY;
            nan |= l[q + v] != l[q + v];
            l[q + v] = tamed(l[q + v]);
        }
    }
    const bool soft = a.score == OPTIM_ROUTE_SOFTMAX;
    float most = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) most = more_of(most, l[v]);
    const float from = most > -INFINITY ? most : 0.0f;
    float total = 0.0f;
    if (soft && !a.renormalise) {
#pragma unroll
        for (int v = 0; v < V; ++v) total += __builtin_amdgcn_exp2f((l[v] - from) * 1.44269504f);
    }
    Key key[V];
    if constexpr (BIAS) {
        double sum = 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            key[v] = soft ? exp((double)l[v] - from) : 1.0 / (1.0 + exp(-(double)l[v]));
            sum += key[v];
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float b = v < a.experts ? a.bias[v] : -INFINITY;
            key[v] = l[v] > -INFINITY && b > -INFINITY ? (soft ? key[v] / sum : key[v]) + (double)b : kShut;
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = l[v];
    }
    float mine[kLaneTopk];
#pragma unroll
    for (int j = 0; j < kLaneTopk; ++j) {
        mine[j] = -INFINITY;
        if (j >= a.topk) continue;
        Key best = kShut;
        int32_t at = -1;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const bool more = key[v] > best;
            best = more ? key[v] : best;
            at = more ? v : at;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const bool it = at == v;
            key[v] = it ? kShut : key[v];
            mine[j] = it ? l[v] : mine[j];
        }
        a.idx[t * a.topk + j] = at;
    }
    float w[kLaneTopk], chosen = -INFINITY;
#pragma unroll
    for (int j = 0; j < kLaneTopk; ++j) chosen = more_of(chosen, mine[j]);
    if (a.renormalise) total = 0.0f;
    else if (!soft) total = 1.0f;
#pragma unroll
    for (int j = 0; j < kLaneTopk; ++j) {
        if (j >= a.topk) continue;
        if (a.renormalise) {
            w[j] = part_of_score(a.score, mine[j], chosen);
            total += w[j];
        } else {
            w[j] = !(mine[j] > -INFINITY) ? 0.0f : soft ? expf(mine[j] - from) : sigmoid(mine[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < kLaneTopk; ++j) {
        if (j >= a.topk) continue;
        float x = mine[j] > -INFINITY ? w[j] / total : 0.0f;
        x *= a.scale;
        a.weights[t * a.topk + j] = nan ? __builtin_nanf("") : x;
    }
}

// ---------------------------------------------------------------- the gradient
// L lanes a token (16, or 64 for more than 16 choices), lane j with choice j.  A
// row passes through registers in chunks of eight, chunk c in lane c mod L, and
// through LDS, where the chosen experts' terms join it.  Only the gradient of the
// whole softmax (WHOLE) reads the row.
template <int L>
__device__ __forceinline__ float lanes_max(float x) { return L == 16 ? max16(x) : wave_max(x); }
template <int L>
__device__ __forceinline__ float lanes_sum(float x) { return L == 16 ? sum16(x) : wave_sum(x); }

template <int L, int C, int DT, bool WHOLE>
__global__ __launch_bounds__(kThreads) void route_grad_kernel(RouteGradArgs a) {
    constexpr int kTokens = 64 / L;  // of a wavefront
    __shared__ __align__(16) float lds[kWaves][kTokens][C * L * 8];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane & (L - 1);
    const int64_t t0 = ((int64_t)blockIdx.x * kWaves + wave) * kTokens;
    if (t0 >= a.tokens) return;
    const int64_t t = t0 + lane / L;
    const bool live = t < a.tokens;
    float *grad = lds[wave][lane / L];
    const char *row = a.logits + (live ? t : t0) * a.ldl;
    const bool slot = live && l < a.topk;
    const int32_t e = slot ? a.idx[t * a.topk + l] : -1;
    const bool chosen = (uint32_t)e < (uint32_t)a.experts;
    Raw8<DT> raw[C];
    if constexpr (WHOLE) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int32_t first = (i * L + l) * 8, n = a.experts - first;
            if (n > 0) raw[i] = get8<DT>(row + (int64_t)first * kElem<DT>, n);
        }
    }
    const float g = chosen ? a.dweights[t * a.topk + l] * a.scale : 0.0f;
    const float mine = chosen ? tamed(logit_at<DT>(row, e)) : -INFINITY;
    // Which of the lanes that name an expert comes first?  Each leaves its number.
    if (chosen) reinterpret_cast<int32_t *>(grad)[e] = l;
    wave_sync();
    const bool twice = __any(chosen && reinterpret_cast<const int32_t *>(grad)[chosen ? e : 0] != l);
    wave_sync();
    float d;             // of the chosen expert, beside the row's own
    float x[C][8];       // the row's own
    float of_top = 0.0f; // the same of an expert with more than half of the score (top)
    bool top = false;
    if constexpr (WHOLE) {
        float most = -INFINITY, total = 0.0f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int32_t n = a.experts - (i * L + l) * 8;
            floats<DT>(raw[i], x[i]);
#pragma unroll
            for (int v = 0; v < 8; ++v) {
                x[i][v] = v < n ? tamed(x[i][v]) : -INFINITY;
                most = more_of(most, x[i][v]);
            }
        }
        most = lanes_max<L>(most);
        const float from = most > -INFINITY ? most : 0.0f;
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int v = 0; v < 8; ++v) {
                x[i][v] = __builtin_amdgcn_exp2f((x[i][v] - from) * 1.44269504f);
                total += x[i][v];
            }
        total = lanes_sum<L>(total);
        const float inv = total > 0.0f ? 1.0f / total : 0.0f;
        const float s = mine > -INFINITY ? expf(mine - from) * inv : 0.0f;
        d = g * s;
        const float by = -(lanes_sum<L>(d) * inv);
        // More than half of the score is one expert's, the only one whose term is 1: its
        // s (g - sum of g s) would be a difference of nearly equal numbers, and is
        // s (g (1 - s) - sum over the others of g s), 1 - s from their terms (what is left
        // of each without whole ones).  Where every row has such an expert that costs,
        // measured, 65536 x 256 bf16 17.5 us for 17.0, x 1024 fp32 120 for 118.
        top = mine == from && s > 0.5f;
        if (__any(top)) {
            float rest = 0.0f;
#pragma unroll
            for (int i = 0; i < C; ++i)
#pragma unroll
                for (int v = 0; v < 8; ++v) rest += __builtin_amdgcn_fractf(x[i][v]);
            rest = lanes_sum<L>(rest);
            of_top = -(lanes_sum<L>(top ? 0.0f : d) * inv);
            d = top ? d * (rest * inv) : d;
        }
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int v = 0; v < 8; ++v) x[i][v] = x[i][v] * by;
    } else if (a.renormalise) {
        const float s = part_of_score(a.score, mine, lanes_max<L>(mine));
        const float total = lanes_sum<L>(s);
        const float w = total > 0.0f ? s / total : 0.0f;
        d = w * (g - lanes_sum<L>(g * w));
        const bool most = w > 0.5f;  // (as above; one lane at most)
        if (__any(most)) {
            const float rest = lanes_sum<L>(most ? 0.0f : s), others = lanes_sum<L>(most ? 0.0f : g * w);
            d = most ? w * (g * (rest / total) - others) : d;
        }
        if (a.score == OPTIM_ROUTE_SIGMOID) d = d * sigmoid(-mine);
    } else {
        d = g * sigmoid(mine) * sigmoid(-mine);
    }
    if (!(mine > -INFINITY)) d = 0.0f;
    bool first = chosen;
    if (twice) {  // the first name's lane adds them up, in order
        float sum = d;
        for (int32_t j = 0; j < a.topk; ++j) {
            const int32_t e2 = __shfl(e, (lane & -L) + j);
            const float d2 = __shfl(d, (lane & -L) + j);
            if (e2 != e || j == l) continue;
            if (j < l) first = false;
            else sum += d2;
        }
        d = sum;
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
        f32x4 *to = reinterpret_cast<f32x4 *>(grad + (i * L + l) * 8);
        to[0] = WHOLE ? f32x4{x[i][0], x[i][1], x[i][2], x[i][3]} : zero;
        to[1] = WHOLE ? f32x4{x[i][4], x[i][5], x[i][6], x[i][7]} : zero;
    }
    wave_sync();
    if (first) grad[e] = (top ? of_top : grad[e]) + d;
    wave_sync();
    if (!live) return;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int32_t at = (i * L + l) * 8, n = a.experts - at;
        if (n <= 0) continue;
        const f32x4 *from = reinterpret_cast<const f32x4 *>(grad + at);
        const f32x4 lo = from[0], hi = from[1];
        const float y[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        put8<DT>(a.dlogits + t * a.ldd + (int64_t)at * kElem<DT>, n, rounded<DT>(y));
    }
}

// A launch takes fewer than 2^32 lanes: calls f(arguments of at most 2^25 tokens).
constexpr int64_t kMostTokens = int64_t(1) << 25;
void advance(RouteArgs &a) {
    a.logits += kMostTokens * a.ldl;
    a.idx += kMostTokens * a.topk;
    a.weights += kMostTokens * a.topk;
}
void advance(RouteGradArgs &a) {
    a.logits += kMostTokens * a.ldl;
    a.idx += kMostTokens * a.topk;
    a.dweights += kMostTokens * a.topk;
    a.dlogits += kMostTokens * a.ldd;
}
template <class A, class F>
hipError_t route_slices(A a, F &&f) {
    for (int64_t left = a.tokens; left > 0; left -= kMostTokens, advance(a)) {
        a.tokens = left < kMostTokens ? left : kMostTokens;
        f(a);
    }
    return hipGetLastError();
}

template <int V>
void launch_route_wave(const RouteArgs &a, int dtype, hipStream_t s) {
    const dim3 grid((unsigned)((a.tokens + kWaves - 1) / kWaves));
    if (dtype == OPTIM_F32)
        hipLaunchKernelGGL((route_wave_kernel<V, OPTIM_F32>), grid, dim3(kThreads), 0, s, a);
    else if (dtype == OPTIM_BF16)
        hipLaunchKernelGGL((route_wave_kernel<V, OPTIM_BF16>), grid, dim3(kThreads), 0, s, a);
    else
        hipLaunchKernelGGL((route_wave_kernel<V, OPTIM_F16>), grid, dim3(kThreads), 0, s, a);
}
template <int V, int D, int DT>
void launch_route_t(const RouteArgs &a, Lay lay, hipStream_t s) {
    const dim3 grid((unsigned)((a.tokens + kWaves * 4 - 1) / (kWaves * 4)));
    if (lay.full)
        hipLaunchKernelGGL((route_kernel<V, D, DT, true>), grid, dim3(kThreads), 0, s, a, lay);
    else
        hipLaunchKernelGGL((route_kernel<V, D, DT, false>), grid, dim3(kThreads), 0, s, a, lay);
}
template <int V, int D>
void launch_route_d(const RouteArgs &a, Lay lay, int dtype, hipStream_t s) {
    lay.full = a.experts == 16 * V;
    if (dtype == OPTIM_F32) return launch_route_t<V, D, OPTIM_F32>(a, lay, s);
    if (dtype == OPTIM_BF16) return launch_route_t<V, D, OPTIM_BF16>(a, lay, s);
    launch_route_t<V, D, OPTIM_F16>(a, lay, s);
}
template <int V, int DT>
void launch_route_lane_t(const RouteArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)((a.tokens + kThreads - 1) / kThreads));
    if (a.bias)
        hipLaunchKernelGGL((route_lane_kernel<V, DT, true>), grid, dim3(kThreads), 0, s, a);
    else
        hipLaunchKernelGGL((route_lane_kernel<V, DT, false>), grid, dim3(kThreads), 0, s, a);
}
template <int V>
void launch_route_lane(const RouteArgs &a, int dtype, hipStream_t s) {
    if (dtype == OPTIM_F32) return launch_route_lane_t<V, OPTIM_F32>(a, s);
    if (dtype == OPTIM_BF16) return launch_route_lane_t<V, OPTIM_BF16>(a, s);
    launch_route_lane_t<V, OPTIM_F16>(a, s);
}
template <int V>
void launch_route_v(const RouteArgs &a, Lay lay, int dtype, hipStream_t s) {
    if constexpr (V < 64)
        if (a.topk <= 8) return launch_route_d<V, 8>(a, lay, dtype, s);
    launch_route_d<V, 16>(a, lay, dtype, s);
}
Lay lay_of(int32_t experts, int32_t groups) {
    int32_t lanes = 16;
    while (lanes > 1 && 16 / lanes < groups) lanes /= 2;
    const int32_t per = experts / groups, n = (per + lanes - 1) / lanes;
    // fours are kept together where that makes them single accesses
    const bool quads = per % 4 == 0;
    return Lay{lanes, per, quads ? (n + 3) / 4 * 4 : n, quads, false};
}

template <int L, int C, int DT>
void launch_route_grad_t(const RouteGradArgs &a, hipStream_t s) {
    constexpr int64_t kTokens = kWaves * 64 / L;
    const dim3 grid((unsigned)((a.tokens + kTokens - 1) / kTokens));
    if (a.score == OPTIM_ROUTE_SOFTMAX && !a.renormalise)
        hipLaunchKernelGGL((route_grad_kernel<L, C, DT, true>), grid, dim3(kThreads), 0, s, a);
    else
        hipLaunchKernelGGL((route_grad_kernel<L, C, DT, false>), grid, dim3(kThreads), 0, s, a);
}
template <int L, int C>
void launch_route_grad_c(const RouteGradArgs &a, int dtype, hipStream_t s) {
    if (dtype == OPTIM_F32) return launch_route_grad_t<L, C, OPTIM_F32>(a, s);
    if (dtype == OPTIM_BF16) return launch_route_grad_t<L, C, OPTIM_BF16>(a, s);
    launch_route_grad_t<L, C, OPTIM_F16>(a, s);
}

}  // namespace

hipError_t launch_route(const RouteArgs &args, int dtype, hipStream_t s) {
    const Lay lay = lay_of(args.experts, args.groups);
    const bool rows16 = args.topk <= (lay.n > 32 ? 15 : 16) && args.groups <= 16 && lay.n <= 64;
    // A lane a token has the shortest way but few wavefronts.  Measured, by lanes and
    // by 16 lanes a token: 65536 x 8 3.7 and 14 us (with a bias 5.7 and 14), x 16 5.6
    // and 14; 16384 x 8 3.5 and 5.4 (5.5 and 5.4), x 16 5.3 and 5.4; 8192 x 16 5.2 and
    // 4.2; 65536 x 32 11.2 (19.7 with a bias) and 13.
    const bool lanes = args.groups == 1 && args.topk <= kLaneTopk && args.experts <= 16 && args.tokens >= 16384;
    return route_slices(args, [&](const RouteArgs &a) {
        if (lanes) return a.experts <= 8 ? launch_route_lane<8>(a, dtype, s) : launch_route_lane<16>(a, dtype, s);
        if (rows16) {
            if (lay.n <= 4) return launch_route_v<4>(a, lay, dtype, s);
            if (lay.n <= 8) return launch_route_v<8>(a, lay, dtype, s);
            if (lay.n <= 16) return launch_route_v<16>(a, lay, dtype, s);
            if (lay.n <= 32) return launch_route_v<32>(a, lay, dtype, s);
            return launch_route_v<64>(a, lay, dtype, s);
        }
        if (a.experts <= 64) return launch_route_wave<1>(a, dtype, s);
        if (a.experts <= 128) return launch_route_wave<2>(a, dtype, s);
        if (a.experts <= 256) return launch_route_wave<4>(a, dtype, s);
        if (a.experts <= 512) return launch_route_wave<8>(a, dtype, s);
        return launch_route_wave<16>(a, dtype, s);
    });
}

hipError_t launch_route_grad(const RouteGradArgs &args, int dtype, hipStream_t s) {
    return route_slices(args, [&](const RouteGradArgs &a) {
        if (a.topk > 16)
            return a.experts <= 512 ? launch_route_grad_c<64, 1>(a, dtype, s) : launch_route_grad_c<64, 2>(a, dtype, s);
        if (a.experts <= 128) return launch_route_grad_c<16, 1>(a, dtype, s);
        if (a.experts <= 256) return launch_route_grad_c<16, 2>(a, dtype, s);
        if (a.experts <= 512) return launch_route_grad_c<16, 4>(a, dtype, s);
        return launch_route_grad_c<16, 8>(a, dtype, s);
    });
}

}  // namespace optim
