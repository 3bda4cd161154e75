// kernels_route.hip -- routing of tokens to experts and its gradient
// (optim_route, optim_route_grad).
//
// One wavefront per token; lane l holds experts l, l + 64, ...  The choice is
// made on keys in fp64: the score plus the bias, or the logit itself.
#include "elems.h"

#include <cfloat>

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

// The largest key and, of equal ones, the lowest expert, over the wavefront.
__device__ __forceinline__ void wave_best(double &k, int32_t &e) {
    for (int m = 32; m; m /= 2) {
        const double k2 = halves(k, [&](int x) { return __shfl_xor(x, m); });
        const int32_t e2 = __shfl_xor(e, m);
        if (k2 > k || (k2 == k && e2 < e)) {
            k = k2;
            e = e2;
        }
    }
}

// The two largest keys of a group, b0 >= b1.
__device__ __forceinline__ void keep_two(double k, double &b0, double &b1) {
    b1 = fmax(b1, fmin(b0, k));
    b0 = fmax(b0, k);
}

// Lane j (below topk) returns choice j, or -1.  V: experts of a lane.
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
        double b0 = kNone, b1 = kNone;
        if (lane < a.groups)
            for (int32_t i = 0; i < per; ++i) keep_two(lds[lane * per + i], b0, b1);
        const double rank = a.group_best > 1 && b1 > kNone ? b0 + b1 : b0;
        int32_t ahead = 0;
        for (int32_t g = 0; g < a.groups; ++g) {
            const double r = halves(rank, [&](int x) { return __shfl(x, g); });
            ahead += r > rank || (r == rank && g < lane) ? 1 : 0;
        }
        const uint64_t kept = __ballot(lane < a.groups && ahead < a.top_groups);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int32_t e = lane + 64 * v;
            if (e < a.experts && !(kept >> (e / per) & 1)) k[v] = kNone;
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
// most: the largest of them; low: below it sigmoids are taken relative to it,
// so that they do not vanish, s_j / s_max = e^(l_j - m) (1 + e^m) / (1 + e^l_j).
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
// Within rows of 16 lanes, values pass between lanes without LDS (DPP).  Each of
// these pairs a lane with one of the other half of its 2, 4, 8 or 16.
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140, kBroadcast = 0x150, kNext = 0x101;
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float x) { return __uint_as_float(dpp<CTRL>(__float_as_uint(x))); }
template <class T, class F>
__device__ __forceinline__ T join16(T x, F &&f) {
    x = f(x, dpp<kXor1>(x));
    x = f(x, dpp<kXor2>(x));
    x = f(x, dpp<kMirror8>(x));
    return f(x, dpp<kMirror16>(x));
}
__device__ __forceinline__ float max16(float x) { return join16(x, [](float a, float b) { return fmaxf(a, b); }); }
__device__ __forceinline__ float min16(float x) { return join16(x, [](float a, float b) { return fminf(a, b); }); }
__device__ __forceinline__ float sum16(float x) { return join16(x, [](float a, float b) { return a + b; }); }

// f(number, value of that lane) for each lane of the 16
template <int I = 0, class F>
__device__ __forceinline__ void each16(float x, F &&f) {
    if constexpr (I < 16) {
        f(I, dpp<kBroadcast + I>(x));
        each16<I + 1>(x, f);
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

// How a row lies in a token's 16 lanes: lane i holds experts n i ... n i + n - 1.
struct Lay {
    int32_t n;
    bool quads;  // four neighbours are one access, all there or none
};
template <int V, int DT>
__device__ __forceinline__ void load_row(const char *row, int32_t experts, Lay lay, int lane, float (&l)[V], bool &nan) {
    const int32_t e0 = lane * lay.n;
    float raw[V];
    if (lay.quads) {
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
            const bool in = q * 4 < lay.n && e0 + q * 4 < experts;
            const char *p = row + (int64_t)(in ? e0 + q * 4 : 0) * kElem<DT>;
            if constexpr (DT == OPTIM_F32) {
                const u32x4 u = *(const GMEM u32x4_at4 *)gp(p);
#pragma unroll
                for (int i = 0; i < 4; ++i) raw[q * 4 + i] = in ? __uint_as_float(u[i]) : -INFINITY;
            } else {
                const u32x2 u = *(const GMEM u32x2_at2 *)gp(p);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t h = u[i / 2] >> (i % 2 * 16) & 0xFFFFu;
                    raw[q * 4 + i] = !in ? -INFINITY : DT == OPTIM_BF16 ? bf16_to_f32(h) : f16_to_f32(h);
                }
            }
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const bool in = v < lay.n && e0 + v < experts;
            const float x = logit_at<DT>(row, in ? e0 + v : 0);
            raw[v] = in ? x : -INFINITY;
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        nan |= raw[v] != raw[v];
        l[v] = tamed(raw[v]);
    }
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
// has |l| s (1 - s) 1.5 <= 0.34 from the exponent, half from the exponential, 3 s
// from the sum and the reciprocal, below 4; a softmax has its terms' |x| + 3, 20
// from the sum (V + 4 terms one after another, V <= 64: 68) and 3 of itself,
// below (V + 32) s as |x| e^-x < 1; the sum with b half of itself.  Twice that is
// allowed for.
template <int V, int D, int DT>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs a, Lay lay) {
    constexpr int V64 = V < 4 ? 1 : V / 4;
    constexpr int kBits = V == 4 ? 6 : V == 8 ? 7 : V == 16 ? 8 : V == 32 ? 9 : 10;  // of an expert's number
    constexpr uint32_t kNumber = (1u << kBits) - 1;
    constexpr float kSteps = (float)((1 << (kBits < 8 ? 24 : 32 - kBits)) - 8);
    __shared__ double lds[kWaves][64 * V64];
    const int lane = threadIdx.x & 63, l16 = lane & 15, wave = threadIdx.x >> 6;
    const bool sums = a.groups > 1 && a.group_best > 1, scored = a.bias || sums;
    const int32_t e0 = l16 * lay.n;
    const int64_t t0 = ((int64_t)blockIdx.x * kWaves + wave) * 4;
    if (t0 >= a.tokens) return;
    uint64_t redo;
    {
        const int64_t t = t0 + (lane >> 4);
        const bool live = t < a.tokens;
        const char *row = a.logits + (live ? t : t0) * a.ldl;
        float c[V];
        bool nan = false;
        load_row<V, DT>(row, a.experts, lay, l16, c, nan);
        // ---- scores, where they count
        const bool soft = a.score == OPTIM_ROUTE_SOFTMAX;
        float most = -INFINITY, total = 1.0f, error = 0.0f;
        if (soft && (scored || !a.renormalise)) {
#pragma unroll
            for (int v = 0; v < V; ++v) most = fmaxf(most, c[v]);
            most = max16(most);
            total = 0.0f;
            const float from = most > -INFINITY ? most : 0.0f;
            if (!scored) {
#pragma unroll
                for (int v = 0; v < V; ++v) total += __builtin_amdgcn_exp2f((c[v] - from) * 1.44269504f);
                total = sum16(total);
            } else {
                float s[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    s[v] = __builtin_amdgcn_exp2f((c[v] - from) * 1.44269504f);
                    total += s[v];
                }
                total = sum16(total);
                const float inv = total > 0.0f ? __builtin_amdgcn_rcpf(total) : 0.0f;
                error = (2.0f * (V + 32)) * inv;
#pragma unroll
                for (int v = 0; v < V; ++v) c[v] = c[v] > -INFINITY ? s[v] * inv : -INFINITY;
            }
        } else if (scored) {
            error = 8.0f;
#pragma unroll
            for (int v = 0; v < V; ++v)
                c[v] = c[v] > -INFINITY ? __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(c[v] * -1.44269504f)) : -INFINITY;
        }
        if (a.bias) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float b = a.bias[v < lay.n && e0 + v < a.experts ? e0 + v : 0];
                c[v] = b > -INFINITY ? c[v] + b : -INFINITY;
            }
        }
        // ---- the row's range
        float hi = -INFINITY, lo = INFINITY;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            hi = fmaxf(hi, c[v]);
            lo = fminf(lo, c[v] > -INFINITY ? c[v] : INFINITY);
        }
        hi = max16(hi);
        lo = min16(lo);
        bool again = scored && !(hi < INFINITY) && hi > -INFINITY;  // an infinite bias
        const bool flat = hi == lo;
        error = scored ? (error + 2.0f * fmaxf(fabsf(hi), fabsf(lo))) * 0x1p-24f : 0.0f;
        const float floor = fmaxf(lo, hi - 32.0f);  // choices far below the largest are one
        const float step = hi > floor ? kSteps / (hi - floor) : 0.0f;
        // ---- keys, sorted
        uint32_t key[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            uint32_t place;
            if (DT != OPTIM_F32 && !scored) {
                const uint32_t u = __float_as_uint(c[v] + 0.0f);  // (-0 is 0)
                place = (u ^ (uint32_t)((int32_t)u >> 31 | INT32_MIN)) >> 13;
            } else {
                place = (uint32_t)(fmaxf(c[v] - floor, 0.0f) * step);
            }
            key[v] = c[v] > -INFINITY ? (place + 1u) << kBits | (kNumber - (uint32_t)(e0 + v)) : 0u;
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
        // ---- groups: 16 / groups lanes each
        if (a.groups > 1) {
            float b0 = -INFINITY, b1 = -INFINITY;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                b1 = __builtin_amdgcn_fmed3f(c[v], b0, b1);
                b0 = fmaxf(b0, c[v]);
            }
            auto with = [&](float o0, float o1) {
                b1 = fmaxf(fminf(b0, o0), fmaxf(b1, o1));
                b0 = fmaxf(b0, o0);
            };
            if (a.groups <= 8) with(dpp<kXor1>(b0), dpp<kXor1>(b1));
            if (a.groups <= 4) with(dpp<kXor2>(b0), dpp<kXor2>(b1));
            if (a.groups <= 2) with(dpp<kMirror8>(b0), dpp<kMirror8>(b1));
            const float mine = sums && b1 > -INFINITY ? b0 + b1 : b0;
            const int32_t lanes = 16 / a.groups, first = l16 / lanes * lanes;
            const float apart = scored ? 4.0f * error : 0.0f;
            int32_t above = 0, near = 0;  // lanes of groups ahead for certain; and of those that may be
            if (scored) {
                each16(mine, [&](int, float r) {
                    above += r > mine + apart;
                    near += r >= mine - apart;
                });
                near -= lanes;
            } else {
                each16(mine, [&](int i, float r) { above += r > mine || (r == mine && i < first); });
                near = above;
            }
            const int32_t bar = a.top_groups * lanes;
            const bool kept = near < bar;
            again |= !kept && above < bar && mine > -INFINITY;
#pragma unroll
            for (int i = 0; i < D; ++i) best[i] = kept ? best[i] : 0u;
#pragma unroll
            for (int v = 0; v < V; ++v) key[v] = kept ? key[v] : 0u;
        }
        absorb_lane<D, kXor1>(best);
        absorb_lane<D, kXor2>(best);
        absorb_lane<D, kMirror8>(best);
        absorb_lane<D, kMirror16>(best);
        // ---- lane j takes choice j; are neighbours far enough apart?
        uint32_t taken = 0u;
#pragma unroll
        for (int i = 0; i < D; ++i) taken = l16 == i ? best[i] : taken;
        if (!(DT != OPTIM_F32 && !scored)) {
            uint32_t next = dpp<kNext>(taken);
            if (V < 64 && a.topk == D) {
                uint32_t behind = 0u;
#pragma unroll
                for (int v = 0; v < V; ++v) behind = key[v] < best[D - 1] && key[v] > behind ? key[v] : behind;
                behind = join16(behind, [](uint32_t x, uint32_t y) { return x > y ? x : y; });
                next = l16 == D - 1 ? behind : next;
            }
            const float least = 2.0f * error * step + 2.0f;  // steps
            const uint32_t margin = !scored ? 0u : least < 1e9f ? (uint32_t)least : 1u << 30;
            again |= l16 < a.topk && next && !(flat && !scored) && (taken >> kBits) - (next >> kBits) <= margin;
        }
        int32_t e = l16 < a.topk && taken ? (int32_t)(kNumber - (taken & kNumber)) : -1;
        redo = __ballot(again && live);
        const bool sure = !(redo >> (lane & 48) & 0xFFFFull);
        // ---- weights
        const float mine = e >= 0 ? tamed(logit_at<DT>(row, e)) : -INFINITY;
        float w;
        if (a.renormalise) {
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
        if (live && sure && l16 < a.topk) {
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

template <int V, int DT>
__global__ __launch_bounds__(kThreads) void route_grad_kernel(RouteGradArgs a) {
    __shared__ float lds[kWaves][64 * V];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float *grad = lds[wave];
    for (int64_t t = (int64_t)blockIdx.x * kWaves + wave; t < a.tokens; t += (int64_t)gridDim.x * kWaves) {
        const char *row = a.logits + t * a.ldl;
        const int32_t e = lane < a.topk ? a.idx[t * a.topk + lane] : -1;
        const bool chosen = (uint32_t)e < (uint32_t)a.experts;
        const float g = chosen ? a.dweights[t * a.topk + lane] * a.scale : 0.0f;
        const float mine = chosen ? tamed(logit_at<DT>(row, e)) : -INFINITY;
        float base[V];  // of every expert
        float d = 0.0f; // of the chosen one beside
#pragma unroll
        for (int v = 0; v < V; ++v) base[v] = 0.0f;
        if (a.score == OPTIM_ROUTE_SOFTMAX && !a.renormalise) {
            float l[V], most = -INFINITY, total = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int32_t x = lane + 64 * v;
                l[v] = x < a.experts ? tamed(logit_at<DT>(row, x)) : -INFINITY;
                most = fmaxf(most, l[v]);
            }
            most = wave_max(most);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                l[v] = l[v] > -INFINITY ? expf(l[v] - most) : 0.0f;
                total += l[v];
            }
            total = wave_sum(total);
            const float inv = total > 0.0f ? 1.0f / total : 0.0f;
            const float s = mine > -INFINITY ? expf(mine - most) * inv : 0.0f;
            const float dot = wave_sum(g * s);
#pragma unroll
            for (int v = 0; v < V; ++v) base[v] = -(l[v] * inv) * dot;
            d = g * s;
        } else if (a.score == OPTIM_ROUTE_SIGMOID && !a.renormalise) {
            d = g * sigmoid(mine) * sigmoid(-mine);
        } else {
            const float s = part_of_score(a.score, mine, wave_max(mine));
            const float total = wave_sum(s);
            const float w = total > 0.0f ? s / total : 0.0f;
            const float dot = wave_sum(g * w);
            d = w * (g - dot);
            if (a.score == OPTIM_ROUTE_SIGMOID) d = d * sigmoid(-mine);
        }
        if (!(mine > -INFINITY)) d = 0.0f;
        // of an expert named twice, the first name's lane writes the sum
        bool first = chosen;
        float sum = d;
        for (int32_t j = 0; j < a.topk; ++j) {
            const int32_t e2 = __shfl(e, j);
            const float d2 = __shfl(d, j);
            if (e2 != e || j == lane) continue;
            if (j < lane) first = false;
            else sum += d2;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) grad[lane + 64 * v] = base[v];
        wave_sync();
        if (first) grad[e] += sum;
        wave_sync();
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int32_t x = lane + 64 * v;
            if (x < a.experts) put_element<DT>(a.dlogits + t * a.ldd + (int64_t)x * kElem<DT>, grad[x]);
        }
        wave_sync();
    }
}

// A launch takes fewer than 2^32 lanes: calls f(arguments of at most 2^25 tokens).
template <class F>
hipError_t route_slices(const RouteArgs &args, F &&f) {
    constexpr int64_t kMost = int64_t(1) << 25;
    RouteArgs a = args;
    for (int64_t left = args.tokens; left > 0; left -= kMost) {
        a.tokens = left < kMost ? left : kMost;
        f(a);
        a.logits += kMost * a.ldl;
        a.idx += kMost * a.topk;
        a.weights += kMost * a.topk;
    }
    return hipGetLastError();
}

unsigned route_grid(int64_t tokens) {
    const int64_t g = (tokens + kWaves - 1) / kWaves;
    return (unsigned)(g < (1 << 23) ? g : 1 << 23);
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
template <int V, int D>
void launch_route_d(const RouteArgs &a, Lay lay, int dtype, hipStream_t s) {
    const dim3 grid((unsigned)((a.tokens + kWaves * 4 - 1) / (kWaves * 4)));
    if (dtype == OPTIM_F32)
        hipLaunchKernelGGL((route_kernel<V, D, OPTIM_F32>), grid, dim3(kThreads), 0, s, a, lay);
    else if (dtype == OPTIM_BF16)
        hipLaunchKernelGGL((route_kernel<V, D, OPTIM_BF16>), grid, dim3(kThreads), 0, s, a, lay);
    else
        hipLaunchKernelGGL((route_kernel<V, D, OPTIM_F16>), grid, dim3(kThreads), 0, s, a, lay);
}
template <int V>
void launch_route_v(const RouteArgs &a, Lay lay, int dtype, hipStream_t s) {
    if constexpr (V < 64)
        if (a.topk <= 8) return launch_route_d<V, 8>(a, lay, dtype, s);
    launch_route_d<V, 16>(a, lay, dtype, s);
}
// Experts of a lane of 16.  Groups are whole lanes; without them fours are kept
// together.
Lay lay_of(int32_t experts, int32_t groups) {
    const int32_t n = (experts + 15) / 16;
    const Lay lay{groups > 1 ? n : (n + 3) / 4 * 4, false};
    return Lay{lay.n, lay.n % 4 == 0 && experts % 4 == 0};
}
template <int V>
hipError_t launch_route_grad_v(const RouteGradArgs &a, int dtype, hipStream_t s) {
    const dim3 grid(route_grid(a.tokens));
    if (dtype == OPTIM_F32)
        hipLaunchKernelGGL((route_grad_kernel<V, OPTIM_F32>), grid, dim3(kThreads), 0, s, a);
    else if (dtype == OPTIM_BF16)
        hipLaunchKernelGGL((route_grad_kernel<V, OPTIM_BF16>), grid, dim3(kThreads), 0, s, a);
    else
        hipLaunchKernelGGL((route_grad_kernel<V, OPTIM_F16>), grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteArgs &args, int dtype, hipStream_t s) {
    const Lay lay = lay_of(args.experts, args.groups);
    const bool rows16 = args.topk <= (lay.n > 32 ? 15 : 16) &&
                        (args.groups == 1 || (16 % args.groups == 0 && args.experts % 16 == 0));
    return route_slices(args, [&](const RouteArgs &a) {
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

hipError_t launch_route_grad(const RouteGradArgs &a, int dtype, hipStream_t s) {
    if (a.experts <= 64) return launch_route_grad_v<1>(a, dtype, s);
    if (a.experts <= 128) return launch_route_grad_v<2>(a, dtype, s);
    if (a.experts <= 256) return launch_route_grad_v<4>(a, dtype, s);
    if (a.experts <= 512) return launch_route_grad_v<8>(a, dtype, s);
    return launch_route_grad_v<16>(a, dtype, s);
}

}  // namespace optim
