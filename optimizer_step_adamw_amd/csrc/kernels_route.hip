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
template <class T>
__device__ __forceinline__ T wave_sum(T x) {
    for (int m = 32; m; m /= 2) x += __shfl_xor(x, m);
    return x;
}

// The largest key and, of equal ones, the lowest expert, over the wavefront.
__device__ __forceinline__ void wave_best(double &k, int32_t &e) {
    for (int m = 32; m; m /= 2) {
        const double k2 = __shfl_xor(k, m);
        const int32_t e2 = __shfl_xor(e, m);
        if (k2 > k || (k2 == k && e2 < e)) {
            k = k2;
            e = e2;
        }
    }
}

// The two largest keys of a group, b0 >= b1.
__device__ __forceinline__ void keep_two(double k, double &b0, double &b1) {
    if (k > b0) {
        b1 = b0;
        b0 = k;
    } else if (k > b1) {
        b1 = k;
    }
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
            total = wave_sum(total);
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
            const double r = __shfl(rank, g);
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

template <int V, int DT>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs a) {
    __shared__ double lds[kWaves][64 * V];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t t = (int64_t)blockIdx.x * kWaves + wave; t < a.tokens; t += (int64_t)gridDim.x * kWaves) {
        const char *row = a.logits + t * a.ldl;
        const int32_t e = choose<V, DT>(a, row, lds[wave], lane);
        const bool chosen = e >= 0;
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
        const float mine = chosen ? tamed(logit_at<DT>(row, e)) : -INFINITY;
        float s;
        if (a.score == OPTIM_ROUTE_SOFTMAX) {
            if (a.renormalise) {  // over the chosen ones
                most = wave_max(mine);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) most = fmaxf(most, l[v]);
                most = wave_max(most);
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (l[v] > -INFINITY) total += expf(l[v] - most);
                total = wave_sum(total);
            }
            s = chosen ? expf(mine - most) : 0.0f;
        } else if (a.renormalise) {
            // relative to the largest, so that small scores do not vanish:
            // s_j / s_max = e^(l_j - m) (1 + e^m) / (1 + e^l_j) for m <= 0
            most = wave_max(mine);
            s = !chosen ? 0.0f : most > 0.0f ? sigmoid(mine) : expf(mine - most) * (1.0f + expf(most)) / (1.0f + expf(mine));
        } else {
            s = chosen ? sigmoid(mine) : 0.0f;
        }
        if (a.renormalise) total = wave_sum(s);
        float w = s;
        if (chosen && (a.renormalise || a.score == OPTIM_ROUTE_SOFTMAX)) w = s / total;
        w *= a.scale;
        if (nan) w = __builtin_nanf("");
        if (lane < a.topk) {
            a.idx[t * a.topk + lane] = e;
            a.weights[t * a.topk + lane] = w;
        }
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
            const float most = wave_max(mine);
            float s;
            if (!(mine > -INFINITY)) s = 0.0f;
            else if (a.score == OPTIM_ROUTE_SOFTMAX) s = expf(mine - most);
            else s = most > 0.0f ? sigmoid(mine) : expf(mine - most) * (1.0f + expf(most)) / (1.0f + expf(mine));
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

unsigned route_grid(int64_t tokens) {
    const int64_t g = (tokens + kWaves - 1) / kWaves;
    return (unsigned)(g < (1 << 23) ? g : 1 << 23);
}

template <int V>
hipError_t launch_route_v(const RouteArgs &a, int dtype, hipStream_t s) {
    const dim3 grid(route_grid(a.tokens));
    if (dtype == OPTIM_F32)
        hipLaunchKernelGGL((route_kernel<V, OPTIM_F32>), grid, dim3(kThreads), 0, s, a);
    else if (dtype == OPTIM_BF16)
        hipLaunchKernelGGL((route_kernel<V, OPTIM_BF16>), grid, dim3(kThreads), 0, s, a);
    else
        hipLaunchKernelGGL((route_kernel<V, OPTIM_F16>), grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
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

hipError_t launch_route(const RouteArgs &a, int dtype, hipStream_t s) {
    if (a.experts <= 64) return launch_route_v<1>(a, dtype, s);
    if (a.experts <= 128) return launch_route_v<2>(a, dtype, s);
    if (a.experts <= 256) return launch_route_v<4>(a, dtype, s);
    if (a.experts <= 512) return launch_route_v<8>(a, dtype, s);
    return launch_route_v<16>(a, dtype, s);
}

hipError_t launch_route_grad(const RouteGradArgs &a, int dtype, hipStream_t s) {
    if (a.experts <= 64) return launch_route_grad_v<1>(a, dtype, s);
    if (a.experts <= 128) return launch_route_grad_v<2>(a, dtype, s);
    if (a.experts <= 256) return launch_route_grad_v<4>(a, dtype, s);
    if (a.experts <= 512) return launch_route_grad_v<8>(a, dtype, s);
    return launch_route_grad_v<16>(a, dtype, s);
}

}  // namespace optim
