// kernels_tokens.hip -- tokens to the experts' rows and back
// (optim_expert_gather, optim_expert_combine, optim_expert_combine_grad).
//
// All three go by token: the token's row is read or written once, and the rows
// of its choices once each.  P lanes share a token, each taking eight neighbouring
// columns at a time.
#include "elems.h"

namespace optim {
namespace {

// The token and the first chunk of eight columns of this lane; P = 1 << lp.
struct Slot {
    int64_t t, dt;   // token, and how far the next one is
    int32_t c, dc;   // chunk, and how far the next one is
};
__device__ __forceinline__ Slot slot(int lp) {
    const int64_t per = kThreads >> lp;
    return Slot{(int64_t)blockIdx.x * per + (threadIdx.x >> lp), (int64_t)gridDim.x * per,
                (int32_t)(threadIdx.x & ((1 << lp) - 1)), 1 << lp};
}

template <int DT, bool WEIGHTS>
__global__ __launch_bounds__(kThreads) void gather_kernel(TokenArgs a, int lp) {
    const int32_t chunks = (a.dim + 7) / 8;
    const Slot s = slot(lp);
    for (int64_t t = s.t; t < a.tokens; t += s.dt) {
        const int32_t *place = a.place + t * a.topk;
        for (int32_t c = s.c; c < chunks; c += s.dc) {
            const int n = a.dim - c * 8;
            const int64_t at = (int64_t)c * (8 * kElem<DT>);
            const Raw8<DT> x = get8<DT>(a.x + t * a.ldx + at, n);
            for (int32_t j = 0; j < a.topk; ++j) {
                const uint32_t r = (uint32_t)place[j];
                if (r >= a.rows) continue;
                char *y = a.dy + r * a.lddy + at;
                if constexpr (WEIGHTS) {
                    float v[8];
                    floats<DT>(x, v);
                    const float w = a.weights[t * a.topk + j];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = v[i] * w;
                    put8<DT>(y, n, rounded<DT>(v));
                } else {
                    put8<DT>(y, n, x);
                }
            }
        }
    }
}

template <int DT, bool DROP>
__global__ __launch_bounds__(kThreads) void combine_kernel(TokenArgs a, int lp) {
    const int32_t chunks = (a.dim + 7) / 8;
    const Slot s = slot(lp);
    const uint32_t step = DROP ? drop_step(a.drop) : 0u;
    for (int64_t t = s.t; t < a.tokens; t += s.dt) {
        const int32_t *place = a.place + t * a.topk;
        for (int32_t c = s.c; c < chunks; c += s.dc) {
            const int n = a.dim - c * 8;
            const int64_t at = (int64_t)c * (8 * kElem<DT>);
            float sum[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
            for (int32_t j = 0; j < a.topk; ++j) {
                const uint32_t r = (uint32_t)place[j];
                if (r >= a.rows) continue;
                float v[8];
                floats<DT>(get8<DT>(a.y + r * a.ldy + at, n), v);
                const float w = a.weights ? a.weights[t * a.topk + j] : 1.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[i] = __builtin_fmaf(w, v[i], sum[i]);
            }
            if constexpr (DROP) drop8(a.drop, step, (uint64_t)(a.drop.first + t * a.dim + c * 8), sum);
            if (a.x) {
                float v[8];
                floats<DT>(get8<DT>(a.x + t * a.ldx + at, n), v);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[i] = v[i] + sum[i];
            }
            put8<DT>(a.out + t * a.ldo + at, n, rounded<DT>(sum));
        }
    }
}

// J choices at a time: their dot products stay in registers over the columns.
constexpr int kGradJ = 8;

template <int DT, bool DROP>
__global__ __launch_bounds__(kThreads) void combine_grad_kernel(TokenArgs a, int lp) {
    __shared__ float part[kThreads / 64][kGradJ];
    const int32_t chunks = (a.dim + 7) / 8;
    const Slot s = slot(lp);
    const uint32_t step = DROP ? drop_step(a.drop) : 0u;
    // (every lane goes through every round: they join their sums at its end)
    for (int64_t t0 = (int64_t)blockIdx.x * (kThreads >> lp); t0 < a.tokens; t0 += s.dt) {
        const int64_t t = t0 + (threadIdx.x >> lp);
        const bool live = t < a.tokens;
        for (int32_t j0 = 0; j0 < a.topk; j0 += kGradJ) {
            uint32_t r[kGradJ];
            float w[kGradJ], dot[kGradJ];
#pragma unroll
            for (int j = 0; j < kGradJ; ++j) {
                const bool in = live && j0 + j < a.topk;
                r[j] = in ? (uint32_t)a.place[t * a.topk + j0 + j] : ~0u;
                w[j] = in && a.weights ? a.weights[t * a.topk + j0 + j] : 1.0f;
                dot[j] = 0.0f;
            }
            for (int32_t c = s.c; live && c < chunks; c += s.dc) {
                const int n = a.dim - c * 8;
                const int64_t at = (int64_t)c * (8 * kElem<DT>);
                float d[8];
                floats<DT>(get8<DT>(a.x + t * a.ldx + at, n), d);
                if constexpr (DROP) drop8(a.drop, step, (uint64_t)(a.drop.first + t * a.dim + c * 8), d);
#pragma unroll
                for (int j = 0; j < kGradJ; ++j) {
                    if (r[j] >= a.rows) continue;
                    float v[8];
                    if (a.dweights) {
                        floats<DT>(get8<DT>(a.y + r[j] * a.ldy + at, n), v);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (i < n) dot[j] = __builtin_fmaf(d[i], v[i], dot[j]);
                    }
                    if (a.dy) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] = w[j] * d[i];
                        put8<DT>(a.dy + r[j] * a.lddy + at, n, rounded<DT>(v));
                    }
                }
            }
            if (!a.dweights) continue;
            const int width = lp < 6 ? 1 << lp : 64;
#pragma unroll
            for (int j = 0; j < kGradJ; ++j)
                for (int m = width / 2; m; m /= 2) dot[j] += __shfl_xor(dot[j], m);
            if (lp > 6) {
                const int wave = threadIdx.x >> 6, per = 1 << (lp - 6);
                __syncthreads();
                if ((threadIdx.x & 63) == 0)
#pragma unroll
                    for (int j = 0; j < kGradJ; ++j) part[wave][j] = dot[j];
                __syncthreads();
                if (s.c == 0)
#pragma unroll
                    for (int j = 0; j < kGradJ; ++j)
                        for (int i = 1; i < per; ++i) dot[j] += part[wave + i][j];
            }
            if (s.c == 0 && live)
#pragma unroll
                for (int j = 0; j < kGradJ; ++j)
                    if (j0 + j < a.topk) a.dweights[t * a.topk + j0 + j] = dot[j];
        }
    }
}

// Lanes for a token's chunks, as a power of two up to a workgroup.
int lanes_log2(int32_t dim, int least) {
    int lp = least;
    while (lp < 8 && (8 << lp) < dim) ++lp;
    return lp;
}
unsigned token_grid(int64_t tokens, int lp) {
    const int64_t per = kThreads >> lp, g = (tokens + per - 1) / per;
    return (unsigned)(g < (1 << 23) ? g : 1 << 23);
}

template <int DT>
hipError_t launch_gather_t(const TokenArgs &a, hipStream_t s) {
    const int lp = lanes_log2(a.dim, 0);
    const dim3 grid(token_grid(a.tokens, lp));
    if (a.weights)
        hipLaunchKernelGGL((gather_kernel<DT, true>), grid, dim3(kThreads), 0, s, a, lp);
    else
        hipLaunchKernelGGL((gather_kernel<DT, false>), grid, dim3(kThreads), 0, s, a, lp);
    return hipGetLastError();
}
template <int DT>
hipError_t launch_combine_t(const TokenArgs &a, hipStream_t s) {
    const int lp = lanes_log2(a.dim, 0);
    const dim3 grid(token_grid(a.tokens, lp));
    if (a.drop.bar)
        hipLaunchKernelGGL((combine_kernel<DT, true>), grid, dim3(kThreads), 0, s, a, lp);
    else
        hipLaunchKernelGGL((combine_kernel<DT, false>), grid, dim3(kThreads), 0, s, a, lp);
    return hipGetLastError();
}
template <int DT>
hipError_t launch_combine_grad_t(const TokenArgs &a, hipStream_t s) {
    const int lp = lanes_log2(a.dim, 0);
    const dim3 grid(token_grid(a.tokens, lp));
    if (a.drop.bar)
        hipLaunchKernelGGL((combine_grad_kernel<DT, true>), grid, dim3(kThreads), 0, s, a, lp);
    else
        hipLaunchKernelGGL((combine_grad_kernel<DT, false>), grid, dim3(kThreads), 0, s, a, lp);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gather(const TokenArgs &a, int dtype, hipStream_t s) {
    if (dtype == OPTIM_F32) return launch_gather_t<OPTIM_F32>(a, s);
    if (dtype == OPTIM_BF16) return launch_gather_t<OPTIM_BF16>(a, s);
    return launch_gather_t<OPTIM_F16>(a, s);
}
hipError_t launch_combine(const TokenArgs &a, int dtype, hipStream_t s) {
    if (dtype == OPTIM_F32) return launch_combine_t<OPTIM_F32>(a, s);
    if (dtype == OPTIM_BF16) return launch_combine_t<OPTIM_BF16>(a, s);
    return launch_combine_t<OPTIM_F16>(a, s);
}
hipError_t launch_combine_grad(const TokenArgs &a, int dtype, hipStream_t s) {
    if (dtype == OPTIM_F32) return launch_combine_grad_t<OPTIM_F32>(a, s);
    if (dtype == OPTIM_BF16) return launch_combine_grad_t<OPTIM_BF16>(a, s);
    return launch_combine_grad_t<OPTIM_F16>(a, s);
}

}  // namespace optim
