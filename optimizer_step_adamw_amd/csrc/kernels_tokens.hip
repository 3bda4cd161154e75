// kernels_tokens.hip -- tokens to the experts' rows and back
// (optim_expert_gather, optim_expert_combine, optim_expert_combine_grad).
//
// All three go by token: the token's row is read or written once, and the rows
// of its choices once each, whatever their order; by row, every token's row would be
// read topk times.  A lane takes eight neighbouring columns (16 bytes of a 16-bit
// row), and a power of two of lanes a token, up to a workgroup; more columns are
// more workgroups, so that one token of a reply is spread as well.  Sums of a token
// are a lane's own, in the order of its choices; the weights' gradients are joined
// over the lanes in a fixed order.
//
// Bound by HBM.  Measured on MI355X: gather 16384 x 2048 bf16 to 8 rows each 114-115
// us (604 MB, 5.3 TB/s), combination of 16384 x 4096 bf16 from 2 with residual and
// dropout 90-97 us (537 MB, 5.5-6.0; 103 at most in a trace), its gradient for 20001
// x 1000 fp16 from 4 63-72 us (361 MB, 5.0-5.8; 104 when each row was asked for
// behind the one before it), for 16384 x 2048 from 8, with dropout, bf16 236 us (4.8)
// and fp32 440 (5.2); one token of 4096 from 8 3.3 us.
#include "elems.h"

namespace optim {
namespace {

// This lane's token, how far the next one is, and its chunk of eight columns; a
// workgroup holds kThreads >> lp tokens, grid.y covers the chunks.
struct Slot {
    int64_t t, dt;
    int32_t c;
};
__device__ __forceinline__ Slot slot(int lp) {
    const int64_t per = kThreads >> lp;
    return Slot{(int64_t)blockIdx.x * per + (threadIdx.x >> lp), (int64_t)gridDim.x * per,
                (int32_t)((blockIdx.y << lp) + (threadIdx.x & ((1 << lp) - 1)))};
}

template <int DT, bool WEIGHTS>
__global__ __launch_bounds__(kThreads) void gather_kernel(TokenArgs a, int lp) {
    const Slot s = slot(lp);
    const int n = a.dim - s.c * 8;
    if (n <= 0) return;
    const int64_t at = (int64_t)s.c * (8 * kElem<DT>);
    for (int64_t t = s.t; t < a.tokens; t += s.dt) {
        const int32_t *place = a.place + t * a.topk;
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

// Choices whose rows are asked for at a time.  A choice without a row reads the
// first one and counts for nothing, so that no load waits for another.
constexpr int kAtOnce = 4;

template <int DT, bool DROP, bool NT>
__global__ __launch_bounds__(kThreads) void combine_kernel(TokenArgs a, int lp) {
    const Slot s = slot(lp);
    const int n = a.dim - s.c * 8;
    if (n <= 0) return;
    const int64_t at = (int64_t)s.c * (8 * kElem<DT>);
    const uint32_t step = DROP ? drop_step(a.drop) : 0u;
    for (int64_t t = s.t; t < a.tokens; t += s.dt) {
        Raw8<DT> res{};
        if (a.x) res = get8<DT, NT>(a.x + t * a.ldx + at, n);
        float sum[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        for (int32_t j0 = 0; j0 < a.topk && a.rows > 0; j0 += kAtOnce) {
            uint32_t r[kAtOnce];
            float w[kAtOnce];
            Raw8<DT> y[kAtOnce];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const int64_t of = t * a.topk + (j0 + j < a.topk ? j0 + j : 0);
                r[j] = j0 + j < a.topk ? (uint32_t)a.place[of] : ~0u;
                w[j] = a.weights ? a.weights[of] : 1.0f;
            }
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) y[j] = get8<DT, NT>(a.y + (r[j] < a.rows ? r[j] : 0u) * a.ldy + at, n);
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                float v[8];
                floats<DT>(y[j], v);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[i] = r[j] < a.rows ? __builtin_fmaf(w[j], v[i], sum[i]) : sum[i];
            }
        }
        if constexpr (DROP) drop8(a.drop, step, (uint64_t)(a.drop.first + t * a.dim + s.c * 8), sum);
        if (a.x) {
            float v[8];
            floats<DT>(res, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] = v[i] + sum[i];
        }
        put8<DT, NT>(a.out + t * a.ldo + at, n, rounded<DT>(sum));
    }
}

// J choices at a time: their dot products stay in registers over the columns.  More
// than J choices, 8 at most, are rounds, each of which reads dout and draws the mask
// again: 8192 x 2048 from 16, with dropout, bf16 242 us (4.6 TB/s of what it cannot do
// without), fp32 469 (4.7).
// `lp`: 1 << lp lanes a token, at most a workgroup, going over its chunks.
template <int J, int DT, bool DROP>
__global__ __launch_bounds__(kThreads) void combine_grad_kernel(TokenArgs a, int lp) {
    __shared__ float part[kThreads / 64][J];
    const int32_t chunks = (a.dim + 7) / 8, per = 1 << lp, l = threadIdx.x & (per - 1);
    const uint32_t step = DROP ? drop_step(a.drop) : 0u;
    // (every lane goes through every round: they join their sums at its end)
    for (int64_t t0 = (int64_t)blockIdx.x * (kThreads >> lp); t0 < a.tokens; t0 += (int64_t)gridDim.x * (kThreads >> lp)) {
        const int64_t t = t0 + (threadIdx.x >> lp);
        const bool live = t < a.tokens;
        for (int32_t j0 = 0; j0 < a.topk; j0 += J) {
            uint32_t r[J];
            float w[J], dot[J];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const bool in = live && j0 + j < a.topk;
                const int64_t of = in ? t * a.topk + j0 + j : 0;
                r[j] = in ? (uint32_t)a.place[of] : ~0u;
                w[j] = a.weights ? a.weights[of] : 1.0f;
                dot[j] = 0.0f;
            }
            // (a choice without a row reads another one of the token's, which no other
            // lane writes where dy is y)
            uint32_t own = ~0u;
#pragma unroll
            for (int j = 0; j < J; ++j) own = r[j] < a.rows ? r[j] : own;
            const bool reads = a.dweights && own < a.rows;
            for (int32_t c = l; live && c < chunks; c += per) {
                const int n = a.dim - c * 8;
                const int64_t at = (int64_t)c * (8 * kElem<DT>);
                const Raw8<DT> dout = get8<DT>(a.x + t * a.ldx + at, n);
                Raw8<DT> y[J];
                if (reads)
#pragma unroll
                    for (int j = 0; j < J; ++j) y[j] = get8<DT>(a.y + (r[j] < a.rows ? r[j] : own) * a.ldy + at, n);
                float d[8];
                floats<DT>(dout, d);
                if constexpr (DROP) drop8(a.drop, step, (uint64_t)(a.drop.first + t * a.dim + c * 8), d);
                if (reads)
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        float v[8];
                        floats<DT>(y[j], v);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            dot[j] = (r[j] < a.rows && i < n) ? __builtin_fmaf(d[i], v[i], dot[j]) : dot[j];
                    }
                if (a.dy)
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        if (r[j] >= a.rows) continue;
                        float v[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] = w[j] * d[i];
                        put8<DT>(a.dy + r[j] * a.lddy + at, n, rounded<DT>(v));
                    }
            }
            if (!a.dweights) continue;
#pragma unroll
            for (int j = 0; j < J; ++j)
                for (int m = (per < 64 ? per : 64) / 2; m; m /= 2) dot[j] += __shfl_xor(dot[j], m);
            if (lp > 6) {
                const int wave = threadIdx.x >> 6;
                __syncthreads();
                if ((threadIdx.x & 63) == 0)
#pragma unroll
                    for (int j = 0; j < J; ++j) part[wave][j] = dot[j];
                __syncthreads();
                if (l == 0)
#pragma unroll
                    for (int j = 0; j < J; ++j)
                        for (int i = 1; i < per >> 6; ++i) dot[j] += part[wave + i][j];
            }
            if (l == 0 && live)
#pragma unroll
                for (int j = 0; j < J; ++j)
                    if (j0 + j < a.topk) a.dweights[t * a.topk + j0 + j] = dot[j];
        }
    }
}

// Lanes for a token's chunks, as a power of two up to `most`.
int lanes_log2(int32_t dim, int most) {
    int lp = 0;
    while (lp < most && (8 << lp) < dim) ++lp;
    return lp;
}
// (a launch has fewer than 2^32 lanes; more tokens go round again)
dim3 token_grid(int64_t tokens, int lp, int32_t dim) {
    const int64_t per = kThreads >> lp, g = (tokens + per - 1) / per, y = ((int64_t)(dim + 7) / 8 + (1 << lp) - 1) >> lp;
    const int64_t most = (int64_t(1) << 23) / y;
    return dim3((unsigned)(g < most ? g : most), (unsigned)y);
}

template <int DT>
hipError_t launch_gather_t(const TokenArgs &a, hipStream_t s) {
    const int lp = lanes_log2(a.dim, 8);
    const dim3 grid = token_grid(a.tokens, lp, a.dim);
    if (a.weights)
        hipLaunchKernelGGL((gather_kernel<DT, true>), grid, dim3(kThreads), 0, s, a, lp);
    else
        hipLaunchKernelGGL((gather_kernel<DT, false>), grid, dim3(kThreads), 0, s, a, lp);
    return hipGetLastError();
}
template <int DT, bool DROP>
hipError_t launch_combine_d(const TokenArgs &a, hipStream_t s) {
    const int lp = lanes_log2(a.dim, 8);
    const dim3 grid = token_grid(a.tokens, lp, a.dim);
    if (a.tokens * (a.topk + (a.x ? 2 : 1)) * a.dim * kElem<DT> > kPastCaches)
        hipLaunchKernelGGL((combine_kernel<DT, DROP, true>), grid, dim3(kThreads), 0, s, a, lp);
    else
        hipLaunchKernelGGL((combine_kernel<DT, DROP, false>), grid, dim3(kThreads), 0, s, a, lp);
    return hipGetLastError();
}
template <int DT>
hipError_t launch_combine_t(const TokenArgs &a, hipStream_t s) {
    return a.drop.bar ? launch_combine_d<DT, true>(a, s) : launch_combine_d<DT, false>(a, s);
}
template <int J, int DT>
hipError_t launch_combine_grad_j(const TokenArgs &a, hipStream_t s) {
    const int lp = lanes_log2(a.dim, 8);
    const dim3 grid(token_grid(a.tokens, lp, 8 << lp).x);
    if (a.drop.bar)
        hipLaunchKernelGGL((combine_grad_kernel<J, DT, true>), grid, dim3(kThreads), 0, s, a, lp);
    else
        hipLaunchKernelGGL((combine_grad_kernel<J, DT, false>), grid, dim3(kThreads), 0, s, a, lp);
    return hipGetLastError();
}
template <int DT>
hipError_t launch_combine_grad_t(const TokenArgs &a, hipStream_t s) {
    if (a.topk <= 2) return launch_combine_grad_j<2, DT>(a, s);
    return a.topk <= 4 ? launch_combine_grad_j<4, DT>(a, s) : launch_combine_grad_j<8, DT>(a, s);
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
