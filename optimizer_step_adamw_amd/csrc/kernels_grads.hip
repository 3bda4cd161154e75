// kernels_grads.hip -- norms of every gradient of a list and of the whole
// list, and clipping of the gradients in place (include/optim_grads.h).
//
// Both are bound by HBM: the norms read every gradient once, the clip reads
// and writes it once.  A workgroup takes one item of the plan's table, a run
// of one tensor's elements, or small tensors, one per wavefront; what it has
// to know stands in one row of a table, so that the data is two memory
// latencies away.  Only one array is walked, so any alignment takes the
// vector path: the elements before the first 16-byte boundary and behind the
// last one go one by one.
//
// Measured on MI355X: norms of 1.1B bf16 372 us (6.1 TB/s; 4 or 16 loads
// of 16 bytes a lane under way instead of 8 are within 2%); norms and clip of
// 667M bf16 569 us (4.0 GB moved, 7.0 TB/s with what the Infinity Cache holds),
// of 4096 x 4096 fp32 38 us; norms of 6000 vectors 9.6 us.
#include "optim_grads.h"

#include "device_common.h"

namespace optim {
namespace {

template <int GK>
constexpr int kGradVec = GK == G_F32 ? 4 : 8;  // elements per 16 bytes
template <int GK>
constexpr int kGradBytes = GK == G_F32 ? 4 : 2;

template <int GK>
__device__ __forceinline__ float grad_value(uint32_t b) {
    if constexpr (GK == G_F32) return __uint_as_float(b);
    else if constexpr (GK == G_BF16) return bf16_to_f32(b);
    else return __half2float(__ushort_as_half((unsigned short)b));
}
template <int GK>
__device__ __forceinline__ uint32_t grad_bits(float x) {
    if constexpr (GK == G_F32) return __float_as_uint(x);
    else if constexpr (GK == G_BF16) return f32_to_bf16_rne(x);
    else return f32_to_f16_rne(x);
}
template <int GK>
__device__ __forceinline__ void unpack(u32x4 u, float (&x)[kGradVec<GK>]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (GK == G_F32) {
            x[i] = grad_value<GK>(u[i]);
        } else {
            x[2 * i] = grad_value<GK>(u[i] & 0xFFFFu);
            x[2 * i + 1] = grad_value<GK>(u[i] >> 16);
        }
    }
}

// Where the 16-byte groups of n elements from p begin, and how many there are.
template <int GK>
__device__ __forceinline__ void grad_groups(const char *p, int32_t n, int32_t &head, int32_t &groups) {
    head = (int32_t)((16 - ((uintptr_t)p & 15)) & 15) / kGradBytes<GK>;
    head = head < n ? head : n;
    groups = (n - head) / kGradVec<GK>;
}

template <int GK>
__device__ __forceinline__ uint32_t grad_load1(const char *p, int64_t e) {
    if constexpr (GK == G_F32) return gp(reinterpret_cast<const uint32_t *>(p))[e];
    else return gp(reinterpret_cast<const uint16_t *>(p))[e];
}
template <int GK>
__device__ __forceinline__ void grad_store1(char *p, int64_t e, uint32_t b) {
    if constexpr (GK == G_F32) gp(reinterpret_cast<uint32_t *>(p))[e] = b;
    else gp(reinterpret_cast<uint16_t *>(p))[e] = (uint16_t)b;
}

// ---------------------------------------------------------------- norms
// A lane's part: the sum in fp64 over fp32 sums of one 16-byte group each, and
// the largest magnitude as fp32 bits, which also tells whether the fp32 part was
// in range and whether all is finite.  A group is a chain of 4 (fp32) or 8
// elements: at most 4 roundings for fp32 squares, the first that of a square;
// 7 for 16-bit ones and for magnitudes, whose first is exact: 7 * 2^-24 of the
// group at most, half of that of a norm of squares, and less on average.  (A
// square in fp64 on every element measured 13% slower on a 1.1B bf16 list.)
struct NormAcc {
    double s = 0.0;
    uint32_t mx = 0;
};

template <int KIND, bool EXACT, int N>
__device__ __forceinline__ void norm_add(const float (&x)[N], NormAcc &a) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t b = __float_as_uint(x[i]) & 0x7FFFFFFFu;
        a.mx = b > a.mx ? b : a.mx;
        if constexpr (KIND == OPTIM_NORM_L2) {
            if constexpr (EXACT) a.s = __builtin_fma((double)x[i], (double)x[i], a.s);
            else t = __builtin_fmaf(x[i], x[i], t);
        } else if constexpr (KIND == OPTIM_NORM_L1) {
            if constexpr (EXACT) a.s += (double)fabsf(x[i]);
            else t += fabsf(x[i]);
        }
    }
    if constexpr (!EXACT && KIND != OPTIM_NORM_INF) a.s += (double)t;
}

// Lane `lane` of `lanes` over n elements from p.
template <int GK, int KIND, bool EXACT, bool KEEP>
__device__ __forceinline__ void norm_walk(const char *p, int32_t n, int32_t lane, int32_t lanes, NormAcc &a) {
    constexpr int V = kGradVec<GK>, U = EXACT ? 1 : 8;
    int32_t head, groups;
    grad_groups<GK>(p, n, head, groups);
    if (lane < head) {
        const float x[1] = {grad_value<GK>(grad_load1<GK>(p, lane))};
        norm_add<KIND, EXACT, 1>(x, a);
    }
    const GMEM u32x4 *q = (const GMEM u32x4 *)gp(p + (int64_t)head * kGradBytes<GK>);
    int32_t i = lane;
    for (; i + (U - 1) * lanes < groups; i += U * lanes) {
        u32x4 u[U];
#pragma unroll
        for (int j = 0; j < U; ++j) u[j] = vload<KEEP ? kStridedKeep : kStrided>(q + i + j * lanes);
#pragma unroll
        for (int j = 0; j < U; ++j) {
            float x[V];
            unpack<GK>(u[j], x);
            norm_add<KIND, EXACT, V>(x, a);
        }
    }
    for (; i < groups; i += lanes) {
        float x[V];
        unpack<GK>(vload<KEEP ? kStridedKeep : kStrided>(q + i), x);
        norm_add<KIND, EXACT, V>(x, a);
    }
    const int32_t e = head + groups * V + lane;
    if (e < n) {
        const float x[1] = {grad_value<GK>(grad_load1<GK>(p, e))};
        norm_add<KIND, EXACT, 1>(x, a);
    }
}

// Magnitudes whose fp32 group sums could leave fp32's range: above 2^62
// eight squares may overflow (a NaN / Inf counts too); where the largest is
// below 2^-40, the others' squares may be subnormal.  Then the elements are
// walked again in fp64.
template <int KIND>
__device__ __forceinline__ bool norm_again(uint32_t mx) {
    if constexpr (KIND == OPTIM_NORM_INF) return false;
    const uint32_t hi = KIND == OPTIM_NORM_L2 ? 0x5E800000u /* 2^62 */ : 0x7B800000u /* 2^120 */;
    return mx >= hi || (mx != 0 && mx < 0x2B800000u /* 2^-40 */);
}

__device__ __forceinline__ void wave_reduce(NormAcc &a) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        a.s += __shfl_xor(a.s, o);
        const uint32_t m = (uint32_t)__shfl_xor((int)a.mx, o);
        a.mx = m > a.mx ? m : a.mx;
    }
}

// What is stored for a tensor or an item: its sum, or its largest
// magnitude's bits (whole numbers, exact in a double; a NaN's are the
// largest).
template <int KIND>
__device__ __forceinline__ double norm_part(const NormAcc &a) {
    return KIND == OPTIM_NORM_INF ? (double)a.mx : a.s;
}
template <int KIND>
__device__ __forceinline__ double norm_join(double x, double y) {
    if constexpr (KIND == OPTIM_NORM_INF) return x > y ? x : y;
    else return x + y;
}
template <int KIND>
__device__ __forceinline__ double norm_of(double sum, double s) {
    if constexpr (KIND == OPTIM_NORM_L2) return sqrt(sum) * s;
    else if constexpr (KIND == OPTIM_NORM_L1) return sum * s;
    else return (double)__uint_as_float((uint32_t)sum) * s;
}

// s * min(1, max_norm / (norm + 1e-6)); s alone without a bar or a finite norm
__device__ __forceinline__ float clip_factor(double norm, double s, double max_norm) {
    double c = 1.0;
    if (max_norm > 0.0 && isfinite(max_norm) && isfinite(norm)) {
        c = max_norm / (norm + 1e-6);
        c = c < 1.0 ? c : 1.0;
    }
    return (float)(s * c);
}

template <int KIND>
__device__ __forceinline__ double block_join(double x, double *red) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) x = norm_join<KIND>(x, __shfl_xor(x, o));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
    __syncthreads();
    double t = red[0];
#pragma unroll
    for (int w = 1; w < kThreads / 64; ++w) t = norm_join<KIND>(t, red[w]);
    __syncthreads();
    return t;
}

// A value that another workgroup of the same launch reads: stored and loaded
// at device scope, past the XCD's own L2.  The writer waits here for its
// store, so an arrival (arrive()) of its workgroup after that means it is
// there; the reader loads after it has seen the arrival.
__device__ __forceinline__ void publish(double *p, double x) {
    __hip_atomic_store(p, x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}
__device__ __forceinline__ double published(const double *p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// body(i, value) for this thread's share of n published values, 8 loads under
// way at a time: each goes to memory past the caches (6000 vectors took 19.8 us
// with one load at a time and the tables behind one more index, 9.6 so).
template <class F>
__device__ __forceinline__ void sums_walk(const double *p, int32_t n, F &&body) {
    constexpr int U = 8;
    for (int32_t i = threadIdx.x; i < n; i += U * kThreads) {
        double y[U];
#pragma unroll
        for (int k = 0; k < U; ++k) y[k] = i + k * kThreads < n ? published(p + i + k * kThreads) : 0.0;
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (i + k * kThreads < n) body(i + k * kThreads, y[k]);
    }
}

// One launch for the whole call.  A workgroup sums its item; the last item
// of a tensor to arrive joins the tensor's partial sums, and the last
// workgroup of the launch turns the tensors' sums into norms, their total
// and the factor.  Every joining runs over the table's order, whoever does
// it, so results repeat bit for bit.
template <int GK, int KIND>
__global__ __launch_bounds__(kThreads) void grad_norms_kernel(GradArgs a, const float *inv_scale, double max_norm,
                                                              float *found_inf, float *norms, float *total,
                                                              float *coef) {
    __shared__ double red[kThreads / 64];
    __shared__ int last;
    if ((int)blockIdx.x < a.nitems) {
        const GradItem it = a.items[blockIdx.x];
        const char *p = static_cast<const char *>(it.g);
        __shared__ uint32_t redm[kThreads / 64];
        NormAcc acc;
        if ((int)blockIdx.x >= a.keep0) norm_walk<GK, KIND, false, true>(p, it.len, threadIdx.x, kThreads, acc);
        else norm_walk<GK, KIND, false, false>(p, it.len, threadIdx.x, kThreads, acc);
#pragma unroll 1
        for (int again = 0;; ++again) {
            wave_reduce(acc);
            if ((threadIdx.x & 63) == 0) {
                red[threadIdx.x >> 6] = acc.s;
                redm[threadIdx.x >> 6] = acc.mx;
            }
            __syncthreads();
            acc = NormAcc{};
#pragma unroll
            for (int w = 0; w < kThreads / 64; ++w) {
                acc.s += red[w];
                acc.mx = redm[w] > acc.mx ? redm[w] : acc.mx;
            }
            __syncthreads();
            if (again || !norm_again<KIND>(acc.mx)) break;
            acc = NormAcc{};
            norm_walk<GK, KIND, true, true>(p, it.len, threadIdx.x, kThreads, acc);
        }
        const double part = norm_part<KIND>(acc);
        if (threadIdx.x == 0) {
            if (found_inf && acc.mx >= 0x7F800000u) *found_inf = 1.0f;
            last = 0;
            if (it.nslots == 1) {
                publish(a.sums + it.tensor, part);
            } else {
                publish(a.partials + it.slot0 + it.slot, part);
                uint32_t *c = a.count + it.tensor;
                if (arrive(c) == (uint32_t)it.nslots - 1) {
                    __hip_atomic_store(c, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                    last = 1;
                }
            }
        }
        __syncthreads();
        if (last) {
            double x = 0.0;
            sums_walk(a.partials + it.slot0, it.nslots, [&](int32_t, double y) { x = norm_join<KIND>(x, y); });
            x = block_join<KIND>(x, red);
            if (threadIdx.x == 0) publish(a.sums + it.tensor, x);
        }
    } else {
        const int32_t k = ((int)blockIdx.x - a.nitems) * (kThreads / 64) + (threadIdx.x >> 6), lane = threadIdx.x & 63;
        if (k < a.nsmall) {
            const GradSmall T = a.small[k];
            const char *p = static_cast<const char *>(T.g);
            NormAcc acc;
            norm_walk<GK, KIND, false, true>(p, T.len, lane, 64, acc);
            wave_reduce(acc);
            if (norm_again<KIND>(acc.mx)) {
                acc = NormAcc{};
                norm_walk<GK, KIND, true, true>(p, T.len, lane, 64, acc);
                wave_reduce(acc);
            }
            if (lane == 0) {
                if (found_inf && acc.mx >= 0x7F800000u) *found_inf = 1.0f;
                publish(a.sums + T.tensor, norm_part<KIND>(acc));
            }
        }
    }
    __syncthreads();  // every wave's sums are out before thread 0 arrives
    if (threadIdx.x == 0) {
        StepArgs step;
        step.done = a.done;  // all that an arrival looks at
        last = last_arrival(step);
    }
    __syncthreads();
    if (!last) return;
    const double s = inv_scale ? (double)*inv_scale : 1.0;
    double x = 0.0;
    sums_walk(a.sums, a.ntensors, [&](int32_t t, double y) {
        if (norms) norms[t] = (float)norm_of<KIND>(y, fabs(s));
        x = norm_join<KIND>(x, y);
    });
    x = block_join<KIND>(x, red);
    if (threadIdx.x == 0) {
        const double n = norm_of<KIND>(x, fabs(s));
        *total = (float)n;
        if (coef) *coef = clip_factor(n, s, max_norm);
    }
}

// ---------------------------------------------------------------- one norm of several
template <int KIND>
__global__ __launch_bounds__(kThreads) void clip_coef_kernel(const float *norms, int64_t count, const float *inv_scale,
                                                             double max_norm, float *total, float *coef) {
    __shared__ double red[kThreads / 64];
    double x = 0.0;
    bool nan = false;
    for (int64_t i = threadIdx.x; i < count; i += kThreads) {
        const double y = (double)norms[i];
        nan |= isnan(y);
        x = norm_join<KIND>(x, KIND == OPTIM_NORM_L2 ? y * y : y);
    }
    x = block_join<KIND>(x, red);
    if (__syncthreads_or(nan)) x = __builtin_nan("");  // a maximum alone would drop it
    if (threadIdx.x == 0) {
        const double s = inv_scale ? (double)*inv_scale : 1.0;
        const double n = KIND == OPTIM_NORM_L2 ? sqrt(x) : x;
        if (total) *total = (float)n;
        if (coef) *coef = clip_factor(n, s, max_norm);
    }
}

// ---------------------------------------------------------------- clip
// The items backwards, with ordinary accesses: the list's end is what the
// norms' read left in the Infinity Cache, and the step that follows meets the
// list's beginning there.  Measured against non-temporal accesses, with the
// norms: 67 MB of fp32 38 us and 43, 1.3 GB of bf16 577 us and 593.
template <int GK>
__device__ __forceinline__ uint32_t clipped(float x, float c) {
    float y = x * c;
    // keeps the product an fp32 value: folded into one instruction with the
    // conversion to fp16 it would not be rounded to fp32 first, and -0 would
    // become +0
    asm("" : "+v"(y));
    return grad_bits<GK>(y);
}

template <int GK>
__device__ __forceinline__ void clip_walk(char *p, int32_t n, int32_t lane, int32_t lanes, float c) {
    constexpr int V = kGradVec<GK>, U = 4;
    int32_t head, groups;
    grad_groups<GK>(p, n, head, groups);
    if (lane < head) grad_store1<GK>(p, lane, clipped<GK>(grad_value<GK>(grad_load1<GK>(p, lane)), c));
    GMEM u32x4 *q = (GMEM u32x4 *)gp(p + (int64_t)head * kGradBytes<GK>);
    auto scaled = [&](u32x4 u) {
        float x[V];
        unpack<GK>(u, x);
        u32x4 y;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (GK == G_F32) y[k] = clipped<GK>(x[k], c);
            else y[k] = clipped<GK>(x[2 * k], c) | clipped<GK>(x[2 * k + 1], c) << 16;
        }
        return y;
    };
    int32_t i = lane;
    for (; i + (U - 1) * lanes < groups; i += U * lanes) {
        u32x4 u[U];
#pragma unroll
        for (int j = 0; j < U; ++j) u[j] = vload<kStridedKeep>(q + i + j * lanes);
#pragma unroll
        for (int j = 0; j < U; ++j) vstore<kStridedKeep>(q + i + j * lanes, scaled(u[j]));
    }
    for (; i < groups; i += lanes) vstore<kStridedKeep>(q + i, scaled(vload<kStridedKeep>(q + i)));
    const int32_t e = head + groups * V + lane;
    if (e < n) grad_store1<GK>(p, e, clipped<GK>(grad_value<GK>(grad_load1<GK>(p, e)), c));
}

template <int GK>
__global__ __launch_bounds__(kThreads) void clip_grads_kernel(GradArgs a, const float *coef, const float *found_inf) {
    const float c = *coef;
    if (c == 1.0f || (found_inf && *found_inf != 0.0f)) return;
    const int32_t b = a.nitems - 1 - (int)blockIdx.x;
    if (b >= 0) {
        const GradItem it = a.items[b];
        clip_walk<GK>(static_cast<char *>(it.g), it.len, threadIdx.x, kThreads, c);
    } else {
        const int32_t k = (-1 - b) * (kThreads / 64) + (threadIdx.x >> 6);
        if (k >= a.nsmall) return;
        const GradSmall T = a.small[k];
        clip_walk<GK>(static_cast<char *>(T.g), T.len, threadIdx.x & 63, 64, c);
    }
}

unsigned grad_grid(const GradArgs &a) { return (unsigned)(a.nitems + (a.nsmall + kThreads / 64 - 1) / (kThreads / 64)); }

template <int GK, int KIND>
void launch_norms_t(const GradArgs &a, const float *inv_scale, double max_norm, float *found_inf, float *norms,
                    float *total, float *coef, hipStream_t s) {
    const unsigned grid = grad_grid(a) > 0 ? grad_grid(a) : 1u;  // an empty list has a total too
    LAUNCH_TRACED((grad_norms_kernel<GK, KIND>), grid, kThreads, s, a, inv_scale, max_norm, found_inf, norms, total,
                  coef);
}

template <int GK>
void launch_norms_k(const GradArgs &a, int kind, const float *inv_scale, double max_norm, float *found_inf,
                    float *norms, float *total, float *coef, hipStream_t s) {
    if (kind == OPTIM_NORM_L2)
        launch_norms_t<GK, OPTIM_NORM_L2>(a, inv_scale, max_norm, found_inf, norms, total, coef, s);
    else if (kind == OPTIM_NORM_L1)
        launch_norms_t<GK, OPTIM_NORM_L1>(a, inv_scale, max_norm, found_inf, norms, total, coef, s);
    else
        launch_norms_t<GK, OPTIM_NORM_INF>(a, inv_scale, max_norm, found_inf, norms, total, coef, s);
}

}  // namespace

hipError_t launch_grad_norms(const GradArgs &a, int gk, int kind, const float *inv_scale, double max_norm,
                             float *found_inf, float *norms, float *total, float *coef, hipStream_t s) {
    if (gk == G_F32)
        launch_norms_k<G_F32>(a, kind, inv_scale, max_norm, found_inf, norms, total, coef, s);
    else if (gk == G_BF16)
        launch_norms_k<G_BF16>(a, kind, inv_scale, max_norm, found_inf, norms, total, coef, s);
    else
        launch_norms_k<G_F16>(a, kind, inv_scale, max_norm, found_inf, norms, total, coef, s);
    return hipGetLastError();
}

hipError_t launch_clip_grads(const GradArgs &a, int gk, const float *coef, const float *found_inf, hipStream_t s) {
    if (grad_grid(a) == 0) return hipSuccess;
    if (gk == G_F32)
        LAUNCH_TRACED((clip_grads_kernel<G_F32>), grad_grid(a), kThreads, s, a, coef, found_inf);
    else if (gk == G_BF16)
        LAUNCH_TRACED((clip_grads_kernel<G_BF16>), grad_grid(a), kThreads, s, a, coef, found_inf);
    else
        LAUNCH_TRACED((clip_grads_kernel<G_F16>), grad_grid(a), kThreads, s, a, coef, found_inf);
    return hipGetLastError();
}

hipError_t launch_clip_coef(const float *norms, int64_t count, int kind, const float *inv_scale, double max_norm,
                            float *total, float *coef, hipStream_t s) {
    if (kind == OPTIM_NORM_L2)
        hipLaunchKernelGGL((clip_coef_kernel<OPTIM_NORM_L2>), dim3(1), dim3(kThreads), 0, s, norms, count, inv_scale,
                           max_norm, total, coef);
    else if (kind == OPTIM_NORM_L1)
        hipLaunchKernelGGL((clip_coef_kernel<OPTIM_NORM_L1>), dim3(1), dim3(kThreads), 0, s, norms, count, inv_scale,
                           max_norm, total, coef);
    else
        hipLaunchKernelGGL((clip_coef_kernel<OPTIM_NORM_INF>), dim3(1), dim3(kThreads), 0, s, norms, count, inv_scale,
                           max_norm, total, coef);
    return hipGetLastError();
}

}  // namespace optim
