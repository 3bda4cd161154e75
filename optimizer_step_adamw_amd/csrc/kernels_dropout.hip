// kernels_dropout.hip -- dropout from a counter (optim_dropout).
//
// A lane takes the elements of one block of the generator, eight neighbours whose
// places begin at a multiple of eight: one call of the generator, 20 products of
// 32 bits for eight draws of 16, so that a mask costs less than the 16 or 32 bytes
// read and written beside it.  (32 bits a draw would double that, for shares finer
// than 1/65536.)  The mask is nowhere in memory, and no lane needs another's.
//
// Bound by HBM: 134M bf16 with residual 124-129 us (805 MB, 6.2-6.5 TB/s), without
// one 88-90 us (537 MB, 6.0), 201M 132 (805 MB, 6.1), 134M fp32 184-187 us (1074 MB,
// 5.8); 999 elements 2.5 us, the launch.  Past the caches (elems.h: NT) where there is
// a residual and much of it: without one it gains nothing (537 MB bf16 88.6-92.7 us
// past them, 89.3-89.8 through them, 805 MB 132.0-133.3 and 131.6-132.0, 1074 MB
// fp32 189 and 186).
#include "elems.h"

namespace optim {
namespace {

template <int DT, bool RES, bool NT>
__global__ __launch_bounds__(kThreads) void dropout_kernel(const char *x, const char *res, char *out, int64_t n, DropArgs d) {
    const uint32_t step = drop_step(d);
    const int64_t lead = d.first & 7;  // places of the first block that lie before element 0
    const int64_t blocks = (lead + n + 7) >> 3;
    for (int64_t b = (int64_t)blockIdx.x * kThreads + threadIdx.x; b < blocks; b += (int64_t)gridDim.x * kThreads) {
        const int64_t e = b * 8 - lead;
        const Words w = philox((uint64_t)((d.first >> 3) + b), step, d.site, d.seed);
        if (e >= 0 && e + 8 <= n) {
            float v[8], r[8];
            floats<DT>(load8<DT, NT>(x + e * kElem<DT>), v);
            if constexpr (RES) floats<DT>(load8<DT, NT>(res + e * kElem<DT>), r);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = draw_of(w, i) < d.bar ? 0.0f : v[i] * d.scale;
                if constexpr (RES) v[i] = r[i] + v[i];
            }
            store8<DT, NT>(out + e * kElem<DT>, rounded<DT>(v));
            continue;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // the first or the last block
            if (e + i < 0 || e + i >= n) continue;
            float v = draw_of(w, i) < d.bar ? 0.0f : element<DT>(x + (e + i) * kElem<DT>) * d.scale;
            if constexpr (RES) v = element<DT>(res + (e + i) * kElem<DT>) + v;
            put_element<DT>(out + (e + i) * kElem<DT>, v);
        }
    }
}

template <int DT, bool RES>
hipError_t launch_dropout_r(const char *x, const char *residual, char *out, int64_t n, const DropArgs &d, hipStream_t s) {
    const int64_t blocks = (n + 14) / 8;
    const int64_t g = (blocks + kThreads - 1) / kThreads;
    const dim3 grid((unsigned)(g < (1 << 23) ? g : 1 << 23));
    if (RES && n * kElem<DT> * 3 > kPastCaches)
        hipLaunchKernelGGL((dropout_kernel<DT, RES, RES>), grid, dim3(kThreads), 0, s, x, residual, out, n, d);
    else
        hipLaunchKernelGGL((dropout_kernel<DT, RES, false>), grid, dim3(kThreads), 0, s, x, residual, out, n, d);
    return hipGetLastError();
}
template <int DT>
hipError_t launch_dropout_t(const char *x, const char *residual, char *out, int64_t n, const DropArgs &d, hipStream_t s) {
    return residual ? launch_dropout_r<DT, true>(x, residual, out, n, d, s) : launch_dropout_r<DT, false>(x, residual, out, n, d, s);
}

}  // namespace

hipError_t launch_dropout(const char *x, const char *residual, char *out, int64_t n, const DropArgs &d, int dtype,
                          hipStream_t s) {
    if (dtype == OPTIM_F32) return launch_dropout_t<OPTIM_F32>(x, residual, out, n, d, s);
    if (dtype == OPTIM_BF16) return launch_dropout_t<OPTIM_BF16>(x, residual, out, n, d, s);
    return launch_dropout_t<OPTIM_F16>(x, residual, out, n, d, s);
}

}  // namespace optim
