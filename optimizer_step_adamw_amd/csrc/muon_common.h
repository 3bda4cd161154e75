// muon_common.h -- what the kernels of the Muon step share: the momentum's
// direction, values as sums of two fp16 numbers, the update.
#pragma once

#include "optim_muon.h"

#include "tiles.h"

namespace optim {
namespace {

// X, A and B are stored times 2^12: bounded by 15 (checked on the host) they
// stay below fp16's 65504, and a typical element of a 4096 x 4096 X, 2^-12 at
// the start and 2^-6 at the end, has both its parts well above fp16's
// smallest subnormal, 2^-24.  An element below 2^-15 may have a subnormal low
// part and is then off by up to 2^-37: rows 1e-6 of the others' size get their
// update to 2e-4 (64 x 64) to 1.3e-2 (4096 x 4096) of it only.  (Low parts with
// a scale of their own would keep 22 bits there, but need sums of their own.)
constexpr float kMuonScale = 4096.0f, kMuonUnscale = 1.0f / 4096.0f;

__device__ __forceinline__ bool skipped(const StepArgs &a) {
    return a.prep.found_inf && *a.prep.found_inf != 0.0f;
}

template <int N>
__device__ __forceinline__ void muon_u(const float (&g)[N], float (&m)[N], float mu, bool nesterov, float (&u)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) u[i] = nesterov ? g[i] + mu * m[i] : m[i];
}

__device__ __forceinline__ void split4(const float (&x)[4], uint2 &hi, uint2 &lo) {
    f16x4 h, l;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        _Float16 a, b;
        split2(x[i], a, b);
        h[i] = a;
        l[i] = b;
    }
    hi = __builtin_bit_cast(uint2, h);
    lo = __builtin_bit_cast(uint2, l);
}

// Factor of the update of a rows x cols matrix.
__device__ __forceinline__ double muon_scale(int32_t kind, double r, double c) {
    return kind == OPTIM_MUON_SCALE_RMS      ? 0.2 * sqrt(r > c ? r : c)
           : kind == OPTIM_MUON_SCALE_ASPECT ? sqrt(r > c ? r / c : 1.0)
                                             : 1.0;
}

// The factor kMuonScale / (||u|| + eps) of a matrix, in fp64: with eps 0 and a
// small u it may leave fp32's range; the scaled u does not.
__device__ __forceinline__ double muon_factor(double sum, double eps) {
    const double n = sqrt(sum) + eps;
    return n == 0.0 ? 0.0 : (double)kMuonScale / n;
}

// A parameter's stores with ordinary accesses: a tile's rows are 64-byte runs,
// which non-temporal stores would write one by one.
template <int PK, int N>
__device__ __forceinline__ void store_p_keep(const TensorDesc &T, int64_t e, const float (&p)[N]) {
    if constexpr (PK == P_F32) {
        stf<N, kStridedKeep>(static_cast<float *>(T.p), e, p);
    } else {
        uint32_t b[N], r[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if constexpr (PK == P_BF16R) rem_split(p[k], b[k], r[k]);
            else b[k] = PK == P_MBF16 ? f32_to_bf16_rne(p[k]) : f32_to_f16_rne(p[k]);
        }
        sth<N, kStridedKeep>(static_cast<uint16_t *>(T.p), e, b);
        if constexpr (PK == P_BF16R) sth<N, kStridedKeep>(T.rem, e, r);
        else stf<N, kStridedKeep>(T.master, e, p);
    }
}

}  // namespace
}  // namespace optim
