// elems.h -- eight neighbouring elements of an fp32, bf16 or fp16 row at a time,
// as raw bits and as floats.  Rows may begin at any element: gfx950 takes
// 16-byte accesses at any element's alignment.
#pragma once

#include "device_common.h"
#include "experts.h"

namespace optim {
namespace {

typedef u32x4 __attribute__((aligned(2))) u32x4_at2;
typedef u32x4 __attribute__((aligned(4))) u32x4_at4;
typedef u32x2 __attribute__((aligned(2))) u32x2_at2;

// DT: OPTIM_F32, OPTIM_BF16 or OPTIM_F16
template <int DT>
constexpr int kElem = DT == OPTIM_F32 ? 4 : 2;

template <int DT>
struct Raw8 {
    u32x4 v[DT == OPTIM_F32 ? 2 : 1];
};

// NT: past the caches, for what is larger than they are.  DT: whose alignment the
// address has.
template <int DT, bool NT>
__device__ __forceinline__ u32x4 load_v(const char *p) {
    if constexpr (DT == OPTIM_F32) {
        const GMEM u32x4_at4 *q = (const GMEM u32x4_at4 *)gp(p);
        if constexpr (NT) return __builtin_nontemporal_load(q);
        else return *q;
    } else {
        const GMEM u32x4_at2 *q = (const GMEM u32x4_at2 *)gp(p);
        if constexpr (NT) return __builtin_nontemporal_load(q);
        else return *q;
    }
}
template <int DT, bool NT>
__device__ __forceinline__ void store_v(char *p, u32x4 x) {
    if constexpr (DT == OPTIM_F32) {
        GMEM u32x4_at4 *q = (GMEM u32x4_at4 *)gp(p);
        if constexpr (NT) __builtin_nontemporal_store(x, q);
        else *q = x;
    } else {
        GMEM u32x4_at2 *q = (GMEM u32x4_at2 *)gp(p);
        if constexpr (NT) __builtin_nontemporal_store(x, q);
        else *q = x;
    }
}
template <int DT, bool NT = false>
__device__ __forceinline__ Raw8<DT> load8(const char *p) {
    Raw8<DT> r;
    if constexpr (DT == OPTIM_F32) {
        r.v[0] = load_v<DT, NT>(p);
        r.v[1] = load_v<DT, NT>(p + 16);
    } else {
        r.v[0] = load_v<DT, NT>(p);
    }
    return r;
}
template <int DT, bool NT = false>
__device__ __forceinline__ void store8(char *p, const Raw8<DT> &r) {
    if constexpr (DT == OPTIM_F32) {
        store_v<DT, NT>(p, r.v[0]);
        store_v<DT, NT>(p + 16, r.v[1]);
    } else {
        store_v<DT, NT>(p, r.v[0]);
    }
}

// The first n (below 8) of eight; the others are zero, or stay as they are.
template <int DT>
__device__ __forceinline__ Raw8<DT> load_some(const char *p, int n) {
    Raw8<DT> r{};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i >= n) continue;
        if constexpr (DT == OPTIM_F32) r.v[i / 4][i % 4] = ((const GMEM uint32_t *)gp(p))[i];
        else r.v[0][i / 2] |= (uint32_t)((const GMEM uint16_t *)gp(p))[i] << (i % 2 * 16);
    }
    return r;
}
template <int DT>
__device__ __forceinline__ void store_some(char *p, int n, const Raw8<DT> &r) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i >= n) continue;
        if constexpr (DT == OPTIM_F32) ((GMEM uint32_t *)gp(p))[i] = r.v[i / 4][i % 4];
        else ((GMEM uint16_t *)gp(p))[i] = (uint16_t)(r.v[0][i / 2] >> (i % 2 * 16));
    }
}
// n: elements from p on that exist.
template <int DT, bool NT = false>
__device__ __forceinline__ Raw8<DT> get8(const char *p, int n) { return n >= 8 ? load8<DT, NT>(p) : load_some<DT>(p, n); }
template <int DT, bool NT = false>
__device__ __forceinline__ void put8(char *p, int n, const Raw8<DT> &r) {
    if (n >= 8) store8<DT, NT>(p, r);
    else store_some<DT>(p, n, r);
}

__device__ __forceinline__ float f16_to_f32(uint32_t h) { return (float)__builtin_bit_cast(_Float16, (uint16_t)h); }

template <int DT>
__device__ __forceinline__ void floats(const Raw8<DT> &r, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (DT == OPTIM_F32) x[i] = __uint_as_float(r.v[i / 4][i % 4]);
        else if constexpr (DT == OPTIM_BF16) x[i] = i % 2 ? __uint_as_float(r.v[0][i / 2] & 0xFFFF0000u) : __uint_as_float(r.v[0][i / 2] << 16);
        else x[i] = f16_to_f32(r.v[0][i / 2] >> (i % 2 * 16) & 0xFFFFu);
    }
}
// Rounded to nearest even, NaN stays NaN.
template <int DT>
__device__ __forceinline__ Raw8<DT> rounded(const float (&x)[8]) {
    Raw8<DT> r;
    if constexpr (DT == OPTIM_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r.v[i / 4][i % 4] = __float_as_uint(x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t lo, hi;
            if constexpr (DT == OPTIM_BF16) {
                lo = __builtin_bit_cast(uint16_t, (__bf16)x[2 * i]);
                hi = __builtin_bit_cast(uint16_t, (__bf16)x[2 * i + 1]);
            } else {
                lo = f32_to_f16_rne(x[2 * i]);
                hi = f32_to_f16_rne(x[2 * i + 1]);
            }
            r.v[0][i] = lo | hi << 16;
        }
    }
    return r;
}

// One element as a float.
template <int DT>
__device__ __forceinline__ float element(const char *p) {
    if constexpr (DT == OPTIM_F32) return *(const GMEM float *)gp(p);
    else if constexpr (DT == OPTIM_BF16) return bf16_to_f32(*(const GMEM uint16_t *)gp(p));
    else return f16_to_f32(*(const GMEM uint16_t *)gp(p));
}
template <int DT>
__device__ __forceinline__ void put_element(char *p, float x) {
    if constexpr (DT == OPTIM_F32) *(GMEM float *)gp(p) = x;
    else if constexpr (DT == OPTIM_BF16) *(GMEM uint16_t *)gp(p) = __builtin_bit_cast(uint16_t, (__bf16)x);
    else *(GMEM uint16_t *)gp(p) = (uint16_t)f32_to_f16_rne(x);
}

__device__ __forceinline__ uint32_t drop_step(const DropArgs &d) { return d.step ? (uint32_t)*d.step : 0u; }

// Eight elements from place q on, dropped or scaled.
__device__ __forceinline__ void drop8(const DropArgs &d, uint32_t step, uint64_t q, float (&x)[8]) {
    const Words w = draws8(q, step, d.site, d.seed);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = draw_of(w, i) < d.bar ? 0.0f : x[i] * d.scale;
}

}  // namespace
}  // namespace optim
