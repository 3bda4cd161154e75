// experts.h -- what the entry points of optim_route.h and optim_dropout.h hand
// to their kernels.
#pragma once

#include "optim_route.h"
#include "philox.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace optim {

// Bytes of a call from which on reads of several arrays and the write pass by the
// caches.  Measured on MI355X, by them and through them: dropout with residual, bf16,
// 260 MB 40.4 and 37.8 us, 384 MB 59.7 and 66.7, 805 MB 128.8 and 141.9; combining
// two rows of 4096 and a residual, 295 MB 50.4 and 46.7, 537 MB 90.0 and 97.9.
constexpr int64_t kPastCaches = int64_t(320) << 20;

constexpr int32_t kMaxExperts = 1024, kMaxTopk = 32, kMaxExpertGroups = 64;

struct RouteArgs {
    const char *logits;
    int64_t ldl;          // bytes between rows
    const float *bias;    // or NULL
    int32_t *idx;
    float *weights;
    int64_t tokens;
    int32_t experts, topk, score, renormalise, groups, top_groups, group_best;
    float scale;
};
hipError_t launch_route(const RouteArgs &a, int dtype, hipStream_t s);

struct RouteGradArgs {
    const char *logits;
    int64_t ldl;          // bytes between rows
    const int32_t *idx;
    const float *dweights;
    char *dlogits;
    int64_t ldd;          // bytes between rows
    int64_t tokens;
    int32_t experts, topk, score, renormalise;
    float scale;
};
hipError_t launch_route_grad(const RouteGradArgs &a, int dtype, hipStream_t s);

hipError_t launch_route_bias(const int32_t *offsets, int32_t experts, float *bias, const float *rate,
                             const float *found_inf, hipStream_t s);

struct RowsArgs {
    const int32_t *idx;
    int32_t *offsets, *place, *order;  // order or NULL
    int32_t *counts;                   // [blocks], rows_workspace() bytes; NULL where one block does it all
    int32_t n, experts, chunk, blocks;
};
// Choices a workgroup takes, a multiple of 1024, and workgroups.
struct RowsShape {
    int32_t chunk, blocks;
};
RowsShape rows_shape(int64_t n);
size_t rows_workspace(RowsShape shape, int32_t experts);
hipError_t launch_rows(const RowsArgs &a, hipStream_t s);

// Matrices of `dim` columns; distances in bytes.
struct TokenArgs {
    const char *x;        // by token: what is gathered, the residual, or dout
    char *out;            // by token
    const char *y;        // rows read
    char *dy;             // rows written
    int64_t ldx, ldo, ldy, lddy;
    const int32_t *place;
    const float *weights;
    float *dweights;
    DropArgs drop;        // bar 0: none
    int64_t tokens;
    int32_t topk, dim;
    uint32_t rows;
};
hipError_t launch_gather(const TokenArgs &a, int dtype, hipStream_t s);
hipError_t launch_combine(const TokenArgs &a, int dtype, hipStream_t s);
hipError_t launch_combine_grad(const TokenArgs &a, int dtype, hipStream_t s);

hipError_t launch_dropout(const char *x, const char *residual, char *out, int64_t n, const DropArgs &d, int dtype,
                          hipStream_t s);

}  // namespace optim
