// api_experts.cpp -- C ABI of routing, the experts' rows and dropout: checks of
// arguments and launches.  Declared in include/optim_route.h and
// include/optim_dropout.h.
#include "api_common.h"
#include "experts.h"
#include "optim_dropout.h"
#include "optim_route.h"

#include <cmath>

using namespace optim;

namespace {

constexpr int64_t kMaxSide = (int64_t(1) << 24) - 1;  // columns, distance between rows
constexpr int64_t kMaxElems = int64_t(1) << 48;
constexpr int64_t kMaxPlace = int64_t(1) << 60;

size_t size_of(int32_t dtype) { return dtype == OPTIM_F32 ? 4 : 2; }

int check_dtype(int32_t dtype) {
    if (dtype != OPTIM_F32 && dtype != OPTIM_BF16 && dtype != OPTIM_F16)
        return fail(OPTIM_EDTYPE, "dtype must be OPTIM_F32, OPTIM_BF16 or OPTIM_F16");
    return OPTIM_OK;
}

int check_choices(int64_t tokens, int32_t topk) {
    if (tokens < 0) return fail(OPTIM_EINVAL, "negative tokens");
    if (topk < 1 || topk > kMaxTopk) return fail(OPTIM_EINVAL, "topk must be in [1, 32]");
    if (tokens > INT32_MAX / topk) return fail(OPTIM_EINVAL, "tokens * topk must be below 2^31");
    return OPTIM_OK;
}

int check_experts(int32_t experts) {
    if (experts < 1 || experts > kMaxExperts) return fail(OPTIM_EINVAL, "experts must be in [1, 1024]");
    return OPTIM_OK;
}

int check_ld(int64_t ld, int64_t cols, const char *what) {
    if (ld < cols || ld > kMaxSide)
        return fail(OPTIM_EINVAL, std::string(what) + " must be at least the row's length, and below 2^24");
    return OPTIM_OK;
}

int check_route_hp(const optim_route_hp *hp, int32_t experts) {
    if (!hp) return fail(OPTIM_EINVAL, "hp is NULL");
    if (hp->score != OPTIM_ROUTE_SOFTMAX && hp->score != OPTIM_ROUTE_SIGMOID) return fail(OPTIM_EINVAL, "unknown score");
    if (hp->groups < 1 || hp->groups > kMaxExpertGroups || experts % hp->groups)
        return fail(OPTIM_EINVAL, "groups must be in [1, 64] and divide experts");
    if (hp->top_groups < 1 || hp->top_groups > hp->groups) return fail(OPTIM_EINVAL, "top_groups must be in [1, groups]");
    if (hp->group_best != 1 && hp->group_best != 2) return fail(OPTIM_EINVAL, "group_best must be 1 or 2");
    if (hp->topk > experts / hp->groups * hp->top_groups)
        return fail(OPTIM_EINVAL, "topk is above the number of experts in top_groups groups");
    if (!std::isfinite((float)hp->scale)) return fail(OPTIM_EINVAL, "scale must be finite, in fp32 as well");
    return OPTIM_OK;
}

// `n` elements of dropout; d.bar 0 where nothing is dropped.
int check_drop(const optim_dropout_hp *hp, const int32_t *step_dev, DropArgs &d) {
    if (!(hp->p >= 0.0 && hp->p < 1.0)) return fail(OPTIM_EINVAL, "p must be in [0, 1)");
    if (hp->first < 0 || hp->first > kMaxPlace) return fail(OPTIM_EINVAL, "first must be in [0, 2^60]");
    if (!aligned(step_dev, 4)) return fail(OPTIM_EALIGN, "step misaligned");
    const double bar = std::floor(65536.0 * hp->p + 0.5);
    d.seed = hp->seed;
    d.first = hp->first;
    d.step = step_dev;
    d.site = hp->site;
    d.bar = bar < 65535.0 ? (uint32_t)bar : 65535u;
    d.scale = (float)(65536.0 / (65536.0 - d.bar));
    return OPTIM_OK;
}

struct Ranges {
    std::vector<Range> all;
    Ranges() { all.reserve(8); }
    void add(const void *p, size_t bytes, bool written, const char *what) {
        if (p && bytes) all.push_back({(uintptr_t)p, (uintptr_t)p + bytes, written, 0, what});
    }
    // rows of `cols` elements, ld elements apart
    void rows(const void *p, int64_t n, int64_t ld, int64_t cols, size_t size, bool written, const char *what) {
        if (n > 0) add(p, ((size_t)(n - 1) * ld + cols) * size, written, what);
    }
};

int check_rows_count(int64_t rows) {
    if (rows < 0 || rows > INT32_MAX) return fail(OPTIM_EINVAL, "rows must be in [0, 2^31)");
    return OPTIM_OK;
}

int check_dim(int64_t dim) {
    if (dim < 0 || dim > kMaxSide) return fail(OPTIM_EINVAL, "dim must be in [0, 2^24)");
    return OPTIM_OK;
}

}  // namespace

extern "C" {

int optim_dropout(const void *x_dev, int32_t dtype, int64_t n, const void *residual_dev, const optim_dropout_hp *hp,
                  const int32_t *step_dev, void *out_dev, void *stream) try {
    if (const int rc = check_dtype(dtype)) return rc;
    if (n < 0 || n > kMaxElems) return fail(OPTIM_EINVAL, "n must be in [0, 2^48]");
    if (!hp) return fail(OPTIM_EINVAL, "hp is NULL");
    DropArgs d{};
    if (const int rc = check_drop(hp, step_dev, d)) return rc;
    if (n == 0) return OPTIM_OK;
    if (!x_dev || !out_dev) return fail(OPTIM_EINVAL, "NULL buffer");
    const size_t sz = size_of(dtype);
    if (!aligned(x_dev, sz) || !aligned(residual_dev, sz) || !aligned(out_dev, sz))
        return fail(OPTIM_EALIGN, "buffer misaligned");
    Ranges r;
    if (x_dev != out_dev) r.add(x_dev, n * sz, false, "x");
    if (residual_dev != out_dev) r.add(residual_dev, n * sz, false, "residual");
    r.add(step_dev, 4, false, "step");
    r.add(out_dev, n * sz, true, "out");
    if (const int rc = check_overlaps(r.all)) return rc;
    HIP_OK(launch_dropout(static_cast<const char *>(x_dev), static_cast<const char *>(residual_dev),
                          static_cast<char *>(out_dev), n, d, dtype, static_cast<hipStream_t>(stream)));
    return OPTIM_OK;
} OPTIM_CATCH

int optim_route(const void *logits_dev, int64_t ldl, int32_t dtype, int64_t tokens, int32_t experts,
                const float *bias_dev, const optim_route_hp *hp, int32_t *idx_dev, float *weights_dev,
                void *stream) try {
    if (const int rc = check_dtype(dtype)) return rc;
    if (const int rc = check_experts(experts)) return rc;
    if (const int rc = check_route_hp(hp, experts)) return rc;
    if (const int rc = check_choices(tokens, hp->topk)) return rc;
    if (const int rc = check_ld(ldl, experts, "ldl")) return rc;
    if (tokens == 0) return OPTIM_OK;
    if (!logits_dev || !idx_dev || !weights_dev) return fail(OPTIM_EINVAL, "NULL buffer");
    const size_t sz = size_of(dtype), slots = (size_t)tokens * hp->topk;
    if (!aligned(logits_dev, sz) || !aligned(bias_dev, 4) || !aligned(idx_dev, 4) || !aligned(weights_dev, 4))
        return fail(OPTIM_EALIGN, "buffer misaligned");
    Ranges r;
    r.rows(logits_dev, tokens, ldl, experts, sz, false, "logits");
    r.add(bias_dev, (size_t)experts * 4, false, "bias");
    r.add(idx_dev, slots * 4, true, "idx");
    r.add(weights_dev, slots * 4, true, "weights");
    if (const int rc = check_overlaps(r.all)) return rc;
    RouteArgs a{};
    a.logits = static_cast<const char *>(logits_dev);
    a.ldl = ldl * (int64_t)sz;
    a.bias = bias_dev;
    a.idx = idx_dev;
    a.weights = weights_dev;
    a.tokens = tokens;
    a.experts = experts;
    a.topk = hp->topk;
    a.score = hp->score;
    a.renormalise = hp->renormalise != 0;
    a.groups = hp->groups;
    a.top_groups = hp->top_groups;
    a.group_best = hp->group_best;
    a.scale = (float)hp->scale;
    HIP_OK(launch_route(a, dtype, static_cast<hipStream_t>(stream)));
    return OPTIM_OK;
} OPTIM_CATCH

int optim_route_grad(const void *logits_dev, int64_t ldl, int32_t dtype, int64_t tokens, int32_t experts,
                     const optim_route_hp *hp, const int32_t *idx_dev, const float *dweights_dev, void *dlogits_dev,
                     int64_t ldd, void *stream) try {
    if (const int rc = check_dtype(dtype)) return rc;
    if (const int rc = check_experts(experts)) return rc;
    if (const int rc = check_route_hp(hp, experts)) return rc;
    if (const int rc = check_choices(tokens, hp->topk)) return rc;
    if (const int rc = check_ld(ldl, experts, "ldl")) return rc;
    if (const int rc = check_ld(ldd, experts, "ldd")) return rc;
    if (tokens == 0) return OPTIM_OK;
    if (!logits_dev || !idx_dev || !dweights_dev || !dlogits_dev) return fail(OPTIM_EINVAL, "NULL buffer");
    const size_t sz = size_of(dtype), slots = (size_t)tokens * hp->topk;
    if (!aligned(logits_dev, sz) || !aligned(idx_dev, 4) || !aligned(dweights_dev, 4) || !aligned(dlogits_dev, sz))
        return fail(OPTIM_EALIGN, "buffer misaligned");
    Ranges r;
    r.rows(logits_dev, tokens, ldl, experts, sz, false, "logits");
    r.add(idx_dev, slots * 4, false, "idx");
    r.add(dweights_dev, slots * 4, false, "dweights");
    r.rows(dlogits_dev, tokens, ldd, experts, sz, true, "dlogits");
    if (const int rc = check_overlaps(r.all)) return rc;
    RouteGradArgs a{};
    a.logits = static_cast<const char *>(logits_dev);
    a.ldl = ldl * (int64_t)sz;
    a.idx = idx_dev;
    a.dweights = dweights_dev;
    a.dlogits = static_cast<char *>(dlogits_dev);
    a.ldd = ldd * (int64_t)sz;
    a.tokens = tokens;
    a.experts = experts;
    a.topk = hp->topk;
    a.score = hp->score;
    a.renormalise = hp->renormalise != 0;
    a.scale = (float)hp->scale;
    HIP_OK(launch_route_grad(a, dtype, static_cast<hipStream_t>(stream)));
    return OPTIM_OK;
} OPTIM_CATCH

int optim_step_route_bias(const int32_t *offsets_dev, int32_t experts, float *bias_dev, const float *rate_dev,
                          const float *found_inf_dev, void *stream) try {
    if (const int rc = check_experts(experts)) return rc;
    if (!offsets_dev || !bias_dev || !rate_dev) return fail(OPTIM_EINVAL, "NULL buffer");
    if (!aligned(offsets_dev, 4) || !aligned(bias_dev, 4) || !aligned(rate_dev, 4) || !aligned(found_inf_dev, 4))
        return fail(OPTIM_EALIGN, "buffer misaligned");
    Ranges r;
    r.add(offsets_dev, ((size_t)experts + 1) * 4, false, "offsets");
    r.add(rate_dev, 4, false, "rate");
    r.add(found_inf_dev, 4, false, "found_inf");
    r.add(bias_dev, (size_t)experts * 4, true, "bias");
    if (const int rc = check_overlaps(r.all)) return rc;
    HIP_OK(launch_route_bias(offsets_dev, experts, bias_dev, rate_dev, found_inf_dev, static_cast<hipStream_t>(stream)));
    return OPTIM_OK;
} OPTIM_CATCH

int optim_route_rows_workspace(int64_t tokens, int32_t topk, int32_t experts, size_t *bytes) try {
    if (!bytes) return fail(OPTIM_EINVAL, "bytes is NULL");
    if (const int rc = check_experts(experts)) return rc;
    if (const int rc = check_choices(tokens, topk)) return rc;
    *bytes = rows_workspace(rows_shape(tokens * topk), experts);
    return OPTIM_OK;
} OPTIM_CATCH

int optim_route_rows(const int32_t *idx_dev, int64_t tokens, int32_t topk, int32_t experts, int32_t *offsets_dev,
                     int32_t *place_dev, int32_t *order_dev, void *workspace, size_t workspace_bytes,
                     void *stream) try {
    if (const int rc = check_experts(experts)) return rc;
    if (const int rc = check_choices(tokens, topk)) return rc;
    const int64_t n = tokens * topk;
    if (!offsets_dev || (n > 0 && (!idx_dev || !place_dev))) return fail(OPTIM_EINVAL, "NULL buffer");
    if (!aligned(idx_dev, 4) || !aligned(offsets_dev, 4) || !aligned(place_dev, 4) || !aligned(order_dev, 4))
        return fail(OPTIM_EALIGN, "buffer misaligned");
    const RowsShape shape = rows_shape(n);
    const size_t need = rows_workspace(shape, experts);
    if (need) {
        if (!workspace || !aligned(workspace, 256))
            return fail(OPTIM_EWORKSPACE, "workspace must be a 256-byte aligned device pointer");
        if (workspace_bytes < need)
            return fail(OPTIM_EWORKSPACE, "workspace too small: need " + std::to_string(need) + " bytes, got " +
                                              std::to_string(workspace_bytes));
    }
    Ranges r;
    r.add(idx_dev, (size_t)n * 4, false, "idx");
    r.add(offsets_dev, ((size_t)experts + 1) * 4, true, "offsets");
    r.add(place_dev, (size_t)n * 4, true, "place");
    r.add(order_dev, (size_t)n * 4, true, "order");
    r.add(need ? workspace : nullptr, need, true, "workspace");
    if (const int rc = check_overlaps(r.all)) return rc;
    RowsArgs a{};
    a.idx = idx_dev;
    a.offsets = offsets_dev;
    a.place = place_dev;
    a.order = order_dev;
    a.counts = need ? static_cast<int32_t *>(workspace) : nullptr;
    a.n = (int32_t)n;
    a.experts = experts;
    a.chunk = shape.chunk;
    a.blocks = shape.blocks;
    HIP_OK(launch_rows(a, static_cast<hipStream_t>(stream)));
    return OPTIM_OK;
} OPTIM_CATCH

int optim_expert_gather(const void *x_dev, int64_t ldx, int32_t dtype, const int32_t *place_dev,
                        const float *weights_dev, int64_t tokens, int32_t topk, int64_t dim, void *y_dev, int64_t ldy,
                        int64_t rows, void *stream) try {
    if (const int rc = check_dtype(dtype)) return rc;
    if (const int rc = check_choices(tokens, topk)) return rc;
    if (const int rc = check_rows_count(rows)) return rc;
    if (const int rc = check_dim(dim)) return rc;
    if (const int rc = check_ld(ldx, dim, "ldx")) return rc;
    if (const int rc = check_ld(ldy, dim, "ldy")) return rc;
    if (tokens == 0 || dim == 0 || rows == 0) return OPTIM_OK;
    if (!x_dev || !place_dev || !y_dev) return fail(OPTIM_EINVAL, "NULL buffer");
    const size_t sz = size_of(dtype), slots = (size_t)tokens * topk;
    if (!aligned(x_dev, sz) || !aligned(place_dev, 4) || !aligned(weights_dev, 4) || !aligned(y_dev, sz))
        return fail(OPTIM_EALIGN, "buffer misaligned");
    Ranges r;
    r.rows(x_dev, tokens, ldx, dim, sz, false, "x");
    r.add(place_dev, slots * 4, false, "place");
    r.add(weights_dev, slots * 4, false, "weights");
    r.rows(y_dev, rows, ldy, dim, sz, true, "y");
    if (const int rc = check_overlaps(r.all)) return rc;
    TokenArgs a{};
    a.x = static_cast<const char *>(x_dev);
    a.ldx = ldx * (int64_t)sz;
    a.dy = static_cast<char *>(y_dev);
    a.lddy = ldy * (int64_t)sz;
    a.place = place_dev;
    a.weights = weights_dev;
    a.tokens = tokens;
    a.topk = topk;
    a.dim = (int32_t)dim;
    a.rows = (uint32_t)rows;
    HIP_OK(launch_gather(a, dtype, static_cast<hipStream_t>(stream)));
    return OPTIM_OK;
} OPTIM_CATCH

int optim_expert_combine(const void *y_dev, int64_t ldy, int64_t rows, int32_t dtype, const int32_t *place_dev,
                         const float *weights_dev, int64_t tokens, int32_t topk, int64_t dim, const void *residual_dev,
                         int64_t ldr, const optim_dropout_hp *drop, const int32_t *step_dev, void *out_dev,
                         int64_t ldo, void *stream) try {
    if (const int rc = check_dtype(dtype)) return rc;
    if (const int rc = check_choices(tokens, topk)) return rc;
    if (const int rc = check_rows_count(rows)) return rc;
    if (const int rc = check_dim(dim)) return rc;
    if (const int rc = check_ld(ldy, dim, "ldy")) return rc;
    if (const int rc = check_ld(ldo, dim, "ldo")) return rc;
    if (residual_dev)
        if (const int rc = check_ld(ldr, dim, "ldr")) return rc;
    TokenArgs a{};
    if (drop)
        if (const int rc = check_drop(drop, step_dev, a.drop)) return rc;
    if (tokens == 0 || dim == 0) return OPTIM_OK;
    if ((rows > 0 && !y_dev) || !place_dev || !out_dev) return fail(OPTIM_EINVAL, "NULL buffer");
    const size_t sz = size_of(dtype), slots = (size_t)tokens * topk;
    if (!aligned(y_dev, sz) || !aligned(place_dev, 4) || !aligned(weights_dev, 4) || !aligned(residual_dev, sz) ||
        !aligned(out_dev, sz))
        return fail(OPTIM_EALIGN, "buffer misaligned");
    if (residual_dev == out_dev && ldr != ldo) return fail(OPTIM_EINVAL, "out is residual, but ldo is not ldr");
    Ranges r;
    r.rows(y_dev, rows, ldy, dim, sz, false, "y");
    r.add(place_dev, slots * 4, false, "place");
    r.add(weights_dev, slots * 4, false, "weights");
    if (residual_dev != out_dev) r.rows(residual_dev, tokens, ldr, dim, sz, false, "residual");
    if (drop) r.add(step_dev, 4, false, "step");
    r.rows(out_dev, tokens, ldo, dim, sz, true, "out");
    if (const int rc = check_overlaps(r.all)) return rc;
    a.x = static_cast<const char *>(residual_dev);
    a.ldx = ldr * (int64_t)sz;
    a.out = static_cast<char *>(out_dev);
    a.ldo = ldo * (int64_t)sz;
    a.y = static_cast<const char *>(y_dev);
    a.ldy = ldy * (int64_t)sz;
    a.place = place_dev;
    a.weights = weights_dev;
    a.tokens = tokens;
    a.topk = topk;
    a.dim = (int32_t)dim;
    a.rows = (uint32_t)rows;
    HIP_OK(launch_combine(a, dtype, static_cast<hipStream_t>(stream)));
    return OPTIM_OK;
} OPTIM_CATCH

int optim_expert_combine_grad(const void *dout_dev, int64_t ldd, int32_t dtype, const void *y_dev, int64_t ldy,
                              int64_t rows, const int32_t *place_dev, const float *weights_dev, int64_t tokens,
                              int32_t topk, int64_t dim, const optim_dropout_hp *drop, const int32_t *step_dev,
                              void *dy_dev, int64_t lddy, float *dweights_dev, void *stream) try {
    if (const int rc = check_dtype(dtype)) return rc;
    if (const int rc = check_choices(tokens, topk)) return rc;
    if (const int rc = check_rows_count(rows)) return rc;
    if (const int rc = check_dim(dim)) return rc;
    if (const int rc = check_ld(ldd, dim, "ldd")) return rc;
    if (dweights_dev)
        if (const int rc = check_ld(ldy, dim, "ldy")) return rc;
    if (dy_dev)
        if (const int rc = check_ld(lddy, dim, "lddy")) return rc;
    TokenArgs a{};
    if (drop)
        if (const int rc = check_drop(drop, step_dev, a.drop)) return rc;
    if (!dweights_dev && !dy_dev && rows > 0) return fail(OPTIM_EINVAL, "neither dy nor dweights is wanted");
    if (tokens == 0) return OPTIM_OK;
    if ((dim > 0 && !dout_dev) || !place_dev || (dweights_dev && rows > 0 && dim > 0 && !y_dev))
        return fail(OPTIM_EINVAL, "NULL buffer");
    const size_t sz = size_of(dtype), slots = (size_t)tokens * topk;
    if (!aligned(dout_dev, sz) || !aligned(y_dev, sz) || !aligned(place_dev, 4) || !aligned(weights_dev, 4) ||
        !aligned(dy_dev, sz) || !aligned(dweights_dev, 4))
        return fail(OPTIM_EALIGN, "buffer misaligned");
    if (dweights_dev && dy_dev == y_dev && dy_dev && lddy != ldy) return fail(OPTIM_EINVAL, "dy is y, but lddy is not ldy");
    Ranges r;
    r.rows(dout_dev, tokens, ldd, dim, sz, false, "dout");
    if (dweights_dev && y_dev != dy_dev) r.rows(y_dev, rows, ldy, dim, sz, false, "y");
    r.add(place_dev, slots * 4, false, "place");
    r.add(weights_dev, slots * 4, false, "weights");
    if (drop) r.add(step_dev, 4, false, "step");
    r.rows(dy_dev, rows, lddy, dim, sz, true, "dy");
    r.add(dweights_dev, slots * 4, true, "dweights");
    if (const int rc = check_overlaps(r.all)) return rc;
    a.x = static_cast<const char *>(dout_dev);
    a.ldx = ldd * (int64_t)sz;
    a.y = static_cast<const char *>(y_dev);
    a.ldy = ldy * (int64_t)sz;
    a.dy = static_cast<char *>(dy_dev);
    a.lddy = lddy * (int64_t)sz;
    a.place = place_dev;
    a.weights = weights_dev;
    a.dweights = dweights_dev;
    a.tokens = tokens;
    a.topk = topk;
    a.dim = (int32_t)dim;
    a.rows = (uint32_t)rows;
    HIP_OK(launch_combine_grad(a, dtype, static_cast<hipStream_t>(stream)));
    return OPTIM_OK;
} OPTIM_CATCH

}  // extern "C"
