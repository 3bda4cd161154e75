// kernels_rows.hip -- the rows of the experts (optim_route_rows): a stable
// counting sort of the choices by expert, and the step of the balance bias
// (optim_step_route_bias).
//
// A workgroup takes a chunk of the choices, each of its wavefronts a run of 64s.
// Choices without an expert are sorted behind the others, as expert E.  Where
// one workgroup takes all, one launch counts, scans and places; otherwise a
// first launch counts each chunk, and every workgroup of the second sums what
// lies before its chunk.  A choice's place among the equal ones of its
// wavefront's 64 comes from ballots over the bits of the expert: no atomics on
// anything whose order could show.
#include "device_common.h"
#include "experts.h"

#include <algorithm>

namespace optim {
namespace {

constexpr int kRowLanes = 512, kRowWaves = kRowLanes / 64;
typedef int32_t __attribute__((ext_vector_type(4))) s32x4;

// What the wavefront's lanes read from LDS they have read, and what they wrote is
// there for all of them.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ int32_t expert_of(const RowsArgs &a, int32_t i) {
    const uint32_t e = (uint32_t)a.idx[i];
    return e < (uint32_t)a.experts ? (int32_t)e : a.experts;
}

// A wavefront's run of the chunk [c0, c1).  (No sum here passes c1, which may lie
// just below 2^31.)
struct Run {
    int32_t begin, end;
};
__device__ __forceinline__ Run wave_run(int32_t c0, int32_t c1, int32_t run) {
    const int32_t wave = threadIdx.x >> 6, n = c1 - c0, lo = wave * run, hi = lo + run;
    return Run{c0 + (lo < n ? lo : n), c0 + (hi < n ? hi : n)};
}

// cnt[wave][expert]: choices of each wavefront's run of the chunk.  The first
// kHeld of a lane's experts stay in registers.
constexpr int kHeld = 8;
__device__ __forceinline__ void count_chunk(const RowsArgs &a, const Run &r, int32_t *cnt, int32_t (&held)[kHeld]) {
    const int32_t E1 = a.experts + 1, lane = threadIdx.x & 63, n = r.end - r.begin;
    int32_t *mine = cnt + (threadIdx.x >> 6) * E1;
#pragma unroll
    for (int h = 0; h < kHeld; ++h) held[h] = h * 64 + lane < n ? expert_of(a, r.begin + h * 64 + lane) : a.experts;
    for (int32_t i = threadIdx.x; i < kRowWaves * E1; i += kRowLanes) cnt[i] = 0;
    __syncthreads();
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
        if (h * 64 + lane < n) atomicAdd(&mine[held[h]], 1);
    for (int32_t i = kHeld * 64 + lane; i < n; i += 64) atomicAdd(&mine[expert_of(a, r.begin + i)], 1);
    __syncthreads();
}

// A chunk's counts lie in rows of whole fours.
__device__ __forceinline__ int32_t count_row(const RowsArgs &a) { return (a.experts + 4) / 4 * 4; }

__global__ __launch_bounds__(kRowLanes) void rows_count_kernel(RowsArgs a) {
    __shared__ int32_t cnt[kRowWaves * (kMaxExperts + 1)];
    const int32_t E1 = a.experts + 1, c0 = (int32_t)blockIdx.x * a.chunk;
    const int32_t c1 = a.n - c0 < a.chunk ? a.n : c0 + a.chunk;
    int32_t held[kHeld];
    count_chunk(a, wave_run(c0, c1, a.chunk / kRowWaves), cnt, held);
    for (int32_t e = threadIdx.x; e < E1; e += kRowLanes) {
        int32_t sum = 0;
        for (int w = 0; w < kRowWaves; ++w) sum += cnt[w * E1 + e];
        a.counts[(int64_t)blockIdx.x * count_row(a) + e] = sum;
    }
}

// The 64 choices that a wavefront's lanes hold, e each (in: there is one): rows
// in the order of lanes, from next[] on, which moves on.
__device__ __forceinline__ void place_64(const RowsArgs &a, int32_t i, int32_t e, bool in, int32_t bits, int32_t *next) {
    const int32_t lane = threadIdx.x & 63;
    uint64_t same = __ballot(in);
    for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot(e >> b & 1);
        same &= e >> b & 1 ? set : ~set;
    }
    const int32_t rank = __popcll(same & ((1ull << lane) - 1));
    const int32_t row = in ? next[e] + rank : 0;
    wave_sync();
    if (in && rank == 0) next[e] += __popcll(same);
    wave_sync();
    if (in) {
        a.place[i] = e < a.experts ? row : -1;
        if (a.order) a.order[row] = e < a.experts ? i : -1;
    }
}

__global__ __launch_bounds__(kRowLanes) void rows_place_kernel(RowsArgs a) {
    __shared__ int32_t cnt[kRowWaves * (kMaxExperts + 1)];
    __shared__ int32_t all[kMaxExperts + 4], before[kMaxExperts + 4];
    const int32_t E1 = a.experts + 1, c0 = (int32_t)blockIdx.x * a.chunk;
    const int32_t c1 = a.n - c0 < a.chunk ? a.n : c0 + a.chunk;
    const int32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const Run r = wave_run(c0, c1, a.chunk / kRowWaves);
    int32_t held[kHeld];
    for (int32_t e = threadIdx.x; e < count_row(a); e += kRowLanes) {
        all[e] = 0;
        before[e] = 0;
    }
    count_chunk(a, r, cnt, held);
    if (a.counts) {
        // Lanes take four experts and every slices-th chunk, eight loads at a time.
        const int32_t quads = count_row(a) / 4, slices = kRowLanes / quads, slice = threadIdx.x / quads, q = threadIdx.x % quads;
        if (slice < slices) {
            s32x4 sum = {0, 0, 0, 0}, low = {0, 0, 0, 0};
            for (int32_t b0 = slice; b0 < a.blocks; b0 += 8 * slices) {
                s32x4 v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int32_t b = b0 + i * slices;
                    v[i] = *(const GMEM s32x4 *)gp(a.counts + ((int64_t)(b < a.blocks ? b : b0) * quads + q) * 4);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int32_t b = b0 + i * slices;
                    if (b < a.blocks) sum += v[i];
                    if (b < (int32_t)blockIdx.x) low += v[i];
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (q * 4 + i < E1) {
                    atomicAdd(&all[q * 4 + i], sum[i]);
                    atomicAdd(&before[q * 4 + i], low[i]);
                }
        }
    } else {
        for (int32_t e = threadIdx.x; e < E1; e += kRowLanes)
            for (int w = 0; w < kRowWaves; ++w) all[e] += cnt[w * E1 + e];
    }
    __syncthreads();
    if (wave == 0) {  // all: number of choices -> first row
        const int32_t per = (E1 + 63) / 64, e0 = lane * per;
        int32_t sum = 0;
        for (int32_t i = e0; i < e0 + per && i < E1; ++i) sum += all[i];
        int32_t first = sum;
        for (int m = 1; m < 64; m *= 2) {
            const int32_t v = __shfl_up(first, m);
            if (lane >= m) first += v;
        }
        first -= sum;
        for (int32_t i = e0; i < e0 + per && i < E1; ++i) {
            const int32_t v = all[i];
            all[i] = first;
            first += v;
        }
    }
    __syncthreads();
    for (int32_t e = threadIdx.x; e < E1; e += kRowLanes) {
        if (blockIdx.x == 0) a.offsets[e] = all[e];
        int32_t at = all[e] + before[e];
        for (int w = 0; w < kRowWaves; ++w) {
            const int32_t v = cnt[w * E1 + e];
            cnt[w * E1 + e] = at;
            at += v;
        }
    }
    __syncthreads();
    const int32_t bits = 32 - __builtin_clz(a.experts), n = r.end - r.begin;
    int32_t *next = cnt + wave * E1;
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
        if (h * 64 >= n) break;
        const bool in = h * 64 + lane < n;
        place_64(a, r.begin + (in ? h * 64 + lane : 0), held[h], in, bits, next);
    }
    for (int32_t i0 = kHeld * 64; i0 < n; i0 += 64) {
        const bool in = i0 + lane < n;
        const int32_t i = r.begin + (in ? i0 + lane : 0);
        place_64(a, i, in ? expert_of(a, i) : 0, in, bits, next);
    }
}

__global__ __launch_bounds__(kMaxExperts) void route_bias_kernel(const int32_t *offsets, int32_t experts, float *bias,
                                                                 const float *rate, const float *found_inf) {
    const int32_t e = threadIdx.x < (uint32_t)experts ? threadIdx.x : 0;
    // (every load before the first is waited for)
    const int32_t first = offsets[0], end = offsets[experts], lo = offsets[e], hi = offsets[e + 1];
    const float b = bias[e], by = *rate;
    if (found_inf && *found_inf != 0.0f) return;
    const int64_t all = (int64_t)end - first, mine = ((int64_t)hi - lo) * experts;
    if (threadIdx.x < (uint32_t)experts && all != mine) bias[e] = b + (all > mine ? by : -by);
}

}  // namespace

RowsShape rows_shape(int64_t n) {
    // 128 workgroups of the second launch sum as many counts each; more of them
    // once each has 16384 choices, 512 at most.
    int64_t chunk = std::max<int64_t>({n / 512, std::min<int64_t>(n / 128, 16384), 4096});
    chunk += kRowLanes - 1;
    chunk -= chunk % kRowLanes;
    return RowsShape{(int32_t)chunk, (int32_t)((n + chunk - 1) / chunk)};
}

size_t rows_workspace(RowsShape shape, int32_t experts) {
    return shape.blocks > 1 ? (size_t)shape.blocks * ((experts + 4) / 4 * 4) * sizeof(int32_t) : 0;
}

hipError_t launch_rows(const RowsArgs &a, hipStream_t s) {
    if (a.counts) hipLaunchKernelGGL(rows_count_kernel, dim3((unsigned)a.blocks), dim3(kRowLanes), 0, s, a);
    hipLaunchKernelGGL(rows_place_kernel, dim3((unsigned)(a.blocks > 0 ? a.blocks : 1)), dim3(kRowLanes), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_route_bias(const int32_t *offsets, int32_t experts, float *bias, const float *rate,
                             const float *found_inf, hipStream_t s) {
    hipLaunchKernelGGL(route_bias_kernel, dim3(1), dim3((unsigned)((experts + 63) / 64 * 64)), 0, s, offsets, experts, bias,
                       rate, found_inf);
    return hipGetLastError();
}

}  // namespace optim
