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

namespace optim {
namespace {

constexpr int kRowLanes = 512, kRowWaves = kRowLanes / 64;

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

// cnt[wave][expert]: choices of each wavefront's run of the chunk.
__device__ __forceinline__ void count_chunk(const RowsArgs &a, int32_t c0, int32_t c1, int32_t run, int32_t *cnt) {
    const int32_t E1 = a.experts + 1, wave = threadIdx.x >> 6;
    for (int32_t i = threadIdx.x; i < kRowWaves * E1; i += kRowLanes) cnt[i] = 0;
    __syncthreads();
    const Run r = wave_run(c0, c1, run);
    for (int32_t i = threadIdx.x & 63; i < r.end - r.begin; i += 64)
        atomicAdd(&cnt[wave * E1 + expert_of(a, r.begin + i)], 1);
    __syncthreads();
}

__global__ __launch_bounds__(kRowLanes) void rows_count_kernel(RowsArgs a) {
    __shared__ int32_t cnt[kRowWaves * (kMaxExperts + 1)];
    const int32_t E1 = a.experts + 1, c0 = (int32_t)blockIdx.x * a.chunk;
    const int32_t c1 = a.n - c0 < a.chunk ? a.n : c0 + a.chunk;
    count_chunk(a, c0, c1, a.chunk / kRowWaves, cnt);
    for (int32_t e = threadIdx.x; e < E1; e += kRowLanes) {
        int32_t sum = 0;
        for (int w = 0; w < kRowWaves; ++w) sum += cnt[w * E1 + e];
        a.counts[(int64_t)blockIdx.x * E1 + e] = sum;
    }
}

__global__ __launch_bounds__(kRowLanes) void rows_place_kernel(RowsArgs a) {
    __shared__ int32_t cnt[kRowWaves * (kMaxExperts + 1)];
    __shared__ int32_t all[kMaxExperts + 1], before[kMaxExperts + 1];
    const int32_t E1 = a.experts + 1, c0 = (int32_t)blockIdx.x * a.chunk, run = a.chunk / kRowWaves;
    const int32_t c1 = a.n - c0 < a.chunk ? a.n : c0 + a.chunk;
    const int32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    count_chunk(a, c0, c1, run, cnt);
    for (int32_t e = threadIdx.x; e < E1; e += kRowLanes) {
        all[e] = 0;
        before[e] = 0;
        if (!a.counts)
            for (int w = 0; w < kRowWaves; ++w) all[e] += cnt[w * E1 + e];
    }
    __syncthreads();
    if (a.counts) {
        // lanes in slices of E1, each summing every slice-th chunk
        const int32_t slices = kRowLanes / E1 > 0 ? kRowLanes / E1 : 1, slice = threadIdx.x / E1;
        if (slice < slices || E1 > kRowLanes)
            for (int32_t e = E1 > kRowLanes ? threadIdx.x : threadIdx.x % E1; e < E1; e += E1 > kRowLanes ? kRowLanes : E1) {
                int32_t sum = 0, low = 0;
                for (int32_t b = E1 > kRowLanes ? 0 : slice; b < a.blocks; b += slices) {
                    const int32_t v = a.counts[(int64_t)b * E1 + e];
                    sum += v;
                    low += b < (int32_t)blockIdx.x ? v : 0;
                }
                atomicAdd(&all[e], sum);
                atomicAdd(&before[e], low);
            }
        __syncthreads();
    }
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
    const int32_t bits = 32 - __builtin_clz(a.experts);
    int32_t *next = cnt + wave * E1;
    const Run r = wave_run(c0, c1, run);
    for (int32_t i0 = 0; i0 < r.end - r.begin; i0 += 64) {
        const bool in = i0 + lane < r.end - r.begin;
        const int32_t i = in ? r.begin + i0 + lane : 0;
        const int32_t e = in ? expert_of(a, i) : 0;
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
}

__global__ __launch_bounds__(kMaxExperts) void route_bias_kernel(const int32_t *offsets, int32_t experts, float *bias,
                                                                 const float *rate, const float *found_inf) {
    if (found_inf && *found_inf != 0.0f) return;
    const int32_t e = threadIdx.x;
    if (e >= experts) return;
    const int64_t all = (int64_t)offsets[experts] - offsets[0], mine = ((int64_t)offsets[e + 1] - offsets[e]) * experts;
    if (all != mine) bias[e] = bias[e] + (all > mine ? *rate : -*rate);
}

}  // namespace

RowsShape rows_shape(int64_t n) {
    constexpr int64_t kMost = 256, kLeast = 2048;  // workgroups, choices of one
    int64_t chunk = (n + kMost - 1) / kMost;
    chunk = (chunk < kLeast ? kLeast : chunk) + kRowLanes - 1;
    chunk -= chunk % kRowLanes;
    return RowsShape{(int32_t)chunk, (int32_t)((n + chunk - 1) / chunk)};
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
