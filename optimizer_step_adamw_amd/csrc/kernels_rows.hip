// kernels_rows.hip -- the rows of the experts (optim_route_rows): a stable
// counting sort of the choices by expert, and the step of the balance bias
// (optim_step_route_bias).
//
// A workgroup takes a chunk of the choices, each of its wavefronts a run of 64s.
// Choices without an expert are sorted behind the others, as expert E.  A choice's
// rank among the equal ones of its 64 comes from ballots over the bits of the
// expert, and the wavefront's count so far from LDS: no atomics on anything whose
// order could show, and none that many lanes would meet in where one expert is
// far more popular.  (The loops are loops: a workgroup goes through this code
// once, and would wait for more of it to be fetched.)  Where one workgroup takes
// all, one launch counts, scans and places; otherwise a first launch counts each
// chunk, and every workgroup of the second sums what lies before its chunk.
//
// Bound by latency, two launches' chains of dependent steps.  Kernels' times in a
// trace, us: 65536 x 8 choices of 256 experts 6.2 and 13.0 (6 MB; of the second one
// reading the choices and the counts takes a third, ranks another), 4096 x 8 of 64
// 3.1 and 8.6; in one launch 1024 x 8 11.6, 256 x 8 6.6, 300 x 2 of 8 4.5.  The
// bias' step behind them 1.4, 4.0 for 256 experts.  Replayed from a graph, where a
// launch begins while the one before ends, all three take 20.1 for 65536 x 8.  The
// tables are as large for 8 experts as for 1024: one workgroup a CU.
#include "device_common.h"
#include "experts.h"

#include <algorithm>

namespace optim {
namespace {

constexpr int kRowLanes = 1024, kRowWaves = kRowLanes / 64;  // of a workgroup, at most
constexpr int kHeld = 16384;                                 // choices of a chunk that stay in LDS, at most
constexpr int kBatch = 10;                                   // rows of counts that a lane asks for at a time
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

// A wavefront's run of this workgroup's chunk.  (No sum here passes the chunk's
// end, which may lie just below 2^31.)
struct Run {
    int32_t begin, n;
};
__device__ __forceinline__ Run wave_run(const RowsArgs &a) {
    const int32_t c0 = (int32_t)blockIdx.x * a.chunk, n = a.n - c0 < a.chunk ? a.n - c0 : a.chunk;
    const int32_t run = a.chunk / (int32_t)(blockDim.x >> 6), lo = (int32_t)(threadIdx.x >> 6) * run, hi = lo + run;
    const int32_t begin = lo < n ? lo : n;
    return Run{c0 + begin, (hi < n ? hi : n) - begin};
}

// Counts the 64 choices that the lanes hold, e each (in: there is one), into the
// wavefront's next[]; returns how many equal ones of the run came before.
// BITS: of an expert's number.
template <int BITS>
__device__ __forceinline__ int32_t count_64(int32_t e, bool in, int32_t *next) {
    const int32_t lane = threadIdx.x & 63;
    const uint64_t there = __ballot(in);
    uint32_t lo = (uint32_t)there, hi = (uint32_t)(there >> 32);
#pragma unroll
    for (int b = 0; b < BITS; ++b) {
        const int32_t bit = (int32_t)((uint32_t)e << (31 - b)) >> 31;  // 0 or all ones
        const uint64_t set = __ballot(bit);
        lo &= ~((uint32_t)set ^ (uint32_t)bit);
        hi &= ~((uint32_t)(set >> 32) ^ (uint32_t)bit);
    }
    const uint64_t same = (uint64_t)hi << 32 | lo;
    const int32_t rank = __popcll(same & ((1ull << lane) - 1)), before = next[e];
    wave_sync();
    if (in && rank == 0) next[e] = before + __popcll(same);
    wave_sync();
    return before + rank;
}

// This workgroup's chunk.
__device__ __forceinline__ Run chunk_of(const RowsArgs &a) {
    const int32_t c0 = (int32_t)blockIdx.x * a.chunk;
    return Run{c0, a.n - c0 < a.chunk ? a.n - c0 : a.chunk};
}

// A lane's first choices of the chunk, kEarly of them asked for at once.
constexpr int kEarly = 4;
struct Early {
    int32_t e[kEarly];
};
__device__ __forceinline__ Early first_choices(const RowsArgs &a, const Run &c) {
    Early x;
#pragma unroll
    for (int i = 0; i < kEarly; ++i) {
        const int32_t at = (int32_t)(threadIdx.x + i * blockDim.x);
        x.e[i] = at < c.n ? expert_of(a, c.begin + at) : 0;
    }
    return x;
}
// f(place in the chunk, expert) for all of this lane's choices
template <class F>
__device__ __forceinline__ void each_choice(const RowsArgs &a, const Run &c, const Early &x, F &&f) {
#pragma unroll
    for (int i = 0; i < kEarly; ++i)
        if ((int32_t)(threadIdx.x + i * blockDim.x) < c.n) f((int32_t)(threadIdx.x + i * blockDim.x), x.e[i]);
#pragma unroll 4
    for (int32_t at = threadIdx.x + kEarly * blockDim.x; at < c.n; at += blockDim.x) f(at, expert_of(a, c.begin + at));
}

// A chunk's counts lie in rows of whole fours.
__device__ __forceinline__ int32_t count_row(const RowsArgs &a) { return (a.experts + 4) / 4 * 4; }

__global__ __launch_bounds__(kRowLanes) void rows_count_kernel(RowsArgs a) {
    constexpr int kCopies = 4;  // that wavefronts count into
    __shared__ int32_t cnt[kCopies * (kMaxExperts + 1)];
    const int32_t E1 = a.experts + 1;
    const Run c = chunk_of(a);
    const Early x = first_choices(a, c);
    for (int32_t i = threadIdx.x; i < kCopies * E1; i += blockDim.x) cnt[i] = 0;
    __syncthreads();
    int32_t *mine = cnt + ((threadIdx.x >> 6) & (kCopies - 1)) * E1;
    each_choice(a, c, x, [&](int32_t, int32_t e) { atomicAdd(&mine[e], 1); });
    __syncthreads();
    for (int32_t e = threadIdx.x; e < E1; e += blockDim.x) {
        int32_t sum = 0;
#pragma unroll
        for (int w = 0; w < kCopies; ++w) sum += cnt[w * E1 + e];
        a.counts[(int64_t)blockIdx.x * count_row(a) + e] = sum;
    }
}

__device__ __forceinline__ void put_row(const RowsArgs &a, int32_t i, int32_t e, int32_t row) {
    a.place[i] = e < a.experts ? row : -1;
    if (a.order) a.order[row] = e < a.experts ? i : -1;
}

template <int BITS>
__global__ __launch_bounds__(kRowLanes) void rows_place_kernel(RowsArgs a) {
    __shared__ int32_t cnt[kRowWaves * (kMaxExperts + 1)];
    __shared__ int32_t all[kMaxExperts + 4], before[kMaxExperts + 4];
    __shared__ uint32_t held[kHeld];  // expert, and rank in the run (below 2^14), of a chunk of no more
    const int32_t E1 = a.experts + 1, waves = blockDim.x >> 6, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const Run c = chunk_of(a), r = wave_run(a);
    const Early x = first_choices(a, c);
    // Lanes take four experts' counts in every slices-th chunk, kBatch loads at a
    // time, the first ones behind the first choices, which return before them.
    const int32_t quads = count_row(a) / 4, slices = (int32_t)blockDim.x / quads, slice = threadIdx.x / quads;
    const int32_t q = threadIdx.x % quads;
    const bool sums = a.counts && slice < slices;
    s32x4 v[kBatch];
    auto load = [&](int32_t b0) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int32_t b = b0 + i * slices;
            v[i] = *(const GMEM s32x4 *)gp(a.counts + ((int64_t)(b < a.blocks ? b : slice) * quads + q) * 4);
        }
    };
    if (sums && slice < a.blocks) load(slice);
    for (int32_t e = threadIdx.x; e < count_row(a); e += blockDim.x) {
        all[e] = 0;
        before[e] = 0;
    }
    // ---- counts of every run, ranks in it
    const bool holds = a.chunk <= kHeld;
    if (holds) each_choice(a, c, x, [&](int32_t i, int32_t e) { held[i] = (uint32_t)e; });
    for (int32_t i = threadIdx.x; i < waves * E1; i += blockDim.x) cnt[i] = 0;
    __syncthreads();
    int32_t *next = cnt + wave * E1;
    uint32_t *mine = held + (r.begin - c.begin);
#pragma unroll 1
    for (int32_t i0 = 0; i0 < r.n; i0 += 64) {
        const bool in = i0 + lane < r.n;
        const int32_t e = !in ? 0 : holds ? (int32_t)mine[i0 + lane] : expert_of(a, r.begin + i0 + lane);
        const int32_t rank = count_64<BITS>(e, in, next);
        if (holds && in) mine[i0 + lane] = (uint32_t)e | (uint32_t)rank << 16;
    }
    // ---- choices of every expert in all chunks, and in those before (element i of
    // a four in the i-th quarter, so that lanes meet different banks)
    if (sums) {
        s32x4 sum = {0, 0, 0, 0}, low = {0, 0, 0, 0};
        for (int32_t b0 = slice; b0 < a.blocks; b0 += kBatch * slices) {
            if (b0 > slice) load(b0);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int32_t b = b0 + i * slices;
                if (b < a.blocks) sum += v[i];
                if (b < (int32_t)blockIdx.x) low += v[i];
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            atomicAdd(&all[i * quads + q], sum[i]);
            atomicAdd(&before[i * quads + q], low[i]);
        }
    }
    __syncthreads();
    auto at = [&](int32_t e) { return (e & 3) * quads + (e >> 2); };
    if (!a.counts) {
        for (int32_t e = threadIdx.x; e < E1; e += blockDim.x) {
            int32_t sum = 0;
            for (int w = 0; w < waves; ++w) sum += cnt[w * E1 + e];
            all[at(e)] = sum;
        }
        __syncthreads();
    }
    if (wave == 0) {  // all: number of choices -> first row
        const int32_t per = (E1 + 63) / 64, e0 = lane * per;
        int32_t sum = 0;
        for (int32_t i = e0; i < e0 + per && i < E1; ++i) sum += all[at(i)];
        int32_t first = sum;
        for (int m = 1; m < 64; m *= 2) {
            const int32_t up = __shfl_up(first, m);
            if (lane >= m) first += up;
        }
        first -= sum;
        for (int32_t i = e0; i < e0 + per && i < E1; ++i) {
            const int32_t n = all[at(i)];
            all[at(i)] = first;
            first += n;
        }
    }
    __syncthreads();
    for (int32_t e = threadIdx.x; e < E1; e += blockDim.x) {
        int32_t row = all[at(e)];
        if (blockIdx.x == 0) a.offsets[e] = row;
        row += before[at(e)];
        for (int w = 0; w < waves; ++w) {  // cnt: number of choices -> the run's first row
            const int32_t n = cnt[w * E1 + e];
            cnt[w * E1 + e] = row;
            row += n;
        }
    }
    __syncthreads();
    if (holds) {
        const int32_t run = a.chunk / waves;
#pragma unroll 1
        for (int32_t i = threadIdx.x; i < c.n; i += blockDim.x) {
            const int32_t e = held[i] & 0xFFFF;  // (64 neighbours are of one run)
            put_row(a, c.begin + i, e, cnt[__builtin_amdgcn_readfirstlane(i) / run * E1 + e] + (int32_t)(held[i] >> 16));
        }
        return;
    }
#pragma unroll 1
    for (int32_t i0 = 0; i0 < r.n; i0 += 64) {
        const bool in = i0 + lane < r.n;
        const int32_t e = in ? expert_of(a, r.begin + i0 + lane) : 0, row = count_64<BITS>(e, in, next);
        if (in) put_row(a, r.begin + i0 + lane, e, row);
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

template <int BITS>
hipError_t launch_rows_t(const RowsArgs &args, hipStream_t s) {
    RowsArgs a = args;
    dim3 lanes(kRowLanes);
    if (!a.counts && a.n <= 1024) {  // fewer wavefronts to wait for
        a.chunk = 1024;
        lanes = dim3(256);
    }
    if (a.counts) hipLaunchKernelGGL(rows_count_kernel, dim3((unsigned)a.blocks), lanes, 0, s, a);
    hipLaunchKernelGGL(rows_place_kernel<BITS>, dim3((unsigned)(a.blocks > 0 ? a.blocks : 1)), lanes, 0, s, a);
    return hipGetLastError();
}

}  // namespace

// One workgroup up to 8192 choices, then 128 of them (each of which reads the
// counts of all), more once each has kHeld, and 512 at most.
RowsShape rows_shape(int64_t n) {
    int64_t chunk = n <= 8192 ? 8192 : std::max<int64_t>({n / 512, std::min<int64_t>(n / 128, kHeld), 4096});
    chunk += kRowLanes - 1;
    chunk -= chunk % kRowLanes;
    return RowsShape{(int32_t)chunk, (int32_t)((n + chunk - 1) / chunk)};
}

size_t rows_workspace(RowsShape shape, int32_t experts) {
    return shape.blocks > 1 ? (size_t)shape.blocks * ((experts + 4) / 4 * 4) * sizeof(int32_t) : 0;
}

hipError_t launch_rows(const RowsArgs &a, hipStream_t s) {
    if (a.experts < 16) return launch_rows_t<4>(a, s);
    if (a.experts < 64) return launch_rows_t<6>(a, s);
    if (a.experts < 256) return launch_rows_t<8>(a, s);
    if (a.experts < 512) return launch_rows_t<9>(a, s);
    return launch_rows_t<11>(a, s);
}

hipError_t launch_route_bias(const int32_t *offsets, int32_t experts, float *bias, const float *rate,
                             const float *found_inf, hipStream_t s) {
    hipLaunchKernelGGL(route_bias_kernel, dim3(1), dim3((unsigned)((experts + 63) / 64 * 64)), 0, s, offsets, experts, bias,
                       rate, found_inf);
    return hipGetLastError();
}

}  // namespace optim
