// plan.h -- device-visible plan tables shared by the C-ABI host layer
// (api.cpp) and the gfx950 kernels (kernels_*.hip).  Internal; not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <deque>
#include <string>
#include <utility>
#include <vector>

namespace optim {

// Work decomposition: every tensor (Adam-mini: every shared-v block) is a
// "span"; a span is cut into units of `tile` consecutive elements (the last
// one ragged).  Units are numbered globally.  By default one workgroup runs
// per unit, so the hardware dispatcher keeps the resident workgroups on one
// narrow, advancing window of every array; a plan may instead ask for a
// persistent grid whose workgroups walk the units grid-stride.
constexpr int kThreads = 256;        // workgroup size (4 wavefronts of 64)
constexpr int64_t kDefaultTile = 2048;
// AdamW / AdEMAMix / Lion plans of more than 2^20 and at most 2^24 elements:
// units of 4096, which the step runs in its early-load form (see
// kernels_adam.hip)
constexpr int64_t kEarlyTile = 4096;
constexpr int64_t kEarlyTileMinElems = int64_t(1) << 20;
constexpr int64_t kEarlyTileMaxElems = int64_t(1) << 24;
constexpr int64_t kAdamMiniTile = 4096;   // also LAMB and the fp16 scaled-state step
// Adam-mini: gradient bytes per segment (a segment's g is read twice, the
// second time mostly from the 256 MB Infinity Cache).  Measured on MI355X,
// Llama-7B-shaped list: 28.1 ms per step in one pass over the list; with
// segments of 160 / 256 / 384 / 512 / 1024 MiB 27.3 / 26.5 / 25.8 / 26.0 /
// 26.8 ms (fewer, larger segments launch less often; past the cache's size
// less of g is found there).  With today's kernels, every size timed in one
// process on the same arrays: 256 / 320 / 384 / 448 / 512 MiB 25.18 /
// 24.95 / 24.88 / 24.99 / 25.06 ms.
constexpr int64_t kMiniSegmentBytes = (int64_t)384 << 20;
// blockwise units, measured best on MI355X over 2^28 elements (4096-16384,
// every size timed in one process on the same arrays, since where the
// driver places a fresh set of arrays moves the step by up to several
// percent): 8-bit separate layout 4096 (757 us against 766 at 8192),
// interleaved 8192 (729 against 751 at 4096), 4-bit 8192 either layout
// (632-634 against 678-684 at 4096 and 653-684 at 16384), AdEMAMix 8-bit
// 8192 (874 against 935 / 895), 4-bit 16384
constexpr int64_t blockwise_tile(bool ademamix, int bits, bool interleaved) {
    return ademamix ? (bits == 8 ? 8192 : 16384) : (bits == 8 && !interleaved) ? 4096 : 8192;
}
// read-only scans (finite check, gradient norm): elements per workgroup;
// measured on MI355X over a 1.1B bf16 gradient list: 8192 -> 5.3 TB/s,
// 32768 -> 6.2 (check) / 6.4 (check + norm), 65536 no better
constexpr int64_t kFiniteCheckElems = 32768;
constexpr int64_t kMinTile = 1024;   // one group of 4 elements per lane
constexpr int64_t kMinBlockwiseTile = 2048;  // one quantizer row: 256 lanes x 8 elements
// AdamW / AdEMAMix interleaved moment layout: blocks of this many elements
// (one group of 4 per lane of a workgroup), m then v (then m2) per block
constexpr int64_t kMomentBlock = 1024;
constexpr int kMaxGroups = 64;    // distinct weight-decay values per plan
constexpr int64_t kMaxNumel = int64_t(1) << 48;  // per tensor (byte sizes stay far from overflow)

// fp32; bf16 + int16 remainder; fp32 master + bf16 or fp16 model copy
enum ParamKind { P_F32 = 0, P_BF16R = 1, P_MBF16 = 2, P_MF16 = 3 };
enum GradKind { G_F32 = 0, G_BF16 = 1, G_F16 = 2 };  // G_F16: gradient lists only
// 16-bit scaled moments (same codes as the public state_dtype values)
enum StateKind { S_BF16 = 1, S_F16 = 2 };

struct TensorDesc {       // 152 bytes
    void *p;              // param (fp32 or bf16 patterns)
    const void *g;        // gradient
    float *m;             // first moment
    float *v;             // second moment (Adam-mini HEAD/SCALAR: per block)
    float *m2;            // AdEMAMix slow EMA
    uint16_t *rem;        // int16 remainder (as raw 16-bit patterns)
    uint8_t *qm, *qv;     // blockwise codes
    float *am, *av;       // blockwise absmax
    int64_t numel;
    int64_t block_len;    // Adam-mini shared-v block length (0 = full v)
    int32_t group;        // weight-decay group
    int32_t kind;         // Adam-mini partition
    int32_t vec_ok;       // every pointer 16-byte aligned
    int32_t pad_;
    uint8_t *qm2;         // blockwise AdEMAMix: codes of m2
    float *am2;           // blockwise AdEMAMix: absmax of m2
    float *master;        // fp32 master of a bf16 / fp16 model param (p)
    float *scale_m;       // 16-bit states: device scale of the stored m
    float *scale_v;       // 16-bit states: device scale of the stored v
};
static_assert(sizeof(TensorDesc) == 152, "TensorDesc layout");

// Packs (AdamW, AdEMAMix and Lion plans): a run of whole tensors of at most
// half a pack each (in list order, empty tensors left out), laid end to end
// as one unit of at most kPackElems elements (or the plan's unit, if
// smaller), each tensor's length rounded up to a multiple of 4.  A
// pack is one span whose tensor field is kPackTensor and whose elem_begin is
// the pack's index; its len is the rounded total.  Packs take the plan's
// last units, after every unit of a single tensor, and have kernels of
// their own (the step kernels of single tensors stay free of their registers
// and LDS).  Member j holds the pack's
// elements [off[j], off[j + 1]), off[j] = pack_off[off_base + j], off[0] = 0,
// off[k] = len; pack_td[td_base + j] is its PackMember record (the fields of
// its tensor descriptor the pack kernels read), so a workgroup loads a
// pack's tables with one contiguous copy into LDS.
constexpr int32_t kPackTensor = -2;
constexpr int32_t kMaxPackTensors = 64;  // members per pack (LDS: 64 descriptors, ~10 KB)
// Pack capacity: 2048 elements, two groups of 4 per lane.  A pack kernel's
// workgroup waits for its member tables before it can load, and per-lane
// member pointers cost registers (4-group packs: 143 VGPRs, 3 waves per
// SIMD; 2-group: 96, 5 waves), so smaller packs in more, leaner workgroups
// hide that wait better.  Measured on MI355X, 2^24 AdamW elements in one
// process on the same arrays (four state sets in turn), 4096- / 2048- /
// 1024-element packs: 65536 tensors of 256 89.6 / 84.5 / 84.5 us, 32768 of
// 512 87.7 / 83.1 / 82.8 us, 262144 of 64 98.5 / 88.4 / 90.6 us.
constexpr int64_t kPackElems = 2048;
// A pack member as the pack kernels see it: its arrays, length, weight-decay
// group and alignment (72 bytes, against 152 for the full TensorDesc; the
// tables are read from HBM once per step, so their size is traffic).
struct PackMember {
    void *p;
    const void *g;
    float *m;
    float *v;
    float *m2;
    uint16_t *rem;
    float *master;
    int32_t numel;        // at most kPackElems / 2
    int32_t group;
    int32_t vec_ok;
    int32_t pad_;
};
static_assert(sizeof(PackMember) == 72, "PackMember layout");
struct PackDesc {         // 16 bytes
    int32_t td_base;      // index of member 0 in pack_td
    int32_t off_base;     // index of off[0] in pack_off
    int32_t k;            // members
    int32_t len;          // elements including the rounding
};
static_assert(sizeof(PackDesc) == 16, "PackDesc layout");

struct SpanDesc {         // 32 bytes
    int64_t unit_begin;   // first global unit number of this span
    int64_t elem_begin;   // first element, relative to the tensor
    int64_t len;          // elements in the span
    int32_t tensor;       // index into the tensor table
    int32_t block;        // Adam-mini global block number, -1 for full v
};
static_assert(sizeof(SpanDesc) == 32, "SpanDesc layout");

// Per-step scalars.  Every workgroup of a step kernel derives them in its
// prologue (fp64, rounded once to fp32) into LDS from the device lr, step
// counter, found_inf and inv_scale.
struct Scalars {
    int32_t skip;         // non-zero: found_inf was set, write nothing
    int32_t t;            // applied-step count including this step
    float lr;
    float step_size;      // fl32(lr / (1 - beta1^t))
    float inv_sqrt_bc2;   // fl32(1 / sqrt(1 - beta2^t))
    float inv_bc1;        // fl32(1 / (1 - beta1^t))
    float b1, c1;         // fl32(beta1), fl32(1 - beta1)
    float b2, c2;
    float b3, c3;         // AdEMAMix
    float alpha;
    float eps;
    float inv_scale;      // gradient multiplier (AMP unscale), 1 if none
    int32_t k;            // schedule iteration read by this step
    double lr64, step_size64, inv_sqrt_bc2_64, eps64, beta2_64, c2_64;
    float lrwd[kMaxGroups];   // fl32(lr * wd_group)
};

// Commit counters: one top counter and kSubCounters sub-counters, each on its
// own 128-byte line, so arrivals of different workgroups spread over lines.
constexpr int kSubCounters = 32;
constexpr int kCounterStride = 32;  // uint32 words between counters
constexpr size_t kCounterBytes = (1 + kSubCounters) * kCounterStride * sizeof(uint32_t);
// fp16 scaled moments: per tensor and moment, the running maximum |x| of
// the step as fp32 bits, kept in kAmaxSlots words on separate lines (a
// workgroup's atomic max goes to one of them); 0 between steps.
constexpr int kAmaxSlots = 16;
constexpr size_t kAmaxBytesPerBlock = 2 * kAmaxSlots * kCounterStride * sizeof(uint32_t);

// Gradient lists (OPTIM_ALGO_GRADS): a workgroup takes an item, a run of one
// tensor's elements, or four small tensors, one per wavefront (6000 vectors
// took 19.8 us so, and 22.4 with 16 a workgroup, when both were measured).
// Items are of kGradItemMax bytes, halved down to kGradItemMin while the list
// has fewer than kGradItems of them.  Measured: 1.1B bf16 430 us with 64 KiB,
// 397 with 128, 390 with 256; 4096 x 4096 fp32 with its clip 49 us with 64 KiB
// (1024 items), 45 with 128, 43 with 256, 49 with 512.
constexpr int64_t kGradItemMax = 256 << 10;
constexpr int64_t kGradItemMin = 64 << 10;
constexpr int64_t kGradItems = 256;
constexpr int64_t kGradMostItems = int64_t(1) << 24;  // a launch has fewer than 2^32 lanes
constexpr int64_t kGradSmall = 4096;   // elements of a small tensor at most
// The list's last bytes are read with ordinary loads, the others non-temporal:
// they stay in the 256 MB Infinity Cache for the clip that follows.  Measured,
// nothing kept, these last bytes, all: norms and clip of 67 MB 49, 43, 43 us,
// of 1.3 GB 577, 569, 573; norms alone of 2.3 GB 380, 373, 412.
constexpr int64_t kGradKeepBytes = int64_t(256) << 20;
struct GradItem {         // 32 bytes
    void *g;              // its first element
    int64_t slot0;        // the tensor's first partial sum
    int32_t tensor;
    int32_t len;          // elements
    int32_t slot;         // which of the tensor's items this is
    int32_t nslots;       // how many it has
};
static_assert(sizeof(GradItem) == 32, "GradItem layout");
struct GradSmall {        // 16 bytes
    void *g;
    int32_t tensor;
    int32_t len;
};
static_assert(sizeof(GradSmall) == 16, "GradSmall layout");

// Muon: a matrix of the list with its arrays in the workspace (byte offsets
// from the region that the runs share).  X is held padded to rp x ld, A and B
// to sp x sp, sides rounded up to multiples of 32.
constexpr int kMuonTile = 128, kMuonWideTile = 256;
constexpr int64_t kMuonUnit = 4096;  // elements of padded X per workgroup of the splitting pass
// Matrices with a side of at most 128 go through slabs: kMuonSlab values of X
// (positions along the longer side times the shorter side padded to 64 or 128)
// that a workgroup holds in LDS.  A matrix of one slab has its whole step in
// one launch; of several (up to kMuonMaxSlabs), their parts of A pass
// through the workspace; unless a plan has more than kMuonSlabRoom slabs of the
// wider kind in such matrices, which then fill the GPU by tiles.  Measured,
// by slabs and by tiles: one 128 x 8192 (64 slabs) 176 and 308 us, 128 x 65536
// (512) 444 and 644, 4 of 128 x 16384 (512) 367 and 481, 64 of 128 x 2048
// (1024) 652 and 530, 16 of 128 x 16384 (2048) 1390 and 926; 64 x 131072 (512)
// 330 and 947, 256 of 64 x 2048 (2048) 847 and 981.
constexpr int32_t kMuonSlab = 16384;
constexpr int64_t kMuonMaxSlabs = 512, kMuonSlabRoom = 768;
// Shorter side of matrices that may take wide tiles (from 400 on, 48 matrices
// of 1000 x 408 took 1267 us instead of 1131).  Right from 768 on, where wide
// tiles gain (64 matrices of 768 x 768 2717 us, 2816 by narrow ones; 4 of 2048 x
// 2048 2373 and 2478); between, a side fills too little of its last tile (64 of 512
// x 512 1145 and 1055, of 520 x 600 1989 and 1502, of 640 x 640 2292 and 1837).
constexpr int64_t kMuonWideMin = 512;
// Tiles of A and of A A are summed in pieces where few workgroups would have
// long sums: a piece is of the steps (of 32) that would share all tiles' steps
// out to the compute units, at least kMuonPieceMin, and only if the longest sum
// is kMuonPieceGain steps longer.  The pieces are joined by a launch of their
// own.  Measured, A whole and in pieces with the joining: 640 x 640 22.8 and
// 17.7 us (20 steps, 2 pieces), 1024 x 1024 27.5 and 18.2, 3981 x 136 66.4 and
// 22.1.  Runs of wide tiles sum whole, also where a short side leaves A few tiles:
// a step of one 512 x 65536 takes 6193 us so, by narrow tiles and pieces 1464; of
// one 1024 x 50304 6513 and 3002.
constexpr int64_t kMuonPieceMin = 8, kMuonPieceGain = 12;
constexpr int64_t kMuonMaxSide = int64_t(1) << 20;
constexpr int64_t kMuonRunBytes = int64_t(4) << 30;  // workspace of one run of launches
struct MuonMat {          // 96 bytes
    int64_t elem0;        // its first element in the tensor
    int64_t x[2], a, b;   // X (read and written in turn), A, B
    int64_t unit0;        // first unit of the splitting pass, within its run
    int32_t tensor;
    int32_t rows, cols;
    int32_t ld, rp;       // padded columns and rows of X
    int32_t sp;           // padded shorter side
    int32_t tall;         // rows > cols
    int32_t slabs;        // of a matrix with a short side (sp 64 or 128)
    int64_t part;         // partial sums of A, then of A A
    int32_t parts[2];     // pieces that tiles of A and of A A are summed in
};
static_assert(sizeof(MuonMat) == 96, "MuonMat layout");
struct MuonTile {         // 8 bytes
    int32_t mat;
    uint16_t i, j;        // tile row and column
};
static_assert(sizeof(MuonTile) == 8, "MuonTile layout");
// Compute units of the GPU that tiles are dealt out to.
constexpr int64_t kMuonSlots = 256;
struct MuonRun {          // matrices [mat0, mat1) that share a run of launches
    int32_t mat0, mat1;
    int64_t units;        // of the splitting pass
    // tiles of the symmetric products, and of X: wide ones, then others
    int64_t sym0, wide_sym, nsym;
    int64_t full0, wide_full, nfull;
    // slabs of matrices of a short side of at most 64 (then 128): of `slabs`
    // in the table from full0 on, the first `narrow`; 0: products by tiles
    int64_t slabs, narrow;
    int32_t wide;         // wide tiles
    int32_t pair_sym, pair_full;  // the others by two groups of wavefronts each
    int32_t most_slabs;   // of one matrix
    int32_t most_parts[2];  // of one matrix
};

// Workspace layout (byte offsets from the workspace base, 256-aligned).
// `counters` holds the arrival counters of the step kernels' commit.
struct Layout {
    size_t counters, group_wd, tensors, spans, codebook, partials, blockfac,
        blockspan, packs, pack_off, pack_td, total;
    // gradient lists: items, small tensors, arrival counters and sums of the
    // tensors
    size_t gitems, gsmall, gcount, gsum;
    // Muon: matrices, tiles of the symmetric products and of X, the region
    // the runs share
    size_t mats, sym, full, muon;
};

// Quantization maps.  A normalised magnitude a in [0, 1] maps to the largest
// j with thr[j] <= a.  The search starts from a bucket table indexed by a's
// exponent and top kLutMantBits mantissa bits over [2^-26, 2): lut[bucket]
// is the index of the bucket's smallest value, and table construction
// checks that no bucket holds more than one threshold, so one comparison
// finishes the search.  Every threshold of every map is above 2^-26.
constexpr int kLutMantBits = 8;
constexpr int kLutBaseExp = 127 - 26;  // biased exponent of 2^-26
constexpr int kLutBinades = 27;        // 2^-26 ... [1, 2)
constexpr int kLutBuckets = kLutBinades << kLutMantBits;

struct QuantMap {
    float vals[256];       // sorted magnitudes (first 2^mb used)
    float thr[260];        // thr[j] = fl32((vals[j-1] + vals[j]) / 2), thr[0] = 0,
                           // thr[2^mb...] = +inf (ends the search)
    uint8_t lut[kLutBuckets];
};

struct Codebook {          // signed map for m, unsigned map for v
    QuantMap m8, v8, m4, v4;
};

struct PrepArgs {
    const double *group_wd;
    int32_t ngroups;
    int32_t sched;        // OPTIM_SCHED_*
    float *lr_dev;
    const float *inv_scale;
    const float *found_inf;
    int32_t *step_dev;
    int32_t *iter_dev;
    double lr_max, lr_min;
    int32_t K;
    double beta1, beta2, beta3, alpha, eps;
};

struct StepArgs {
    PrepArgs prep;            // inputs of the per-step scalars
    uint32_t *done;           // arrival counters (workspace), 0 between steps
    int32_t commit;           // this kernel publishes step / lr / iteration
    const TensorDesc *tensors;
    const SpanDesc *spans;    // nspans + 1 entries (sentinel at the end)
    int32_t nspans;
    int64_t unit0;            // this launch covers units [unit0, nunits)
    int64_t nunits;
    int64_t tile;             // elements per unit
    double *partials;         // Adam-mini: one per unit; LAMB: two per unit;
                              // gradient norm: one per workgroup (+ stage 2)
    int64_t npartials;        // capacity of partials
    float *blockfac;          // per block: Adam-mini lr/bc1/h, LAMB lr*trust;
                              // fp16 scaled moments: the maxima slots
    const int32_t *blockspan; // span index of each block (Adam-mini shared-v
                              // block; LAMB or scaled-moment tensor)
    int32_t block0;           // Adam-mini finalize: blocks [block0, nblocks)
    int32_t nblocks;
    const Codebook *codebook;
    int32_t bits, block;
    int32_t interleaved;      // blockwise 2-state: m and v codes (and absmax)
                              // side by side in qm (absmax_m); AdamW /
                              // AdEMAMix: the moments of a tensor in one
                              // array, in blocks of kMomentBlock elements
    float *found_inf;         // finite check output
    int32_t cus;              // compute units of the device
    const PackDesc *packs;    // packs of small tensors (elementwise plans)
    const int32_t *pack_off;
    const PackMember *pack_td;
    int64_t pack_unit0;       // units [pack_unit0, nunits) of the plan are packs
    int32_t grid_request;     // persistent workgroups (0 = see units_per_wg)
    int32_t units_per_wg;     // without a persistent grid: consecutive units
                              // per workgroup (set by the launcher)
};

// Kernel trace of a plan (optim_plan_trace): while one of a traced plan's
// entry points runs, g_trace points at its trace and every launch takes the
// next start / stop event pair, which the kernel's dispatch stamps itself
// (hipExtLaunchKernel); nothing is added to the stream.
struct TraceRec {
    const char *name;  // the launch site's kernel expression (a literal)
    int64_t grid;      // workgroups
    hipEvent_t start, stop;
};
struct Trace {
    std::vector<TraceRec> recs;  // capacity: one pair per launch
    size_t used = 0;
    int64_t dropped = 0;         // launches after the trace was full
    std::deque<std::pair<const char *, std::string>> names;  // cleaned names (stable addresses)
};
extern thread_local Trace *g_trace;
// The event pair for the next launch of `name` over `grid` workgroups, or
// nullptr (no trace, or the trace is full).
TraceRec *trace_slot(const char *name, int64_t grid);

// Launchers (kernels_*.hip).  Return the hipError_t of the launch.  Step
// launchers always start at least one workgroup (the commit must run even
// for an empty plan).
hipError_t launch_adamw(const StepArgs &a, int pk, int gk, hipStream_t s);
hipError_t launch_ademamix(const StepArgs &a, int pk, int gk, hipStream_t s);
// Adam-mini runs its three kernels segment by segment: a segment is a run of
// whole tensors (units [unit_begin, unit_end), shared-v blocks
// [block_begin, block_end)), either all with shared v and at most a bounded
// number of gradient bytes, or all with full v (no block sums).
struct MiniSegment {
    int64_t unit_begin, unit_end;
    int32_t block_begin, block_end;
};
hipError_t launch_adam_mini(const StepArgs &a, int pk, int gk, const MiniSegment *segs, int32_t nsegs,
                            hipStream_t s);
hipError_t launch_lion(const StepArgs &a, int pk, int gk, hipStream_t s);
// AdamW with 16-bit moments and per-tensor scales (sk: S_F16 / S_BF16)
hipError_t launch_adamw_scaled(const StepArgs &a, int pk, int gk, int sk, hipStream_t s);
hipError_t launch_lamb(const StepArgs &a, int pk, int gk, hipStream_t s);
hipError_t launch_blockwise(const StepArgs &a, int gk, bool ademamix, hipStream_t s);
hipError_t launch_check_finite(const StepArgs &a, int gk, hipStream_t s);
// Workgroups of the finite check / gradient norm pass for a plan.
int64_t finite_pass_grid(int64_t nunits, int64_t tile, int32_t grid_request);
// Partial sums the gradient norm pass needs (both reduction stages).
int64_t norm_partials(int64_t nunits, int64_t tile, int32_t grid_request);
hipError_t launch_grad_norm(const StepArgs &a, int gk, const float *inv_scale, double max_norm,
                            float *norm_out, float *clip_out, hipStream_t s);
// Muon (kernels_muon.hip)
struct MuonArgs {
    const MuonMat *mats;
    const MuonTile *sym, *full;
    char *ws;             // the region the runs share
    int32_t mat0, mat1;   // this run's matrices
    int32_t tiles;        // of the symmetric products, per piece
    float qa, qb, qc;     // the quintic
    int32_t scale_kind;
    // matrices of one slab: [lone0, nmats), the first lone_narrow of them of
    // sp 64; units from lone_unit0 on
    int32_t lone0, lone_narrow, nmats;
    int64_t lone_unit0;
};
hipError_t launch_muon_slabs(const StepArgs &a, const MuonArgs &ma, const MuonRun &R, int pk, int gk, int32_t steps,
                             int32_t nesterov, bool commit, hipStream_t s);
hipError_t launch_muon_lone(const StepArgs &a, const MuonArgs &ma, int pk, int gk, int32_t steps, int32_t nesterov,
                            hipStream_t s);
hipError_t launch_muon(const StepArgs &a, const MuonArgs &ma, int pk, int gk, int32_t steps, int32_t nesterov,
                       const MuonRun *runs, int32_t nruns, hipStream_t s);

// Gradient lists (kernels_grads.hip).  kind: OPTIM_NORM_*.
struct GradArgs {
    const GradItem *items;
    const GradSmall *small;
    uint32_t *count;       // per tensor: items that have arrived, 0 between calls
    uint32_t *done;        // arrival counters of the launch, 0 between calls
    double *partials;      // one per item of a tensor of several
    double *sums;          // one per tensor
    int32_t ntensors;
    int32_t nitems;
    int32_t nsmall;
    int32_t keep0;         // items from here on are left in the cache
};
hipError_t launch_grad_norms(const GradArgs &a, int gk, int kind, const float *inv_scale, double max_norm,
                             float *found_inf, float *norms, float *total, float *coef, hipStream_t s);
hipError_t launch_clip_grads(const GradArgs &a, int gk, const float *coef, const float *found_inf, hipStream_t s);
hipError_t launch_clip_coef(const float *norms, int64_t count, int kind, const float *inv_scale, double max_norm,
                            float *total, float *coef, hipStream_t s);
// Experts' weight gradients (kernels_expert.hip)
struct ExpertArgs {
    const char *x, *dy;
    int64_t ldx, ldy;     // bytes between rows
    const int32_t *offsets;
    char *dw;
    float *parts;         // partial sums [pieces][experts][m][n], or NULL
    const float *scale;
    int32_t experts, tokens, m, n;
    int32_t mt, nt;       // tiles of one expert's dW
    int32_t pieces;       // pieces of a run
    int32_t accumulate;
    int32_t out_vec;      // four neighbouring elements of dW are one access
};
int32_t expert_pieces(int32_t experts, int64_t tokens, int64_t m, int64_t n);
hipError_t launch_expert_grad(const ExpertArgs &a, bool bf16, bool out_f32, bool direct, hipStream_t s);
hipError_t launch_scaler_update(float *scale, float *inv_scale, int32_t *tracker, const float *found_inf,
                                double growth, double backoff, int32_t interval, hipStream_t s);
hipError_t launch_quantize(const Codebook *cb, int bits, int block, int is_signed, const float *x,
                           int64_t n, uint8_t *codes, float *absmax, hipStream_t s);
hipError_t launch_dequantize(const Codebook *cb, int bits, int block, int is_signed, const uint8_t *codes,
                             const float *absmax, int64_t n, float *x, hipStream_t s);
hipError_t launch_remainder_split(const float *x, uint16_t *b, int16_t *r, int64_t n,
                                  hipStream_t s);
hipError_t launch_remainder_reconstruct(const uint16_t *b, const int16_t *r, float *x,
                                        int64_t n, hipStream_t s);

}  // namespace optim
