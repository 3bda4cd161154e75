// api.cpp -- C ABI of the fused AdamW-family optimizer step: validation,
// plan tables (tensor descriptors, unit spans, weight-decay groups,
// quantization tables), workspace layout and launches.  Declared in
// include/optim_step.h, which documents each entry point and its sources,
// include/optim_grads.h and include/optim_muon.h.
#include "optim_grads.h"
#include "optim_muon.h"
#include "optim_step.h"
#include "plan.h"

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <memory>
#include <mutex>
#include <string>
#include <vector>

using namespace optim;

namespace optim {
thread_local Trace *g_trace = nullptr;

TraceRec *trace_slot(const char *name, int64_t grid) {
    Trace *t = g_trace;
    if (!t) return nullptr;
    if (t->used >= t->recs.size()) {
        ++t->dropped;
        return nullptr;
    }
    TraceRec &r = t->recs[t->used++];
    r.name = name;
    r.grid = grid;
    return &r;
}
}  // namespace optim

namespace {

thread_local std::string g_err;

int fail(int code, const std::string &msg) {
    g_err = msg;
    return code;
}

// What an entry point's body throws (the host is out of memory) becomes a status:
// no exception leaves the library.
int out_of_memory() noexcept {
    try {
        g_err = "the host is out of memory";
    } catch (...) {
        g_err = "no host memory";  // short enough to need none
    }
    return OPTIM_EINVAL;
}
#define OPTIM_CATCH \
    catch (...) { return out_of_memory(); }

#define HIP_OK(expr)                                                                 \
    do {                                                                             \
        hipError_t e_ = (expr);                                                      \
        if (e_ != hipSuccess)                                                        \
            return fail(OPTIM_EHIP, std::string(#expr) + ": " + hipGetErrorString(e_)); \
    } while (0)

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// ---------------------------------------------------------------- codebook
// Dynamic map with mb magnitude bits (see optim_quant_codebook).
void dynamic_map(int mb, float *vals, float *thr) {
    std::vector<float> M;
    M.reserve(size_t(1) << mb);
    M.push_back(0.0f);
    for (int e = 0; e < mb; ++e) {
        const int nk = 1 << (mb - 1 - e);
        const double dec = std::pow(10.0, -(double)e);
        for (int k = 0; k < nk; ++k)
            M.push_back((float)(dec * (0.1 + 0.9 * (double)(k + 1) / (double)nk)));
    }
    std::sort(M.begin(), M.end());
    for (size_t j = 0; j < M.size(); ++j) {
        vals[j] = M[j];
        thr[j] = j == 0 ? 0.0f : (float)(((double)M[j - 1] + (double)M[j]) * 0.5);
    }
}

float bits_to_float(uint32_t u) {
    float f;
    std::memcpy(&f, &u, sizeof f);
    return f;
}

// Largest j >= 1 with thr[j] <= a, else 0 (the threshold rule itself).
int threshold_index(const float *thr, int count, float a) {
    int idx = 0;
    for (int j = 1; j < count; ++j)
        if (thr[j] <= a) idx = j;
    return idx;
}

// Values, thresholds and the bucket table of one map.  Returns false if a
// bucket would hold two thresholds or a threshold lies below the table.
bool build_map(int mb, QuantMap &q) {
    std::memset(&q, 0, sizeof q);
    dynamic_map(mb, q.vals, q.thr);
    const int count = 1 << mb;
    for (int j = count; j < (int)(sizeof q.thr / sizeof q.thr[0]); ++j) q.thr[j] = INFINITY;
    const uint32_t shift = 23 - kLutMantBits;
    if (threshold_index(q.thr, count, bits_to_float(((uint32_t)kLutBaseExp << 23) - 1)) != 0) return false;
    for (int b = 0; b < kLutBuckets; ++b) {
        const uint32_t lo = (uint32_t)(b + (kLutBaseExp << kLutMantBits)) << shift;
        const uint32_t hi = lo + (1u << shift) - 1u;
        const int ilo = threshold_index(q.thr, count, bits_to_float(lo));
        const int ihi = threshold_index(q.thr, count, bits_to_float(hi));
        if (ihi - ilo > 1) return false;
        q.lut[b] = (uint8_t)ilo;
    }
    return true;
}

// ---------------------------------------------------------------- plan build
struct Built {
    std::vector<TensorDesc> tensors;
    std::vector<SpanDesc> spans;  // with sentinel
    std::vector<int32_t> blockspan;
    std::vector<double> group_wd;
    int64_t nunits = 0;
    int64_t tile = 0;
    int32_t grid = 0;        // requested persistent workgroups
    bool states16 = false;   // AdamW moments stored in 16 bits with scales
    int64_t npartials = 0;   // capacity of the partials region
    int32_t nblocks = 0;
    std::vector<MiniSegment> segs;  // Adam-mini launch segments
    bool interleaved = false;       // blockwise: interleaved state layout
    std::vector<PackDesc> packs;    // packs of small tensors
    std::vector<int32_t> pack_off;
    std::vector<PackMember> pack_td;
    int64_t pack_unit0 = 0;         // first pack unit (packs come last)
    std::vector<GradItem> gitems;      // gradient lists
    std::vector<GradSmall> gsmall;
    int64_t gbytes = 0;
    int32_t gkeep0 = 0;
    std::vector<MuonMat> mats;      // Muon
    std::vector<MuonTile> sym, full;
    std::vector<MuonRun> runs;
    int64_t muon_bytes = 0;         // of the region the runs share
    int64_t muon_tiles = 0, muon_end = 0;
    int run_kind = -1;
    int32_t lone0 = -1, lone_narrow = 0;  // matrices of one slab
    int64_t lone_unit0 = 0;
    Layout L{};
};

struct Range {
    uintptr_t lo, hi;
    bool written;
    int tensor;
    const char *what;
};

// no written buffer may overlap any other buffer of the plan
int check_overlaps(std::vector<Range> &ranges) {
    std::sort(ranges.begin(), ranges.end(), [](const Range &a, const Range &b) { return a.lo < b.lo; });
    uintptr_t end_all = 0, end_w = 0;
    const Range *cov_all = nullptr, *cov_w = nullptr;
    for (const Range &r : ranges) {
        const Range *hit = nullptr;
        if (r.written && r.lo < end_all) hit = cov_all;
        else if (!r.written && r.lo < end_w) hit = cov_w;
        if (hit)
            return fail(OPTIM_EINVAL, "buffers overlap: tensor " + std::to_string(hit->tensor) + " " +
                                          hit->what + " and tensor " + std::to_string(r.tensor) + " " +
                                          r.what);
        if (r.hi > end_all) { end_all = r.hi; cov_all = &r; }
        if (r.written && r.hi > end_w) { end_w = r.hi; cov_w = &r; }
    }
    return OPTIM_OK;
}

int check_hp_beta(double b, const char *name) {
    if (!(b >= 0.0 && b < 1.0))
        return fail(OPTIM_EINVAL, std::string("invalid ") + name + " (need 0 <= beta < 1)");
    return OPTIM_OK;
}

bool is_blockwise(int32_t algo) { return algo == OPTIM_ALGO_BLOCKWISE || algo == OPTIM_ALGO_BLOCKWISE_ADEMAMIX; }

int64_t count_of(int64_t n, int64_t of) { return (n + of - 1) / of; }
int64_t round_up(int64_t n, int64_t to) { return count_of(n, to) * to; }
// Whether a matrix may take wide tiles (in a plan with enough of them): below,
// padding to whole wide tiles costs more than they gain.
bool wide_matrix(int64_t rows, int64_t cols) { return std::min(rows, cols) >= kMuonWideMin; }

// Workgroup b runs on XCD b mod kXcds, each with an L2 of its own.
constexpr int kXcds = 8;

// Appends a run's tiles in launch order.  Blocks of up to 4 x 4 tiles of one
// matrix (`block` numbers them) stay on one XCD, whose L2 then holds their
// operands once; a block goes to the XCD with the fewest tiles, and single
// tiles then move until all XCDs have as many (but for one: -1 fills up).
// Measured against tiles dealt out one by one: 48 matrices of 1000 x 408 56 us
// a Gram matrix and 64, 8 of 512 x 512 a step 335 us and 367.  Fewer than 8
// blocks are dealt out so.
void order_tiles(const std::vector<std::pair<int64_t, MuonTile>> &tiles, std::vector<MuonTile> &out) {
    std::vector<MuonTile> of[kXcds];
    const bool blocks = !tiles.empty() && tiles.back().first - tiles.front().first + 1 >= kXcds;
    int x = 0;
    for (size_t k = 0; k < tiles.size(); ++k) {
        if (k == 0 || !blocks || tiles[k].first != tiles[k - 1].first) {
            x = 0;
            for (int y = 1; y < kXcds; ++y)
                if (of[y].size() < of[x].size()) x = y;
        }
        of[x].push_back(tiles[k].second);
    }
    for (;;) {
        int most = 0, least = 0;
        for (int y = 1; y < kXcds; ++y) {
            if (of[y].size() > of[most].size()) most = y;
            if (of[y].size() < of[least].size()) least = y;
        }
        if (of[most].size() <= of[least].size() + 1) break;
        of[least].push_back(of[most].back());
        of[most].pop_back();
    }
    size_t longest = 0;
    for (const auto &v : of) longest = std::max(longest, v.size());
    for (size_t k = 0; k < longest; ++k)
        for (const auto &v : of) out.push_back(k < v.size() ? v[k] : MuonTile{-1, 0, 0});
    while (!out.empty() && out.back().mat < 0 && !tiles.empty()) out.pop_back();
}

// A run's tiles of one product, in whole rounds of wide tiles over the GPU and,
// where they are at most half a round, the rest as four narrow tiles each: a
// round of a few wide tiles takes as long as a full one (4 of 4096 x 4096: a
// round of A 305 us, the rest of 32 wide tiles as 121 narrow ones 110).
// upper: tiles on and above the diagonal of square arrays.
void add_product(const Built &B, const MuonRun &R, bool upper, std::vector<MuonTile> &out, int64_t &first,
                 int64_t &wide, int64_t &narrow) {
    typedef std::vector<std::pair<int64_t, MuonTile>> Tiles;
    Tiles tiles, rest;
    const int64_t tile = R.wide ? kMuonWideTile : kMuonTile;
    int64_t block = 0;
    for (int32_t m = R.mat0; m < R.mat1; ++m) {
        const MuonMat &M = B.mats[m];
        const int64_t rows = count_of(upper ? M.sp : M.rp, tile), cols = count_of(upper ? M.sp : M.ld, tile);
        for (int64_t a = 0; a < rows; a += 4)
            for (int64_t b = upper ? a : 0; b < cols; b += 4, ++block)
                for (int64_t i = a; i < std::min(a + 4, rows); ++i)
                    for (int64_t j = upper ? std::max(b, i) : b; j < std::min(b + 4, cols); ++j)
                        tiles.push_back({block, MuonTile{m, (uint16_t)i, (uint16_t)j}});
    }
    first = (int64_t)out.size();
    if (!R.wide) {
        std::swap(tiles, rest);
    } else {
        const size_t over = tiles.size() % kMuonSlots;
        if (over <= kMuonSlots / 2) {
            for (size_t k = tiles.size() - over; k < tiles.size(); ++k) {
                const MuonTile t = tiles[k].second;
                const MuonMat &M = B.mats[t.mat];
                for (int i = 0; i < 2; ++i)
                    for (int j = upper && t.i == t.j ? i : 0; j < 2; ++j)
                        if ((2 * t.i + i) * kMuonTile < (upper ? M.sp : M.rp) && (2 * t.j + j) * kMuonTile < (upper ? M.sp : M.ld))
                            rest.push_back({tiles[k].first, MuonTile{t.mat, (uint16_t)(2 * t.i + i), (uint16_t)(2 * t.j + j)}});
            }
            tiles.resize(tiles.size() - over);
        }
    }
    order_tiles(tiles, out);
    wide = (int64_t)out.size() - first;
    order_tiles(rest, out);
    narrow = (int64_t)out.size() - first - wide;
}

// The pieces of the sums of A and A A (see kMuonPieceMin); partial sums as 128 x
// 128 tiles of fp32 [piece][tile row][tile column].  (Decided for the plan too.)
void add_pieces(Built &B) {
    auto steps = [](const MuonMat &M, int k) { return (int64_t)((k ? M.sp : std::max(M.rp, M.ld)) / 32); };
    int64_t total[2] = {0, 0}, longest[2] = {0, 0}, piece[2];
    for (int k = 0; k < 2; ++k) {
        for (const MuonMat &M : B.mats) {
            if (M.slabs) continue;
            const int64_t nt = count_of(M.sp, kMuonTile);
            total[k] += nt * (nt + 1) / 2 * steps(M, k);
            longest[k] = std::max(longest[k], steps(M, k));
        }
        piece[k] = std::max(kMuonPieceMin, count_of(total[k], kMuonSlots));
    }
    int64_t most = 0;
    for (MuonRun &R : B.runs) {
        R.most_parts[0] = R.most_parts[1] = 1;
        int64_t used = 0;
        for (int32_t m = R.mat0; m < R.mat1; ++m) {
            MuonMat &M = B.mats[m];
            M.part = B.muon_bytes + used;
            for (int k = 0; k < 2; ++k) {
                M.parts[k] = 1;
                if (!R.slabs && !R.wide && longest[k] >= piece[k] + kMuonPieceGain)
                    M.parts[k] = (int32_t)std::max<int64_t>(1, steps(M, k) / piece[k]);
                R.most_parts[k] = std::max(R.most_parts[k], M.parts[k]);
            }
            const int64_t nt = count_of(M.sp, kMuonTile), parts = std::max(M.parts[0], M.parts[1]);
            if (parts > 1) used += parts * nt * nt * kMuonTile * kMuonTile * 4;
        }
        most = std::max(most, used);
    }
    B.muon_bytes += most;
}

// The tile tables of the runs, from their matrices.  Plans whose products
// have fewer narrow tiles than there are compute units give each tile two
// groups of wavefronts (a lone group takes 0.66 us a step, two on a compute
// unit 0.8 us for a step of each).  (Decided for the plan, not run by run: the
// groups sum in another order, and results do not depend on the bound on a
// run.)
void add_tiles(Built &B) {
    int64_t sym = 0, full = 0;
    for (const MuonMat &M : B.mats) {
        if (M.slabs) continue;
        const int64_t nt = count_of(M.sp, kMuonTile);
        sym += nt * (nt + 1) / 2;
        full += count_of(M.rp, kMuonTile) * count_of(M.ld, kMuonTile);
    }
    for (MuonRun &R : B.runs) {
        if (R.slabs) {
            R.full0 = (int64_t)B.full.size();
            for (int32_t m = R.mat0; m < R.mat1; ++m)
                for (int32_t k = 0; k < B.mats[m].slabs; ++k) B.full.push_back(MuonTile{m, (uint16_t)k, 0});
            continue;
        }
        add_product(B, R, true, B.sym, R.sym0, R.wide_sym, R.nsym);
        add_product(B, R, false, B.full, R.full0, R.wide_full, R.nfull);
        R.pair_sym = sym <= kMuonSlots;
        R.pair_full = full <= kMuonSlots;
    }
    add_pieces(B);
}

// How a matrix is multiplied: by wide tiles, by tiles, through several slabs or
// through one, of a short side padded to 64 or 128.
enum MuonKind { kWide = 0, kTiles, kSlabs64, kSlabs128, kLone64, kLone128, kMuonKinds };

int64_t muon_slabs(int64_t rows, int64_t cols) {
    const int64_t sp = std::min(rows, cols) <= 64 ? 64 : 128, l = kMuonSlab / sp;
    return (std::max(rows, cols) + l - 1) / l;
}

MuonKind muon_kind(int64_t rows, int64_t cols, bool wide, bool slabs128) {
    const int64_t s = std::min(rows, cols), p = muon_slabs(rows, cols);
    if (s <= 128 && p == 1) return s <= 64 ? kLone64 : kLone128;
    if (s <= 64 && p <= kMuonMaxSlabs) return kSlabs64;
    if (s <= 128 && p <= kMuonMaxSlabs && slabs128) return kSlabs128;
    return wide && wide_matrix(rows, cols) ? kWide : kTiles;
}

// Muon: the matrices of tensor i and their arrays.  A run takes matrices of
// one kind (slabs: of both) until their arrays pass `cap` bytes.
int add_matrices(const std::string &ti, int i, int64_t numel, int64_t rows, int64_t cols, MuonKind kind, int64_t cap,
                 Built &B) {
    if (numel % (rows * cols) != 0) return fail(OPTIM_EINVAL, ti + "numel must be a multiple of rows * cols");
    const int64_t count = numel / (rows * cols);
    const bool slabs = kind >= kSlabs64, lone = kind >= kLone64;
    const int run_kind = slabs ? kSlabs64 : kind;
    const int64_t tile = kind == kWide ? kMuonWideTile : kMuonTile;
    const int64_t rp = round_up(rows, 32), ld = round_up(cols, 32);
    const int64_t sp = !slabs ? std::min(rp, ld) : kind == kSlabs64 || kind == kLone64 ? 64 : 128;
    const int64_t p = slabs ? muon_slabs(rows, cols) : 0;
    // X twice (slabs: once, in place), A and B (slabs: two sets of parts of A)
    const int64_t xbytes = lone ? 0 : slabs ? p * kMuonSlab * 4 : rp * ld * 4;
    const int64_t abytes = lone ? 0 : slabs ? p * sp * sp * 4 : sp * sp * 4;
    const int64_t bytes = (slabs ? 1 : 2) * xbytes + 2 * abytes;
    const int64_t nt = count_of(sp, tile);
    const int64_t tiles = slabs ? p : nt * (nt + 1) / 2 + count_of(rp, tile) * count_of(ld, tile);
    if (count > INT32_MAX / 4 || (int64_t)B.mats.size() + count >= ((int64_t)1 << 23) ||
        tiles > (((int64_t)1 << 26) - B.muon_tiles) / count)
        return fail(OPTIM_EUNSUPPORTED, ti + "too many matrices or tiles");
    B.muon_tiles += tiles * count;
    for (int64_t k = 0; k < count; ++k) {
        int64_t used = B.muon_end;
        if (!lone && (B.runs.empty() || B.run_kind != run_kind || used + bytes > cap)) {
            const int32_t m = (int32_t)B.mats.size();
            MuonRun R{};
            R.mat0 = R.mat1 = m;
            R.wide = kind == kWide;
            B.runs.push_back(R);
            B.run_kind = run_kind;
            used = 0;
        }
        MuonMat M{};
        M.elem0 = k * rows * cols;
        M.x[0] = used;
        M.x[1] = M.x[0] + (slabs ? 0 : xbytes);
        M.a = M.x[1] + xbytes;
        M.b = M.a + abytes;
        M.tensor = i;
        M.rows = (int32_t)rows;
        M.cols = (int32_t)cols;
        M.ld = (int32_t)ld;
        M.rp = (int32_t)rp;
        M.sp = (int32_t)sp;
        M.tall = rows > cols;
        M.slabs = (int32_t)p;
        const int32_t m = (int32_t)B.mats.size();
        if (!lone) {
            MuonRun &R = B.runs.back();
            M.unit0 = R.units;
            R.mat1 = m + 1;
            if (slabs) {
                R.slabs += p;
                R.most_slabs = std::max(R.most_slabs, (int32_t)p);
                if (sp == 64) R.narrow += p;
            } else {
                R.units += count_of(rp * ld, kMuonUnit);
            }
            B.muon_end = used + bytes;
            B.muon_bytes = std::max(B.muon_bytes, B.muon_end);
        } else if (B.lone0 < 0) {
            B.lone0 = m;
            B.lone_unit0 = B.nunits;
        }
        if (kind == kLone64) ++B.lone_narrow;
        B.mats.push_back(M);
        // a span per matrix: its units' sums of squares give its norm
        B.blockspan.push_back((int32_t)B.spans.size());
        B.spans.push_back(SpanDesc{B.nunits, M.elem0, rows * cols, i, B.nblocks});
        B.nunits += (rows * cols + B.tile - 1) / B.tile;
        ++B.nblocks;
    }
    return OPTIM_OK;
}

// Muon: the matrices of the list, kind by kind, so that a run's are of one
// kind; wide tiles where all matrices that may take them make a round of the
// GPU, slabs of the wider kind where all of them are few.
int add_muon(const optim_tensor_list *list, int64_t cap, Built &B) {
    int64_t wide_full = 0, slabs128 = 0;
    for (int i = 0; i < list->n; ++i) {
        if (list->numel[i] == 0) continue;
        const int64_t r = list->rows[i], c = list->cols[i];
        if (r < 1 || c < 1 || r > kMuonMaxSide || c > kMuonMaxSide)
            return fail(OPTIM_EINVAL, "tensor " + std::to_string(i) + ": rows and cols must be in [1, 2^20]");
        const MuonKind kind = muon_kind(r, c, true, true);
        if (kind == kSlabs128) slabs128 += std::min(list->numel[i] / (r * c), kMuonSlabRoom + 1) * muon_slabs(r, c);
        if (kind == kWide)
            wide_full += list->numel[i] / (r * c) * count_of(r, kMuonWideTile) * count_of(c, kMuonWideTile);
    }
    for (int kind = 0; kind < kMuonKinds; ++kind)
        for (int i = 0; i < list->n; ++i) {
            if (list->numel[i] == 0) continue;
            const int64_t r = list->rows[i], c = list->cols[i];
            if (muon_kind(r, c, wide_full >= kMuonSlots, slabs128 <= kMuonSlabRoom) != kind) continue;
            if (const int rc = add_matrices("tensor " + std::to_string(i) + ": ", i, list->numel[i], r, c, (MuonKind)kind,
                                            cap, B))
                return rc;
        }
    if (B.lone0 < 0) {
        B.lone0 = (int32_t)B.mats.size();
        B.lone_unit0 = B.nunits;
    }
    add_tiles(B);
    return OPTIM_OK;
}

// Gradient lists: the item table (see GradItem) and its workspace.
int build_grads(const optim_tensor_list *list, const optim_plan_opts *opts, Built &B) {
    const int n = list->n;
    if (n < 0) return fail(OPTIM_EINVAL, "negative tensor count");
    if (list->grad_dtype != OPTIM_F32 && list->grad_dtype != OPTIM_BF16 && list->grad_dtype != OPTIM_F16)
        return fail(OPTIM_EDTYPE, "grad_dtype must be OPTIM_F32, OPTIM_BF16 or OPTIM_F16");
    if (opts && (opts->grid || opts->tile || opts->state_dtype || opts->state_layout))
        return fail(OPTIM_EUNSUPPORTED, "gradient lists take no grid, tile, state_dtype or state_layout");
    if (n > 0 && (!list->numel || !list->grad)) return fail(OPTIM_EINVAL, "numel and grad arrays are required");
    const size_t gsz = list->grad_dtype == OPTIM_F32 ? 4 : 2;
    std::vector<Range> ranges;
    for (int i = 0; i < n; ++i) {
        const std::string ti = "tensor " + std::to_string(i) + ": ";
        const int64_t numel = list->numel[i];
        if (numel < 0) return fail(OPTIM_EINVAL, ti + "negative numel");
        if (numel > kMaxNumel) return fail(OPTIM_EINVAL, ti + "numel above 2^48");
        void *g = const_cast<void *>(list->grad[i]);
        if (numel > 0 && !g) return fail(OPTIM_EINVAL, ti + "NULL grad");
        if (!aligned(g, gsz)) return fail(OPTIM_EALIGN, ti + "grad misaligned");
        if (numel == 0) continue;
        ranges.push_back({(uintptr_t)g, (uintptr_t)g + (size_t)numel * gsz, true, i, "grad"});
        B.gbytes += numel * (int64_t)gsz;
    }
    int64_t item = kGradItemMax;
    while (item > kGradItemMin && B.gbytes < item * kGradItems) item /= 2;
    while (B.gbytes / item >= kGradMostItems / 2) item *= 2;
    item /= (int64_t)gsz;  // elements
    for (int i = 0; i < n; ++i) {
        const int64_t numel = list->numel[i];
        if (numel == 0) continue;
        char *g = static_cast<char *>(const_cast<void *>(list->grad[i]));
        if (numel <= kGradSmall) {
            B.gsmall.push_back(GradSmall{g, i, (int32_t)numel});
            continue;
        }
        const int64_t items = (numel + item - 1) / item;
        if (items + (int64_t)B.gitems.size() >= kGradMostItems) return fail(OPTIM_EUNSUPPORTED, "too many gradients in one list");
        for (int64_t k = 0; k < items; ++k)
            B.gitems.push_back(GradItem{g + k * item * (int64_t)gsz, B.npartials, i,
                                        (int32_t)std::min(item, numel - k * item), (int32_t)k, (int32_t)items});
        if (items > 1) B.npartials += items;
    }
    int64_t kept = 0;
    B.gkeep0 = (int32_t)B.gitems.size();
    while (B.gkeep0 > 0 && kept < kGradKeepBytes) kept += B.gitems[--B.gkeep0].len * (int64_t)gsz;
    if ((int64_t)(B.gitems.size() + B.gsmall.size() / 4 + 1) >= kGradMostItems)
        return fail(OPTIM_EUNSUPPORTED, "too many gradients in one list");
    if (const int rc = check_overlaps(ranges)) return rc;

    Layout &L = B.L;
    size_t off = 0;
    L.counters = off; off += align256(kCounterBytes);
    L.group_wd = L.tensors = L.spans = L.codebook = L.blockspan = L.packs = L.pack_off = L.pack_td = L.blockfac = off;
    L.gitems = off; off += align256(std::max<size_t>(1, B.gitems.size()) * sizeof(GradItem));
    L.gsmall = off; off += align256(std::max<size_t>(1, B.gsmall.size()) * sizeof(GradSmall));
    L.gcount = off; off += align256(std::max<size_t>(1, (size_t)n) * sizeof(uint32_t));
    L.gsum = off; off += align256(std::max<size_t>(1, (size_t)n) * sizeof(double));
    L.partials = off;  // the uploaded image ends here
    off += align256(std::max<int64_t>(1, B.npartials) * sizeof(double));
    L.total = off;
    return OPTIM_OK;
}

int build(const optim_tensor_list *list, int32_t algo, const optim_plan_opts *opts, Built &B) {
    if (!list) return fail(OPTIM_EINVAL, "tensor list is NULL");
    if (algo == OPTIM_ALGO_GRADS) return build_grads(list, opts, B);
    if (algo < OPTIM_ALGO_ADAMW || algo > OPTIM_ALGO_MUON)
        return fail(OPTIM_EINVAL, "unknown algorithm");
    const bool muon = algo == OPTIM_ALGO_MUON;
    const int n = list->n;
    if (n < 0) return fail(OPTIM_EINVAL, "negative tensor count");
    const int32_t pdt = list->param_dtype;
    if (pdt != OPTIM_F32 && pdt != OPTIM_BF16 && pdt != OPTIM_F16)
        return fail(OPTIM_EDTYPE, "param_dtype must be OPTIM_F32, OPTIM_BF16 or OPTIM_F16");
    if (list->grad_dtype != OPTIM_F32 && list->grad_dtype != OPTIM_BF16)
        return fail(OPTIM_EDTYPE, "grad_dtype must be OPTIM_F32 or OPTIM_BF16");
    const bool masterw = list->master != nullptr;
    if (masterw && pdt == OPTIM_F32) return fail(OPTIM_EINVAL, "master weights need a BF16 or F16 model param");
    if (pdt == OPTIM_F16 && !masterw) return fail(OPTIM_EUNSUPPORTED, "F16 params need fp32 master weights");
    if (masterw && algo != OPTIM_ALGO_ADAMW && algo != OPTIM_ALGO_ADEMAMIX && !muon)
        return fail(OPTIM_EUNSUPPORTED, "master weights are supported for AdamW, AdEMAMix and Muon");
    const bool bf16p = pdt == OPTIM_BF16 && !masterw;  // bf16 + remainder
    if (pdt != OPTIM_F32 && is_blockwise(algo))
        return fail(OPTIM_EUNSUPPORTED, "blockwise states take fp32 params only");
    int bits = 0, block = 0;
    if (is_blockwise(algo)) {
        if (!opts) return fail(OPTIM_EINVAL, "blockwise plans need opts (bits, block)");
        bits = opts->bits;
        block = opts->block;
        // a block is L = block/E lanes of one wavefront (E = 4 codes per lane
        // up to block 256, else 8), L a power of two in [16, 64]
        if (bits != 8 && bits != 4) return fail(OPTIM_EINVAL, "bits must be 8 or 4");
        const bool ok = bits == 8 ? (block == 64 || block == 128 || block == 256)
                                  : (block == 128 || block == 256 || block == 512);
        if (!ok)
            return fail(OPTIM_EINVAL, bits == 8 ? "8-bit block must be 64, 128 or 256"
                                                : "4-bit block must be 128, 256 or 512");
    }
    const int32_t layout = opts ? opts->state_layout : OPTIM_LAYOUT_SEPARATE;
    if (layout != OPTIM_LAYOUT_SEPARATE && layout != OPTIM_LAYOUT_INTERLEAVED)
        return fail(OPTIM_EINVAL, "unknown state_layout");
    const bool adam_like = algo == OPTIM_ALGO_ADAMW || algo == OPTIM_ALGO_ADEMAMIX;
    if (layout == OPTIM_LAYOUT_INTERLEAVED && algo != OPTIM_ALGO_BLOCKWISE && !adam_like)
        return fail(OPTIM_EUNSUPPORTED,
                    "the interleaved state layout is for AdamW, AdEMAMix and the 2-state blockwise step");
    // blockwise: m and v codes side by side; AdamW / AdEMAMix: the moments
    // of each tensor in one array, in blocks of kMomentBlock elements
    const bool il = layout == OPTIM_LAYOUT_INTERLEAVED && algo == OPTIM_ALGO_BLOCKWISE;
    const bool mom_il = layout == OPTIM_LAYOUT_INTERLEAVED && adam_like;
    B.interleaved = il || mom_il;
    if (opts && opts->grid < 0) return fail(OPTIM_EINVAL, "negative grid");
    if (opts && opts->grid && muon) return fail(OPTIM_EUNSUPPORTED, "Muon takes no persistent grid");
    B.grid = opts ? opts->grid : 0;
    if (opts && opts->tile < 0) return fail(OPTIM_EINVAL, "negative tile");
    if (opts && opts->segment_bytes < 0) return fail(OPTIM_EINVAL, "negative segment_bytes");
    const int64_t seg_cap = (opts && opts->segment_bytes > 0) ? opts->segment_bytes
                            : muon                            ? kMuonRunBytes
                                                              : kMiniSegmentBytes;
    bool seg_shared = false;
    int64_t seg_gbytes = 0;
    const int32_t sdt = opts ? opts->state_dtype : OPTIM_F32;
    if (sdt != OPTIM_F32 && sdt != OPTIM_F16 && sdt != OPTIM_BF16)
        return fail(OPTIM_EDTYPE, "state_dtype must be OPTIM_F32, OPTIM_F16 or OPTIM_BF16");
    const bool states16 = sdt != OPTIM_F32;
    if (states16 && algo != OPTIM_ALGO_ADAMW) return fail(OPTIM_EUNSUPPORTED, "16-bit states are for AdamW plans");
    if (states16 && masterw) return fail(OPTIM_EUNSUPPORTED, "16-bit states take fp32 or bf16 + remainder params");
    if (states16 && mom_il) return fail(OPTIM_EUNSUPPORTED, "the interleaved moment layout holds fp32 moments");
    if (n > 0 && states16 && (!list->scale_m || !list->scale_v))
        return fail(OPTIM_EINVAL, "16-bit states need scale_m and scale_v arrays");
    B.states16 = states16;
    // measured on MI355X: 2048 elements per workgroup (two groups of 4 per
    // lane, loaded at once) stream best for AdamW / AdEMAMix / Lion;
    // Adam-mini, LAMB and the two-pass fp16-state step prefer 4096 (per-unit
    // reductions), and the blockwise step amortises its LDS tables and
    // prologue over larger units
    const bool unit_sums = algo == OPTIM_ALGO_ADAM_MINI || algo == OPTIM_ALGO_LAMB || sdt == OPTIM_F16;
    // AdamW / AdEMAMix (fp32 moments) and Lion plans of (2^20, 2^24]
    // elements take the units of the early-load kernel form
    int64_t total = 0;  // elements, counted only up to past the bound
    if (n > 0 && list->numel)
        for (int i = 0; i < n && total <= kEarlyTileMaxElems; ++i)
            total += std::min<int64_t>(std::max<int64_t>(list->numel[i], 0), kMaxNumel);
    const bool early_units = (algo == OPTIM_ALGO_ADAMW || algo == OPTIM_ALGO_ADEMAMIX || algo == OPTIM_ALGO_LION) &&
                             !states16 &&
                             total > kEarlyTileMinElems && total <= kEarlyTileMaxElems;
    const int64_t tile = (opts && opts->tile > 0) ? opts->tile
                         : is_blockwise(algo) ? blockwise_tile(algo == OPTIM_ALGO_BLOCKWISE_ADEMAMIX, bits, il)
                         : unit_sums          ? kAdamMiniTile
                         : early_units        ? kEarlyTile
                                              : kDefaultTile;
    if (tile < kMinTile || tile > (1 << 24) || (tile & (tile - 1)))
        return fail(OPTIM_EINVAL, "tile must be a power of two in [1024, 2^24]");
    if (is_blockwise(algo) && tile < kMinBlockwiseTile)
        return fail(OPTIM_EINVAL, "blockwise tile must be at least 2048");
    B.tile = tile;
    if (n > 0 && (!list->numel || !list->param || !list->grad || !list->weight_decay))
        return fail(OPTIM_EINVAL, "numel, param, grad and weight_decay arrays are required");
    const bool need_mv = !is_blockwise(algo) && algo != OPTIM_ALGO_LION && !muon;
    if (n > 0 && need_mv && (!list->m || (!mom_il && !list->v)))
        return fail(OPTIM_EINVAL, mom_il ? "the m array is required" : "m and v arrays are required");
    if (n > 0 && algo == OPTIM_ALGO_LION && !list->m) return fail(OPTIM_EINVAL, "Lion needs the m array");
    if (n > 0 && muon && (!list->m || !list->rows || !list->cols))
        return fail(OPTIM_EINVAL, "Muon needs the m, rows and cols arrays");
    if (n > 0 && algo == OPTIM_ALGO_ADEMAMIX && !mom_il && !list->m2)
        return fail(OPTIM_EINVAL, "AdEMAMix needs the m2 array");
    if (n > 0 && is_blockwise(algo) && (!list->qm || (!il && !list->qv) || !list->absmax_m || (!il && !list->absmax_v)))
        return fail(OPTIM_EINVAL, il ? "interleaved blockwise plans need qm and absmax_m"
                                     : "blockwise plans need qm, qv, absmax_m and absmax_v");
    if (n > 0 && algo == OPTIM_ALGO_BLOCKWISE_ADEMAMIX && (!list->qm2 || !list->absmax_m2))
        return fail(OPTIM_EINVAL, "blockwise AdEMAMix plans need qm2 and absmax_m2");
    if (n > 0 && algo == OPTIM_ALGO_ADAM_MINI && (!list->mini_kind || !list->head_numel))
        return fail(OPTIM_EINVAL, "Adam-mini needs mini_kind and head_numel arrays");
    if (n > 0 && bf16p && !list->remainder)
        return fail(OPTIM_EUNSUPPORTED, "bf16 params need int16 remainders (fp32 master)");

    const size_t psz = pdt == OPTIM_F32 ? 4 : 2, gsz = list->grad_dtype == OPTIM_BF16 ? 2 : 4;
    std::vector<Range> ranges;
    B.tensors.assign(n, TensorDesc{});
    B.spans.clear();
    B.blockspan.clear();
    B.group_wd.clear();
    B.nunits = 0;
    B.nblocks = 0;
    B.segs.clear();
    B.packs.clear();
    B.pack_off.clear();
    B.pack_td.clear();
    // Packs: AdamW / AdEMAMix (fp32 moments) and Lion plans lay runs of
    // tensors of at most half a pack end to end in shared units of up to
    // pack_cap elements, so a workgroup serves many small tensors (one
    // prologue, every lane busy) instead of one each.
    const bool packable = (algo == OPTIM_ALGO_ADAMW || algo == OPTIM_ALGO_ADEMAMIX || algo == OPTIM_ALGO_LION) &&
                          !states16;
    const int64_t pack_cap = std::min<int64_t>(tile, kPackElems);
    std::vector<int32_t> open_pack;  // members of the pack being filled
    int64_t open_len = 0;
    auto close_pack = [&]() {
        if (open_pack.empty()) return;
        if (open_pack.size() == 1) {  // a lone member: an ordinary span
            const int32_t t = open_pack[0];
            B.spans.push_back(SpanDesc{B.nunits, 0, B.tensors[t].numel, t, -1});
        } else {
            PackDesc P{(int32_t)B.pack_td.size(), (int32_t)B.pack_off.size(), (int32_t)open_pack.size(),
                       (int32_t)open_len};
            int32_t off = 0;
            for (int32_t t : open_pack) {
                const TensorDesc &T = B.tensors[t];
                B.pack_td.push_back(PackMember{T.p, T.g, T.m, T.v, T.m2, T.rem, T.master, (int32_t)T.numel, T.group,
                                               T.vec_ok, 0});
                B.pack_off.push_back(off);
                off += (int32_t)((B.tensors[t].numel + 3) / 4 * 4);
            }
            B.pack_off.push_back(off);
            B.packs.push_back(P);  // its span is laid after all single-tensor units
        }
        if (open_pack.size() == 1) B.nunits += 1;
        open_pack.clear();
        open_len = 0;
    };
    for (int i = 0; i < n; ++i) {
        const std::string ti = "tensor " + std::to_string(i) + ": ";
        TensorDesc &T = B.tensors[i];
        const int64_t numel = list->numel[i];
        if (numel < 0) return fail(OPTIM_EINVAL, ti + "negative numel");
        if (numel > kMaxNumel) return fail(OPTIM_EINVAL, ti + "numel above 2^48");
        const double wd = list->weight_decay[i];
        if (!(wd >= 0.0) || !std::isfinite(wd)) return fail(OPTIM_EINVAL, ti + "invalid weight_decay");
        auto git = std::find(B.group_wd.begin(), B.group_wd.end(), wd);
        if (git == B.group_wd.end()) {
            if ((int)B.group_wd.size() >= kMaxGroups)
                return fail(OPTIM_EUNSUPPORTED, "more than 64 distinct weight_decay values");
            B.group_wd.push_back(wd);
            git = B.group_wd.end() - 1;
        }
        T.group = (int32_t)(git - B.group_wd.begin());
        T.numel = numel;
        T.p = list->param[i];
        T.g = list->grad[i];
        if (numel > 0 && (!T.p || !T.g)) return fail(OPTIM_EINVAL, ti + "NULL param or grad");
        if (!aligned(T.p, psz) || !aligned(T.g, gsz)) return fail(OPTIM_EALIGN, ti + "param/grad misaligned");
        bool vec = aligned(T.p, 16) && aligned(T.g, 16);
        auto add = [&](const void *ptr, size_t bytes, bool written, const char *what) {
            if (ptr && bytes) ranges.push_back({(uintptr_t)ptr, (uintptr_t)ptr + bytes, written, i, what});
        };
        add(T.p, numel * psz, true, "param");
        add(T.g, numel * gsz, false, "grad");
        if (bf16p) {
            T.rem = static_cast<uint16_t *>(list->remainder[i]);
            if (numel > 0 && !T.rem) return fail(OPTIM_EINVAL, ti + "NULL remainder");
            if (!aligned(T.rem, 2)) return fail(OPTIM_EALIGN, ti + "remainder misaligned");
            vec = vec && aligned(T.rem, 16);
            add(T.rem, numel * 2, true, "remainder");
        } else if (list->remainder && list->remainder[i]) {
            return fail(OPTIM_EINVAL, ti + (masterw ? "remainder given with master weights"
                                                    : "remainder given for fp32 params"));
        }
        if (masterw) {
            T.master = list->master[i];
            if (numel > 0 && !T.master) return fail(OPTIM_EINVAL, ti + "NULL master");
            if (!aligned(T.master, 4)) return fail(OPTIM_EALIGN, ti + "master misaligned");
            vec = vec && aligned(T.master, 16);
            add(T.master, numel * 4, true, "master");
        }
        int32_t kind = OPTIM_MINI_FULL_V;
        int64_t vlen = numel;
        if (algo == OPTIM_ALGO_ADAM_MINI) {
            kind = list->mini_kind[i];
            if (kind == OPTIM_MINI_HEAD) {
                const int64_t h = list->head_numel[i];
                if (h <= 0 || numel % h != 0)
                    return fail(OPTIM_EINVAL, ti + "head_numel must be > 0 and divide numel");
                T.block_len = h;
                vlen = numel / h;
            } else if (kind == OPTIM_MINI_SCALAR) {
                T.block_len = numel;
                vlen = numel > 0 ? 1 : 0;
            } else if (kind == OPTIM_MINI_FULL_V) {
                T.block_len = 0;
            } else {
                return fail(OPTIM_EINVAL, ti + "unknown mini_kind");
            }
        }
        T.kind = kind;
        if (mom_il) {
            // m, v (, m2) of each block of kMomentBlock elements side by side
            // in m: K kMomentBlock floats per block, the last block whole
            const int K = algo == OPTIM_ALGO_ADEMAMIX ? 3 : 2;
            if ((list->v && list->v[i]) || (list->m2 && list->m2[i]))
                return fail(OPTIM_EINVAL, ti + "interleaved moments: v and m2 must be NULL (they live in m)");
            T.m = static_cast<float *>(list->m[i]);
            if (numel > 0 && !T.m) return fail(OPTIM_EINVAL, ti + "NULL m");
            if (!aligned(T.m, 4)) return fail(OPTIM_EALIGN, ti + "m misaligned");
            T.v = T.m ? T.m + kMomentBlock : nullptr;
            T.m2 = T.m && K == 3 ? T.m + 2 * kMomentBlock : nullptr;
            vec = vec && aligned(T.m, 16);
            add(T.m, (numel + kMomentBlock - 1) / kMomentBlock * K * kMomentBlock * 4, true, "m");
        } else if (need_mv) {
            T.m = static_cast<float *>(list->m[i]);
            T.v = static_cast<float *>(list->v[i]);
            if (numel > 0 && (!T.m || !T.v)) return fail(OPTIM_EINVAL, ti + "NULL m or v");
            const size_t ssz = states16 ? 2 : 4;  // bytes per stored moment
            if (!aligned(T.m, ssz) || !aligned(T.v, ssz)) return fail(OPTIM_EALIGN, ti + "m/v misaligned");
            vec = vec && aligned(T.m, 16) && (kind != OPTIM_MINI_FULL_V || aligned(T.v, 16));
            add(T.m, numel * ssz, true, "m");
            add(T.v, vlen * ssz, true, "v");
            if (states16) {
                T.scale_m = list->scale_m[i];
                T.scale_v = list->scale_v[i];
                if (numel > 0 && (!T.scale_m || !T.scale_v)) return fail(OPTIM_EINVAL, ti + "NULL state scale");
                if (!aligned(T.scale_m, 4) || !aligned(T.scale_v, 4))
                    return fail(OPTIM_EALIGN, ti + "state scale misaligned");
                add(T.scale_m, 4, true, "scale_m");
                add(T.scale_v, 4, true, "scale_v");
            }
        }
        if (algo == OPTIM_ALGO_LION || muon) {
            T.m = static_cast<float *>(list->m[i]);
            if (numel > 0 && !T.m) return fail(OPTIM_EINVAL, ti + "NULL m");
            if (!aligned(T.m, 4)) return fail(OPTIM_EALIGN, ti + "m misaligned");
            vec = vec && aligned(T.m, 16);
            add(T.m, numel * 4, true, "m");
        }
        if (algo == OPTIM_ALGO_ADEMAMIX && !mom_il) {
            T.m2 = static_cast<float *>(list->m2[i]);
            if (numel > 0 && !T.m2) return fail(OPTIM_EINVAL, ti + "NULL m2");
            if (!aligned(T.m2, 4)) return fail(OPTIM_EALIGN, ti + "m2 misaligned");
            vec = vec && aligned(T.m2, 16);
            add(T.m2, numel * 4, true, "m2");
        }
        if (is_blockwise(algo) && il) {
            // m and v codes side by side in qm, (absmax m, absmax v) pairs in am
            if ((list->qv && list->qv[i]) || (list->absmax_v && list->absmax_v[i]))
                return fail(OPTIM_EINVAL, ti + "interleaved layout: qv and absmax_v must be NULL");
            T.qm = static_cast<uint8_t *>(list->qm[i]);
            T.am = list->absmax_m[i];
            if (numel > 0 && (!T.qm || !T.am)) return fail(OPTIM_EINVAL, ti + "NULL code or absmax buffer");
            if (!aligned(T.am, 8)) return fail(OPTIM_EALIGN, ti + "interleaved absmax must be 8-byte aligned");
            vec = vec && aligned(T.qm, 16);
            add(T.qm, numel * 2 * bits / 8, true, "qm");
            add(T.am, (numel + block - 1) / block * 8, true, "absmax_m");
        } else if (is_blockwise(algo)) {
            T.qm = static_cast<uint8_t *>(list->qm[i]);
            T.qv = static_cast<uint8_t *>(list->qv[i]);
            T.am = list->absmax_m[i];
            T.av = list->absmax_v[i];
            if (numel > 0 && (!T.qm || !T.qv || !T.am || !T.av))
                return fail(OPTIM_EINVAL, ti + "NULL code or absmax buffer");
            if (!aligned(T.am, 4) || !aligned(T.av, 4)) return fail(OPTIM_EALIGN, ti + "absmax misaligned");
            vec = vec && aligned(T.qm, 16) && aligned(T.qv, 16);
            const int64_t cbytes = (numel * bits + 7) / 8;
            const int64_t nblk = (numel + block - 1) / block;
            add(T.qm, cbytes, true, "qm");
            add(T.qv, cbytes, true, "qv");
            add(T.am, nblk * 4, true, "absmax_m");
            add(T.av, nblk * 4, true, "absmax_v");
            if (algo == OPTIM_ALGO_BLOCKWISE_ADEMAMIX) {
                T.qm2 = static_cast<uint8_t *>(list->qm2[i]);
                T.am2 = list->absmax_m2[i];
                if (numel > 0 && (!T.qm2 || !T.am2)) return fail(OPTIM_EINVAL, ti + "NULL qm2 or absmax_m2");
                if (!aligned(T.am2, 4)) return fail(OPTIM_EALIGN, ti + "absmax_m2 misaligned");
                vec = vec && aligned(T.qm2, 16);
                add(T.qm2, cbytes, true, "qm2");
                add(T.am2, nblk * 4, true, "absmax_m2");
            }
        }
        T.vec_ok = vec ? 1 : 0;
        if (numel == 0) continue;
        const int64_t units_before = B.nunits;
        const int32_t blocks_before = B.nblocks;
        // spans
        if (algo == OPTIM_ALGO_ADAM_MINI && kind != OPTIM_MINI_FULL_V) {
            for (int64_t s = 0; s < numel; s += T.block_len) {
                SpanDesc sp{B.nunits, s, T.block_len, i, B.nblocks};
                B.blockspan.push_back((int32_t)B.spans.size());
                B.spans.push_back(sp);
                B.nunits += (T.block_len + tile - 1) / tile;
                if (B.nblocks == INT32_MAX) return fail(OPTIM_EUNSUPPORTED, "too many blocks");
                ++B.nblocks;
            }
        } else if (muon) {
            // (their spans are added below, run by run)
        } else if (algo == OPTIM_ALGO_LAMB || states16) {
            // one block per tensor: its trust ratio, or its state scales
            B.blockspan.push_back((int32_t)B.spans.size());
            B.spans.push_back(SpanDesc{B.nunits, 0, numel, i, B.nblocks});
            B.nunits += (numel + tile - 1) / tile;
            ++B.nblocks;
        } else if (packable && numel <= pack_cap / 2) {
            const int64_t r = (numel + 3) / 4 * 4;
            if (open_len + r > pack_cap || (int32_t)open_pack.size() >= kMaxPackTensors) close_pack();
            open_pack.push_back(i);
            open_len += r;
        } else {
            close_pack();
            B.spans.push_back(SpanDesc{B.nunits, 0, numel, i, -1});
            B.nunits += (numel + tile - 1) / tile;
        }
        // Adam-mini segments: runs of whole tensors, all with shared v and
        // at most seg_cap gradient bytes (a larger tensor alone), or all
        // with full v
        if (algo == OPTIM_ALGO_ADAM_MINI) {
            const bool shared = kind != OPTIM_MINI_FULL_V;
            const int64_t gb = numel * (int64_t)gsz;
            if (B.segs.empty() || shared != seg_shared || (shared && seg_gbytes + gb > seg_cap)) {
                B.segs.push_back(MiniSegment{units_before, B.nunits, blocks_before, B.nblocks});
                seg_shared = shared;
                seg_gbytes = gb;
            } else {
                B.segs.back().unit_end = B.nunits;
                B.segs.back().block_end = B.nblocks;
                seg_gbytes += gb;
            }
        }
    }
    if (muon)
        if (const int rc = add_muon(list, seg_cap, B)) return rc;
    close_pack();
    B.pack_unit0 = B.nunits;
    for (size_t k = 0; k < B.packs.size(); ++k) {
        B.spans.push_back(SpanDesc{B.nunits, (int64_t)k, B.packs[k].len, kPackTensor, -1});
        B.nunits += 1;
    }
    if (B.spans.size() >= (size_t)INT32_MAX || B.pack_off.size() >= (size_t)INT32_MAX)
        return fail(OPTIM_EUNSUPPORTED, "too many spans");
    B.spans.push_back(SpanDesc{B.nunits, 0, 0, -1, -1});  // sentinel

    if (const int rc = check_overlaps(ranges)) return rc;

    Layout &L = B.L;
    size_t off = 0;
    L.counters = off; off += align256(kCounterBytes);
    L.group_wd = off; off += align256(kMaxGroups * sizeof(double));
    L.tensors = off; off += align256(std::max<size_t>(1, B.tensors.size()) * sizeof(TensorDesc));
    L.spans = off; off += align256(B.spans.size() * sizeof(SpanDesc));
    L.codebook = off; off += is_blockwise(algo) ? align256(sizeof(Codebook)) : 0;
    L.blockspan = off; off += align256(std::max<size_t>(1, B.blockspan.size()) * sizeof(int32_t));
    L.packs = off; off += align256(B.packs.size() * sizeof(PackDesc));
    L.pack_off = off; off += align256(B.pack_off.size() * sizeof(int32_t));
    L.pack_td = off; off += align256(B.pack_td.size() * sizeof(PackMember));
    L.mats = off; off += align256(B.mats.size() * sizeof(MuonMat));
    L.sym = off; off += align256(B.sym.size() * sizeof(MuonTile));
    L.full = off; off += align256(B.full.size() * sizeof(MuonTile));
    // partial sums: Adam-mini's block sums (one per unit) and the gradient
    // norm pass (one per workgroup) share the region; they never overlap in
    // stream order
    L.partials = off;
    // (LAMB: two per unit, sums of p^2 and u^2)
    B.npartials = std::max<int64_t>(algo == OPTIM_ALGO_ADAM_MINI || muon ? B.nunits
                                    : algo == OPTIM_ALGO_LAMB    ? 2 * B.nunits
                                                                 : 0,
                                    norm_partials(B.nunits, B.tile, B.grid));
    off += align256(std::max<int64_t>(1, B.npartials) * sizeof(double));
    // per-block factors; 16-bit states: the maxima slots of each tensor
    // (zero in the uploaded image)
    L.blockfac = off;
    off += align256(B.states16 ? std::max<int32_t>(1, B.nblocks) * kAmaxBytesPerBlock
                               : std::max<int32_t>(1, 2 * B.nblocks) * sizeof(float));
    L.muon = off; off += align256((size_t)B.muon_bytes);
    L.total = off;
    return OPTIM_OK;
}

}  // namespace

struct optim_plan {
    int32_t algo;
    int32_t pk, gk;
    int32_t bits, block;
    int32_t grid;  // requested persistent workgroups (0 = one per unit)
    int32_t cus;
    int32_t nspans, nblocks, ngroups;
    int64_t nunits;
    int64_t tile;
    int64_t npartials;
    int32_t state_dtype;
    char *ws;
    Layout L;
    std::vector<MiniSegment> segs;  // Adam-mini launch segments
    std::vector<MuonRun> runs;      // Muon: runs of launches
    int32_t lone0, lone_narrow;     // Muon: matrices of one slab (MuonArgs)
    int64_t lone_unit0;
    int32_t interleaved;            // blockwise: interleaved state layout
    int32_t sched;
    double lr_max, lr_min;
    int32_t K;
    int32_t *iter_dev;
    // plans on the static workspace: the device and the creation number
    // (0 for a plan on a caller's workspace)
    int32_t static_dev;
    uint64_t static_gen;
    Trace *trace;  // kernel trace (optim_plan_trace), or NULL
    int64_t pack_unit0;  // first pack unit
    int32_t ngrads, ngitems, ngsmall;  // gradient lists: tensors, items, small tensors
    int32_t gkeep0;           // first item that is left in the cache
};

extern "C" {

const char *optim_last_error(void) { return g_err.c_str(); }

int optim_quant_codebook(int32_t bits, int32_t is_signed, float *values, float *thresholds) try {
    if (bits != 8 && bits != 4) return fail(OPTIM_EINVAL, "bits must be 8 or 4");
    if (!values || !thresholds) return fail(OPTIM_EINVAL, "NULL output");
    dynamic_map(is_signed ? bits - 1 : bits, values, thresholds);
    return OPTIM_OK;
} OPTIM_CATCH

int optim_plan_workspace_size(const optim_tensor_list *list, int32_t algo,
                              const optim_plan_opts *opts, size_t *bytes) try {
    if (!bytes) return fail(OPTIM_EINVAL, "bytes is NULL");
    Built B;
    const int rc = build(list, algo, opts, B);
    if (rc) return rc;
    *bytes = B.L.total;
    return OPTIM_OK;
} OPTIM_CATCH

}  // extern "C"

namespace {

// ---------------------------------------------------------------- static workspace
// The workspace of plans made by optim_plan_create_static, for callers that
// cannot allocate device memory.  One array per device (each device that
// loads the library holds its own copy at its own address until the process
// ends).  In host code `scratch` is only a stand-in for the symbol: its
// device address is looked up once per device with hipGetSymbolAddress and
// kept in g_scratch_ptr, and only that address is ever handed to the device.
__device__ __align__(256) unsigned char scratch[OPTIM_STATIC_WORKSPACE_BYTES];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void *g_scratch_ptr[kMaxDevices];
// creation number of the live static plan of each device; a plan made
// earlier on the same device has been overwritten and is refused
std::atomic<uint64_t> g_static_gen[kMaxDevices];

int scratch_of_device(int dev, void **ptr) {
    if (dev < 0 || dev >= kMaxDevices)
        return fail(OPTIM_EUNSUPPORTED, "static workspace: device index " + std::to_string(dev) + " above 63");
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (!g_scratch_ptr[dev]) {
        void *p = nullptr;
        HIP_OK(hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)));
        if (!p || !aligned(p, 256)) return fail(OPTIM_EHIP, "static workspace: no 256-byte aligned device address");
        g_scratch_ptr[dev] = p;
    }
    *ptr = g_scratch_ptr[dev];
    return OPTIM_OK;
}

// Refuses a static plan whose tables a later optim_plan_create_static on the
// same device has overwritten (its kernels would walk another plan's tables).
int check_live(const optim_plan *P, const char *fn) {
    if (P->static_gen && P->static_gen != g_static_gen[P->static_dev].load(std::memory_order_acquire))
        return fail(OPTIM_EINVAL, std::string(fn) +
                                      ": this static plan was superseded by a later optim_plan_create_static "
                                      "on its device (the static workspace holds one plan at a time)");
    return OPTIM_OK;
}

// ---------------------------------------------------------------- kernel trace
void free_trace(optim_plan *P) {
    if (!P->trace) return;
    for (TraceRec &r : P->trace->recs) {
        if (r.start) (void)hipEventDestroy(r.start);
        if (r.stop) (void)hipEventDestroy(r.stop);
    }
    delete P->trace;
    P->trace = nullptr;
}

// "(mini_update_kernel<PK, GK>)" -> "mini_update_kernel"; kept in the trace
// so the returned pointers live until the trace is freed.
const char *clean_name(Trace *t, const char *raw) {
    for (const auto &kv : t->names)
        if (kv.first == raw) return kv.second.c_str();
    std::string s(raw ? raw : "");
    s.erase(std::remove(s.begin(), s.end(), '('), s.end());
    const size_t lt = s.find('<');
    if (lt != std::string::npos) s.resize(lt);
    while (!s.empty() && (s.back() == ')' || s.back() == ' ')) s.pop_back();
    t->names.emplace_back(raw, s);
    return t->names.back().second.c_str();
}

// Points the launches of one entry point at its plan's trace.
struct TraceScope {
    explicit TraceScope(const optim_plan *P) { g_trace = P ? P->trace : nullptr; }
    ~TraceScope() { g_trace = nullptr; }
};

// Plan creation on a given workspace (the caller's, or the static one).
int create_on(const Built &B, const optim_tensor_list *list, int32_t algo, const optim_plan_opts *opts,
              void *workspace, hipStream_t s, int dev, optim_plan **out) {
    // host image of the table region [0, partials); with 16-bit states the
    // whole workspace, so the maxima slots start at zero
    std::vector<char> img(B.states16 ? B.L.total : B.L.partials, 0);
    std::memcpy(img.data() + B.L.group_wd, B.group_wd.data(), B.group_wd.size() * sizeof(double));
    std::memcpy(img.data() + B.L.tensors, B.tensors.data(), B.tensors.size() * sizeof(TensorDesc));
    std::memcpy(img.data() + B.L.spans, B.spans.data(), B.spans.size() * sizeof(SpanDesc));
    std::memcpy(img.data() + B.L.blockspan, B.blockspan.data(), B.blockspan.size() * sizeof(int32_t));
    std::memcpy(img.data() + B.L.packs, B.packs.data(), B.packs.size() * sizeof(PackDesc));
    std::memcpy(img.data() + B.L.pack_off, B.pack_off.data(), B.pack_off.size() * sizeof(int32_t));
    std::memcpy(img.data() + B.L.pack_td, B.pack_td.data(), B.pack_td.size() * sizeof(PackMember));
    std::memcpy(img.data() + B.L.mats, B.mats.data(), B.mats.size() * sizeof(MuonMat));
    std::memcpy(img.data() + B.L.sym, B.sym.data(), B.sym.size() * sizeof(MuonTile));
    std::memcpy(img.data() + B.L.full, B.full.data(), B.full.size() * sizeof(MuonTile));
    std::memcpy(img.data() + B.L.gitems, B.gitems.data(), B.gitems.size() * sizeof(GradItem));
    std::memcpy(img.data() + B.L.gsmall, B.gsmall.data(), B.gsmall.size() * sizeof(GradSmall));
    if (is_blockwise(algo)) {
        Codebook *cb = reinterpret_cast<Codebook *>(img.data() + B.L.codebook);
        if (!build_map(7, cb->m8) || !build_map(8, cb->v8) || !build_map(3, cb->m4) || !build_map(4, cb->v4))
            return fail(OPTIM_EUNSUPPORTED, "quantization map does not fit the bucket table");
    }
    std::unique_ptr<optim_plan> owner(new optim_plan{});
    optim_plan *P = owner.get();
    P->segs = B.segs;
    P->runs = B.runs;
    int cus = 0;
    HIP_OK(hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev));
    HIP_OK(hipMemcpyAsync(workspace, img.data(), img.size(), hipMemcpyHostToDevice, s));
    HIP_OK(hipStreamSynchronize(s));

    P->algo = algo;
    P->pk = list->param_dtype == OPTIM_F32 ? P_F32
            : !list->master                 ? P_BF16R
            : list->param_dtype == OPTIM_BF16 ? P_MBF16
                                              : P_MF16;
    P->gk = list->grad_dtype == OPTIM_BF16 ? G_BF16 : list->grad_dtype == OPTIM_F16 ? G_F16 : G_F32;
    P->bits = opts ? opts->bits : 0;
    P->block = opts ? opts->block : 0;
    P->grid = opts ? opts->grid : 0;
    P->cus = cus;
    P->nspans = (int32_t)B.spans.size() - 1;
    P->nblocks = B.nblocks;
    P->ngroups = (int32_t)B.group_wd.size();
    P->nunits = B.nunits;
    P->tile = B.tile;
    P->npartials = B.npartials;
    P->state_dtype = opts ? opts->state_dtype : OPTIM_F32;
    P->ws = static_cast<char *>(workspace);
    P->L = B.L;
    P->lone0 = B.lone0;
    P->lone_narrow = B.lone_narrow;
    P->lone_unit0 = B.lone_unit0;
    P->interleaved = B.interleaved ? 1 : 0;
    P->sched = OPTIM_SCHED_NONE;
    P->static_dev = dev;
    P->static_gen = 0;
    P->pack_unit0 = B.pack_unit0;
    P->ngrads = list->n;
    P->ngitems = (int32_t)B.gitems.size();
    P->ngsmall = (int32_t)B.gsmall.size();
    P->gkeep0 = B.gkeep0;
    *out = owner.release();
    return OPTIM_OK;
}

}  // namespace

extern "C" {

int optim_plan_create(const optim_tensor_list *list, int32_t algo, const optim_plan_opts *opts,
                      void *workspace, size_t workspace_bytes, void *stream, optim_plan **out) try {
    if (!out) return fail(OPTIM_EINVAL, "out is NULL");
    *out = nullptr;
    Built B;
    int rc = build(list, algo, opts, B);
    if (rc) return rc;
    if (!workspace || !aligned(workspace, 256))
        return fail(OPTIM_EWORKSPACE, "workspace must be a 256-byte aligned device pointer");
    if (workspace_bytes < B.L.total)
        return fail(OPTIM_EWORKSPACE, "workspace too small: need " + std::to_string(B.L.total) +
                                          " bytes, got " + std::to_string(workspace_bytes));
    int dev = 0;
    HIP_OK(hipGetDevice(&dev));
    return create_on(B, list, algo, opts, workspace, static_cast<hipStream_t>(stream), dev, out);
} OPTIM_CATCH

int optim_plan_create_static(const optim_tensor_list *list, int32_t algo, const optim_plan_opts *opts,
                             void *stream, optim_plan **out) try {
    if (!out) return fail(OPTIM_EINVAL, "out is NULL");
    *out = nullptr;
    Built B;
    int rc = build(list, algo, opts, B);
    if (rc) return rc;
    if (B.L.total > (size_t)OPTIM_STATIC_WORKSPACE_BYTES)
        return fail(OPTIM_EWORKSPACE, "optim_plan_create_static: the plan needs " + std::to_string(B.L.total) +
                                          " bytes of workspace; the static workspace holds " +
                                          std::to_string((size_t)OPTIM_STATIC_WORKSPACE_BYTES) +
                                          " (use optim_plan_create with a caller workspace)");
    int dev = 0;
    HIP_OK(hipGetDevice(&dev));
    void *ws = nullptr;
    if ((rc = scratch_of_device(dev, &ws))) return rc;
    // every earlier static plan of this device is superseded from here on,
    // also if this creation fails after overwriting part of the tables
    const uint64_t gen = g_static_gen[dev].fetch_add(1, std::memory_order_acq_rel) + 1;
    optim_plan *P = nullptr;
    if ((rc = create_on(B, list, algo, opts, ws, static_cast<hipStream_t>(stream), dev, &P))) return rc;
    P->static_gen = gen;
    *out = P;
    return OPTIM_OK;
} OPTIM_CATCH

int optim_plan_destroy(optim_plan *plan) try {
    if (plan) free_trace(plan);
    delete plan;
    return OPTIM_OK;
} OPTIM_CATCH

int optim_plan_trace(optim_plan *plan, int32_t capacity) try {
    if (!plan) return fail(OPTIM_EINVAL, "plan is NULL");
    if (capacity < 0) return fail(OPTIM_EINVAL, "negative trace capacity");
    free_trace(plan);
    if (capacity == 0) return OPTIM_OK;
    std::unique_ptr<Trace> t(new Trace{});
    t->recs.reserve((size_t)capacity);
    for (int32_t i = 0; i < capacity; ++i) {
        TraceRec r{nullptr, 0, nullptr, nullptr};
        hipError_t e = hipEventCreate(&r.start);
        if (e == hipSuccess) {
            e = hipEventCreate(&r.stop);
            if (e != hipSuccess) (void)hipEventDestroy(r.start);
        }
        if (e != hipSuccess) {
            plan->trace = t.release();
            free_trace(plan);
            return fail(OPTIM_EHIP, std::string("hipEventCreate: ") + hipGetErrorString(e));
        }
        t->recs.push_back(r);
    }
    plan->trace = t.release();
    return OPTIM_OK;
} OPTIM_CATCH

int optim_plan_trace_read(optim_plan *plan, optim_kernel_time *out, int32_t max, int32_t *count,
                          int64_t *dropped) try {
    if (!plan || !count) return fail(OPTIM_EINVAL, "plan and count are required");
    if (max < 0 || (max > 0 && !out)) return fail(OPTIM_EINVAL, "need out[max], max >= 0");
    Trace *t = plan->trace;
    if (!t) return fail(OPTIM_EINVAL, "the plan has no trace (optim_plan_trace)");
    const size_t n = t->used;
    t->used = 0;
    const int64_t lost = t->dropped;
    t->dropped = 0;
    for (size_t i = 0; i < n; ++i) {
        const TraceRec &r = t->recs[i];
        HIP_OK(hipEventSynchronize(r.stop));
        float ms = 0.0f;
        HIP_OK(hipEventElapsedTime(&ms, r.start, r.stop));
        if ((int64_t)i < (int64_t)max) out[i] = optim_kernel_time{clean_name(t, r.name), r.grid, (double)ms};
    }
    *count = (int32_t)n;
    if (dropped) *dropped = lost;
    return OPTIM_OK;
} OPTIM_CATCH

int optim_plan_set_schedule(optim_plan *plan, int32_t kind, double lr_max, double lr_min, int32_t K,
                            int32_t *iter_dev) try {
    if (!plan) return fail(OPTIM_EINVAL, "plan is NULL");
    if (kind == OPTIM_SCHED_NONE) {
        plan->sched = OPTIM_SCHED_NONE;
        plan->iter_dev = nullptr;
        return OPTIM_OK;
    }
    if (kind != OPTIM_SCHED_COSINE) return fail(OPTIM_EINVAL, "unknown schedule kind");
    if (!(lr_max >= 0.0) || !(lr_min >= 0.0) || !std::isfinite(lr_max) || !std::isfinite(lr_min))
        return fail(OPTIM_EINVAL, "invalid learning rate (need 0 <= lr, finite)");
    if (K <= 0) return fail(OPTIM_EINVAL, "schedule length K must be > 0");
    if (!iter_dev || !aligned(iter_dev, 4)) return fail(OPTIM_EINVAL, "iter_dev must be an aligned device int32");
    plan->sched = kind;
    plan->lr_max = lr_max;
    plan->lr_min = lr_min;
    plan->K = K;
    plan->iter_dev = iter_dev;
    return OPTIM_OK;
} OPTIM_CATCH

}  // extern "C"

namespace {

StepArgs step_args(optim_plan *P) {
    StepArgs a{};
    a.done = reinterpret_cast<uint32_t *>(P->ws + P->L.counters);
    a.commit = 1;
    a.tensors = reinterpret_cast<const TensorDesc *>(P->ws + P->L.tensors);
    a.spans = reinterpret_cast<const SpanDesc *>(P->ws + P->L.spans);
    a.nspans = P->nspans;
    a.nunits = P->nunits;
    a.tile = P->tile;
    a.partials = reinterpret_cast<double *>(P->ws + P->L.partials);
    a.npartials = P->npartials;
    a.blockfac = reinterpret_cast<float *>(P->ws + P->L.blockfac);
    a.blockspan = reinterpret_cast<const int32_t *>(P->ws + P->L.blockspan);
    a.packs = reinterpret_cast<const PackDesc *>(P->ws + P->L.packs);
    a.pack_off = reinterpret_cast<const int32_t *>(P->ws + P->L.pack_off);
    a.pack_td = reinterpret_cast<const PackMember *>(P->ws + P->L.pack_td);
    a.pack_unit0 = P->pack_unit0;
    a.nblocks = P->nblocks;
    a.codebook = reinterpret_cast<const Codebook *>(P->ws + P->L.codebook);
    a.bits = P->bits;
    a.block = P->block;
    a.interleaved = P->interleaved;
    a.cus = P->cus;
    a.grid_request = P->grid;
    a.units_per_wg = 1;
    return a;
}

// Validates the per-step device scalars and fills the inputs every step
// kernel derives its scalars from.
int step_inputs(optim_plan *P, double b1, double b2, double b3, double alpha, double eps, float *lr_dev,
                const float *inv_scale, const float *found_inf, int32_t *step_dev, StepArgs &a) {
    if (!lr_dev || !aligned(lr_dev, 4)) return fail(OPTIM_EINVAL, "lr_dev must be an aligned device float");
    if (!step_dev || !aligned(step_dev, 4)) return fail(OPTIM_EINVAL, "step_dev must be an aligned device int32");
    if (!aligned(inv_scale, 4) || !aligned(found_inf, 4)) return fail(OPTIM_EALIGN, "scalar pointer misaligned");
    if (!(eps >= 0.0) || !std::isfinite(eps)) return fail(OPTIM_EINVAL, "invalid eps (need finite eps >= 0)");
    a = step_args(P);
    PrepArgs &p = a.prep;
    p.group_wd = reinterpret_cast<const double *>(P->ws + P->L.group_wd);
    p.ngroups = P->ngroups;
    p.sched = P->sched;
    p.lr_dev = lr_dev;
    p.inv_scale = inv_scale;
    p.found_inf = found_inf;
    p.step_dev = step_dev;
    p.iter_dev = P->iter_dev;
    p.lr_max = P->lr_max;
    p.lr_min = P->lr_min;
    p.K = P->K;
    p.beta1 = b1;
    p.beta2 = b2;
    p.beta3 = b3;
    p.alpha = alpha;
    p.eps = eps;
    return OPTIM_OK;
}

int check_plan(optim_plan *P, int32_t algo, const char *fn) {
    if (!P) return fail(OPTIM_EINVAL, std::string(fn) + ": plan is NULL");
    if (P->algo != algo) return fail(OPTIM_EINVAL, std::string(fn) + ": plan was built for another algorithm");
    return check_live(P, fn);
}

// The largest |x| over |s| <= R of s (a + b s^2 + c s^4), and of b s^2 +
// c s^4: each is monotone between its critical points, which are roots of
// quadratics in s^2.
void quintic_bounds(double a, double b, double c, double R, double &x, double &y) {
    double at[4] = {R * R, 0.0, 0.0, 0.0};  // values of s^2
    int n = 1;
    auto add = [&](double t) {
        if (t > 0.0 && t < R * R) at[n++] = t;
    };
    if (c != 0.0) {
        add(-b / (2.0 * c));
        const double d = 9.0 * b * b - 20.0 * a * c;
        if (d >= 0.0) {
            add((-3.0 * b + std::sqrt(d)) / (10.0 * c));
            add((-3.0 * b - std::sqrt(d)) / (10.0 * c));
        }
    } else if (b != 0.0) {
        add(-a / (3.0 * b));
    }
    x = y = 0.0;
    for (int i = 0; i < n; ++i) {
        x = std::max(x, std::sqrt(at[i]) * std::fabs(a + at[i] * (b + c * at[i])));
        y = std::max(y, at[i] * std::fabs(b + c * at[i]));
    }
}

int check_muon_hp(const optim_muon_hp *hp) {
    if (!hp) return fail(OPTIM_EINVAL, "hyperparameters are NULL");
    if (const int rc = check_hp_beta(hp->momentum, "momentum")) return rc;
    if (!std::isfinite(hp->a) || !std::isfinite(hp->b) || !std::isfinite(hp->c))
        return fail(OPTIM_EINVAL, "invalid polynomial (need finite a, b, c)");
    if (hp->steps < 1 || hp->steps > 16) return fail(OPTIM_EINVAL, "steps must be in [1, 16]");
    if (hp->scale_kind < OPTIM_MUON_SCALE_NONE || hp->scale_kind > OPTIM_MUON_SCALE_RMS)
        return fail(OPTIM_EINVAL, "unknown scale_kind");
    double R = 1.0;
    for (int i = 0; i < hp->steps; ++i) {
        double x, y;
        quintic_bounds(hp->a, hp->b, hp->c, R, x, y);
        if (!(x <= 15.0) || !(y <= 15.0) || !(R * R <= 15.0))
            return fail(OPTIM_EINVAL, "the polynomial leaves the range of its 16-bit parts (|X|, |A|, |B| <= 15)");
        R = std::max(1.0, x);
    }
    return OPTIM_OK;
}

constexpr int64_t kExpertMaxSide = (int64_t(1) << 24) - 1;

int check_expert_sizes(int32_t experts, int64_t tokens, int64_t m, int64_t n) {
    if (experts < 0 || tokens < 0 || m < 0 || n < 0) return fail(OPTIM_EINVAL, "negative size");
    if (tokens > INT32_MAX) return fail(OPTIM_EINVAL, "tokens must be below 2^31");
    if (m > kExpertMaxSide || n > kExpertMaxSide) return fail(OPTIM_EINVAL, "m and n must be below 2^24");
    // a launch has fewer than 2^32 lanes: 16 tiles a block, up to 512 lanes each
    const int64_t blocks = ((m + 511) / 512) * ((n + 511) / 512);
    if (blocks * experts >= int64_t(1) << 18 || (experts > 0 && m > 0 && n > kMaxNumel / m / experts))
        return fail(OPTIM_EUNSUPPORTED, "dW has too many experts or elements");
    return OPTIM_OK;
}

GradArgs grad_args(optim_plan *P) {
    GradArgs a{};
    a.items = reinterpret_cast<const GradItem *>(P->ws + P->L.gitems);
    a.small = reinterpret_cast<const GradSmall *>(P->ws + P->L.gsmall);
    a.count = reinterpret_cast<uint32_t *>(P->ws + P->L.gcount);
    a.done = reinterpret_cast<uint32_t *>(P->ws + P->L.counters);
    a.partials = reinterpret_cast<double *>(P->ws + P->L.partials);
    a.sums = reinterpret_cast<double *>(P->ws + P->L.gsum);
    a.ntensors = P->ngrads;
    a.nitems = P->ngitems;
    a.nsmall = P->ngsmall;
    a.keep0 = P->gkeep0;
    return a;
}

int check_norm_args(int32_t kind, const float *inv_scale, double max_norm, const float *total, const float *coef) {
    if (kind != OPTIM_NORM_L2 && kind != OPTIM_NORM_L1 && kind != OPTIM_NORM_INF)
        return fail(OPTIM_EINVAL, "unknown norm kind");
    if (std::isnan(max_norm)) return fail(OPTIM_EINVAL, "max_norm is NaN");
    if (!aligned(inv_scale, 4) || !aligned(total, 4) || !aligned(coef, 4))
        return fail(OPTIM_EALIGN, "scalar pointer misaligned");
    return OPTIM_OK;
}

// the quantize / dequantize helpers take either blockwise plan
int check_blockwise_plan(optim_plan *P, const char *fn) {
    if (!P) return fail(OPTIM_EINVAL, std::string(fn) + ": plan is NULL");
    if (!is_blockwise(P->algo)) return fail(OPTIM_EINVAL, std::string(fn) + ": plan is not blockwise");
    return check_live(P, fn);
}

int check_ademamix_hp(const optim_ademamix_hp *hp) {
    if (!hp) return fail(OPTIM_EINVAL, "hyperparameters are NULL");
    int rc;
    if ((rc = check_hp_beta(hp->beta1, "beta1")) || (rc = check_hp_beta(hp->beta2, "beta2")) ||
        (rc = check_hp_beta(hp->beta3, "beta3")))
        return rc;
    if (!std::isfinite(hp->alpha) || hp->alpha < 0.0) return fail(OPTIM_EINVAL, "invalid alpha (need finite alpha >= 0)");
    return OPTIM_OK;
}

int check_adamw_hp(const optim_adamw_hp *hp) {
    if (!hp) return fail(OPTIM_EINVAL, "hyperparameters are NULL");
    int rc = check_hp_beta(hp->beta1, "beta1");
    if (rc) return rc;
    return check_hp_beta(hp->beta2, "beta2");
}

}  // namespace

extern "C" {

int optim_step_adamw(optim_plan *plan, const optim_adamw_hp *hp, float *lr_dev, const float *inv_scale_dev,
                     const float *found_inf_dev, int32_t *step_dev, void *stream) try {
    int rc = check_plan(plan, OPTIM_ALGO_ADAMW, "optim_step_adamw");
    if (!rc) rc = check_adamw_hp(hp);
    if (rc) return rc;
    StepArgs a;
    rc = step_inputs(plan, hp->beta1, hp->beta2, 0.0, 0.0, hp->eps, lr_dev, inv_scale_dev, found_inf_dev,
                     step_dev, a);
    if (rc) return rc;
    const TraceScope ts(plan);
    if (plan->state_dtype != OPTIM_F32)
        HIP_OK(launch_adamw_scaled(a, plan->pk, plan->gk, plan->state_dtype == OPTIM_F16 ? S_F16 : S_BF16,
                                   static_cast<hipStream_t>(stream)));
    else
        HIP_OK(launch_adamw(a, plan->pk, plan->gk, static_cast<hipStream_t>(stream)));
    return OPTIM_OK;
} OPTIM_CATCH

int optim_step_ademamix(optim_plan *plan, const optim_ademamix_hp *hp, float *lr_dev,
                        const float *inv_scale_dev, const float *found_inf_dev, int32_t *step_dev,
                        void *stream) try {
    int rc = check_plan(plan, OPTIM_ALGO_ADEMAMIX, "optim_step_ademamix");
    if (!rc) rc = check_ademamix_hp(hp);
    if (rc) return rc;
    StepArgs a;
    rc = step_inputs(plan, hp->beta1, hp->beta2, hp->beta3, hp->alpha, hp->eps, lr_dev, inv_scale_dev,
                     found_inf_dev, step_dev, a);
    if (rc) return rc;
    const TraceScope ts(plan);
    HIP_OK(launch_ademamix(a, plan->pk, plan->gk, static_cast<hipStream_t>(stream)));
    return OPTIM_OK;
} OPTIM_CATCH

int optim_step_adam_mini(optim_plan *plan, const optim_adamw_hp *hp, float *lr_dev, const float *inv_scale_dev,
                         const float *found_inf_dev, int32_t *step_dev, void *stream) try {
    int rc = check_plan(plan, OPTIM_ALGO_ADAM_MINI, "optim_step_adam_mini");
    if (!rc) rc = check_adamw_hp(hp);
    if (rc) return rc;
    StepArgs a;
    rc = step_inputs(plan, hp->beta1, hp->beta2, 0.0, 0.0, hp->eps, lr_dev, inv_scale_dev, found_inf_dev,
                     step_dev, a);
    if (rc) return rc;
    const TraceScope ts(plan);
    HIP_OK(launch_adam_mini(a, plan->pk, plan->gk, plan->segs.data(), (int32_t)plan->segs.size(),
                            static_cast<hipStream_t>(stream)));
    return OPTIM_OK;
} OPTIM_CATCH

int optim_step_lion(optim_plan *plan, const optim_lion_hp *hp, float *lr_dev, const float *inv_scale_dev,
                    const float *found_inf_dev, int32_t *step_dev, void *stream) try {
    int rc = check_plan(plan, OPTIM_ALGO_LION, "optim_step_lion");
    if (rc) return rc;
    if (!hp) return fail(OPTIM_EINVAL, "hyperparameters are NULL");
    if ((rc = check_hp_beta(hp->beta1, "beta1")) || (rc = check_hp_beta(hp->beta2, "beta2"))) return rc;
    StepArgs a;
    rc = step_inputs(plan, hp->beta1, hp->beta2, 0.0, 0.0, 0.0, lr_dev, inv_scale_dev, found_inf_dev, step_dev, a);
    if (rc) return rc;
    const TraceScope ts(plan);
    HIP_OK(launch_lion(a, plan->pk, plan->gk, static_cast<hipStream_t>(stream)));
    return OPTIM_OK;
} OPTIM_CATCH

int optim_step_lamb(optim_plan *plan, const optim_adamw_hp *hp, float *lr_dev, const float *inv_scale_dev,
                    const float *found_inf_dev, int32_t *step_dev, void *stream) try {
    int rc = check_plan(plan, OPTIM_ALGO_LAMB, "optim_step_lamb");
    if (!rc) rc = check_adamw_hp(hp);
    if (rc) return rc;
    StepArgs a;
    rc = step_inputs(plan, hp->beta1, hp->beta2, 0.0, 0.0, hp->eps, lr_dev, inv_scale_dev, found_inf_dev,
                     step_dev, a);
    if (rc) return rc;
    const TraceScope ts(plan);
    HIP_OK(launch_lamb(a, plan->pk, plan->gk, static_cast<hipStream_t>(stream)));
    return OPTIM_OK;
} OPTIM_CATCH

int optim_step_muon(optim_plan *plan, const optim_muon_hp *hp, float *lr_dev, const float *inv_scale_dev,
                    const float *found_inf_dev, int32_t *step_dev, void *stream) try {
    int rc = check_plan(plan, OPTIM_ALGO_MUON, "optim_step_muon");
    if (!rc) rc = check_muon_hp(hp);
    if (rc) return rc;
    StepArgs a;
    rc = step_inputs(plan, hp->momentum, 0.0, 0.0, 0.0, hp->eps, lr_dev, inv_scale_dev, found_inf_dev, step_dev, a);
    if (rc) return rc;
    MuonArgs ma{};
    ma.mats = reinterpret_cast<const MuonMat *>(plan->ws + plan->L.mats);
    ma.sym = reinterpret_cast<const MuonTile *>(plan->ws + plan->L.sym);
    ma.full = reinterpret_cast<const MuonTile *>(plan->ws + plan->L.full);
    ma.ws = plan->ws + plan->L.muon;
    ma.qa = (float)hp->a;
    ma.qb = (float)hp->b;
    ma.qc = (float)hp->c;
    ma.scale_kind = hp->scale_kind;
    ma.lone0 = plan->lone0;
    ma.lone_narrow = plan->lone_narrow;
    ma.lone_unit0 = plan->lone_unit0;
    ma.nmats = plan->nblocks;
    const TraceScope ts(plan);
    HIP_OK(launch_muon(a, ma, plan->pk, plan->gk, hp->steps, hp->nesterov != 0, plan->runs.data(),
                       (int32_t)plan->runs.size(), static_cast<hipStream_t>(stream)));
    return OPTIM_OK;
} OPTIM_CATCH

int optim_step_8bit_blockwise(optim_plan *plan, const optim_adamw_hp *hp, int32_t bits, int32_t block,
                              float *lr_dev, const float *inv_scale_dev, const float *found_inf_dev,
                              int32_t *step_dev, void *stream) try {
    int rc = check_plan(plan, OPTIM_ALGO_BLOCKWISE, "optim_step_8bit_blockwise");
    if (!rc) rc = check_adamw_hp(hp);
    if (rc) return rc;
    if (bits != plan->bits || block != plan->block)
        return fail(OPTIM_EINVAL, "bits/block differ from the plan's");
    StepArgs a;
    rc = step_inputs(plan, hp->beta1, hp->beta2, 0.0, 0.0, hp->eps, lr_dev, inv_scale_dev, found_inf_dev,
                     step_dev, a);
    if (rc) return rc;
    const TraceScope ts(plan);
    HIP_OK(launch_blockwise(a, plan->gk, false, static_cast<hipStream_t>(stream)));
    return OPTIM_OK;
} OPTIM_CATCH

int optim_step_8bit_blockwise_ademamix(optim_plan *plan, const optim_ademamix_hp *hp, int32_t bits, int32_t block,
                                       float *lr_dev, const float *inv_scale_dev, const float *found_inf_dev,
                                       int32_t *step_dev, void *stream) try {
    int rc = check_plan(plan, OPTIM_ALGO_BLOCKWISE_ADEMAMIX, "optim_step_8bit_blockwise_ademamix");
    if (!rc) rc = check_ademamix_hp(hp);
    if (rc) return rc;
    if (bits != plan->bits || block != plan->block)
        return fail(OPTIM_EINVAL, "bits/block differ from the plan's");
    StepArgs a;
    rc = step_inputs(plan, hp->beta1, hp->beta2, hp->beta3, hp->alpha, hp->eps, lr_dev, inv_scale_dev,
                     found_inf_dev, step_dev, a);
    if (rc) return rc;
    const TraceScope ts(plan);
    HIP_OK(launch_blockwise(a, plan->gk, true, static_cast<hipStream_t>(stream)));
    return OPTIM_OK;
} OPTIM_CATCH

int optim_check_finite(optim_plan *plan, float *found_inf_dev, void *stream) try {
    if (!plan) return fail(OPTIM_EINVAL, "plan is NULL");
    if (int rc = check_live(plan, "optim_check_finite")) return rc;
    if (plan->algo == OPTIM_ALGO_GRADS)
        return fail(OPTIM_EINVAL, "optim_check_finite: a gradient list is checked by optim_grad_norms");
    if (!found_inf_dev || !aligned(found_inf_dev, 4))
        return fail(OPTIM_EINVAL, "found_inf_dev must be an aligned device float");
    if (plan->nunits == 0) return OPTIM_OK;
    StepArgs a = step_args(plan);
    a.commit = 0;
    a.found_inf = found_inf_dev;
    const TraceScope ts(plan);
    HIP_OK(launch_check_finite(a, plan->gk, static_cast<hipStream_t>(stream)));
    return OPTIM_OK;
} OPTIM_CATCH

int optim_grad_norm(optim_plan *plan, const float *inv_scale_dev, double max_norm, float *found_inf_dev,
                    float *norm_dev, float *clip_inv_scale_dev, void *stream) try {
    if (!plan) return fail(OPTIM_EINVAL, "plan is NULL");
    if (int rc = check_live(plan, "optim_grad_norm")) return rc;
    if (plan->algo == OPTIM_ALGO_GRADS)
        return fail(OPTIM_EINVAL, "optim_grad_norm: the norms of a gradient list are taken by optim_grad_norms");
    if (!found_inf_dev || !aligned(found_inf_dev, 4))
        return fail(OPTIM_EINVAL, "found_inf_dev must be an aligned device float");
    if (!clip_inv_scale_dev || !aligned(clip_inv_scale_dev, 4))
        return fail(OPTIM_EINVAL, "clip_inv_scale_dev must be an aligned device float");
    if (!aligned(inv_scale_dev, 4) || !aligned(norm_dev, 4)) return fail(OPTIM_EALIGN, "scalar pointer misaligned");
    if (std::isnan(max_norm)) return fail(OPTIM_EINVAL, "max_norm is NaN");
    StepArgs a = step_args(plan);
    a.commit = 0;
    a.found_inf = found_inf_dev;
    const TraceScope ts(plan);
    HIP_OK(launch_grad_norm(a, plan->gk, inv_scale_dev, max_norm, norm_dev, clip_inv_scale_dev,
                            static_cast<hipStream_t>(stream)));
    return OPTIM_OK;
} OPTIM_CATCH

int optim_grad_norms(optim_plan *plan, int32_t kind, const float *inv_scale_dev, double max_norm,
                     float *found_inf_dev, float *norms_dev, float *total_dev, float *coef_dev, void *stream) try {
    if (const int rc = check_plan(plan, OPTIM_ALGO_GRADS, "optim_grad_norms")) return rc;
    if (const int rc = check_norm_args(kind, inv_scale_dev, max_norm, total_dev, coef_dev)) return rc;
    if (!total_dev) return fail(OPTIM_EINVAL, "total_dev must be an aligned device float");
    if (!aligned(found_inf_dev, 4) || !aligned(norms_dev, 4)) return fail(OPTIM_EALIGN, "scalar pointer misaligned");
    const TraceScope ts(plan);
    HIP_OK(launch_grad_norms(grad_args(plan), plan->gk, kind, inv_scale_dev, max_norm, found_inf_dev, norms_dev,
                             total_dev, coef_dev, static_cast<hipStream_t>(stream)));
    return OPTIM_OK;
} OPTIM_CATCH

int optim_clip_coef(const float *norms_dev, int64_t count, int32_t kind, const float *inv_scale_dev, double max_norm,
                    float *total_dev, float *coef_dev, void *stream) try {
    if (count < 0) return fail(OPTIM_EINVAL, "negative count");
    if (count > 0 && !norms_dev) return fail(OPTIM_EINVAL, "NULL norms");
    if (!aligned(norms_dev, 4)) return fail(OPTIM_EALIGN, "norms misaligned");
    if (const int rc = check_norm_args(kind, inv_scale_dev, max_norm, total_dev, coef_dev)) return rc;
    HIP_OK(launch_clip_coef(norms_dev, count, kind, inv_scale_dev, max_norm, total_dev, coef_dev,
                            static_cast<hipStream_t>(stream)));
    return OPTIM_OK;
} OPTIM_CATCH

int optim_clip_grads(optim_plan *plan, const float *coef_dev, const float *found_inf_dev, void *stream) try {
    if (const int rc = check_plan(plan, OPTIM_ALGO_GRADS, "optim_clip_grads")) return rc;
    if (!coef_dev || !aligned(coef_dev, 4)) return fail(OPTIM_EINVAL, "coef_dev must be an aligned device float");
    if (!aligned(found_inf_dev, 4)) return fail(OPTIM_EALIGN, "scalar pointer misaligned");
    const TraceScope ts(plan);
    HIP_OK(launch_clip_grads(grad_args(plan), plan->gk, coef_dev, found_inf_dev, static_cast<hipStream_t>(stream)));
    return OPTIM_OK;
} OPTIM_CATCH

int optim_expert_grad_workspace(int32_t experts, int64_t tokens, int64_t m, int64_t n, size_t *bytes) try {
    if (!bytes) return fail(OPTIM_EINVAL, "bytes is NULL");
    if (const int rc = check_expert_sizes(experts, tokens, m, n)) return rc;
    const int32_t pieces = expert_pieces(experts, tokens, m, n);
    *bytes = pieces > 1 ? (size_t)pieces * experts * m * n * sizeof(float) : 0;
    return OPTIM_OK;
} OPTIM_CATCH

int optim_expert_grad(const void *x_dev, int64_t ldx, const void *dy_dev, int64_t ldy, int32_t in_dtype,
                      const int32_t *offsets_dev, int32_t experts, int64_t tokens, int64_t m, int64_t n, void *dw_dev,
                      int32_t dw_dtype, int32_t accumulate, const float *scale_dev, void *workspace,
                      size_t workspace_bytes, void *stream) try {
    if (const int rc = check_expert_sizes(experts, tokens, m, n)) return rc;
    if (in_dtype != OPTIM_BF16 && in_dtype != OPTIM_F16)
        return fail(OPTIM_EDTYPE, "in_dtype must be OPTIM_BF16 or OPTIM_F16");
    if (dw_dtype != OPTIM_F32 && dw_dtype != OPTIM_BF16)
        return fail(OPTIM_EDTYPE, "dw_dtype must be OPTIM_F32 or OPTIM_BF16");
    if (ldx < m || ldy < n || ldx > kExpertMaxSide || ldy > kExpertMaxSide)
        return fail(OPTIM_EINVAL, "ldx and ldy must be at least m and n, and below 2^24");
    if (experts == 0 || m == 0 || n == 0) return OPTIM_OK;
    if (!offsets_dev || !dw_dev || (tokens > 0 && (!x_dev || !dy_dev))) return fail(OPTIM_EINVAL, "NULL buffer");
    const size_t osz = dw_dtype == OPTIM_F32 ? 4 : 2;
    if (!aligned(x_dev, 2) || !aligned(dy_dev, 2) || !aligned(offsets_dev, 4) || !aligned(dw_dev, osz) ||
        !aligned(scale_dev, 4))
        return fail(OPTIM_EALIGN, "buffer misaligned");
    int32_t pieces = workspace ? expert_pieces(experts, tokens, m, n) : 1;
    const size_t need = pieces > 1 ? (size_t)pieces * experts * m * n * sizeof(float) : 0;
    if (need) {
        if (!aligned(workspace, 256))
            return fail(OPTIM_EWORKSPACE, "workspace must be a 256-byte aligned device pointer");
        if (workspace_bytes < need)
            return fail(OPTIM_EWORKSPACE, "workspace too small: need " + std::to_string(need) + " bytes, got " +
                                              std::to_string(workspace_bytes));
    }
    std::vector<Range> ranges;
    auto add = [&](const void *p, size_t bytes, bool written, const char *what) {
        if (p && bytes) ranges.push_back({(uintptr_t)p, (uintptr_t)p + bytes, written, 0, what});
    };
    if (tokens > 0) {
        add(x_dev, ((size_t)(tokens - 1) * ldx + m) * 2, false, "x");
        add(dy_dev, ((size_t)(tokens - 1) * ldy + n) * 2, false, "dy");
    }
    add(offsets_dev, ((size_t)experts + 1) * 4, false, "offsets");
    add(dw_dev, (size_t)experts * m * n * osz, true, "dw");
    add(need ? workspace : nullptr, need, true, "workspace");
    if (const int rc = check_overlaps(ranges)) return rc;
    ExpertArgs a{};
    a.x = static_cast<const char *>(x_dev);
    a.dy = static_cast<const char *>(dy_dev);
    a.ldx = ldx * 2;
    a.ldy = ldy * 2;
    a.offsets = offsets_dev;
    a.dw = static_cast<char *>(dw_dev);
    a.parts = need ? static_cast<float *>(workspace) : nullptr;
    a.scale = scale_dev;
    a.experts = experts;
    a.tokens = (int32_t)tokens;
    a.m = (int32_t)m;
    a.n = (int32_t)n;
    a.pieces = pieces;
    a.accumulate = accumulate != 0;
    a.out_vec = n % 4 == 0 && aligned(dw_dev, 4 * osz);
    const bool direct = m % 8 == 0 && n % 8 == 0 && ldx % 8 == 0 && ldy % 8 == 0 && aligned(x_dev, 16) && aligned(dy_dev, 16);
    HIP_OK(launch_expert_grad(a, in_dtype == OPTIM_BF16, dw_dtype == OPTIM_F32, direct,
                              static_cast<hipStream_t>(stream)));
    return OPTIM_OK;
} OPTIM_CATCH

int optim_scaler_update(float *scale_dev, float *inv_scale_dev, int32_t *growth_tracker_dev,
                        const float *found_inf_dev, double growth_factor, double backoff_factor,
                        int32_t growth_interval, void *stream) try {
    if (!scale_dev || !growth_tracker_dev || !found_inf_dev)
        return fail(OPTIM_EINVAL, "scale, growth tracker and found_inf are required");
    if (!aligned(scale_dev, 4) || !aligned(inv_scale_dev, 4) || !aligned(growth_tracker_dev, 4) ||
        !aligned(found_inf_dev, 4))
        return fail(OPTIM_EALIGN, "scalar pointer misaligned");
    if (!(growth_factor > 1.0) || !std::isfinite(growth_factor))
        return fail(OPTIM_EINVAL, "growth_factor must be finite and > 1");
    if (!(backoff_factor > 0.0 && backoff_factor < 1.0)) return fail(OPTIM_EINVAL, "backoff_factor must be in (0, 1)");
    if (growth_interval < 1) return fail(OPTIM_EINVAL, "growth_interval must be >= 1");
    HIP_OK(launch_scaler_update(scale_dev, inv_scale_dev, growth_tracker_dev, found_inf_dev, growth_factor,
                                backoff_factor, growth_interval, static_cast<hipStream_t>(stream)));
    return OPTIM_OK;
} OPTIM_CATCH

int optim_quantize_blockwise(optim_plan *plan, int32_t is_signed, const float *x_dev, int64_t n,
                             uint8_t *codes_dev, float *absmax_dev, void *stream) try {
    int rc = check_blockwise_plan(plan, "optim_quantize_blockwise");
    if (rc) return rc;
    if (n < 0) return fail(OPTIM_EINVAL, "negative n");
    if (n == 0) return OPTIM_OK;
    if (!x_dev || !codes_dev || !absmax_dev) return fail(OPTIM_EINVAL, "NULL buffer");
    if (!aligned(x_dev, 4) || !aligned(absmax_dev, 4)) return fail(OPTIM_EALIGN, "buffer misaligned");
    HIP_OK(launch_quantize(reinterpret_cast<const Codebook *>(plan->ws + plan->L.codebook), plan->bits,
                           plan->block, is_signed ? 1 : 0, x_dev, n, codes_dev, absmax_dev,
                           static_cast<hipStream_t>(stream)));
    return OPTIM_OK;
} OPTIM_CATCH

int optim_dequantize_blockwise(optim_plan *plan, int32_t is_signed, const uint8_t *codes_dev,
                               const float *absmax_dev, int64_t n, float *x_dev, void *stream) try {
    int rc = check_blockwise_plan(plan, "optim_dequantize_blockwise");
    if (rc) return rc;
    if (n < 0) return fail(OPTIM_EINVAL, "negative n");
    if (n == 0) return OPTIM_OK;
    if (!x_dev || !codes_dev || !absmax_dev) return fail(OPTIM_EINVAL, "NULL buffer");
    if (!aligned(x_dev, 4) || !aligned(absmax_dev, 4)) return fail(OPTIM_EALIGN, "buffer misaligned");
    HIP_OK(launch_dequantize(reinterpret_cast<const Codebook *>(plan->ws + plan->L.codebook), plan->bits,
                             plan->block, is_signed ? 1 : 0, codes_dev, absmax_dev, n, x_dev,
                             static_cast<hipStream_t>(stream)));
    return OPTIM_OK;
} OPTIM_CATCH

int optim_remainder_split(const float *master_dev, uint16_t *bf16_dev, int16_t *rem_dev, int64_t n,
                          void *stream) try {
    if (n < 0) return fail(OPTIM_EINVAL, "negative n");
    if (n == 0) return OPTIM_OK;
    if (!master_dev || !bf16_dev || !rem_dev) return fail(OPTIM_EINVAL, "NULL buffer");
    if (!aligned(master_dev, 4) || !aligned(bf16_dev, 2) || !aligned(rem_dev, 2))
        return fail(OPTIM_EALIGN, "buffer misaligned");
    HIP_OK(launch_remainder_split(master_dev, bf16_dev, rem_dev, n, static_cast<hipStream_t>(stream)));
    return OPTIM_OK;
} OPTIM_CATCH

int optim_remainder_reconstruct(const uint16_t *bf16_dev, const int16_t *rem_dev, float *master_dev, int64_t n,
                                void *stream) try {
    if (n < 0) return fail(OPTIM_EINVAL, "negative n");
    if (n == 0) return OPTIM_OK;
    if (!master_dev || !bf16_dev || !rem_dev) return fail(OPTIM_EINVAL, "NULL buffer");
    if (!aligned(master_dev, 4) || !aligned(bf16_dev, 2) || !aligned(rem_dev, 2))
        return fail(OPTIM_EALIGN, "buffer misaligned");
    HIP_OK(launch_remainder_reconstruct(bf16_dev, rem_dev, master_dev, n, static_cast<hipStream_t>(stream)));
    return OPTIM_OK;
} OPTIM_CATCH

}  // extern "C"
