// expert_rows.h -- which rows of an expert's run a workgroup of
// kernels_expert.hip sums, and in what steps.  Plain arithmetic on counts below
// 2^31, here so that its limits are checked on the CPU as well.
#pragma once

#include <cstdint>

namespace optim {

constexpr int32_t kStepRows = 64;  // rows of a step of the product

struct Rows {
    int32_t first, end;
};

// Rows [begin, end) of `tokens`: both clamped to [0, tokens], the end to the
// beginning as well.
constexpr Rows expert_run(int32_t begin, int32_t end, int32_t tokens) {
    const int32_t b = begin < 0 ? 0 : (begin < tokens ? begin : tokens);
    return Rows{b, end < b ? b : (end < tokens ? end : tokens)};
}

// Piece `piece` of `pieces` of a run: whole steps but for the run's last.
constexpr Rows expert_piece(Rows run, int32_t pieces, int32_t piece) {
    const int32_t steps = (int32_t)(((int64_t)run.end - run.first + kStepRows - 1) / kStepRows);
    const int32_t each = (steps + pieces - 1) / pieces;
    const int64_t lo = run.first + (int64_t)piece * each * kStepRows, hi = lo + (int64_t)each * kStepRows;
    return Rows{(int32_t)(lo < run.end ? lo : run.end), (int32_t)(hi < run.end ? hi : run.end)};
}

// Goes on from the step at `done` (below rows) to the next one of `rows` rows,
// where there is one.  (`done` never passes `rows`: it could pass 2^31.)
constexpr bool next_step(int32_t &done, int32_t rows) {
    if (rows - done <= kStepRows) return false;
    done += kStepRows;
    return true;
}

}  // namespace optim
