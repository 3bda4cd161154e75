"""The rows that the experts' kernel takes (csrc/expert_rows.h), at its limits,
on the CPU.  The checks are evaluated by the compiler as constant expressions,
in which a signed overflow is an error.

From any step of a run of up to 2^31 - 1 rows the walk comes to its last step
and stops; clamped runs lie inside [0, tokens]; the pieces of a run are its rows,
each once and in order."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include "expert_rows.h"
#include <initializer_list>
using namespace optim;
constexpr int32_t kMost = INT32_MAX;

// Steps from `done` to the end of `rows` rows, at most `limit`.
constexpr int walk(int32_t done, int32_t rows, int limit) {
    int steps = 1;
    while (steps < limit && next_step(done, rows)) ++steps;
    return steps;
}
constexpr bool ends(int32_t rows) {
    const int32_t last = (rows - 1) / 64;  // the last step's number
    for (int32_t k = last < 3 ? 0 : last - 3; k <= last; ++k)
        if (walk(k * 64, rows, 10) != last - k + 1) return false;
    return true;
}
constexpr bool all_end() {
    for (int32_t r = 1; r <= 300; ++r)
        if (!ends(r)) return false;
    for (int32_t r = kMost - 300; r < kMost; ++r)
        if (!ends(r)) return false;
    return ends(kMost);
}
static_assert(all_end(), "a walk goes on behind the last rows");

constexpr bool inside(Rows r, int32_t tokens) { return 0 <= r.first && r.first <= r.end && r.end <= tokens; }
constexpr bool tiles(Rows run, int32_t pieces) {
    int32_t at = run.first;
    for (int32_t p = 0; p < pieces; ++p) {
        const Rows r = expert_piece(run, pieces, p);
        if (r.first != at || r.end < r.first || r.end > run.end) return false;
        if (r.end != run.end && (r.end - run.first) % kStepRows != 0) return false;
        at = r.end;
    }
    return at == run.end;
}
constexpr bool runs() {
    const int32_t bounds[] = {INT32_MIN, -1, 0, 1, 63, 64, 65, 1000, kMost - 64, kMost - 1, kMost};
    for (int32_t tokens : {0, 1, 64, 1000, kMost - 63, kMost})
        for (int32_t b : bounds)
            for (int32_t e : bounds) {
                const Rows run = expert_run(b, e, tokens);
                if (!inside(run, tokens)) return false;
                if (0 <= b && b <= e && e <= tokens && (run.first != b || run.end != e)) return false;
                for (int32_t pieces : {1, 2, 3, 16, 512})
                    if (!tiles(run, pieces)) return false;
            }
    return true;
}
static_assert(runs(), "a run or its pieces");
int main() {}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not found")
def test_rows_of_a_run(tmp_path):
    src = tmp_path / "rows.cpp"
    src.write_text(PROGRAM)
    r = subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-fconstexpr-ops-limit=100000000",
                        "-I", os.path.join(ROOT, "optimizer_step_adamw_amd", "csrc"), str(src), "-o", str(tmp_path / "rows")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
