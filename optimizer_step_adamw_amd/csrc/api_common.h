// api_common.h -- what the C entry points share: statuses with their message,
// and the check that no written buffer overlaps another.  Internal.
#pragma once

#include "optim_step.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <string>
#include <vector>

namespace optim {

// Keeps the message for optim_last_error() and returns the code.
int fail(int code, const std::string &msg);

// What an entry point's body throws (the host is out of memory) becomes a status:
// no exception leaves the library.
int out_of_memory() noexcept;
#define OPTIM_CATCH \
    catch (...) { return out_of_memory(); }

#define HIP_OK(expr)                                                                 \
    do {                                                                             \
        hipError_t e_ = (expr);                                                      \
        if (e_ != hipSuccess)                                                        \
            return fail(OPTIM_EHIP, std::string(#expr) + ": " + hipGetErrorString(e_)); \
    } while (0)

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Range {
    uintptr_t lo, hi;
    bool written;
    int tensor;
    const char *what;
};

// no written buffer may overlap any other buffer of the call or plan
int check_overlaps(std::vector<Range> &ranges);

}  // namespace optim
