// grkan_check.h -- argument checks shared by the C ABI's sources: alignment,
// overlapping byte ranges, HIP errors as statuses.  Internal.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "grkan.h"

namespace grkan {

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A byte range an argument covers; empty if absent.
struct Range {
    const void *p;
    size_t n;
};

inline bool overlap(const Range &a, const Range &b) {
    if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.n && y < x + a.n;
}

// Every output apart from every other argument.
inline bool outputs_overlap(const Range *outs, int no, const Range *ins, int ni) {
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j)
            if (overlap(outs[i], ins[j])) return true;
        for (int j = i + 1; j < no; ++j)
            if (overlap(outs[i], outs[j])) return true;
    }
    return false;
}

inline grkan_status_t from_hip(hipError_t e) { return e == hipSuccess ? GRKAN_OK : GRKAN_ERR_HIP; }

}  // namespace grkan
