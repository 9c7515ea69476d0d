// Host-side argument checks shared by the C ABI sources (gdr_api.cpp, layer_api.cpp).
#pragma once

#include <stdint.h>

#include <initializer_list>

#include "../../include/gdr.h"

namespace gdr {

// the text behind gdr_last_error()
extern thread_local char g_last_error[512];

// records the text and returns s
gdr_status_t fail(gdr_status_t s, const char *fmt, ...);

struct Range {
    const char *name;
    uintptr_t lo, hi;  // [lo, hi)
    bool present() const { return lo != 0 && hi > lo; }
};

inline Range rng(const char *name, const void *p, int64_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{name, lo, lo + (uintptr_t)(bytes > 0 ? bytes : 0)};
}

inline bool overlap(const Range &a, const Range &b) {
    return a.present() && b.present() && a.lo < b.hi && b.lo < a.hi;
}

inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

// product of non-negative sizes, or -1 on overflow past 2^62
inline int64_t prod(std::initializer_list<int64_t> xs) {
    int64_t r = 1;
    for (int64_t x : xs) {
        if (x < 0) return -1;
        if (x != 0 && r > (INT64_C(1) << 62) / x) return -1;
        r *= x;
    }
    return r;
}

inline int64_t elem_size(int32_t dtype) { return dtype == GDR_BF16 ? 2 : 4; }

}  // namespace gdr
