// Argument checks shared by the C ABI's translation units.
#pragma once

#include "nm_internal.h"

namespace nm {

inline int64_t esize(nm_dtype d) { return d == NM_BF16 ? 2 : (d == NM_I8 || d == NM_FP8) ? 1 : 4; }
inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
inline bool aligned_to(const void* p, int64_t bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

struct Range {
    uintptr_t lo, hi;
};
// Byte range touched by a row-major [rows, cols] view with leading dimension ld.
inline Range span(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t es) {
    if (!p || rows <= 0 || cols <= 0) return {0, 0};
    const uintptr_t b = (uintptr_t)p;
    return {b, b + (uintptr_t)(((rows - 1) * ld + cols) * es)};
}
inline bool overlap(Range a, Range b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

#define NM_REQ(cond, st, ...)                                                \
    do {                                                                     \
        if (!(cond)) return set_error(st, __VA_ARGS__);                      \
    } while (0)

}  // namespace nm
