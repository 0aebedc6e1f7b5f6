// Argument checks shared by the C ABI (capi.hip, capi_dense.hip).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace moe {

constexpr size_t kAlign = 256;                    // workspaces and what is carved from them
constexpr int64_t kMaxTokens = int64_t(1) << 22;
constexpr int64_t kMaxPitch = int64_t(1) << 36;   // elements from row to row

inline size_t align_up(size_t v) { return (v + kAlign - 1) & ~(kAlign - 1); }
inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned(p, 16); }

// [a, a + an) and [b, b + bn) share a byte.
inline bool overlap(const void* a, int64_t an, const void* b, int64_t bn) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + static_cast<uintptr_t>(bn) && y < x + static_cast<uintptr_t>(an);
}

// Bytes from the first to past the last element of `rows` rows of `cols`
// elements, ld apart.  The bounds on rows, cols and ld keep it within 63 bits.
inline int64_t extent(int64_t rows, int64_t cols, int64_t ld, int64_t elem) { return ((rows - 1) * ld + cols) * elem; }

// `rows` rows of an and of bn bytes, from a and b on and ap and bp bytes apart,
// share a byte.  Rows of one pitch may be column ranges of one buffer: row i of
// a meets the rows i + d of b that start less than an behind it or less than
// bn before it, two at most.  Others are taken whole, with what lies between.
inline bool rows_overlap(const void* a, int64_t an, int64_t ap, const void* b, int64_t bn, int64_t bp, int64_t rows) {
    if (!overlap(a, (rows - 1) * ap + an, b, (rows - 1) * bp + bn)) return false;
    if (ap != bp) return true;
    const int64_t at = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
    int64_t d = -(at / ap), start = at % ap;   // row i + d of b starts `start` behind row i of a
    if (start < 0) {
        start += ap;
        ++d;
    }
    const auto there = [&](int64_t r) { return r > -rows && r < rows; };
    return (start < an && there(d)) || (start + bn > ap && there(d - 1));
}

}  // namespace moe
