// rog_head_checks.h -- what the host planners of the vocabulary-side operators
// check their arguments with.  Pure host code.
#pragma once

#include "rog_head.h"

namespace rog {

inline uintptr_t addr(const void *p) { return reinterpret_cast<uintptr_t>(p); }
inline uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }
inline uint32_t esize(rog_dtype t) { return t == ROG_DTYPE_F32 ? 4 : 2; }
inline bool known(rog_dtype t) { return t == ROG_DTYPE_F32 || t == ROG_DTYPE_BF16 || t == ROG_DTYPE_F16; }

// `rows` runs of `width` bytes, `stride` bytes apart.
struct Strip {
    uintptr_t at;
    uint64_t rows, stride, width;
    uint64_t extent() const { return rows && width ? (rows - 1) * stride + width : 0; }
};
inline Strip flat(const void *p, uint64_t bytes) { return Strip{addr(p), 1, 0, bytes}; }

// Whether two strips share a byte.  Strips of one stride whose runs fit in it
// (column slices of one matrix) are compared run by run; others by their
// extents, which may call two interleaved strips overlapping.
inline bool overlap(const Strip &a, const Strip &b) {
    const uint64_t na = a.extent(), nb = b.extent();
    if (!na || !nb || a.at >= b.at + nb || b.at >= a.at + na) return false;
    if (a.rows > 1 && b.rows > 1 && a.stride == b.stride && a.width <= a.stride && b.width <= a.stride) {
        const uint64_t s = a.stride;
        const uint64_t d = b.at >= a.at ? (b.at - a.at) % s : (s - (a.at - b.at) % s) % s;   // b's place in a's period
        return d < a.width || d + b.width > s;
    }
    return true;
}

// Address range of a strip inside the address space, sizes without overflow.
inline bool fits(uintptr_t at, uint64_t rows, uint64_t stride, uint64_t width) {
    if (!rows || !width) return true;
    if (stride && rows - 1 > (uint64_t(1) << 62) / stride) return false;
    const uint64_t n = (rows - 1) * stride + width;
    return at <= UINTPTR_MAX - n;
}

}  // namespace rog
