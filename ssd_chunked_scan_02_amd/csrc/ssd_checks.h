// Argument checks that the C entry points of the attention layer, the delta rule, the 8-bit cache and the rotation share (host only).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "ssd.h"

namespace ssd {
namespace checks {

// one token axis: in-sequence positions, and positions one tile past an end, are 32-bit in the kernels
constexpr int64_t kMaxTokens = ((int64_t)1 << 31) - 1025;
constexpr int64_t kMaxHeads = 1 << 16;

inline bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
template <size_t N> bool all_aligned(const void* const (&pointers)[N], uintptr_t n) {
    for (const void* p : pointers)
        if (!aligned(p, n)) return false;
    return true;
}
template <size_t N> bool any_null(const void* const (&pointers)[N]) {
    for (const void* p : pointers)
        if (!p) return true;
    return false;
}

// Whether an output is one of the inputs (kernels read inputs after their first stores to outputs) or another output.
template <size_t N, size_t M> bool shared(const void* const (&outputs)[N], const void* const (&inputs)[M]) {
    for (size_t o = 0; o < N; ++o) {
        if (!outputs[o]) continue;
        for (const void* i : inputs)
            if (outputs[o] == i) return true;
        for (size_t i = 0; i < o; ++i)
            if (outputs[o] == outputs[i]) return true;
    }
    return false;
}

// Elements from one token to the next, as given or dense (a tile's byte offsets are 32-bit: 64 rows of up to 2^24
// four-byte elements).
inline int stride(int64_t given, int64_t dense, int64_t elem, int64_t& out) {
    if (given == 0) {
        out = dense;
        return SSD_OK;
    }
    if (given < dense || given >= ((int64_t)1 << 24)) return SSD_ERR_INVALID;
    if (given * elem % 16 != 0) return SSD_ERR_ALIGN;
    out = given;
    return SSD_OK;
}

// HIP counts the threads of a launch in 32 bits.
inline bool launchable(int64_t groups, int threads) { return groups < ((int64_t)1 << 32) / threads; }

inline int code(int rc) { return rc == 0 ? SSD_OK : rc == -2 ? SSD_ERR_UNSUPPORTED : SSD_ERR_HIP; }

inline size_t align16(size_t n) { return (n + 15) & ~(size_t)15; }

}  // namespace checks
}  // namespace ssd
