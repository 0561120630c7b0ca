// The tiles of all sequences, one sequence behind the other, cut into equal ranges whatever the lengths.
#pragma once

#include "kv_device.h"

namespace lorapool {

// The ranges: R of them (no more than there are tiles), base tiles each and one more in the first `rem`.
struct Ranges {
    int64_t base;
    int32_t rem, R;
    __device__ __forceinline__ int64_t start(int64_t r) const { return r * base + (r < rem ? r : rem); }
    __device__ __forceinline__ int32_t of(int64_t tile) const {            // the range a tile lies in
        const int64_t longer = rem * (base + 1);
        return tile < longer ? (int32_t)div(tile, base + 1) : rem + (int32_t)div(tile - longer, base);
    }
    static __device__ __forceinline__ int64_t div(int64_t a, int64_t b) {  // 32 bits as a rule: a third of the time
        return (a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
    }
};
__device__ __forceinline__ Ranges ranges_of(int64_t total, int32_t R) {
    Ranges r;
    r.R = (int32_t)(total < R ? total : R);
    r.base = r.R ? Ranges::div(total, r.R) : 0;
    r.rem = (int32_t)(total - r.base * r.R);
    return r;
}

// Pieces of the sequence whose tiles are [t0, t1): from range r0's slot s0, then slot 0 of r0 + 1 .. r1.
// r0 == r1: one wave saw it whole.
struct Pieces {
    int32_t r0, r1, s0;
};
__device__ __forceinline__ Pieces pieces_of(int64_t t0, int64_t t1, const Ranges &rg) {
    Pieces p;
    p.r0 = rg.of(t0);
    p.r1 = rg.of(t1 - 1);
    p.s0 = rg.start(p.r0) == t0 ? 0 : 1;
    return p;
}

}  // namespace lorapool
