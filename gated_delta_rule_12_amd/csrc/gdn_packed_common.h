// Where packed sequences and their chunks lie, shared by the packed forward
// (gdn_packed.hip) and backward (gdn_bwd_chunk.hip).  Internal to libgdn.
//
// Lengths are known on the device only.  Chunks (or segments) of 2^shift
// tokens of sequence s get consecutive places from cu[s] / 2^shift + s on:
// ceil(n / 2^shift) of them never reach the next sequence's first place, and
// N / 2^shift + S places are enough, so no kernel has to lay out a table.
// Offsets are clamped to 0 .. N and to rising order, so no content of cu leads
// out of bounds.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdn {
namespace {

struct Offsets {
    const int32_t* cu;  // [S + 1]
    int64_t N, S;
};
__device__ __forceinline__ int64_t cu_at(const Offsets& p, int64_t s) {
    const int64_t x = p.cu[s];
    return x < 0 ? 0 : x > p.N ? p.N : x;
}
struct Span {
    int64_t begin;
    int64_t n;
};
__device__ __forceinline__ Span span_of(const Offsets& p, int64_t s) {
    const int64_t a = cu_at(p, s), b = cu_at(p, s + 1);
    return {a, b > a ? b - a : 0};
}
// The sequence whose places hold `place` (2^shift tokens a place), found by
// a whole wave: 64 candidates a round.
__device__ __forceinline__ int64_t seq_of_place(const Offsets& p, int64_t place, int shift, int lane) {
    int64_t lo = 0, cnt = p.S;
    while (cnt > 1) {
        const int64_t step = (cnt + 63) >> 6;
        bool le = false;
        if (lane * step < cnt) {
            const int64_t s = lo + lane * step;
            le = (cu_at(p, s) >> shift) + s <= place;
        }
        // (the count is unsigned: none of them has to give 0 too, as in front
        // of the first sequence)
        const int hits = (int)__popcll(__ballot(le));
        const int64_t k = hits > 0 ? hits - 1 : 0;
        lo += k * step;
        cnt = min(step, cnt - k * step);
    }
    return lo;
}

}  // namespace
}  // namespace gdn
