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

// The sequences by falling length (classes a quarter of an octave of 64-token
// chunks wide; within a class in no particular order, which no result depends
// on), so that the kernels that carry a state through a sequence start the
// longest first.  By one workgroup of `threads`; hist: 2 x kLenClasses ints of
// LDS.
constexpr int kLenClasses = 128;
__device__ __forceinline__ int len_class(int64_t n) {
    const unsigned c = (unsigned)((n + 63) >> 6) + 1;
    const int e = 31 - __clz(c);
    const int key = 4 * e + (e >= 2 ? (c >> (e - 2)) & 3 : (c << (2 - e)) & 3);
    return max(kLenClasses - 1 - key, 0);
}
__device__ __forceinline__ void order_sequences(const Offsets& p, int32_t* order, int* hist, int tid, int threads) {
    for (int i = tid; i < 2 * kLenClasses; i += threads) hist[i] = 0;
    __syncthreads();
    for (int64_t s = tid; s < p.S; s += threads) atomicAdd(&hist[len_class(span_of(p, s).n)], 1);
    __syncthreads();
    if (tid == 0) {
        int at = 0;
        for (int i = 0; i < kLenClasses; ++i) {
            hist[kLenClasses + i] = at;
            at += hist[i];
        }
    }
    __syncthreads();
    for (int64_t s = tid; s < p.S; s += threads)
        order[atomicAdd(&hist[kLenClasses + len_class(span_of(p, s).n)], 1)] = (int32_t)s;
}
// Segments of 2^shift tokens of sequences of at least min_len tokens, counted
// over the sequences in that order: first[r] those before rank r, first[S] all
// of them.  By the workgroup that ordered them; sums: `threads` ints of LDS.
__device__ __forceinline__ void count_segments(const Offsets& p, const int32_t* order, int shift, int64_t min_len,
                                               int32_t* first, int* sums, int tid, int threads) {
    const int64_t run = (p.S + threads - 1) / threads, r0 = tid * run, r1 = min(r0 + run, p.S);
    auto segments = [&](int64_t r) {
        const int64_t n = span_of(p, order[r]).n;
        return n < min_len ? 0 : (int)((n + ((int64_t)1 << shift) - 1) >> shift);
    };
    int mine = 0;
    for (int64_t r = r0; r < r1; ++r) mine += segments(r);
    sums[tid] = mine;
    __syncthreads();
    if (tid == 0) {
        int at = 0;
        for (int i = 0; i < threads; ++i) {
            const int x = sums[i];
            sums[i] = at;
            at += x;
        }
        first[p.S] = at;
    }
    __syncthreads();
    int at = sums[tid];
    for (int64_t r = r0; r < r1; ++r) {
        first[r] = at;
        at += segments(r);
    }
}
// The rank whose segments hold the i-th (i < first[S]), by a whole wave.
__device__ __forceinline__ int64_t rank_of_segment(const int32_t* first, int64_t S, int i, int lane) {
    int64_t lo = 0, cnt = S;
    while (cnt > 1) {
        const int64_t step = (cnt + 63) >> 6;
        const bool le = lane * step < cnt && first[lo + lane * step] <= i;
        const int hits = (int)__popcll(__ballot(le));
        const int64_t k = hits > 0 ? hits - 1 : 0;
        lo += k * step;
        cnt = min(step, cnt - k * step);
    }
    return lo;
}

}  // namespace
}  // namespace gdn
