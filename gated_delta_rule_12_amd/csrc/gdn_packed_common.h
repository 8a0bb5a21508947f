// Where packed sequences and their chunks lie, shared by the packed forward
// (gdn_packed.hip) and backward (gdn_bwd_chunk.hip).  Internal to libgdn.
//
// Lengths are known on the device only.  Chunks of 64 tokens of sequence s get
// consecutive places from cu[s] / 64 + s on: ceil(n / 64) of them never reach
// the next sequence's first place, and N / 64 + S places are enough, so no
// kernel has to lay out a table.  Where only sequences of 32 tokens or more
// have chunks, cu[s] / 32 serves as well, with N / 32 places however many
// shorter ones there are: ceil(n / 64) <= floor(n / 32) from n = 32 on.
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
// The rule of the chunks' places
struct Places {
    int shift;  // 6: cu / 64 + s; 5: cu / 32
    int each;   // 1; 0
    __device__ int64_t first(int64_t begin, int64_t s) const { return (begin >> shift) + s * each; }
};
__host__ __device__ __forceinline__ Places chunk_places() { return {6, 1}; }
// The sequence whose places hold `place`, found by a whole wave: 64 candidates
// a round.
__device__ __forceinline__ int64_t seq_of_place(const Offsets& p, int64_t place, const Places& rule, int lane) {
    int64_t lo = 0, cnt = p.S;
    while (cnt > 1) {
        const int64_t step = (cnt + 63) >> 6;
        bool le = false;
        if (lane * step < cnt) {
            const int64_t s = lo + lane * step;
            le = rule.first(cu_at(p, s), s) <= place;
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
// K counts of every sequence, counts(s, c), summed over the sequences in that
// order: out[k][r] those before rank r, out[k][S] all of them, INT32_MAX where
// there are more (lengths of offsets out of order can sum to any number).  By
// the workgroup that ordered them; sums: K a wave in LDS.
__device__ __forceinline__ uint32_t add_up_to_max(uint32_t a, uint32_t b) { return min(a + b, (uint32_t)INT32_MAX); }
template <int K, class F>
__device__ __forceinline__ void count_ranks(int S, const int32_t* order, F counts, int32_t* const (&out)[K],
                                            uint32_t* sums, int tid, int threads) {
    const int run = (S + threads - 1) / threads, r0 = min(tid * run, S), r1 = min(r0 + run, S);
    const int w = tid >> 6, lane = tid & 63;
    uint32_t at[K] = {}, c[K];
#pragma unroll 1
    for (int r = r0; r < r1; ++r) {
        counts(order[r], c);
#pragma unroll
        for (int k = 0; k < K; ++k) at[k] = add_up_to_max(at[k], c[k]);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t y = __shfl_up(at[k], o, 64);
            if (lane >= o) at[k] = add_up_to_max(at[k], y);
        }
        if (lane == 63) sums[w * K + k] = at[k];
        at[k] = __shfl_up(at[k], 1, 64);
        if (lane == 0) at[k] = 0;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
        for (int i = 0; i < w; ++i) at[k] = add_up_to_max(at[k], sums[i * K + k]);
#pragma unroll 1
    for (int r = r0; r < r1; ++r) {
        counts(order[r], c);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            out[k][r] = (int32_t)at[k];
            at[k] = add_up_to_max(at[k], c[k]);
        }
    }
    if (tid == threads - 1) {
#pragma unroll
        for (int k = 0; k < K; ++k) out[k][S] = (int32_t)at[k];
    }
}
// The rank whose things hold the i-th (i < first[S]), by a whole wave.
__device__ __forceinline__ int64_t rank_holding(const int32_t* first, int64_t S, int i, int lane) {
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
