// Linear attention with a decay for each head over packed ragged sequences,
// forward and backward (gdn_linear_fwd, gdn_linear_backward).
//
// Per value head with decay a (state S is dv x dk):
//   S_t = a S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t
// which over a segment of n tokens (i, j counted in it, S its start state) is
//   o_i = scale (sum_{j<=i} a^{i-j} (q_i.k_j) v_j + a^{i+1} S q_i)
//   S'  = a^n S + sum_j a^{n-1-j} v_j k_j^T
// and, with do' = scale do and G the gradient of S',
//   dq_i = sum_{j<=i} a^{i-j} (do'_i.v_j) k_j + a^{i+1} S^T do'_i
//   dv_j = sum_{i>=j} a^{i-j} (q_i.k_j) do'_i + a^{n-1-j} G k_j
//   dk_j = sum_{i>=j} a^{i-j} (do'_i.v_j) q_i + a^{n-1-j} G^T v_j
//   dS   = a^n G + sum_i a^{i+1} do'_i q_i^T
//   da   = sum_{i>j} (i-j) a^{i-j-1} (q_i.k_j) (do'_i.v_j) + sum_i (i+1) a^i do'_i.S q_i
//        + sum_j (n-1-j) a^{n-2-j} v_j.G k_j + n a^{n-1} <G, S>
// No term divides by a power of a, and each term of da has its power of a as a
// factor, so any a from 0 to 1 is right and none of the sums cancels by
// construction.
//
// Why segments of 256: their states are written once and read twice (64 KiB a head
// of 128, as much as 256 tokens of it in one array), and what is quadratic in a
// segment grows with its length.  512 tokens: outputs 122 instead of 88 us, the scan
// 20 instead of 33, additions 43 instead of 45 (one sequence of 65531 tokens, 4
// heads of 128, bf16; fp32, where products cost eight times as much, was not
// measured with others).
//
// Forward: k_lin_plan (where the segments lie), k_lin_add (what each adds to its
// state; short sequences beside that), k_lin_scan (the states between), k_lin_out (the
// outputs, a segment's 128 rows a workgroup), k_lin_end (in place: the last
// segments' states).  Backward: k_lin_bfirst, k_lin_badd and k_lin_bscan do the same
// for states and gradients of states at once, k_lin_grads has all rows, k_lin_join
// sums addends.  Sequences of few tokens: k_lin_rec alone.
//
// Kernel times in us, and what bounds them (bf16, heads of 128; averages of a kernel
// trace of 45 calls behind 5, from a device that was idle: such calls take 200, 185
// and 558 us without a trace as well, the same in a long row 179, 170 and 526; 6.05
// TB/s is the rate of a copy on this card):
//   40 sequences, 16384 tokens, 16 heads: plan 6, add 69 (short sequences inside), scan
//     29, out 96; in place 6, 54, 25, 93, end 25
//   one sequence of 65531 tokens, 4 heads: 5, add 46 (201 MB moved: 4.4 TB/s; without
//     products 43, without stores 36, with few loads 37), scan 36 (134 MB, one chain
//     of 256 segments an element), out 96 (335 MB: 55 at least); in place 5, 46, 36,
//     92, end 16.  Best times of the outputs with waves of 32 rows: 88, loads alone 66,
//     without tiles of tokens 46, without the start states 71, with scores of one
//     term 80
//   7 sequences, 16384 tokens, 16 heads, backward: 6, add 82 (260 MB moved), scan 58
//     (235 MB), gradients 403 (870 MB from and to HBM take 145; matrix cores are busy
//     21 % of the time, vector ALU 28 %, LDS 19 %; waves wait for memory and barriers
//     37 % and for each other's issue 34 %; 27 of 256 registers a lane are spilled),
//     join 5
//   a step of 256 single tokens, 16 heads: 92 (the states at 5.8 TB/s)
#include "gdn_elements.h"
#include "gdn_internal.h"
#include "gdn_mfma_common.h"
#include "gdn_packed_common.h"
#include "../../include/gdn.h"

namespace gdn {
namespace {

// Sequences of fewer tokens go token by token (forward): a chain of latencies that
// many sequences share a chip for, against one pass of a segment.  Heads of 128, 16
// heads, tokens against segments: bf16 16 sequences of 32 tokens 29.6 and 30 us,
// 256 of 32 352 and 322, 256 of 48 516 and 357; fp32 (an eighth of the matrix
// rate) 16 of 48 37 and 60, 256 of 48 532 and 852, 16 of 200 142 and 110, 256 of
// 200 1894 and 1621: about even from 64 tokens (few) to 130 (many) on.
constexpr int lin_min(int dtype) { return dtype == GDN_BF16 ? 32 : 64; }
// Tokens of a segment.
constexpr int kSeg = 256;

// A segment: its tokens, its sequence, whether it is that one's first or last.
struct Seg {
    int begin, n, seq, ends;
};
constexpr int kFirst = 1, kLast = 2;

struct Lin {
    Linear p;
    Offsets at;
    int Hv, group;
    int state;           // elements of a state
    int64_t chunk_min;   // sequences of fewer tokens have no segments
    int64_t nrank, nseg; // the most sequences with segments, and segments
    int32_t* count;      // [2]: such sequences, segments
    int32_t* seqs;       // [nrank]: the sequences with segments
    int32_t* first;      // [nrank + 1]: segments before each of them
    Seg* segs;           // [nseg], without tokens behind the last
    float* log2a;        // [Hv]: of the decays
    float* s_seg;        // [nseg, Hv] states: what a segment adds, then the state behind it
    bool late;           // end states are written behind the outputs (in place)
    // backward
    const void* dout;
    const float* ds_out;
    void *dq, *dk, *dv;
    float *dalpha, *ds0;
    float* g_seg;        // [nseg, Hv]: what a segment adds to its start state's gradient, then all of that
    float* part;         // [Hv, parts]: addends of dalpha
    int64_t parts;
    int64_t part_dv, part_pairs, part_scan;  // behind dq's: where dv's, the pairs' and the scan's begin
    int splits;          // parts that a key head's value heads are summed in for dq and dk
    float* split;        // [2 (dk, dq), splits, N, Hk, dk]: these sums, where there is more than one
};

// Segment si, in scalar registers
__device__ __forceinline__ Seg segment(const Lin& a, int64_t si) {
    const Seg x = a.segs[si];
    auto same = [](int y) { return __builtin_amdgcn_readfirstlane(y); };
    return Seg{same(x.begin), same(x.n), same(x.seq), same(x.ends)};
}
__device__ __forceinline__ const float* start_of(const Lin& a, int64_t s, int64_t h) {
    const Linear& p = a.p;
    const int64_t slot = p.slots_in ? (int64_t)p.slots_in[s] : s;
    if (!p.s_in || slot < 0 || slot >= p.n_in) return nullptr;
    return p.s_in + (slot * a.Hv + h) * a.state;
}
__device__ __forceinline__ float* end_of(const Lin& a, int64_t s, int64_t h) {
    const Linear& p = a.p;
    const int64_t slot = p.slots_out ? (int64_t)p.slots_out[s] : s;
    if (!p.s_out || slot < 0 || slot >= p.n_out) return nullptr;
    return p.s_out + (slot * a.Hv + h) * a.state;
}

// The state in front of segment si, or null (zero)
__device__ __forceinline__ const float* state_before(const Lin& a, const Seg& sg, int64_t si, int h) {
    return sg.ends & kFirst ? start_of(a, sg.seq, h) : a.s_seg + ((si - 1) * a.Hv + h) * (int64_t)a.state;
}

// Powers of a decay: e^(x log a), with a^0 = 1 for a zero decay too.  The
// exponent's rounding leaves an error of |x log2 a| 2^-24 relative to the power,
// less than 2^-24 of a weight of one wherever the power counts.
struct Decay {
    float a, log2a;
    __device__ Decay(const Lin& l, int h) : a(l.p.alpha[h]), log2a(l.log2a[h]) {}
    __device__ float operator()(int x) const { return x == 0 ? 1.f : exp2f((float)x * log2a); }
};

// ---------------------------------------------------------------------------
// where the segments lie
// ---------------------------------------------------------------------------
// By one workgroup.  Counts saturate and are cut to the tables' sizes, so that no
// content of the offsets leads out of them.
constexpr int kPlanThreads = 1024;
constexpr int kPlanLds = 2048;  // ranks whose counts the search finds in LDS
__device__ __forceinline__ void plan_segments(const Lin& a, int tid) {
    __shared__ uint32_t sums[2 * kPlanThreads / 64];
    __shared__ int lfirst[kPlanLds];
    for (int h = tid; h < a.Hv; h += kPlanThreads) a.log2a[h] = (float)log2((double)a.p.alpha[h]);
    const int64_t S = a.at.S, run = (S + kPlanThreads - 1) / kPlanThreads, r0 = min(tid * run, S), r1 = min(r0 + run, S);
    const int w = tid >> 6, lane = tid & 63;
    auto segs_of = [&](int64_t n) { return (uint32_t)((n + kSeg - 1) / kSeg); };
    uint32_t at[2] = {0, 0};
    for (int64_t s = r0; s < r1; ++s) {
        const int64_t n = span_of(a.at, s).n;
        if (n < a.chunk_min) continue;
        at[0] += 1;
        at[1] = add_up_to_max(at[1], segs_of(n));
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t y = __shfl_up(at[k], o, 64);
            if (lane >= o) at[k] = add_up_to_max(at[k], y);
        }
        if (lane == 63) sums[2 * w + k] = at[k];
        at[k] = __shfl_up(at[k], 1, 64);
        if (lane == 0) at[k] = 0;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k)
        for (int i = 0; i < w; ++i) at[k] = add_up_to_max(at[k], sums[2 * i + k]);
    auto put = [&](uint32_t rank, uint32_t first) {
        if (rank <= a.nrank) a.first[rank] = (int32_t)first;
        if (rank < kPlanLds) lfirst[rank] = (int)first;
    };
    for (int64_t s = r0; s < r1; ++s) {
        const int64_t n = span_of(a.at, s).n;
        if (n < a.chunk_min) continue;
        put(at[0], at[1]);
        if (at[0] < a.nrank) a.seqs[at[0]] = (int32_t)s;
        at[0] += 1;
        at[1] = add_up_to_max(at[1], segs_of(n));
    }
    __shared__ int total[2];
    if (tid == kPlanThreads - 1) {
        put(at[0], at[1]);
        total[0] = (int)min<int64_t>(at[0], a.nrank);
        total[1] = (int)min<int64_t>(at[1], a.nseg);
        a.count[0] = total[0];
        a.count[1] = total[1];
    }
    __threadfence_block();
    __syncthreads();
    const int ranks = total[0];
    for (int64_t i = total[1] + tid; i < a.nseg; i += kPlanThreads) a.segs[i] = Seg{0, 0, 0, 0};
    for (int i = tid; i < total[1]; i += kPlanThreads) {
        int lo = 0, hi = ranks;  // first[lo] <= i, first[hi] > i or none
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            const int f = mid < kPlanLds ? lfirst[mid] : a.first[mid];
            if (f <= i) lo = mid;
            else hi = mid;
        }
        const int s = a.seqs[lo];
        const Span sp = span_of(a.at, s);
        const int64_t from = (int64_t)(i - (lo < kPlanLds ? lfirst[lo] : a.first[lo])) * kSeg;
        Seg x;
        x.n = (int)max<int64_t>(min<int64_t>(kSeg, sp.n - from), 0);
        x.begin = x.n > 0 ? (int)(sp.begin + from) : 0;
        x.seq = s;
        // (where the table ends, so does the sequence: no segment looks behind it)
        x.ends = (from == 0 ? kFirst : 0) | (from + kSeg >= sp.n || i + 1 == total[1] ? kLast : 0);
        a.segs[i] = x;
    }
}

// ---------------------------------------------------------------------------
// token by token
// ---------------------------------------------------------------------------
// LPR lanes hold a row of S, four elements each, and kLinR rows one behind the
// other: a token's v and o of a lane's rows are one piece each.
constexpr int kLinR = 4, kFlight = 4;
template <int LPR>
constexpr int rec_rows() {
    return 4 * (64 / LPR) * kLinR;  // rows a workgroup
}
template <int DT, int LPR>
__device__ __forceinline__ void rec_sequence(const Lin& a, unsigned block, unsigned blocks) {
    constexpr int RB = rec_rows<LPR>();
    const Linear& p = a.p;
    const int dk = (int)p.dk, dv = (int)p.dv;
    const unsigned nrb = ((unsigned)dv + RB - 1) / RB;
    const unsigned id0 = on_one_xcd(block, blocks, nrb * a.Hv), id = id0 / nrb;
    const int rb = id0 - id * nrb, s = id / a.Hv, h = id - s * a.Hv, hk = h / a.group;
    const Span sp = span_of(a.at, s);
    const float* src = start_of(a, s, h);
    float* dst = end_of(a, s, h);
    if (sp.n >= a.chunk_min || (sp.n == 0 && src == dst)) return;
    const int c = threadIdx.x % LPR, row = rb * RB + threadIdx.x / LPR * kLinR;
    // (lanes behind the row's end and rows behind the last repeat the last piece
    // and store nothing; what such lanes add to a sum is zero, whatever they hold)
    const bool on = 4 * c < dk, in = row < dv;
    const int col = on ? 4 * c : dk - 4, r0 = in ? row : dv - kLinR;
    f32x4 S[kLinR];
#pragma unroll
    for (int j = 0; j < kLinR; ++j)
        S[j] = src ? __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(src + (r0 + j) * dk + col)) : zero4();
    const float alpha = p.alpha[h];
    // the next kFlight tokens' rows are in flight
    R4<DT> k[kFlight], q[kFlight], v[kFlight];
    auto fetch = [&](int u, int64_t t) {
        if (t >= sp.n) return;
        t += sp.begin;
        k[u] = ldr<DT>(p.k, t * p.k_stride + hk * dk + col);
        q[u] = ldr<DT>(p.q, t * p.q_stride + hk * dk + col);
        v[u] = ldr<DT>(p.v, t * p.v_stride + h * dv + r0);
    };
#pragma unroll
    for (int u = 0; u < kFlight; ++u) fetch(u, u);
    for (int64_t t0 = 0; t0 < sp.n; t0 += kFlight)
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            if (t0 + u >= sp.n) break;
            const f32x4 kt = cvt<DT>(k[u]), qt = cvt<DT>(q[u]), vt = cvt<DT>(v[u]);
            f32x4 o;
#pragma unroll
            for (int j = 0; j < kLinR; ++j) {
                S[j] = alpha * S[j] + vt[j] * kt;
                o[j] = p.scale * row_sum<LPR>(on ? dot4e(S[j], qt) : 0.f);
            }
            fetch(u, t0 + u + kFlight);
            if (c == 0 && in) {
                const int64_t at = ((sp.begin + t0 + u) * a.Hv + h) * dv + row;
                if constexpr (DT == GDN_BF16)
                    st_g(static_cast<uint16_t*>(p.out) + at, u32x2{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])});
                else
                    st_g(static_cast<float*>(p.out) + at, o);
            }
        }
    if (!dst || !on || !in) return;
#pragma unroll
    for (int j = 0; j < kLinR; ++j)
        __builtin_nontemporal_store(S[j], reinterpret_cast<f32x4*>(dst + (row + j) * dk + col));
}
template <int DT, int LPR>
__global__ __launch_bounds__(kThreads) void k_lin_rec(Lin a) {
    rec_sequence<DT, LPR>(a, blockIdx.x, gridDim.x);
}
__global__ __launch_bounds__(kPlanThreads) void k_lin_plan(Lin a) { plan_segments(a, threadIdx.x); }
// the segments' places, and the gradients' rows outside every sequence
__global__ __launch_bounds__(kPlanThreads) void k_lin_bfirst(Lin a) {
    if (blockIdx.x == 0) {
        plan_segments(a, threadIdx.x);
        return;
    }
    const Linear& p = a.p;
    const int64_t c0 = cu_at(a.at, 0), c1 = max(cu_at(a.at, p.S), c0);
    const int64_t e = p.dtype == GDN_BF16 ? 2 : 4, bk = p.Hk * p.dk * e, bv = p.Hv * p.dv * e;
    for (int64_t i = blockIdx.x - 1; i < c0 + (p.N - c1); i += gridDim.x - 1) {
        const int64_t t = i < c0 ? i : c1 + (i - c0);
        for (int64_t b = 16 * threadIdx.x; b < bk; b += 16 * kPlanThreads) {
            st_g(static_cast<char*>(a.dq) + t * bk + b, u32x4{0, 0, 0, 0});
            st_g(static_cast<char*>(a.dk) + t * bk + b, u32x4{0, 0, 0, 0});
        }
        for (int64_t b = 16 * threadIdx.x; b < bv; b += 16 * kPlanThreads)
            st_g(static_cast<char*>(a.dv) + t * bv + b, u32x4{0, 0, 0, 0});
    }
}

// ---------------------------------------------------------------------------
// operands of the matrix cores
// ---------------------------------------------------------------------------
// Lane l = 16 g + i.  A step contracts KS indices; the lane holds KS / 4 of row
// (or column) i: those from (KS / 4) g on.  bf16 elements are exact operands;
// what fp32 arithmetic made is split into TERMS of them.  (Blocks of 32 x 32, whose
// instructions do twice the work in the same time, were no faster: additions of a
// training step of 16384 tokens 85 instead of 82 us, outputs of a mixed batch 94
// instead of 90, gradients 450 instead of 430.  Products are not what these
// kernels wait for.)
template <int DT>
struct El;
template <>
struct El<GDN_BF16> {
    using T = uint16_t;
    using Op = u16x8;
    static constexpr int KS = 32, TT = 32, PAD = 16, TERMS = 2;  // TT: tokens a tile
};
template <>
struct El<GDN_F32> {
    using T = float;
    using Op = f32x4;
    static constexpr int KS = 16, TT = 32, PAD = 4, TERMS = 1;
};

__device__ __forceinline__ f32x4 mm(const u16x8& a, const u16x8& b, const f32x4& c) { return mfma(a, b, c); }
__device__ __forceinline__ f32x4 mm(const f32x4& a, const f32x4& b, f32x4 c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = mfma_f32(a[e], b[e], c);
    return c;
}

// of the row that `at` points into
template <int DT>
__device__ __forceinline__ typename El<DT>::Op row_op(const typename El<DT>::T* at, int g) {
    return *reinterpret_cast<const typename El<DT>::Op*>(at + El<DT>::KS / 4 * g);
}
// of column c0 + i, rows k0 ..
template <int DT>
__device__ __forceinline__ typename El<DT>::Op col_op(const typename El<DT>::T* tile, int ld, int k0, int c0, int g, int i) {
    if constexpr (DT == GDN_BF16) {
        const uint16_t* at = tile + (k0 + 8 * g + (i >> 2)) * ld + c0 + 4 * (i & 3);
        return cat(lds_column4(at), lds_column4(at + 4 * ld));
    } else {
        const float* at = tile + (k0 + 4 * g) * ld + c0 + i;
        return f32x4{at[0], at[ld], at[2 * ld], at[3 * ld]};
    }
}
// the same for 32 rows (16 in fp32) in the order in which two accumulators (one)
// hold theirs: rows 4 g .. of each 16
template <int DT>
__device__ __forceinline__ typename El<DT>::Op col_op_acc(const typename El<DT>::T* tile, int ld, int k0, int c0, int g, int i) {
    if constexpr (DT == GDN_BF16) {
        const uint16_t* at = tile + (k0 + 4 * g + (i >> 2)) * ld + c0 + 4 * (i & 3);
        return cat(lds_column4(at), lds_column4(at + 16 * ld));
    } else {
        return col_op<DT>(tile, ld, k0, c0, g, i);
    }
}

// Bytes from `base` (the same for the wave) on, as far as `bytes`; a load past them
// gives zero, without a branch.
typedef __amdgpu_buffer_rsrc_t Bytes;
__device__ __forceinline__ Bytes bytes_from(const void* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00027000);
}
__device__ __forceinline__ u32x4 ld_bytes(Bytes from, uint32_t at) {
    return __builtin_amdgcn_raw_buffer_load_b128(from, (int)at, 0, 0);
}
constexpr uint32_t kNowhere = 0xFFFFFFF0u;  // behind every buffer
// `rows` rows (none below one) of d elements of e bytes, `stride` bytes apart
__device__ __forceinline__ uint32_t rows_bytes(int rows, uint32_t stride, int d, int e) {
    return rows > 0 ? (uint32_t)(rows - 1) * stride + (uint32_t)(d * e) : 0u;
}

// No instruction moves across this.  The products below ask for a batch of
// operands from LDS and only then work on the one before it (left to itself, the
// compiler keeps few operands in few registers and waits for each), and tiles on
// their way are asked for in the order in which they are waited for, on every path
// into a loop (else its waits are for all of them).
template <int DT = GDN_BF16>
__device__ __forceinline__ void in_order() {
    // (fp32 operands take twice the registers and their products eight times as
    // long: there the compiler may order them)
    if (DT == GDN_BF16) __builtin_amdgcn_sched_barrier(0);
}

// A tile of TT tokens' rows of D features (d of them real) on its way to LDS;
// rows behind the last and features past d are zero there.
template <int DT, int D, int NT>
struct Tile {
    using T = typename El<DT>::T;
    static constexpr int TT = El<DT>::TT, LD = D + El<DT>::PAD, V = 16 / sizeof(T), PPR = D / V, ALL = TT * PPR;
    static constexpr int NP = ALL < NT ? 1 : ALL / NT;  // (fewer pieces than threads: the rest has none)
    static constexpr int kSize = TT * LD;
    static_assert(ALL < NT || (NP * NT == ALL && NT % PPR == 0), "whole rounds of whole rows");
    struct At {  // a thread's pieces
        uint32_t stride, first;
        int d;
        __device__ __forceinline__ At(int64_t elements, int d, int tid) : stride((uint32_t)(elements * sizeof(T))), d(d) {
            const int c = V * (tid % PPR);
            first = c < d && tid < ALL ? (uint32_t)(tid / PPR) * stride + (uint32_t)(c * sizeof(T)) : kNowhere;
        }
    };
    u32x4 r[NP];
    __device__ __forceinline__ void fetch(const T* from, const At& at, int rows) {
        const Bytes b = bytes_from(from, rows_bytes(min(rows, TT), at.stride, at.d, sizeof(T)));
#pragma unroll
        for (int k = 0; k < NP; ++k)
            r[k] = ld_bytes(b, at.first == kNowhere ? kNowhere : at.first + (uint32_t)k * (NT / PPR) * at.stride);
    }
    __device__ __forceinline__ void put(T* tile, int tid) const {
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            const int p = tid + NT * k;
            if (ALL < NT && p >= ALL) return;
            *reinterpret_cast<u32x4*>(tile + p / PPR * LD + V * (p % PPR)) = r[k];
        }
    }
    // Whether one of the pieces holds an infinity or a NaN: its exponent is all ones,
    // and one more carries into the sign's place
    __device__ __forceinline__ bool odd() const {
        constexpr uint32_t ones = sizeof(T) == 2 ? 0x7F807F80u : 0x7F800000u, one = sizeof(T) == 2 ? 0x00800080u : 0x00800000u;
        uint32_t x = 0;
#pragma unroll
        for (int k = 0; k < NP; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) x |= (r[k][j] & ones) + one;
        return (x & (sizeof(T) == 2 ? 0x80008000u : 0x80000000u)) != 0;
    }
    // Sets infinities and NaN of the thread's pieces in LDS to zero and the bit of their
    // row in their feature's word of `mask`
    static __device__ __forceinline__ void clear_odd(T* tile, uint32_t* mask, int tid) {
        asm volatile("" ::: "memory");  // (they were put as vectors of another type)
#pragma unroll 1
        for (int x = 0; x < NP * V; ++x) {
            const int p = tid + x / V * NT, row = p / PPR, f = V * (p % PPR) + x % V;
            if (ALL < NT && p >= ALL) return;
            T* at = tile + row * LD + f;
            uint32_t exponent;
            if constexpr (sizeof(T) == 2) exponent = (uint32_t)*at << 16;
            else exponent = __float_as_uint(*at);
            if ((exponent & 0x7F800000u) != 0x7F800000u) continue;
            *at = T(0);
            atomicOr(mask + f, 1u << row);
        }
    }
};

// ---------------------------------------------------------------------------
// what a segment adds
// ---------------------------------------------------------------------------
// M[r][c] = sum_j w_j X[j][r] Y[j][c] over a segment: to its end state (X = v,
// Y = k, w_j = a^{n-1-j}) or to the gradient of its start state (X = do, Y = q,
// w_j = scale a^{j+1}).  Y is an exact operand; w_j X[j] is an fp32 value, which
// three bf16 terms hold to the last bit (above 2^-102, where the third is no
// subnormal), so that states are as exact as fp32 arithmetic makes them.
__device__ __forceinline__ void split3(float x0, float x1, uint32_t& h, uint32_t& m, uint32_t& l) {
    auto top = [](float x) { return __uint_as_float(__float_as_uint(x) & 0xFFFF0000u); };
    auto two = [](float x, float y) { return __builtin_amdgcn_perm(__float_as_uint(y), __float_as_uint(x), 0x07060302u); };
    h = two(x0, x1);
    const float r0 = x0 - top(x0), r1 = x1 - top(x1);
    m = two(r0, r1);
    l = two(r0 - top(r0), r1 - top(r1));
}

// to(row, col, four columns' sums) takes them.
template <int DT, int DV, int DK>
constexpr int add_lds() {
    return 2 * (Tile<DT, DV, kThreads>::kSize + Tile<DT, DK, kThreads>::kSize);
}
template <int DT, int DV, int DK, class F>
__device__ __forceinline__ void add_segment(const Lin& a, const Seg& sg, int h, bool rev, typename El<DT>::T* lds, float* wt, F to) {
    using E = El<DT>;
    using T = typename E::T;
    using Op = typename E::Op;
    constexpr int TT = E::TT, KS = E::KS, RT = DV / 64, CT = DK / 16;
    using TX = Tile<DT, DV, kThreads>;
    using TY = Tile<DT, DK, kThreads>;
    const Linear& p = a.p;
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), g = (tid & 63) >> 4, i = tid & 15;
    const int dk = (int)p.dk, dv = (int)p.dv;
    const Decay decay(a, h);
    for (int j = tid; j < kSeg; j += kThreads)
        wt[j] = j >= sg.n ? 0.f : rev ? p.scale * decay(j + 1) : decay(sg.n - 1 - j);
    const int hk = h / a.group;
    const int64_t xs = rev ? (int64_t)a.Hv * dv : p.v_stride, ys = rev ? p.q_stride : p.k_stride;
    const T* x = static_cast<const T*>(rev ? a.dout : p.v) + sg.begin * xs + (int64_t)h * dv;
    const T* y = static_cast<const T*>(rev ? p.q : p.k) + sg.begin * ys + (int64_t)hk * dk;

    f32x4 acc[RT][CT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[r][c] = zero4();
    TX tx[2];
    TY ty[2];
    const typename TX::At ax(xs, dv, tid);
    const typename TY::At ay(ys, dk, tid);
    const int nt = (sg.n + TT - 1) / TT;
    auto fetch = [&](int t, int b) {
        tx[b].fetch(x + t * TT * xs, ax, sg.n - t * TT);
        ty[b].fetch(y + t * TT * ys, ay, sg.n - t * TT);
    };
    auto step = [&](int t, int b) {
        T *bx = lds + b * TX::kSize, *by = lds + 2 * TX::kSize + b * TY::kSize;
        tx[b].put(bx, tid);
        ty[b].put(by, tid);
        in_order();
        fetch(t + 2, b);
        in_order();
        __syncthreads();
#pragma unroll
        for (int k0 = 0; k0 < TT; k0 += KS) {
            const float* wk = wt + t * TT + k0 + KS / 4 * g;
            Op bt[RT][DT == GDN_BF16 ? 3 : 1];
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const Op raw = col_op<DT>(bx, TX::LD, k0, 16 * (RT * w + r), g, i);
                if constexpr (DT == GDN_BF16) {
                    uint32_t t3[3][4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        split3(wk[2 * e] * gdn_bf16_to_f32(raw[2 * e]), wk[2 * e + 1] * gdn_bf16_to_f32(raw[2 * e + 1]),
                               t3[0][e], t3[1][e], t3[2][e]);
#pragma unroll
                    for (int e = 0; e < 3; ++e) bt[r][e] = __builtin_bit_cast(u16x8, u32x4{t3[e][0], t3[e][1], t3[e][2], t3[e][3]});
                } else {
                    bt[r][0] = raw * *reinterpret_cast<const f32x4*>(wk);
                }
            }
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                const Op col = col_op<DT>(by, TY::LD, k0, 16 * c, g, i);
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int e = (DT == GDN_BF16 ? 2 : 0); e >= 0; --e) acc[r][c] = mm(col, bt[r][e], acc[r][c]);
            }
        }
    };
    // two tiles ahead
    in_order();
    fetch(0, 0);
    in_order();
    fetch(1, 1);
    in_order();
    // (a step behind the loop, not a way out of its middle: that would be taken for
    // a way back to its start, with other loads in flight)
    int t = 0;
    for (; t + 1 < nt; t += 2) {
        step(t, 0);
        step(t + 1, 1);
    }
    if (t < nt) step(t, 0);
    // the accumulator: column 4 g .. of 16 c, row i of the wave's
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            const int row = 16 * (RT * w + r) + i, col = 16 * c + 4 * g;
            if (row < dv && col < dk) to(row, col, acc[r][c]);
        }
}

// The end state of the sequence whose last segment is si: f * (the state before) +
// what the segment adds.
template <int DT, int DV, int DK>
__device__ __forceinline__ void end_state(const Lin& a, const Seg& sg, int64_t si, int h, typename El<DT>::T* lds, float* wt) {
    float* dst = end_of(a, sg.seq, h);
    if (!dst) return;
    const float* before = state_before(a, sg, si, h);
    const float f = Decay(a, h)(sg.n);
    add_segment<DT, DV, DK>(a, sg, h, false, lds, wt, [&](int row, int col, const f32x4& x) {
        const int at = row * (int)a.p.dk + col;
        st_g(dst + at, before ? f * ld_g<f32x4>(before + at) + x : x);
    });
}

// What every segment adds (blockIdx.y 1: to the gradients, the first one's only
// where that is wanted).  A sequence of one segment is done with that.  The first
// `recs` workgroups work the short sequences off beside that: chains of tokens'
// latencies, which cost 17 us in a launch of their own in a mixed batch of 16384
// tokens.
template <int DT, int DV, int DK>
__global__ __launch_bounds__(kThreads, 2) void k_lin_add(Lin a, unsigned recs) {
    __shared__ __attribute__((aligned(16))) typename El<DT>::T lds[add_lds<DT, DV, DK>()];
    __shared__ __attribute__((aligned(16))) float wt[kSeg];
    if (blockIdx.x < recs) {
        rec_sequence<DT, DK == 128 ? 32 : 16>(a, blockIdx.x, recs);
        return;
    }
    const bool rev = blockIdx.y == 1;
    const unsigned id = on_one_xcd(blockIdx.x - recs, gridDim.x - recs, a.group);
    const int64_t si = id / a.Hv;
    const int h = id - si * a.Hv;
    const Seg sg = segment(a, si);
    if (sg.n == 0) return;
    if (rev ? (sg.ends & kFirst) && !a.ds0 : (sg.ends & kLast) && (a.late || !a.p.s_out)) return;
    if (!rev && sg.ends == (kFirst | kLast)) {
        end_state<DT, DV, DK>(a, sg, si, h, lds, wt);
        return;
    }
    float* out = (rev ? a.g_seg : a.s_seg) + (si * a.Hv + h) * (int64_t)a.state;
    add_segment<DT, DV, DK>(a, sg, h, rev, lds, wt, [&](int row, int col, const f32x4& x) { st_g(out + row * (int)a.p.dk + col, x); });
}

// In place, a sequence's end state goes where the outputs of its first rows are
// read from: it waits for them (k_lin_out is in front of this).
template <int DT, int DV, int DK>
__global__ __launch_bounds__(kThreads, 2) void k_lin_end(Lin a) {
    __shared__ __attribute__((aligned(16))) typename El<DT>::T lds[add_lds<DT, DV, DK>()];
    __shared__ __attribute__((aligned(16))) float wt[kSeg];
    const unsigned id = on_one_xcd(blockIdx.x, gridDim.x, a.group);
    const int r = id / a.Hv, h = id - r * a.Hv;
    if (r >= a.count[0]) return;
    const int64_t si = (int64_t)min(a.first[r + 1], a.count[1]) - 1;
    if (si >= a.first[r]) end_state<DT, DV, DK>(a, segment(a, si), si, h, lds, wt);
}

// ---------------------------------------------------------------------------
// the states between the segments
// ---------------------------------------------------------------------------
// S <- a^n S + (what the segment adds), element by element, each segment's place
// holding the state behind it afterwards.  AHEAD segments' pieces are in flight
// (long_chains).
template <int AHEAD, bool BACK, class F>
__device__ __forceinline__ void scan_places(const float* from, int64_t stride, int count, F step) {
    f32x4 x[AHEAD], y[AHEAD];
    auto fetch = [&](f32x4 (&r)[AHEAD], int g0) {
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int g = BACK ? count - 1 - (g0 + u) : g0 + u;
            if (g0 + u < count) r[u] = ld_g<f32x4>(from + g * stride);
        }
    };
    fetch(x, 0);
    for (int g0 = 0; g0 < count; g0 += AHEAD) {
        if (g0 + AHEAD < count) fetch(y, g0 + AHEAD);
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (g0 + u < count) step(BACK ? count - 1 - (g0 + u) : g0 + u, x[u]);
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) x[u] = y[u];
    }
}

struct ScanAt {
    int r, h, s, f, G, e;
    Span sp;
    bool on;
};
__device__ __forceinline__ ScanAt scan_at(const Lin& a, int tid) {
    ScanAt x{};
    const unsigned per = ((unsigned)a.state + 4 * kThreads - 1) / (4 * kThreads), id = blockIdx.x / per;
    x.e = 4 * (kThreads * (blockIdx.x - id * per) + tid);
    x.r = id / a.Hv;
    x.h = id - x.r * a.Hv;
    x.on = x.r < a.count[0] && x.e < a.state;
    if (x.r < a.count[0]) {
        x.s = a.seqs[x.r];
        x.sp = span_of(a.at, x.s);
        x.f = min(a.first[x.r], a.count[1]);
        x.G = min(a.first[x.r + 1], a.count[1]) - x.f;
    }
    return x;
}

template <int AHEAD>
__global__ __launch_bounds__(kThreads) void k_lin_scan(Lin a) {
    const ScanAt x = scan_at(a, threadIdx.x);
    if (!x.on || x.G < 2) return;
    const float* src = start_of(a, x.s, x.h);
    float* dst = a.late ? nullptr : end_of(a, x.s, x.h);
    f32x4 S = src ? ld_g<f32x4>(src + x.e) : zero4();
    const Decay decay(a, x.h);
    const float whole = decay(kSeg), rest = decay((int)(x.sp.n - (int64_t)(x.G - 1) * kSeg));
    const int64_t stride = (int64_t)a.Hv * a.state;
    float* at = a.s_seg + ((int64_t)x.f * a.Hv + x.h) * a.state + x.e;
    scan_places<AHEAD, false>(at, stride, dst ? x.G : x.G - 1, [&](int g, const f32x4& add) {
        S = (g == x.G - 1 ? rest : whole) * S + add;
        if (g == x.G - 1) st_g(dst + x.e, S);
        else st_g(at + g * stride, S);
    });
}

// The workgroup's sum of x, in a fixed order, written by one thread.
template <int NT>
__device__ __forceinline__ void sum_to(float x, float* sums, float* to, int tid) {
    x = xor32_sum(row_sum<32>(x));
    if ((tid & 63) == 0) sums[tid >> 6] = x;
    __syncthreads();
    if (tid == 0) {
        x = 0.f;
        for (int i = 0; i < NT / 64; ++i) x += sums[i];
        *to = x;
    }
    __syncthreads();
}

// Backward: the states behind the segments, then the gradients behind them, and
// n a^{n-1} <G, S> of each for dalpha.
template <int AHEAD>
__global__ __launch_bounds__(kThreads) void k_lin_bscan(Lin a) {
    __shared__ float sums[kThreads / 64];
    const int tid = threadIdx.x;
    const ScanAt x = scan_at(a, tid);
    float da = 0.f;
    if (x.on) {
        const Decay decay(a, x.h);
        const int n_last = (int)(x.sp.n - (int64_t)(x.G - 1) * kSeg);
        const float whole = decay(kSeg), rest = x.G > 0 ? decay(n_last) : 1.f;
        const int64_t stride = (int64_t)a.Hv * a.state, off = ((int64_t)x.f * a.Hv + x.h) * a.state + x.e;
        const float* src = start_of(a, x.s, x.h);
        const f32x4 S0 = src ? ld_g<f32x4>(src + x.e) : zero4();
        f32x4 S = S0;
        float* at = a.s_seg + off;
        scan_places<AHEAD, false>(at, stride, x.G - 1, [&](int g, const f32x4& add) {
            S = whole * S + add;
            st_g(at + g * stride, S);
        });
        const int64_t own = ((int64_t)x.s * a.Hv + x.h) * a.state + x.e;
        f32x4 G = a.ds_out ? ld_g<f32x4>(a.ds_out + own) : zero4();
        float* ga = a.g_seg + off;
        // (without a gradient of the start state the first segment adds nothing)
        const int lowest = a.ds0 ? 0 : 1;
        const float dw = (float)kSeg * decay(kSeg - 1), dr = (float)n_last * decay(n_last - 1);
        scan_places<AHEAD, true>(ga + lowest * stride, stride, x.G - lowest, [&](int g, const f32x4& add) {
            g += lowest;
            if (a.dalpha) {
                const f32x4 from = g > 0 ? ld_g<f32x4>(at + (g - 1) * stride) : S0;
                da += (g == x.G - 1 ? dr : dw) * dot4e(G, from);
            }
            G = (g == x.G - 1 ? rest : whole) * G + add;
            st_g(ga + g * stride, G);
        });
        if (a.dalpha && lowest > 0 && x.G > 0) da += (x.G == 1 ? dr : dw) * dot4e(G, S0);
        if (a.ds0) st_g(a.ds0 + own, G);
    }
    if (a.dalpha) {
        const unsigned per = ((unsigned)a.state + 4 * kThreads - 1) / (4 * kThreads), id = blockIdx.x / per;
        const int64_t r = id / a.Hv, h = id - r * a.Hv;
        sum_to<kThreads>(da, sums, a.part + h * a.parts + a.part_scan + r * per + (blockIdx.x - id * per), tid);
    }
}

// dalpha of a head (the first `heads` workgroups) and, where they were made in
// parts, dk and dq: their addends in a fixed order
__device__ __forceinline__ void join_parts(const Lin& a, int64_t at) {
    const Linear& p = a.p;
    const int64_t row = p.Hk * p.dk, all = p.N * row;
    const int which = 4 * at >= all;
    const int64_t e = 4 * at - which * all, t = e / row;
    // (rows outside every sequence are zero already)
    if (e >= all || t < cu_at(a.at, 0) || t >= cu_at(a.at, p.S)) return;
    const float* from = a.split + which * a.splits * all + e;
    f32x4 x = ld_g<f32x4>(from);
#pragma unroll 4
    for (int z = 1; z < a.splits; ++z) x += ld_g<f32x4>(from + z * all);
    void* to = which ? a.dq : a.dk;
    if (p.dtype == GDN_BF16) st_g(static_cast<uint16_t*>(to) + e, u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])});
    else st_g(static_cast<float*>(to) + e, x);
}
__global__ __launch_bounds__(1024) void k_lin_join(Lin a, unsigned heads) {
    __shared__ double sums[1024];
    const int tid = threadIdx.x;
    if (blockIdx.x >= heads) {
        join_parts(a, (int64_t)(blockIdx.x - heads) * 1024 + tid);
        return;
    }
    const float* part = a.part + (int64_t)blockIdx.x * a.parts;
    double s = 0.;
    for (int64_t i = tid; i < a.parts; i += 1024) s += (double)part[i];
    sums[tid] = s;
    for (int o = 512; o > 0; o >>= 1) {
        __syncthreads();
        if (tid < o) sums[tid] += sums[tid + o];
    }
    if (tid == 0) a.dalpha[blockIdx.x] = (float)sums[0];
}

// ---------------------------------------------------------------------------
// rows of the results
// ---------------------------------------------------------------------------
// All of them have one form: row i of a segment is
//   Y_i = sum_j a^{|i-j|} (X_i.A_j) B_j + a^{e_i} M X_i
// over the tokens j up to i (o: X = q, A = k, B = v, M = S; dq: do, v, k, S^T) or
// from i on (dv: k, q, do, G; dk: v, do, q, G^T).  A wave has 16 IT rows, one a
// lane i; scores are formed as (keys x rows), so that an accumulator's four
// values belong to four keys of the lane's row and serve, weighted and split into
// two bf16 terms, as the right operand of the product with B as they stand; Y
// is accumulated as (features x rows).
//
// Weights: with blocks of 16 rows and 16 keys D > 0 blocks apart, |i - j| - 1 is a
// lane's constant (up to i: i in its block; from i on: 15 - i) plus an exponent
// that a table holds for each D and place of the key; no exponent is negative,
// so nothing overflows.  In the block itself the four powers of a lane are
// constants, zero on the other side.
template <bool REV>
struct Weights {
    float ul, rl;   // the row's factor, without and with one more a
    f32x4 dw, du;   // in the block itself: a^d, and d a^(d-1) for dalpha
    const float* tab;
    __device__ __forceinline__ void set(const Decay& decay, float scale, const float* table, int g, int i) {
        ul = scale * decay(REV ? 15 - i : i);
        rl = decay.a * ul;
        tab = table;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int d = REV ? 4 * g + e - i : i - 4 * g - e;
            dw[e] = d >= 0 ? scale * decay(d) : 0.f;
            du[e] = d > 0 ? scale * (float)d * decay(d - 1) : 0.f;
        }
    }
    static __device__ __forceinline__ void fill(const Decay& decay, float* table, int n, int tid, int threads) {
        for (int x = tid; x < n; x += threads) table[x] = decay(REV ? x : x + 15 - 2 * (x & 15));
    }
    __device__ __forceinline__ bool seen(int g, int i, int e) const { return REV ? 4 * g + e >= i : i >= 4 * g + e; }
    // factors of the scores of a block of keys D blocks from the rows'
    __device__ __forceinline__ f32x4 factors(int D, int g) const {
        return D > 0 ? rl * *reinterpret_cast<const f32x4*>(tab + 16 * (D - 1) + 4 * g) : dw;
    }
    // the scores p times them; zero on the other side, whatever p is
    __device__ __forceinline__ f32x4 weighted(const f32x4& p, const f32x4& f, int D, int g, int i) const {
        f32x4 y = p * f;
        if (D <= 0)
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = D == 0 && seen(g, i, e) ? y[e] : 0.f;
        return y;
    }
    // their derivatives with respect to a
    __device__ __forceinline__ f32x4 slope(int D, int g, int i) const {
        if (D < 0) return zero4();
        if (D == 0) return du;
        const f32x4 u = ul * *reinterpret_cast<const f32x4*>(tab + 16 * (D - 1) + 4 * g);
        f32x4 y;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = u[e] * (float)(REV ? 16 * D + 4 * g + e - i : 16 * D + i - 4 * g - e);
        return y;
    }
};

// A wave's 16 IT rows as right operands, straight from memory (zero behind the
// last); from: the wave's first row, rows: as many as there are from it on
template <int DT, int D, int IT>
__device__ __forceinline__ void load_rows(typename El<DT>::Op (&x)[IT][D / El<DT>::KS], const typename El<DT>::T* from,
                                          int64_t stride, int rows, int d, int g, int i) {
    using Op = typename El<DT>::Op;
    constexpr int KS = El<DT>::KS, e = sizeof(typename El<DT>::T);
    const uint32_t sb = (uint32_t)(stride * e);
    const Bytes b = bytes_from(from, rows_bytes(min(rows, 16 * IT), sb, d, e));
#pragma unroll
    for (int it = 0; it < IT; ++it)
#pragma unroll
        for (int k = 0; k < D / KS; ++k) {
            const int c = KS * k + KS / 4 * g;
            x[it][k] = __builtin_bit_cast(Op, ld_bytes(b, c < d ? (uint32_t)(16 * it + i) * sb + (uint32_t)(c * e) : kNowhere));
        }
}

// Four features from c on of a wave's row i, from a buffer of its rows
template <int DT>
__device__ __forceinline__ R4<DT> row_piece(Bytes rows, uint32_t stride, int i, int c) {
    if constexpr (DT == GDN_BF16)
        return __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rows, (int)((uint32_t)i * stride + 2u * c), 0, 0));
    else
        return __builtin_bit_cast(f32x4, ld_bytes(rows, (uint32_t)i * stride + 4u * c));
}

// p[jt]: scores of the tile's 32 keys and the wave's rows
template <int DT, int D>
struct ScoreOps {
    using Op = typename El<DT>::Op;
    static constexpr int KS = El<DT>::KS, LD = D + El<DT>::PAD, N = D / KS;
    Op op[2][N];
    __device__ __forceinline__ void load(const typename El<DT>::T* tile, int g, int i) {
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int jt = 0; jt < 2; ++jt) op[jt][k] = row_op<DT>(tile + (16 * jt + i) * LD + KS * k, g);
    }
    __device__ __forceinline__ void times(f32x4 (&p)[2], const Op (&x)[N]) const {
        p[0] = p[1] = zero4();
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int jt = 0; jt < 2; ++jt) p[jt] = mm(op[jt][k], x[k], p[jt]);
    }
};
// acc[mt] += (columns 16 mt .. of the tile's 32 rows) p, B columns' blocks a batch
template <int DT, int D>
struct ColumnOps {
    using Op = typename El<DT>::Op;
    static constexpr int LD = D + El<DT>::PAD, PER = DT == GDN_BF16 ? 1 : 2, B = 4 / PER, N = D / 16 / B;
    Op op[B][PER];
    __device__ __forceinline__ void load(const typename El<DT>::T* tile, int n, int g, int i) {
#pragma unroll
        for (int m = 0; m < B; ++m)
#pragma unroll
            for (int j = 0; j < PER; ++j) op[m][j] = col_op_acc<DT>(tile, LD, 16 * j, 16 * (n * B + m), g, i);
    }
};
template <int DT, int D, int IT>
__device__ __forceinline__ void gather(f32x4 (&acc)[IT][D / 16], const f32x4 (&p)[IT][2], ColumnOps<DT, D>& first,
                                       const typename El<DT>::T* tile, int g, int i) {
    using C = ColumnOps<DT, D>;
    typename El<DT>::Op t[IT][2];  // the terms (bf16), the two blocks (fp32)
#pragma unroll
    for (int it = 0; it < IT; ++it) {
        if constexpr (DT == GDN_BF16) {
            u16x4 h0, l0, h1, l1;
            split4(p[it][0], h0, l0);
            split4(p[it][1], h1, l1);
            t[it][0] = cat(l0, l1);
            t[it][1] = cat(h0, h1);
        } else {
            t[it][0] = p[it][0];
            t[it][1] = p[it][1];
        }
    }
    C next;
#pragma unroll
    for (int n = 0; n < C::N; ++n) {
        C &now = n & 1 ? next : first, &then = n & 1 ? first : next;
        if (n + 1 < C::N) then.load(tile, n + 1, g, i);
        in_order<DT>();
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int m = 0; m < C::B; ++m)
#pragma unroll
                for (int it = 0; it < IT; ++it)
                    acc[it][n * C::B + m] = mm(now.op[m][e % C::PER], t[it][e], acc[it][n * C::B + m]);
        in_order<DT>();
    }
}

// As split4, each element's terms formed from itself alone: there an infinity or a
// NaN makes its neighbour's low term a NaN too.
__device__ __forceinline__ void split4_apart(const f32x4& x, u16x4& hi, u16x4& lo) {
    auto low = [](uint32_t h, float a, float b) {
        return pack_bf16(a - __uint_as_float(h << 16), b - __uint_as_float(h & 0xFFFF0000u));
    };
    const uint32_t h0 = pack_bf16(x[0], x[1]), h1 = pack_bf16(x[2], x[3]);
    hi = __builtin_bit_cast(u16x4, u32x2{h0, h1});
    lo = __builtin_bit_cast(u16x4, u32x2{low(h0, x[0], x[1]), low(h1, x[2], x[3])});
}

// 32 rows (TR: columns) of a state [dv][dk] on their way to LDS, where they lie
// split into terms, and their products with a wave's rows.
template <int DT, int DV, int DK, bool TR, int NT, int TERMS>
struct Slab {
    using T = typename El<DT>::T;
    using Op = typename El<DT>::Op;
    static constexpr int DX = TR ? DV : DK;  // what is contracted
    static constexpr int W = TR ? 32 : DK, LD = TR ? 36 : DK + El<DT>::PAD, ROWS = TR ? DV : 32, LO = ROWS * LD;
    static constexpr int kSize = TERMS * LO, NP = 8 * DX / NT;
    f32x4 r[NP];
    __device__ __forceinline__ void fetch(const float* M, int m0, int dv, int dk, int tid) {
        const Bytes b = bytes_from(M, (uint32_t)(dv * dk * 4));
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            const int p = tid + NT * k, row = p / (W / 4) + (TR ? 0 : m0), c = 4 * (p % (W / 4)) + (TR ? m0 : 0);
            r[k] = __builtin_bit_cast(f32x4, ld_bytes(b, c < dk ? (uint32_t)(row * dk + c) * 4u : kNowhere));
        }
    }
    __device__ __forceinline__ void put(T* slab, int tid) const {
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            const int p = tid + NT * k;
            T* to = slab + p / (W / 4) * LD + 4 * (p % (W / 4));
            if constexpr (TERMS == 3) {
                u32x2 t[3];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint32_t h, m, l;
                    split3(r[k][2 * e], r[k][2 * e + 1], h, m, l);
                    t[0][e] = h, t[1][e] = m, t[2][e] = l;
                }
#pragma unroll
                for (int e = 0; e < 3; ++e) *reinterpret_cast<u32x2*>(to + e * LO) = t[e];
            } else if constexpr (TERMS == 2) {
                u16x4 hi, lo;
                if (TR) split4_apart(r[k], hi, lo);  // (neighbours are features of two results)
                else split4(r[k], hi, lo);  // (of one sum)
                *reinterpret_cast<u16x4*>(to) = hi;
                *reinterpret_cast<u16x4*>(to + LO) = lo;
            } else {
                *reinterpret_cast<f32x4*>(to) = r[k];
            }
        }
    }
};
// Rows (TR: columns) 16 m .. of a state that lies in LDS in terms LO elements
// apart, LD elements a row, as operands; K of them contract all features.
template <int DT, int D, bool TR, int LD, int LO, int TERMS>
struct StateOps {
    using Op = typename El<DT>::Op;
    static constexpr int KS = El<DT>::KS, K = D / KS;
    Op op[K][TERMS];
    __device__ __forceinline__ void load(const typename El<DT>::T* at, int m, int g, int i) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < TERMS; ++e)
                op[k][e] = TR ? col_op<DT>(at + e * LO, LD, KS * k, 16 * m, g, i)
                              : row_op<DT>(at + e * LO + (16 * m + i) * LD + KS * k, g);
    }
    __device__ __forceinline__ f32x4 times(const Op (&x)[K]) const {
        f32x4 t[TERMS];
#pragma unroll
        for (int e = 0; e < TERMS; ++e) t[e] = zero4();
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < TERMS; ++e) t[e] = mm(op[k][e], x[k], t[e]);
#pragma unroll
        for (int e = TERMS - 1; e > 0; --e) t[e - 1] += t[e];
        return t[0];
    }
};

// Four features of a row, rounded once
template <int DT>
__device__ __forceinline__ void st4(typename El<DT>::T* to, const f32x4& x) {
    if constexpr (DT == GDN_BF16) st_g(to, u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])});
    else st_g(to, x);
}

// The gradient of the state behind segment si, or null (zero)
__device__ __forceinline__ const float* gradient_behind(const Lin& a, const Seg& sg, int64_t si, int h) {
    if (!(sg.ends & kLast)) return a.g_seg + ((si + 1) * a.Hv + h) * (int64_t)a.state;
    return a.ds_out ? a.ds_out + ((int64_t)sg.seq * a.Hv + h) * a.state : nullptr;
}

// The four results and what they are made of
enum Kind { kOut, kDq, kDk, kDv };
template <int KIND>
struct Made {
    static constexpr bool REV = KIND == kDk || KIND == kDv;  // over the tokens from i on
    static constexpr bool TR = KIND == kDq || KIND == kDk;   // the state's transpose
    static constexpr bool SUM = TR;                          // of a key head, over its value heads
};
struct Rows {  // an array's rows, one behind the other by token
    const void* at;
    int64_t stride;
    bool key;  // heads are key heads
};
template <int KIND>
__device__ __forceinline__ void made_of(const Lin& a, Rows& x, Rows& left, Rows& right) {
    const Linear& p = a.p;
    const Rows q{p.q, p.q_stride, true}, k{p.k, p.k_stride, true}, v{p.v, p.v_stride, false},
        o{a.dout, (int64_t)a.Hv * p.dv, false};
    x = KIND == kOut ? q : KIND == kDq ? o : KIND == kDk ? v : k;
    left = KIND == kOut ? k : KIND == kDq ? v : KIND == kDk ? o : q;
    right = KIND == kOut ? v : KIND == kDq ? k : KIND == kDk ? q : o;
}

// x, not known to be what it was: what a loop's body derives from it is formed
// anew in every round and holds no registers across it.
__device__ __forceinline__ int anew(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

// A workgroup has 128 rows of a head (fp32: 64); dq's and dk's are a key head's,
// its value heads one after the other in one sum.  Four waves of 32 rows (fp32: 16)
// read each operand from LDS for twice as many products as eight of 16: gradients
// of a training step 430 instead of 615 us (heads of 128; the loop over value heads
// takes registers: the four waves spill 27 of 256, the eight more of their 128, so
// that this says nothing of eight waves without the loop), outputs with values of 64
// 68 instead of 76 us.  Outputs with values of 128 are made by eight, whose registers
// let sixteen waves share a compute unit (best times: one sequence of 65531 84 instead
// of 88 us, a mixed batch 86 instead of 88).  With 256 rows a workgroup, tiles are
// read once but waves wait for the last rows' (94 instead of 92, 100 instead of 88).
template <int DT>
struct Shape {
    static constexpr int NT = 256, IT = DT == GDN_BF16 ? 2 : 1, ROWS = NT / 4 * IT, WAVES = 2;
};
template <int DT, int DV>
struct OutShape {
    static constexpr int IT = DV > 64 ? 1 : Shape<DT>::IT, NT = 4 * Shape<DT>::ROWS / IT, WAVES = NT / 128;
};
// Terms of the states.  Rows of bf16 results are far from seeing an error of
// 2^-17; dalpha, an fp32 sum over all tokens, is not (two terms left it 1e-6 to 9e-6
// off on inputs where three leave 1e-8 to 4e-7; where terms of both signs nearly
// cancel, three leave up to 2e-6, as fp32 sums do), and three hold an fp32 state
// exactly (above 2^-102).
template <int DT, bool SLOPES>
constexpr int state_terms() {
    return DT == GDN_BF16 && SLOPES ? 3 : El<DT>::TERMS;
}
template <int DT, int DK, int DV, bool SLOPES>
constexpr int rows_lds() {
    constexpr int tiles = 2 * (Tile<DT, DK, kThreads>::kSize + Tile<DT, DV, kThreads>::kSize), TERMS = state_terms<DT, SLOPES>();
    return std::max(tiles, 2 * std::max(Slab<DT, DV, DK, false, kThreads, TERMS>::kSize, Slab<DT, DV, DK, true, kThreads, TERMS>::kSize));
}
// The tiles of keys that a workgroup's own rows lie in are seen in part: the keys
// behind a row (REV: in front of it) have a weight of zero, and zero times an infinity
// or a NaN would be a NaN in a row that does not see it.  What is not finite in B is
// set to zero in these tiles (PARTS of them) and noted, and behind the last tile the
// rows that see it are made NaN in its feature.  Looking for it costs 1 to 3 % of a
// call (one of 65531 tokens 2, a training step of 16384 1.5, prompts with heads of 64 3).
template <int PARTS>
struct Odd {
    int found;
    uint32_t mask[PARTS][128];  // of each feature, the tile's rows
    template <int NT>
    __device__ __forceinline__ void clear(int tid) {
        if (tid == 0) found = 0;
        for (int x = tid; x < PARTS * 128; x += NT) (&mask[0][0])[x] = 0;
    }
};
template <int DT, int DK, int DV, int NT, int IT, int KIND, bool SLOPES>
__device__ __forceinline__ void rows_of(const Lin& a, unsigned block, unsigned blocks, typename El<DT>::T* lds, float* tab,
                                        Odd<Shape<DT>::ROWS / El<DT>::TT>& odd, float* sums) {
    using E = El<DT>;
    using T = typename E::T;
    using Op = typename E::Op;
    constexpr bool REV = Made<KIND>::REV, TR = Made<KIND>::TR, SUM = Made<KIND>::SUM;
    constexpr int DX = TR ? DV : DK, DM = TR ? DK : DV, TT = E::TT, kBlockRows = NT / 4 * IT, PARTS = kBlockRows / TT;
    using TA = Tile<DT, DX, NT>;
    using TB = Tile<DT, DM, NT>;
    constexpr int TERMS = state_terms<DT, SLOPES>();
    using SL = Slab<DT, DV, DK, TR, NT, TERMS>;
    using SO = StateOps<DT, DX, TR, SL::LD, SL::LO, TERMS>;
    const Linear& p = a.p;
    const int heads = SUM ? (int)p.Hk : a.Hv, nh = SUM ? a.group : 1, splits = SUM ? a.splits : 1;
    constexpr unsigned nrb = kSeg / kBlockRows;
    const unsigned b = on_one_xcd(block, blocks, nrb * (SUM ? splits : a.group)), id0 = b / nrb, id = id0 / splits;
    const int rb = b - id0 * nrb, hh = id % heads, z = id0 - id * splits;
    const int from = z * nh / splits, to = (z + 1) * nh / splits;  // of the value heads
    const int64_t si = id / heads;
    const int thread = threadIdx.x, w = __builtin_amdgcn_readfirstlane(thread >> 6);
    const Seg sg = segment(a, si);
    float* part = SLOPES ? a.part + (int64_t)hh * nh * a.parts + (KIND == kDv ? a.part_dv : 0) + si * nrb + rb : nullptr;
    if (rb * kBlockRows >= sg.n) {
        for (int j = from + thread; SLOPES && j < to; j += NT) part[j * a.parts] = 0.f;
        return;
    }
    const int dk = (int)p.dk, dv = (int)p.dv, dx = TR ? dv : dk, dm = TR ? dk : dv;
    Rows X, A, B;
    made_of<KIND>(a, X, A, B);
    const int row0 = rb * kBlockRows + 16 * IT * w, rblk = row0 / 16;
    // tiles of keys
    const int first = REV ? rb * kBlockRows / TT : 0, nkeys = REV ? sg.n : min(sg.n, (rb + 1) * kBlockRows),
              nt = (nkeys + TT - 1) / TT;

    f32x4 acc[IT][DM / 16];
#pragma unroll
    for (int it = 0; it < IT; ++it)
#pragma unroll
        for (int mt = 0; mt < DM / 16; ++mt) acc[it][mt] = zero4();
    odd.template clear<NT>(thread);  // (the barrier in front of the first tile is behind this)
    for (int j = from; j < to; ++j) {
        const int tid = SUM ? anew(thread) : thread, g = (tid & 63) >> 4, i = tid & 15;
        const int h = hh * nh + j, hk = SUM ? hh : hh / a.group;
        const T* xp = static_cast<const T*>(X.at) + (sg.begin + row0) * X.stride + (int64_t)(X.key ? hk : h) * dx;
        const T* ap = static_cast<const T*>(A.at) + sg.begin * A.stride + (int64_t)(A.key ? hk : h) * dx;
        const T* bp = static_cast<const T*>(B.at) + sg.begin * B.stride + (int64_t)(B.key ? hk : h) * dm;
        const float* M = REV ? gradient_behind(a, sg, si, h) : state_before(a, sg, si, h);
        SL sl;
        if (M) sl.fetch(M, 0, dv, dk, tid);
        Op x[IT][DX / E::KS];
        load_rows<DT, DX, IT>(x, xp, X.stride, sg.n - row0, dx, g, i);
        const Decay decay(a, h);
        if (j > from) __syncthreads();
        Weights<REV>::fill(decay, tab, kSeg, tid, NT);
        Weights<REV> weight;
        weight.set(decay, p.scale, tab, g, i);
        float da = 0.f;
        const typename TA::At aa(A.stride, dx, tid);
        const typename TB::At ab(B.stride, dm, tid);
        TA ta[2];
        TB tb[2];
        auto fetch = [&](int t, int b) {
            in_order();
            ta[b].fetch(ap + t * TT * A.stride, aa, nkeys - t * TT);
            tb[b].fetch(bp + t * TT * B.stride, ab, nkeys - t * TT);
            in_order();
        };
        if (M) {
            float f[IT], df[IT];
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const int row = row0 + 16 * it + i, e = REV ? sg.n - 1 - row : row + 1;  // (below zero: no row)
                const float scale = REV ? 1.f : p.scale;
                f[it] = e >= 0 ? scale * decay(e) : 0.f;
                df[it] = e > 0 ? scale * (float)e * decay(e - 1) : 0.f;
            }
            // rows that the product is multiplied with for dalpha: q, v
            const Rows W = KIND == kDq ? Rows{p.q, p.q_stride, true} : Rows{p.v, p.v_stride, false};
            const uint32_t ws = (uint32_t)(W.stride * sizeof(T));
            const Bytes wb = bytes_from(static_cast<const T*>(W.at) + (sg.begin + row0) * W.stride + (int64_t)(W.key ? hk : h) * dm,
                                        rows_bytes(min(sg.n - row0, 16 * IT), ws, dm, sizeof(T)));
#pragma unroll
            for (int s = 0; s < DM / 32; ++s) {
                if (32 * s >= dm) break;
                T* slab = lds + (s & 1) * SL::kSize;
                sl.put(slab, tid);
                if (s + 1 < DM / 32) sl.fetch(M, 32 * (s + 1), dv, dk, tid);
                R4<DT> wr[SLOPES ? 2 : 1][SLOPES ? IT : 1];
                if constexpr (SLOPES)
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int it = 0; it < IT; ++it) wr[m][it] = row_piece<DT>(wb, ws, 16 * it + i, 32 * s + 16 * m + 4 * g);
                in_order();
                __syncthreads();
                SO so;
                so.load(slab, 0, g, i);
                in_order<DT>();
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    f32x4 t[IT];
#pragma unroll
                    for (int it = 0; it < IT; ++it) t[it] = so.times(x[it]);
                    if (m == 0) so.load(slab, 1, g, i);
                    in_order<DT>();
#pragma unroll
                    for (int it = 0; it < IT; ++it) {
                        acc[it][2 * s + m] += f[it] * t[it];
                        if constexpr (SLOPES && (KIND == kDq || KIND == kDv))
                            if (32 * s + 16 * m < dm) da += df[it] * dot4e(t[it], cvt<DT>(wr[m][it]));
                    }
                }
                in_order<DT>();
            }
        }
        __syncthreads();
        fetch(first, 0);
        fetch(first + 1, 1);
        auto step = [&](int t, int b) {
            T *ba = lds + b * TA::kSize, *bb = lds + 2 * TA::kSize + b * TB::kSize;
            ta[b].put(ba, tid);
            tb[b].put(bb, tid);
            const unsigned part = t - rb * kBlockRows / TT;
            if (__builtin_expect(part < PARTS && tb[b].odd(), 0)) {
                odd.found = 1;
                TB::clear_odd(bb, odd.mask[part], anew(tid));
            }
            fetch(t + 2, b);
            __syncthreads();
            const int kblk = t * TT / 16;
            if (REV ? kblk + 1 < rblk : kblk > rblk + IT - 1) return;
            auto between = [&](int it, int jt) { return REV ? kblk + jt - rblk - it : rblk + it - kblk - jt; };
            ScoreOps<DT, DX> ops;
            ops.load(ba, g, i);
            in_order<DT>();
            f32x4 s[IT][2];
#pragma unroll
            for (int it = 0; it < IT; ++it) ops.times(s[it], x[it]);
            ColumnOps<DT, DM> cols;
            cols.load(bb, 0, g, i);
            in_order<DT>();
#pragma unroll
            for (int it = 0; it < IT; ++it)
#pragma unroll
                for (int jt = 0; jt < 2; ++jt)
                    s[it][jt] = weight.weighted(s[it][jt], weight.factors(between(it, jt), g), between(it, jt), g, i);
            gather<DT, DM, IT>(acc, s, cols, bb, g, i);
        };
        int t = first;
        for (; t + 1 < nt; t += 2) {
            step(t, 0);
            step(t + 1, 1);
        }
        if (t < nt) step(t, 0);
        if (__builtin_expect(odd.found, 0)) {
            const int own = anew(tid), g = (own & 63) >> 4, i = own & 15;
#pragma unroll
            for (int it = 0; it < IT; ++it)
#pragma unroll 1
                for (int part = 0; part < PARTS; ++part) {
                    const int x = 16 * (rblk + it) - (rb * kBlockRows + part * TT) + i;  // the row's own place in the tile
                    const uint32_t see = REV ? (x > 31 ? 0u : ~0u << max(x, 0)) : (x < 0 ? 0u : ~0u >> (31 - min(x, 31)));
#pragma unroll
                    for (int mt = 0; mt < DM / 16; ++mt) {
                        in_order();  // (few registers)
                        const uint32_t* m = odd.mask[part] + 16 * mt + 4 * g;
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[it][mt][e] = m[e] & see ? __builtin_nanf("") : acc[it][mt][e];
                    }
                }
            if (j + 1 < to) {
                __syncthreads();
                odd.template clear<NT>(own);
            }
        }
        if constexpr (SLOPES) sum_to<NT>(da, sums, part + j * a.parts, tid);
    }
    T* out = static_cast<T*>(KIND == kOut ? p.out : KIND == kDq ? a.dq : KIND == kDk ? a.dk : a.dv) + (int64_t)hh * dm;
    const int64_t os = (int64_t)heads * dm;
    const int g = (thread & 63) >> 4;
    if (SUM && splits > 1) {
        float* sum = a.split + ((int64_t)(KIND == kDq ? splits : 0) + z) * p.N * os + (int64_t)hh * dm;
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            const int row = row0 + 16 * it + (thread & 15);
            if (row < sg.n)
#pragma unroll
                for (int mt = 0; mt < DM / 16; ++mt)
                    if (16 * mt < dm) st_g(sum + (sg.begin + row) * os + 16 * mt + 4 * g, acc[it][mt]);
        }
        return;
    }
#pragma unroll
    for (int it = 0; it < IT; ++it) {
        const int row = row0 + 16 * it + (thread & 15);
        if (row < sg.n)
#pragma unroll
            for (int mt = 0; mt < DM / 16; ++mt)
                if (16 * mt < dm) st4<DT>(out + (sg.begin + row) * os + 16 * mt + 4 * g, acc[it][mt]);
    }
}

template <int DT, int DK, int DV>
__global__ __launch_bounds__((OutShape<DT, DV>::NT), (DK + DV > 128 ? OutShape<DT, DV>::WAVES : 4)) void k_lin_out(Lin a) {
    __shared__ __attribute__((aligned(16))) typename El<DT>::T lds[rows_lds<DT, DK, DV, false>()];
    __shared__ __attribute__((aligned(16))) float tab[kSeg];
    __shared__ Odd<Shape<DT>::ROWS / El<DT>::TT> odd;
    rows_of<DT, DK, DV, OutShape<DT, DV>::NT, OutShape<DT, DV>::IT, kOut, false>(a, blockIdx.x, gridDim.x, lds, tab, odd, nullptr);
}
// dalpha's pairs of tokens: sum over i > j of (i - j) a^(i-j-1) (q_i.k_j)
// (do_i.v_j), rows j of a value head, both kinds of scores at once.
template <int DT, int DK, int DV, int NT, int IT>
__device__ __forceinline__ void slopes_of(const Lin& a, unsigned block, unsigned blocks, typename El<DT>::T* lds, float* tab,
                                          float* sums) {
    using E = El<DT>;
    using T = typename E::T;
    using Op = typename E::Op;
    constexpr int TT = E::TT, kBlockRows = NT / 4 * IT;
    using TQ = Tile<DT, DK, NT>;
    using TO = Tile<DT, DV, NT>;
    const Linear& p = a.p;
    constexpr unsigned nrb = kSeg / kBlockRows;
    const unsigned b = on_one_xcd(block, blocks, nrb * a.group), id = b / nrb;
    const int rb = b - id * nrb, h = id % a.Hv, hk = h / a.group;
    const int64_t si = id / a.Hv;
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), g = (tid & 63) >> 4, i = tid & 15;
    const Seg sg = segment(a, si);
    float* part = a.part + (int64_t)h * a.parts + a.part_pairs + si * nrb + rb;
    if (rb * kBlockRows >= sg.n) {
        if (tid == 0) *part = 0.f;
        return;
    }
    const int dk = (int)p.dk, dv = (int)p.dv;
    const int64_t os = (int64_t)a.Hv * dv;
    const int row0 = rb * kBlockRows + 16 * IT * w, rblk = row0 / 16;
    const int first = rb * kBlockRows / TT, nt = (sg.n + TT - 1) / TT;
    const T* qp = static_cast<const T*>(p.q) + sg.begin * p.q_stride + (int64_t)hk * dk;
    const T* op = static_cast<const T*>(a.dout) + sg.begin * os + (int64_t)h * dv;
    Op xk[IT][DK / E::KS], xv[IT][DV / E::KS];
    load_rows<DT, DK, IT>(xk, static_cast<const T*>(p.k) + (sg.begin + row0) * p.k_stride + (int64_t)hk * dk, p.k_stride,
                          sg.n - row0, dk, g, i);
    load_rows<DT, DV, IT>(xv, static_cast<const T*>(p.v) + (sg.begin + row0) * p.v_stride + (int64_t)h * dv, p.v_stride,
                          sg.n - row0, dv, g, i);
    const typename TQ::At aq(p.q_stride, dk, tid);
    const typename TO::At ao(os, dv, tid);
    TQ tq[2];
    TO to[2];
    auto fetch = [&](int t, int b) {
        in_order();
        tq[b].fetch(qp + t * TT * p.q_stride, aq, sg.n - t * TT);
        to[b].fetch(op + t * TT * os, ao, sg.n - t * TT);
        in_order();
    };
    fetch(first, 0);
    fetch(first + 1, 1);
    const Decay decay(a, h);
    Weights<true>::fill(decay, tab, kSeg, tid, NT);
    Weights<true> weight;
    weight.set(decay, p.scale, tab, g, i);
    float da = 0.f;
    auto step = [&](int t, int b) {
        T *bq = lds + b * TQ::kSize, *bo = lds + 2 * TQ::kSize + b * TO::kSize;
        tq[b].put(bq, tid);
        to[b].put(bo, tid);
        fetch(t + 2, b);
        __syncthreads();
        const int kblk = t * TT / 16;
        if (kblk + 1 < rblk) return;
        ScoreOps<DT, DK> qops;
        ScoreOps<DT, DV> oops;
        qops.load(bq, g, i);
        oops.load(bo, g, i);
        in_order<DT>();
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            f32x4 s[2], r[2];
            qops.times(s, xk[it]);
            oops.times(r, xv[it]);
#pragma unroll
            for (int jt = 0; jt < 2; ++jt) {
                const int D = kblk + jt - rblk - it;
                const f32x4 u = weight.slope(D, g, i);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    da += D > 0 || (D == 0 && weight.seen(g, i, e)) ? u[e] * s[jt][e] * r[jt][e] : 0.f;
            }
        }
    };
    int t = first;
    for (; t + 1 < nt; t += 2) {
        step(t, 0);
        step(t + 1, 1);
    }
    if (t < nt) step(t, 0);
    sum_to<NT>(da, sums, part, tid);
}

// dk and dq of the key heads (blocks_k of each), dv of the value heads and, with
// SLOPES, dalpha's addends (blocks_v of each)
template <int DT, int DK, int DV, bool SLOPES>
__global__ __launch_bounds__(Shape<DT>::NT, Shape<DT>::WAVES) void k_lin_grads(Lin a, unsigned blocks_k, unsigned blocks_v) {
    constexpr int NT = Shape<DT>::NT, IT = Shape<DT>::IT;
    __shared__ __attribute__((aligned(16))) typename El<DT>::T lds[rows_lds<DT, DK, DV, SLOPES>()];
    __shared__ __attribute__((aligned(16))) float tab[kSeg];
    __shared__ Odd<Shape<DT>::ROWS / El<DT>::TT> odd;
    __shared__ float sums[NT / 64];
    unsigned b = blockIdx.x;
    if (b < blocks_k) {
        rows_of<DT, DK, DV, NT, IT, kDk, false>(a, b, blocks_k, lds, tab, odd, sums);
    } else if ((b -= blocks_k) < blocks_k) {
        rows_of<DT, DK, DV, NT, IT, kDq, SLOPES>(a, b, blocks_k, lds, tab, odd, sums);
    } else if ((b -= blocks_k) < blocks_v) {
        rows_of<DT, DK, DV, NT, IT, kDv, SLOPES>(a, b, blocks_v, lds, tab, odd, sums);
    } else if constexpr (SLOPES) {
        slopes_of<DT, DK, DV, NT, IT>(a, b - blocks_v, blocks_v, lds, tab, sums);
    }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
// What a batch has at most: ranks of sequences of `least` tokens or more (0:
// empty ones too), and their segments.
struct LinSizes {
    int64_t nrank, nseg;
};
LinSizes sizes(const Linear& p, int64_t least) {
    LinSizes z;
    z.nrank = least > 0 ? std::min(p.S, p.N / least) : p.S;
    z.nseg = p.N / kSeg + std::min(p.S, p.N / std::max<int64_t>(least, 1));
    return z;
}
int64_t scan_blocks(const Linear& p) { return (p.dk * p.dv + 4 * kThreads - 1) / (4 * kThreads); }
// Whether a sequence may have many segments: few workgroups then carry long chains
// (one of 65531 tokens, 4 heads: 34 us with 8 pieces in flight, 31.6 with 16; 40
// sequences of 16384 tokens, 16 heads: 36 and 50).  The gradients' call knows no bound
// on the lengths: more than 8192 tokens count as one sequence there.
bool long_chains(const Linear& p) { return std::min(p.N, p.max_len) > 32 * kSeg; }
bool overlap(const Linear& p) {
    const char *a = reinterpret_cast<const char*>(p.s_in), *b = reinterpret_cast<const char*>(p.s_out);
    const int64_t one = p.Hv * p.dv * p.dk * 4;
    return a && b && a < b + p.n_out * one && b < a + p.n_in * one;
}
bool in_chunks(const Linear& p) { return std::min(p.N, p.max_len) >= lin_min(p.dtype); }

struct LinLayout {
    size_t count, seqs, first, segs, log2a, s_seg, g_seg, part, split, total;
    int64_t parts, part_dv, part_pairs, part_scan;
    int splits;
};
// dq's and dk's workgroups work a key head's value heads off one by one, the
// others have one each: that sum is split where all of them together fill the
// chip's 512 places less often than that (1500 tokens, 16 value heads of one key
// head: 275 us unsplit, 74 split; 16384 tokens: not split).  The parts hold 32 MiB
// at most.
int head_splits(const Linear& p, int64_t rows) {
    const int64_t group = p.Hv / p.Hk, at_once = std::min(group, (4 * rows * p.Hv + 511) / 512);
    return at_once > 0 ? (int)((group + at_once - 1) / at_once) : 1;
}
LinLayout layout(const Linear& p, const LinSizes& z, bool back) {
    LinLayout L{};
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += align256(bytes);
        return at;
    };
    L.count = take(8);
    L.seqs = take(4 * (size_t)z.nrank);
    L.first = take(4 * ((size_t)z.nrank + 1));
    L.segs = take(sizeof(Seg) * (size_t)z.nseg);
    L.log2a = take(4 * (size_t)p.Hv);
    const size_t head = sizeof(float) * (size_t)(p.Hv * p.dk * p.dv);
    L.s_seg = take(head * z.nseg);
    if (back) {
        L.g_seg = take(head * z.nseg);
        L.part_dv = z.nseg * (kSeg / (p.dtype == GDN_BF16 ? Shape<GDN_BF16>::ROWS : Shape<GDN_F32>::ROWS));
        L.splits = head_splits(p, L.part_dv);
        L.part_pairs = 2 * L.part_dv;
        L.part_scan = 3 * L.part_dv;
        L.parts = L.part_scan + z.nrank * scan_blocks(p);
        L.part = take(sizeof(float) * (size_t)(L.parts * p.Hv));
        if (L.splits > 1) L.split = take(sizeof(float) * 2 * (size_t)(L.splits * p.N * p.Hk * p.dk));
    }
    L.total = off;
    return L;
}
Lin arguments(const Linear& p) {
    Lin a{};
    a.p = p;
    a.at = {p.cu, p.N, p.S};
    a.Hv = (int)p.Hv;
    a.group = (int)(p.Hv / p.Hk);
    a.state = (int)(p.dk * p.dv);
    return a;
}
void place(Lin& a, const LinSizes& z, const LinLayout& L, char* base) {
    a.nrank = z.nrank;
    a.nseg = z.nseg;
    a.count = reinterpret_cast<int32_t*>(base + L.count);
    a.seqs = reinterpret_cast<int32_t*>(base + L.seqs);
    a.first = reinterpret_cast<int32_t*>(base + L.first);
    a.segs = reinterpret_cast<Seg*>(base + L.segs);
    a.log2a = reinterpret_cast<float*>(base + L.log2a);
    a.s_seg = reinterpret_cast<float*>(base + L.s_seg);
}

template <class K, class... More>
hipError_t launch(const char* name, K kernel, dim3 grid, int threads, const Lin& a, hipStream_t st, More... more) {
    if (grid.x == 0) return hipSuccess;
    prof_begin(a.p.timer, name, st);
    hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, st, a, more...);
    prof_end(a.p.timer, st);
    return hipGetLastError();
}
unsigned rec_blocks(const Linear& p, int lpr) {
    const int rows = 4 * (64 / lpr) * kLinR;
    return (unsigned)(p.S * p.Hv * ((p.dv + rows - 1) / rows));
}
template <int DT, int LPR>
hipError_t tokens(const Lin& a, hipStream_t st) {
    return launch("k_lin_rec", k_lin_rec<DT, LPR>, dim3(rec_blocks(a.p, LPR)), kThreads, a, st);
}
template <int DT>
hipError_t tokens_by_size(const Lin& a, hipStream_t st) {
    return a.p.dk > 64 ? tokens<DT, 32>(a, st) : a.p.dk > 32 ? tokens<DT, 16>(a, st) : tokens<DT, 8>(a, st);
}
template <int DT, int DK, int DV>
hipError_t forward_chunks(const Lin& a, hipStream_t st) {
    const Linear& p = a.p;
    hipError_t e = launch("k_lin_plan", k_lin_plan, dim3(1), kPlanThreads, a, st);
    if (e != hipSuccess) return e;
    const unsigned recs = rec_blocks(p, DK == 128 ? 32 : 16);
    e = launch("k_lin_add", k_lin_add<DT, DV, DK>, dim3(recs + (unsigned)(a.nseg * p.Hv)), kThreads, a, st, recs);
    if (e != hipSuccess) return e;
    e = launch("k_lin_scan", long_chains(p) ? k_lin_scan<16> : k_lin_scan<8>, dim3((unsigned)(a.nrank * p.Hv * scan_blocks(p))),
               kThreads, a, st);
    if (e != hipSuccess) return e;
    e = launch("k_lin_out", k_lin_out<DT, DK, DV>, dim3((unsigned)(a.nseg * (kSeg / Shape<DT>::ROWS) * p.Hv)),
               OutShape<DT, DV>::NT, a, st);
    if (e != hipSuccess || !a.late) return e;
    return launch("k_lin_end", k_lin_end<DT, DV, DK>, dim3((unsigned)(a.nrank * p.Hv)), kThreads, a, st);
}
template <int DT, int DK, int DV>
hipError_t backward_chunks(const Lin& a, hipStream_t st) {
    const Linear& p = a.p;
    hipError_t e = launch("k_lin_badd", k_lin_add<DT, DV, DK>, dim3((unsigned)(a.nseg * p.Hv), 2), kThreads, a, st, 0u);
    if (e != hipSuccess) return e;
    e = launch("k_lin_bscan", long_chains(p) ? k_lin_bscan<16> : k_lin_bscan<8>,
               dim3((unsigned)(a.nrank * p.Hv * scan_blocks(p))), kThreads, a, st);
    if (e != hipSuccess) return e;
    const int64_t rows = a.nseg * (kSeg / Shape<DT>::ROWS);
    const unsigned bk = (unsigned)(rows * p.Hk * a.splits), bv = (unsigned)(rows * p.Hv);
    e = a.dalpha ? launch("k_lin_grads", k_lin_grads<DT, DK, DV, true>, dim3(2 * bk + 2 * bv), Shape<DT>::NT, a, st, bk, bv)
                 : launch("k_lin_grads", k_lin_grads<DT, DK, DV, false>, dim3(2 * bk + bv), Shape<DT>::NT, a, st, bk, bv);
    if (e != hipSuccess) return e;
    const unsigned heads = a.dalpha ? (unsigned)p.Hv : 0, joins = a.splits > 1 ? (unsigned)((p.N * p.Hk * p.dk / 2 + 1023) / 1024) : 0;
    return launch("k_lin_join", k_lin_join, dim3(heads + joins), 1024, a, st, heads);
}
// (tiles of 64 or 128 features, the ones behind the real ones zero)
template <int DT>
hipError_t forward_by_size(const Lin& a, hipStream_t st) {
    const bool k = a.p.dk > 64, v = a.p.dv > 64;
    if (k) return v ? forward_chunks<DT, 128, 128>(a, st) : forward_chunks<DT, 128, 64>(a, st);
    return v ? forward_chunks<DT, 64, 128>(a, st) : forward_chunks<DT, 64, 64>(a, st);
}
template <int DT>
hipError_t backward_by_size(const Lin& a, hipStream_t st) {
    const bool k = a.p.dk > 64, v = a.p.dv > 64;
    if (k) return v ? backward_chunks<DT, 128, 128>(a, st) : backward_chunks<DT, 128, 64>(a, st);
    return v ? backward_chunks<DT, 64, 128>(a, st) : backward_chunks<DT, 64, 64>(a, st);
}

}  // namespace

bool linear_in_chunks(const Linear& p) { return in_chunks(p); }

size_t linear_workspace(const Linear& p) {
    return in_chunks(p) ? layout(p, sizes(p, lin_min(p.dtype)), false).total : 0;
}

hipError_t linear_forward(const Linear& p, void* ws, hipStream_t st) {
    Lin a = arguments(p);
    const bool chunks = in_chunks(p);
    a.chunk_min = chunks ? lin_min(p.dtype) : INT64_MAX;
    if (chunks) {
        const LinSizes z = sizes(p, lin_min(p.dtype));
        const LinLayout L = layout(p, z, false);
        place(a, z, L, static_cast<char*>(ws));
        a.late = overlap(p);
    }
    const bool bf16 = p.dtype == GDN_BF16;
    if (!chunks) return bf16 ? tokens_by_size<GDN_BF16>(a, st) : tokens_by_size<GDN_F32>(a, st);
    return bf16 ? forward_by_size<GDN_BF16>(a, st) : forward_by_size<GDN_F32>(a, st);
}

size_t linear_backward_workspace(const Linear& p) { return layout(p, sizes(p, 0), true).total; }

hipError_t linear_backward(const LinearBwd& b, void* ws, hipStream_t st) {
    const Linear& p = b.p;
    Lin a = arguments(p);
    a.chunk_min = 0;
    const LinSizes z = sizes(p, 0);
    const LinLayout L = layout(p, z, true);
    char* base = static_cast<char*>(ws);
    place(a, z, L, base);
    a.g_seg = reinterpret_cast<float*>(base + L.g_seg);
    a.part = reinterpret_cast<float*>(base + L.part);
    a.splits = L.splits;
    a.split = reinterpret_cast<float*>(base + L.split);
    a.parts = L.parts;
    a.part_dv = L.part_dv;
    a.part_pairs = L.part_pairs;
    a.part_scan = L.part_scan;
    a.dout = b.dout;
    a.ds_out = b.ds_out;
    a.dq = b.dq;
    a.dk = b.dk;
    a.dv = b.dv;
    a.dalpha = b.dalpha;
    a.ds0 = b.ds0;
    const hipError_t e = launch("k_lin_bfirst", k_lin_bfirst, dim3(1 + (unsigned)std::min<int64_t>(std::max<int64_t>(p.N, 1), 256)), kPlanThreads, a, st);
    if (e != hipSuccess) return e;
    return p.dtype == GDN_BF16 ? backward_by_size<GDN_BF16>(a, st) : backward_by_size<GDN_F32>(a, st);
}

}  // namespace gdn
