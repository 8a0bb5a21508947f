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
// factor, so any a >= 0 is right and none of the sums cancels by construction.
#include "gdn_elements.h"
#include "gdn_internal.h"
#include "gdn_mfma_common.h"
#include "gdn_packed_common.h"
#include "../../include/gdn.h"

namespace gdn {
namespace {

// Sequences of fewer tokens go token by token (forward).
constexpr int kLinMin = 32;
// Tokens of a segment at most.
constexpr int kSegMax = 512;

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
    int seg;             // tokens a segment
    int64_t chunk_min;   // sequences of fewer tokens have no segments
    int64_t nrank, nseg; // the most sequences with segments, and segments
    int32_t* count;      // [2]: such sequences, segments
    int32_t* seqs;       // [nrank]: the sequences with segments
    int32_t* first;      // [nrank + 1]: segments before each of them
    Seg* segs;           // [nseg]
    float* s_seg;        // [nseg, Hv] states: what a segment adds, then the state behind it
    float* s_copy;       // [nrank, Hv]: start states of a call in place, or null
    // backward
    const void* dout;
    const float* ds_out;
    void *dq, *dk, *dv;
    float *dalpha, *ds0;
    float* g_seg;        // [nseg, Hv]: what a segment adds to its start state's gradient, then all of that
    float* part;         // [Hv, parts]: addends of dalpha
    int64_t parts;
    int64_t part_dkv, part_scan;  // where those of the key and value rows and of the scan begin
};

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

// Powers of a decay: e^(x log a), with a^0 = 1 for a zero decay too.  The
// exponent's rounding leaves an error of |x log2 a| 2^-24 relative to the power,
// less than 2^-24 of a weight of one wherever the power counts.
struct Decay {
    float a, log2a;
    __device__ explicit Decay(float alpha) : a(alpha), log2a((float)log2((double)alpha)) {}
    __device__ float operator()(int x) const { return x == 0 ? 1.f : exp2f((float)x * log2a); }
};

// ---------------------------------------------------------------------------
// where the segments lie
// ---------------------------------------------------------------------------
// By one workgroup.  Counts saturate and are cut to the tables' sizes, so that no
// content of the offsets leads out of them.
constexpr int kPlanLds = 1024;  // ranks whose counts the search finds in LDS
__device__ __forceinline__ void plan_segments(const Lin& a, int tid) {
    __shared__ uint32_t sums[2 * kThreads / 64];
    __shared__ int lfirst[kPlanLds];
    const int64_t S = a.at.S, run = (S + kThreads - 1) / kThreads, r0 = min(tid * run, S), r1 = min(r0 + run, S);
    const int w = tid >> 6, lane = tid & 63;
    auto segs_of = [&](int64_t n) { return (uint32_t)((n + a.seg - 1) / a.seg); };
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
    if (tid == kThreads - 1) {
        put(at[0], at[1]);
        total[0] = (int)min<int64_t>(at[0], a.nrank);
        total[1] = (int)min<int64_t>(at[1], a.nseg);
        a.count[0] = total[0];
        a.count[1] = total[1];
    }
    __threadfence_block();
    __syncthreads();
    const int ranks = total[0];
    for (int i = tid; i < total[1]; i += kThreads) {
        int lo = 0, hi = ranks;  // first[lo] <= i, first[hi] > i or none
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            const int f = mid < kPlanLds ? lfirst[mid] : a.first[mid];
            if (f <= i) lo = mid;
            else hi = mid;
        }
        const int s = a.seqs[lo];
        const Span sp = span_of(a.at, s);
        const int64_t from = (int64_t)(i - (lo < kPlanLds ? lfirst[lo] : a.first[lo])) * a.seg;
        Seg x;
        x.n = (int)max<int64_t>(min<int64_t>(a.seg, sp.n - from), 0);
        x.begin = x.n > 0 ? (int)(sp.begin + from) : 0;
        x.seq = s;
        // (where the table ends, so does the sequence: no segment looks behind it)
        x.ends = (from == 0 ? kFirst : 0) | (from + a.seg >= sp.n || i + 1 == total[1] ? kLast : 0);
        a.segs[i] = x;
    }
}

// ---------------------------------------------------------------------------
// token by token
// ---------------------------------------------------------------------------
// LPR lanes hold one row of S, four elements each, R rows a thread.
constexpr int kLinR = 4;
template <int LPR>
constexpr int rec_rows() {
    return 4 * (64 / LPR) * kLinR;  // rows a workgroup
}
template <int DT, int LPR>
__device__ __forceinline__ void rec_sequence(const Lin& a, unsigned block, unsigned blocks) {
    constexpr int RPW = 64 / LPR, RB = rec_rows<LPR>();
    const Linear& p = a.p;
    const int dk = (int)p.dk, dv = (int)p.dv;
    const unsigned nrb = ((unsigned)dv + RB - 1) / RB;
    const unsigned id0 = on_one_xcd(block, blocks, nrb * a.Hv), id = id0 / nrb;
    const int rb = id0 - id * nrb, s = id / a.Hv, h = id - s * a.Hv, hk = h / a.group;
    const Span sp = span_of(a.at, s);
    const float* src = start_of(a, s, h);
    float* dst = end_of(a, s, h);
    if (sp.n >= a.chunk_min || (sp.n == 0 && src == dst)) return;
    const int w = threadIdx.x >> 6, l = threadIdx.x & 63, c = l % LPR;
    const bool on = 4 * c < dk;
    const float alpha = p.alpha[h];
    int row[kLinR];
    f32x4 S[kLinR];
#pragma unroll
    for (int j = 0; j < kLinR; ++j) {
        row[j] = rb * RB + (j * 4 + w) * RPW + l / LPR;
        S[j] = zero4();
        if (src && on && row[j] < dv) S[j] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(src + row[j] * dk + 4 * c));
    }
    for (int64_t t = sp.begin; t < sp.begin + sp.n; ++t) {
        const f32x4 k = on ? ld4e<DT>(p.k, t * p.k_stride + hk * dk + 4 * c) : zero4();
        const f32x4 q = on ? ld4e<DT>(p.q, t * p.q_stride + hk * dk + 4 * c) : zero4();
        float v[kLinR], o[kLinR];
#pragma unroll
        for (int j = 0; j < kLinR; ++j) v[j] = row[j] < dv ? gdn_ld<DT>(p.v, t * p.v_stride + h * dv + row[j]) : 0.f;
#pragma unroll
        for (int j = 0; j < kLinR; ++j) {
            S[j] = alpha * S[j] + v[j] * k;
            o[j] = p.scale * row_sum<LPR>(dot4e(S[j], q));
        }
        if (c == 0)
#pragma unroll
            for (int j = 0; j < kLinR; ++j)
                if (row[j] < dv) st_out<DT>(p.out, (t * a.Hv + h) * dv + row[j], o[j]);
    }
    if (!dst) return;
#pragma unroll
    for (int j = 0; j < kLinR; ++j)
        if (on && row[j] < dv) __builtin_nontemporal_store(S[j], reinterpret_cast<f32x4*>(dst + row[j] * dk + 4 * c));
}
template <int DT, int LPR>
__global__ __launch_bounds__(kThreads) void k_lin_rec(Lin a) {
    rec_sequence<DT, LPR>(a, blockIdx.x, gridDim.x);
}
// the segments' places, and the short sequences beside that
template <int DT, int LPR>
__global__ __launch_bounds__(kThreads) void k_lin_first(Lin a) {
    if (blockIdx.x == 0) plan_segments(a, threadIdx.x);
    else rec_sequence<DT, LPR>(a, blockIdx.x - 1, gridDim.x - 1);
}
// the segments' places, and the gradients' rows outside every sequence
__global__ __launch_bounds__(kThreads) void k_lin_bfirst(Lin a) {
    if (blockIdx.x == 0) {
        plan_segments(a, threadIdx.x);
        return;
    }
    const Linear& p = a.p;
    const int64_t c0 = cu_at(a.at, 0), c1 = max(cu_at(a.at, p.S), c0);
    const int64_t e = p.dtype == GDN_BF16 ? 2 : 4, bk = p.Hk * p.dk * e, bv = p.Hv * p.dv * e;
    for (int64_t i = blockIdx.x - 1; i < c0 + (p.N - c1); i += gridDim.x - 1) {
        const int64_t t = i < c0 ? i : c1 + (i - c0);
        for (int64_t b = 16 * threadIdx.x; b < bk; b += 16 * kThreads) {
            st_g(static_cast<char*>(a.dq) + t * bk + b, u32x4{0, 0, 0, 0});
            st_g(static_cast<char*>(a.dk) + t * bk + b, u32x4{0, 0, 0, 0});
        }
        for (int64_t b = 16 * threadIdx.x; b < bv; b += 16 * kThreads)
            st_g(static_cast<char*>(a.dv) + t * bv + b, u32x4{0, 0, 0, 0});
    }
}

// ---------------------------------------------------------------------------
// operands of the matrix cores
// ---------------------------------------------------------------------------
// Lane l = 16 g + i.  A step contracts KS indices; the lane holds KS / 4 of row
// (or column) i: those from (KS / 4) g on.  bf16 elements are exact operands;
// what fp32 arithmetic made is split into TERMS of them.
template <int DT>
struct El;
template <>
struct El<GDN_BF16> {
    using T = uint16_t;
    using Op = u16x8;
    static constexpr int KS = 32, TT = 64, PAD = 16, TERMS = 2;  // TT: tokens a tile
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

// A tile of TT tokens' rows of D features (d of them real) on its way to LDS;
// rows behind the last and features past d are zero there.
template <int DT, int D>
struct Tile {
    using T = typename El<DT>::T;
    static constexpr int TT = El<DT>::TT, LD = D + El<DT>::PAD, V = 16 / sizeof(T), PPR = D / V, NP = TT * PPR / kThreads;
    static constexpr int kSize = TT * LD;
    static_assert(NP * kThreads == TT * PPR, "whole rounds");
    u32x4 r[NP];
    __device__ __forceinline__ void fetch(const T* from, int64_t stride, int rows, int d, int tid) {
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            const int p = tid + kThreads * k, t = p / PPR, c = V * (p % PPR);
            r[k] = u32x4{0, 0, 0, 0};
            if (t < rows && c < d) r[k] = ld_g<u32x4>(from + t * stride + c);
        }
    }
    __device__ __forceinline__ void put(T* tile, int tid) const {
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            const int p = tid + kThreads * k;
            *reinterpret_cast<u32x4*>(tile + p / PPR * LD + V * (p % PPR)) = r[k];
        }
    }
};

// ---------------------------------------------------------------------------
// what a segment adds
// ---------------------------------------------------------------------------
// M[r][c] = sum_j w_j X[j][r] Y[j][c] over a segment: to its end state (X = v,
// Y = k, w_j = a^{n-1-j}) or to the gradient of its start state (X = do, Y = q,
// w_j = scale a^{j+1}).  Y is an exact operand; w_j X[j] is an fp32 value, which
// three bf16 terms hold to the last bit, so that states are as exact as fp32
// arithmetic makes them.
__device__ __forceinline__ void split3(float x0, float x1, uint32_t& h, uint32_t& m, uint32_t& l) {
    auto top = [](float x) { return __uint_as_float(__float_as_uint(x) & 0xFFFF0000u); };
    auto two = [](float x, float y) { return __builtin_amdgcn_perm(__float_as_uint(y), __float_as_uint(x), 0x07060302u); };
    h = two(x0, x1);
    const float r0 = x0 - top(x0), r1 = x1 - top(x1);
    m = two(r0, r1);
    l = two(r0 - top(r0), r1 - top(r1));
}

template <int DT, int DV, int DK>
__global__ __launch_bounds__(kThreads) void k_lin_add(Lin a) {
    using E = El<DT>;
    using T = typename E::T;
    using Op = typename E::Op;
    constexpr int TT = E::TT, KS = E::KS, RT = DV / 64, CT = DK / 16;
    using TX = Tile<DT, DV>;
    using TY = Tile<DT, DK>;
    __shared__ __attribute__((aligned(16))) T lx[2][TX::kSize];
    __shared__ __attribute__((aligned(16))) T ly[2][TY::kSize];
    __shared__ __attribute__((aligned(16))) float wt[kSegMax];
    const Linear& p = a.p;
    const bool rev = blockIdx.y == 1;
    const unsigned id = on_one_xcd(blockIdx.x, gridDim.x, a.group);
    const int64_t si = id / a.Hv;
    const int h = id - si * a.Hv;
    if (si >= a.count[1]) return;
    const Seg sg = a.segs[si];
    // (a last segment's end, where no one wants it; a first one's start gradient)
    if (rev ? (sg.ends & kFirst) && !a.ds0 : (sg.ends & kLast) && !(p.s_out && end_of(a, sg.seq, h))) return;
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, g = l >> 4, i = l & 15;
    const int dk = (int)p.dk, dv = (int)p.dv;
    const Decay decay(p.alpha[h]);
    for (int j = tid; j < a.seg; j += kThreads)
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
    TX tx;
    TY ty;
    const int nt = (sg.n + TT - 1) / TT;
    tx.fetch(x, xs, sg.n, dv, tid);
    ty.fetch(y, ys, sg.n, dk, tid);
    for (int t = 0; t < nt; ++t) {
        const T *bx = lx[t & 1], *by = ly[t & 1];
        tx.put(lx[t & 1], tid);
        ty.put(ly[t & 1], tid);
        if (t + 1 < nt) {
            tx.fetch(x + (t + 1) * TT * xs, xs, sg.n - (t + 1) * TT, dv, tid);
            ty.fetch(y + (t + 1) * TT * ys, ys, sg.n - (t + 1) * TT, dk, tid);
        }
        __syncthreads();
#pragma unroll
        for (int k0 = 0; k0 < TT; k0 += KS) {
            const float* wk = wt + t * TT + k0 + KS / 4 * g;
            Op b[RT][DT == GDN_BF16 ? 3 : 1];
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
                    for (int e = 0; e < 3; ++e) b[r][e] = __builtin_bit_cast(u16x8, u32x4{t3[e][0], t3[e][1], t3[e][2], t3[e][3]});
                } else {
                    b[r][0] = raw * *reinterpret_cast<const f32x4*>(wk);
                }
            }
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                const Op col = col_op<DT>(by, TY::LD, k0, 16 * c, g, i);
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int e = (DT == GDN_BF16 ? 2 : 0); e >= 0; --e) acc[r][c] = mm(col, b[r][e], acc[r][c]);
            }
        }
    }
    // the accumulator: column 4 g .. of 16 c, row i of the wave's
    float* out = (rev ? a.g_seg : a.s_seg) + (si * a.Hv + h) * (int64_t)a.state;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            const int row = 16 * (RT * w + r) + i, col = 16 * c + 4 * g;
            if (row < dv && col < dk) st_g(out + row * dk + col, acc[r][c]);
        }
}

// ---------------------------------------------------------------------------
// the states between the segments
// ---------------------------------------------------------------------------
// S <- a^n S + (what the segment adds), element by element, each segment's place
// holding the state behind it afterwards.  kAhead segments' pieces are in flight.
constexpr int kAhead = 8;
template <bool BACK, class F>
__device__ __forceinline__ void scan_places(const float* from, int64_t stride, int count, F step) {
    f32x4 x[kAhead], y[kAhead];
    auto fetch = [&](f32x4 (&r)[kAhead], int g0) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int g = BACK ? count - 1 - (g0 + u) : g0 + u;
            if (g0 + u < count) r[u] = ld_g<f32x4>(from + g * stride);
        }
    };
    fetch(x, 0);
    for (int g0 = 0; g0 < count; g0 += kAhead) {
        if (g0 + kAhead < count) fetch(y, g0 + kAhead);
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (g0 + u < count) step(BACK ? count - 1 - (g0 + u) : g0 + u, x[u]);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) x[u] = y[u];
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

__global__ __launch_bounds__(kThreads) void k_lin_scan(Lin a) {
    const ScanAt x = scan_at(a, threadIdx.x);
    if (!x.on) return;
    const float* src = start_of(a, x.s, x.h);
    float* dst = end_of(a, x.s, x.h);
    f32x4 S = zero4();
    if (src) {
        S = ld_g<f32x4>(src + x.e);
        if (a.s_copy) st_g(a.s_copy + ((int64_t)x.r * a.Hv + x.h) * a.state + x.e, S);
    }
    const Decay decay(a.p.alpha[x.h]);
    const float whole = decay(a.seg), rest = decay((int)(x.sp.n - (int64_t)(x.G - 1) * a.seg));
    const int64_t stride = (int64_t)a.Hv * a.state;
    float* at = a.s_seg + ((int64_t)x.f * a.Hv + x.h) * a.state + x.e;
    scan_places<false>(at, stride, dst ? x.G : x.G - 1, [&](int g, const f32x4& add) {
        S = (g == x.G - 1 ? rest : whole) * S + add;
        if (g == x.G - 1) st_g(dst + x.e, S);
        else st_g(at + g * stride, S);
    });
}

// The workgroup's sum of x, in a fixed order, written by one thread.
__device__ __forceinline__ void sum_to(float x, float* sums, float* to, int tid) {
    x = xor32_sum(row_sum<32>(x));
    if ((tid & 63) == 0) sums[tid >> 6] = x;
    __syncthreads();
    if (tid == 0) *to = (sums[0] + sums[1]) + (sums[2] + sums[3]);
    __syncthreads();
}

// Backward: the states behind the segments, then the gradients behind them, and
// n a^{n-1} <G, S> of each for dalpha.
__global__ __launch_bounds__(kThreads) void k_lin_bscan(Lin a) {
    __shared__ float sums[kThreads / 64];
    const int tid = threadIdx.x;
    const ScanAt x = scan_at(a, tid);
    float da = 0.f;
    if (x.on) {
        const Decay decay(a.p.alpha[x.h]);
        const int n_last = (int)(x.sp.n - (int64_t)(x.G - 1) * a.seg);
        const float whole = decay(a.seg), rest = x.G > 0 ? decay(n_last) : 1.f;
        const int64_t stride = (int64_t)a.Hv * a.state, off = ((int64_t)x.f * a.Hv + x.h) * a.state + x.e;
        const float* src = start_of(a, x.s, x.h);
        const f32x4 S0 = src ? ld_g<f32x4>(src + x.e) : zero4();
        f32x4 S = S0;
        float* at = a.s_seg + off;
        scan_places<false>(at, stride, x.G - 1, [&](int g, const f32x4& add) {
            S = whole * S + add;
            st_g(at + g * stride, S);
        });
        const int64_t own = ((int64_t)x.s * a.Hv + x.h) * a.state + x.e;
        f32x4 G = a.ds_out ? ld_g<f32x4>(a.ds_out + own) : zero4();
        float* ga = a.g_seg + off;
        // (without a gradient of the start state the first segment adds nothing)
        const int lowest = a.ds0 ? 0 : 1;
        const float dw = (float)a.seg * decay(a.seg - 1), dr = (float)n_last * decay(n_last - 1);
        scan_places<true>(ga + lowest * stride, stride, x.G - lowest, [&](int g, const f32x4& add) {
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
        sum_to(da, sums, a.part + h * a.parts + a.part_scan + r * per + (blockIdx.x - id * per), tid);
    }
}

// dalpha of a head: its addends in a fixed order
__global__ __launch_bounds__(1024) void k_lin_dalpha(Lin a) {
    __shared__ double sums[1024];
    const int tid = threadIdx.x;
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
    static __device__ __forceinline__ void fill(const Decay& decay, float* table, int n, int tid) {
        for (int x = tid; x < n; x += kThreads) table[x] = decay(REV ? x : x + 15 - 2 * (x & 15));
    }
    __device__ __forceinline__ bool seen(int g, int i, int e) const { return REV ? 4 * g + e >= i : i >= 4 * g + e; }
    // scores of keys of block kb and rows of block rb, weighted
    __device__ __forceinline__ f32x4 operator()(const f32x4& p, int D, int g, int i) const {
        if (D > 0) return p * (rl * *reinterpret_cast<const f32x4*>(tab + 16 * (D - 1) + 4 * g));
        f32x4 y;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = D == 0 && seen(g, i, e) ? p[e] * dw[e] : 0.f;
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

// A wave's rows as right operands, straight from memory (zero behind the last)
template <int DT, int D, int IT>
__device__ __forceinline__ void load_rows(typename El<DT>::Op (&x)[IT][D / El<DT>::KS], const typename El<DT>::T* from,
                                          int64_t stride, int row0, int rows, int d, int g, int i) {
    using Op = typename El<DT>::Op;
    constexpr int KS = El<DT>::KS;
#pragma unroll
    for (int it = 0; it < IT; ++it)
#pragma unroll
        for (int k = 0; k < D / KS; ++k) {
            const int row = row0 + 16 * it + i, c = KS * k + KS / 4 * g;
            x[it][k] = Op{};
            if (row < rows && c < d) x[it][k] = ld_g<Op>(from + row * stride + c);
        }
}

// p[jt][it]: scores of 32 keys from k0 of the tile on and the wave's rows
template <int DT, int D, int IT>
__device__ __forceinline__ void scores(f32x4 (&p)[2][IT], const typename El<DT>::T* tile, int k0,
                                       const typename El<DT>::Op (&x)[IT][D / El<DT>::KS], int g, int i) {
    constexpr int KS = El<DT>::KS, LD = D + El<DT>::PAD;
#pragma unroll
    for (int jt = 0; jt < 2; ++jt) {
#pragma unroll
        for (int it = 0; it < IT; ++it) p[jt][it] = zero4();
#pragma unroll
        for (int k = 0; k < D / KS; ++k) {
            const auto op = row_op<DT>(tile + (k0 + 16 * jt + i) * LD + KS * k, g);
#pragma unroll
            for (int it = 0; it < IT; ++it) p[jt][it] = mm(op, x[it][k], p[jt][it]);
        }
    }
}
// acc[it][mt] += (columns of 32 rows of the tile) p
template <int DT, int D, int IT>
__device__ __forceinline__ void gather(f32x4 (&acc)[IT][D / 16], const f32x4 (&p)[2][IT], const typename El<DT>::T* tile,
                                       int k0, int g, int i) {
    constexpr int LD = D + El<DT>::PAD;
    if constexpr (DT == GDN_BF16) {
        u16x8 hi[IT], lo[IT];
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            u16x4 h0, l0, h1, l1;
            split4(p[0][it], h0, l0);
            split4(p[1][it], h1, l1);
            hi[it] = cat(h0, h1);
            lo[it] = cat(l0, l1);
        }
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
            const u16x8 col = col_op_acc<DT>(tile, LD, k0, 16 * mt, g, i);
#pragma unroll
            for (int it = 0; it < IT; ++it) acc[it][mt] = mm(col, hi[it], mm(col, lo[it], acc[it][mt]));
        }
    } else {
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
            for (int jt = 0; jt < 2; ++jt) {
                const f32x4 col = col_op_acc<DT>(tile, LD, k0 + 16 * jt, 16 * mt, g, i);
#pragma unroll
                for (int it = 0; it < IT; ++it) acc[it][mt] = mm(col, p[jt][it], acc[it][mt]);
            }
    }
}

// M X for the state's product, 32 rows of M (TR: columns) at a time through LDS,
// split into terms there; use(mt, it, t): rows 16 mt .. of M X.  M has dm rows and
// dx columns, TR: dx rows and dm columns.
template <int DT, int DX, int DM, bool TR>
constexpr int slab_size() {
    constexpr int PAD = El<DT>::PAD;
    return El<DT>::TERMS * (TR ? DX * (32 + PAD) : 32 * (DX + PAD));
}
template <int DT, int DX, int DM, int IT, bool TR, class F>
__device__ __forceinline__ void state_rows(const float* M, typename El<DT>::T* slab,
                                           const typename El<DT>::Op (&x)[IT][DX / El<DT>::KS], int dx, int dm, int tid, F use) {
    using Op = typename El<DT>::Op;
    constexpr int KS = El<DT>::KS, NP = DX / 32, LD = TR ? 32 + El<DT>::PAD : DX + El<DT>::PAD;
    constexpr int LO = slab_size<DT, DX, DM, TR>() / El<DT>::TERMS;
    const int l = tid & 63, g = l >> 4, i = l & 15;
    f32x4 r[NP];
    auto fetch = [&](int m0) {
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            const int p = tid + kThreads * k, row = TR ? p / 8 : p / (DX / 4), c = 4 * (TR ? p % 8 : p % (DX / 4));
            r[k] = zero4();
            if (TR ? row < dx && m0 + c < dm : m0 + row < dm && c < dx)
                r[k] = ld_g<f32x4>(M + (TR ? row * dm + m0 + c : (m0 + row) * dx + c));
        }
    };
    fetch(0);
#pragma unroll
    for (int m0 = 0; m0 < DM; m0 += 32) {
        if (m0 >= dm) break;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            const int p = tid + kThreads * k, row = TR ? p / 8 : p / (DX / 4), c = 4 * (TR ? p % 8 : p % (DX / 4));
            auto* to = slab + row * LD + c;
            if constexpr (DT == GDN_BF16) {
                u16x4 hi, lo;
                split4(r[k], hi, lo);
                *reinterpret_cast<u16x4*>(to) = hi;
                *reinterpret_cast<u16x4*>(to + LO) = lo;
            } else {
                *reinterpret_cast<f32x4*>(to) = r[k];
            }
        }
        if (m0 + 32 < dm) fetch(m0 + 32);
        __syncthreads();
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            f32x4 t[IT];
#pragma unroll
            for (int it = 0; it < IT; ++it) t[it] = zero4();
#pragma unroll
            for (int k = 0; k < DX / KS; ++k)
#pragma unroll
                for (int e = El<DT>::TERMS - 1; e >= 0; --e) {
                    const Op op = TR ? col_op<DT>(slab + e * LO, LD, KS * k, 16 * m, g, i)
                                     : row_op<DT>(slab + e * LO + (16 * m + i) * LD + KS * k, g);
#pragma unroll
                    for (int it = 0; it < IT; ++it) t[it] = mm(op, x[it][k], t[it]);
                }
            use(m0 / 16 + m, t);
        }
    }
    __syncthreads();
}

// Four features of a row, rounded once
template <int DT>
__device__ __forceinline__ void st4(typename El<DT>::T* to, const f32x4& x) {
    if constexpr (DT == GDN_BF16) st_g(to, u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])});
    else st_g(to, x);
}

// The state in front of segment si, or null (zero)
__device__ __forceinline__ const float* state_before(const Lin& a, const Seg& sg, int64_t si, int h) {
    if (!(sg.ends & kFirst)) return a.s_seg + ((si - 1) * a.Hv + h) * (int64_t)a.state;
    const float* src = start_of(a, sg.seq, h);
    if (!src || !a.s_copy) return src;
    // (its rank: the first segments before it are counted in a.first)
    int lo = 0, hi = a.count[0];
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.first[mid] <= si) lo = mid;
        else hi = mid;
    }
    return a.s_copy + ((int64_t)lo * a.Hv + h) * a.state;
}

// Rows up to i: the forward's outputs (BACK false; a workgroup a value head) and
// dq (a workgroup a key head, its value heads one after the other in one sum).
constexpr int kIT = 2, kBlockRows = 64 * kIT;
template <int DT, int DX, int DM, bool BACK>
__global__ __launch_bounds__(kThreads, 2) void k_lin_rows(Lin a) {
    using E = El<DT>;
    using T = typename E::T;
    using Op = typename E::Op;
    constexpr int TT = E::TT, IT = kIT;
    using TA = Tile<DT, DX>;
    using TB = Tile<DT, DM>;
    static_assert(slab_size<DT, DX, DM, BACK>() <= 2 * TA::kSize, "a slab of the state fits the tiles");
    __shared__ __attribute__((aligned(16))) T la[2 * TA::kSize];
    __shared__ __attribute__((aligned(16))) T lb[2 * TB::kSize];
    __shared__ __attribute__((aligned(16))) float tab[kSegMax];
    __shared__ float sums[kThreads / 64];
    const Linear& p = a.p;
    const int heads = BACK ? (int)p.Hk : a.Hv, nh = BACK ? a.group : 1;
    const unsigned nrb = (a.seg + kBlockRows - 1) / kBlockRows;
    const unsigned block = on_one_xcd(blockIdx.x, gridDim.x, BACK ? nrb : nrb * a.group), id = block / nrb;
    const int rb = block - id * nrb, hh = id % heads;
    const int64_t si = id / heads;
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, g = l >> 4, i = l & 15;
    const Seg sg = si < a.count[1] ? a.segs[si] : Seg{0, 0, 0, 0};
    const bool slopes = BACK && a.dalpha;
    float* part = slopes ? a.part + (int64_t)hh * nh * a.parts + si * nrb + rb : nullptr;
    if (rb * kBlockRows >= sg.n) {
        for (int j = tid; slopes && j < nh; j += kThreads) part[j * a.parts] = 0.f;
        return;
    }
    const int dx = (int)(BACK ? p.dv : p.dk), dm = (int)(BACK ? p.dk : p.dv);
    const int64_t xs = BACK ? (int64_t)a.Hv * p.dv : p.q_stride, as = BACK ? p.v_stride : p.k_stride,
                  bs = BACK ? p.k_stride : p.v_stride;
    const int row0 = rb * kBlockRows + 16 * IT * w, rblk = row0 / 16;
    const int nkeys = min(sg.n, (rb + 1) * kBlockRows), nt = (nkeys + TT - 1) / TT;

    f32x4 acc[IT][DM / 16];
#pragma unroll
    for (int it = 0; it < IT; ++it)
#pragma unroll
        for (int mt = 0; mt < DM / 16; ++mt) acc[it][mt] = zero4();
    for (int j = 0; j < nh; ++j) {
        const int h = hh * nh + j, hk = BACK ? hh : hh / a.group;
        const T* xp = static_cast<const T*>(BACK ? a.dout : p.q) + sg.begin * xs + (int64_t)(BACK ? h : hk) * dx;
        const T* ap = static_cast<const T*>(BACK ? p.v : p.k) + sg.begin * as + (int64_t)(BACK ? h : hk) * dx;
        const T* bp = static_cast<const T*>(BACK ? p.k : p.v) + sg.begin * bs + (int64_t)(BACK ? hk : h) * dm;
        const Decay decay(p.alpha[h]);
        if (j > 0) __syncthreads();
        Weights<false>::fill(decay, tab, a.seg, tid);
        Weights<false> weight;
        weight.set(decay, p.scale, tab, g, i);
        Op x[IT][DX / E::KS];
        load_rows<DT, DX, IT>(x, xp, xs, row0, sg.n, dx, g, i);
        TA ta;
        TB tb;
        const float* M = state_before(a, sg, si, h);
        float da = 0.f;
        if (M) {
            float f[IT], df[IT];
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const int row = row0 + 16 * it + i;
                df[it] = p.scale * (float)(row + 1) * decay(row);
                f[it] = p.scale * decay(row + 1);
            }
            state_rows<DT, DX, DM, IT, BACK>(M, la, x, dx, dm, tid, [&](int mt, const f32x4 (&t)[IT]) {
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    acc[it][mt] += f[it] * t[it];
                    if constexpr (BACK) {
                        const int row = row0 + 16 * it + i, c = 16 * mt + 4 * g;
                        if (slopes && row < sg.n && c < dm)
                            da += df[it] * dot4e(t[it], ld4e<DT>(p.q, (sg.begin + row) * p.q_stride + hk * dm + c));
                    }
                }
            });
        }
        ta.fetch(ap, as, nkeys, dx, tid);
        tb.fetch(bp, bs, nkeys, dm, tid);
        for (int t = 0; t < nt; ++t) {
            T *ba = la + (t & 1) * TA::kSize, *bb = lb + (t & 1) * TB::kSize;
            ta.put(ba, tid);
            tb.put(bb, tid);
            if (t + 1 < nt) {
                ta.fetch(ap + (t + 1) * TT * as, as, nkeys - (t + 1) * TT, dx, tid);
                tb.fetch(bp + (t + 1) * TT * bs, bs, nkeys - (t + 1) * TT, dm, tid);
            }
            __syncthreads();
#pragma unroll
            for (int k0 = 0; k0 < TT; k0 += 32) {
                const int kblk = (t * TT + k0) / 16;
                if (kblk > rblk + IT - 1) continue;
                f32x4 s[2][IT];
                scores<DT, DX, IT>(s, ba, k0, x, g, i);
#pragma unroll
                for (int jt = 0; jt < 2; ++jt)
#pragma unroll
                    for (int it = 0; it < IT; ++it) s[jt][it] = weight(s[jt][it], rblk + it - kblk - jt, g, i);
                gather<DT, DM, IT>(acc, s, bb, k0, g, i);
            }
        }
        if (slopes) sum_to(da, sums, part + j * a.parts, tid);
    }
    T* out = static_cast<T*>(BACK ? a.dq : p.out) + (int64_t)hh * dm;
    const int64_t os = (int64_t)heads * dm;
#pragma unroll
    for (int it = 0; it < IT; ++it) {
        const int row = row0 + 16 * it + i;
        if (row < sg.n)
#pragma unroll
            for (int mt = 0; mt < DM / 16; ++mt)
                if (16 * mt < dm) st4<DT>(out + (sg.begin + row) * os + 16 * mt + 4 * g, acc[it][mt]);
    }
}

// Rows from j on: dk and dv together, whose products read the same tiles of q and
// do.  A workgroup a key head; dk is summed over its value heads.
template <int DT, int DK, int DV, int IT>
__global__ __launch_bounds__(kThreads) void k_lin_dkv(Lin a) {
    using E = El<DT>;
    using T = typename E::T;
    using Op = typename E::Op;
    constexpr int TT = E::TT, kRows = 64 * IT;
    using TQ = Tile<DT, DK>;
    using TO = Tile<DT, DV>;
    constexpr int SLAB = std::max(slab_size<DT, DK, DV, false>(), slab_size<DT, DV, DK, true>());
    static_assert(SLAB <= 2 * TQ::kSize + 2 * TO::kSize, "a slab of the state fits the tiles");
    __shared__ __attribute__((aligned(16))) T tiles[2 * TQ::kSize + 2 * TO::kSize];
    __shared__ __attribute__((aligned(16))) float tab[kSegMax];
    __shared__ float sums[kThreads / 64];
    T *lq = tiles, *lo = tiles + 2 * TQ::kSize;
    const Linear& p = a.p;
    const unsigned nrb = (a.seg + kRows - 1) / kRows;
    const unsigned block = on_one_xcd(blockIdx.x, gridDim.x, nrb), id = block / nrb;
    const int rb = block - id * nrb, hk = id % (int)p.Hk;
    const int64_t si = id / (int)p.Hk;
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, g = l >> 4, i = l & 15;
    const Seg sg = si < a.count[1] ? a.segs[si] : Seg{0, 0, 0, 0};
    const bool slopes = a.dalpha;
    float* part = slopes ? a.part + (int64_t)hk * a.group * a.parts + a.part_dkv + si * nrb + rb : nullptr;
    if (rb * kRows >= sg.n) {
        for (int j = tid; slopes && j < a.group; j += kThreads) part[j * a.parts] = 0.f;
        return;
    }
    const int dk = (int)p.dk, dv = (int)p.dv;
    const int64_t os = (int64_t)a.Hv * dv;
    const int row0 = rb * kRows + 16 * IT * w, rblk = row0 / 16;
    const int first = rb * kRows / TT, nt = (sg.n + TT - 1) / TT;

    Op xk[IT][DK / E::KS];
    load_rows<DT, DK, IT>(xk, static_cast<const T*>(p.k) + sg.begin * p.k_stride + (int64_t)hk * dk, p.k_stride, row0, sg.n, dk,
                          g, i);
    const T* qp = static_cast<const T*>(p.q) + sg.begin * p.q_stride + (int64_t)hk * dk;
    f32x4 ak[IT][DK / 16];
#pragma unroll
    for (int it = 0; it < IT; ++it)
#pragma unroll
        for (int mt = 0; mt < DK / 16; ++mt) ak[it][mt] = zero4();
    for (int j = 0; j < a.group; ++j) {
        const int h = hk * a.group + j;
        const T* vp = static_cast<const T*>(p.v) + sg.begin * p.v_stride + (int64_t)h * dv;
        const T* op = static_cast<const T*>(a.dout) + sg.begin * os + (int64_t)h * dv;
        const Decay decay(p.alpha[h]);
        if (j > 0) __syncthreads();
        Weights<true>::fill(decay, tab, a.seg, tid);
        Weights<true> weight;
        weight.set(decay, p.scale, tab, g, i);
        Op xv[IT][DV / E::KS];
        load_rows<DT, DV, IT>(xv, vp, p.v_stride, row0, sg.n, dv, g, i);
        f32x4 av[IT][DV / 16];
#pragma unroll
        for (int it = 0; it < IT; ++it)
#pragma unroll
            for (int mt = 0; mt < DV / 16; ++mt) av[it][mt] = zero4();
        const float* G = !(sg.ends & kLast) ? a.g_seg + ((si + 1) * a.Hv + h) * (int64_t)a.state
                         : a.ds_out         ? a.ds_out + ((int64_t)sg.seq * a.Hv + h) * a.state
                                            : nullptr;
        float da = 0.f;
        if (G) {
            float f[IT], df[IT];
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const int e = sg.n - 1 - (row0 + 16 * it + i);  // (below zero: no row)
                f[it] = e >= 0 ? decay(e) : 0.f;
                df[it] = e > 0 ? (float)e * decay(e - 1) : 0.f;
            }
            state_rows<DT, DK, DV, IT, false>(G, tiles, xk, dk, dv, tid, [&](int mt, const f32x4 (&t)[IT]) {
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    av[it][mt] += f[it] * t[it];
                    const int row = row0 + 16 * it + i, c = 16 * mt + 4 * g;
                    if (slopes && row < sg.n && c < dv)
                        da += df[it] * dot4e(t[it], ld4e<DT>(p.v, (sg.begin + row) * p.v_stride + (int64_t)h * dv + c));
                }
            });
            state_rows<DT, DV, DK, IT, true>(G, tiles, xv, dv, dk, tid, [&](int mt, const f32x4 (&t)[IT]) {
#pragma unroll
                for (int it = 0; it < IT; ++it) ak[it][mt] += f[it] * t[it];
            });
        }
        TQ tq;
        TO to;
        tq.fetch(qp + first * TT * p.q_stride, p.q_stride, sg.n - first * TT, dk, tid);
        to.fetch(op + first * TT * os, os, sg.n - first * TT, dv, tid);
        for (int t = first; t < nt; ++t) {
            T *bq = lq + (t & 1) * TQ::kSize, *bo = lo + (t & 1) * TO::kSize;
            tq.put(bq, tid);
            to.put(bo, tid);
            if (t + 1 < nt) {
                tq.fetch(qp + (t + 1) * TT * p.q_stride, p.q_stride, sg.n - (t + 1) * TT, dk, tid);
                to.fetch(op + (t + 1) * TT * os, os, sg.n - (t + 1) * TT, dv, tid);
            }
            __syncthreads();
#pragma unroll
            for (int k0 = 0; k0 < TT; k0 += 32) {
                const int kblk = (t * TT + k0) / 16;
                if (kblk + 1 < rblk) continue;
                f32x4 s[2][IT], r[2][IT];
                scores<DT, DK, IT>(s, bq, k0, xk, g, i);
                scores<DT, DV, IT>(r, bo, k0, xv, g, i);
#pragma unroll
                for (int jt = 0; jt < 2; ++jt)
#pragma unroll
                    for (int it = 0; it < IT; ++it) {
                        const int D = kblk + jt - rblk - it;
                        if (slopes) {
                            const f32x4 u = weight.slope(D, g, i);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                da += D > 0 || (D == 0 && weight.seen(g, i, e)) ? u[e] * s[jt][it][e] * r[jt][it][e] : 0.f;
                        }
                        s[jt][it] = weight(s[jt][it], D, g, i);
                        r[jt][it] = weight(r[jt][it], D, g, i);
                    }
                gather<DT, DV, IT>(av, s, bo, k0, g, i);
                gather<DT, DK, IT>(ak, r, bq, k0, g, i);
            }
        }
        T* out = static_cast<T*>(a.dv) + (int64_t)h * dv;
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            const int row = row0 + 16 * it + i;
            if (row < sg.n)
#pragma unroll
                for (int mt = 0; mt < DV / 16; ++mt)
                    if (16 * mt < dv) st4<DT>(out + (sg.begin + row) * os + 16 * mt + 4 * g, av[it][mt]);
        }
        if (slopes) sum_to(da, sums, part + j * a.parts, tid);
    }
    T* out = static_cast<T*>(a.dk) + (int64_t)hk * dk;
#pragma unroll
    for (int it = 0; it < IT; ++it) {
        const int row = row0 + 16 * it + i;
        if (row < sg.n)
#pragma unroll
            for (int mt = 0; mt < DK / 16; ++mt)
                if (16 * mt < dk) st4<DT>(out + (sg.begin + row) * (p.Hk * dk) + 16 * mt + 4 * g, ak[it][mt]);
    }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
int seg_for(const Linear&) { return 256; }

// What a batch has at most: ranks of sequences of `least` tokens or more (0:
// empty ones too), and their segments.
struct LinSizes {
    int seg;
    int64_t nrank, nseg;
};
LinSizes sizes(const Linear& p, int64_t least) {
    LinSizes z;
    z.seg = seg_for(p);
    z.nrank = least > 0 ? std::min(p.S, p.N / least) : p.S;
    z.nseg = p.N / z.seg + std::min(p.S, p.N / std::max<int64_t>(least, 1));
    return z;
}
int64_t scan_blocks(const Linear& p) { return (p.dk * p.dv + 4 * kThreads - 1) / (4 * kThreads); }
bool overlap(const Linear& p) {
    const char *a = reinterpret_cast<const char*>(p.s_in), *b = reinterpret_cast<const char*>(p.s_out);
    const int64_t one = p.Hv * p.dv * p.dk * 4;
    return a && b && a < b + p.n_out * one && b < a + p.n_in * one;
}
bool in_chunks(const Linear& p) { return std::min(p.N, p.max_len) >= kLinMin; }

struct LinLayout {
    size_t count, seqs, first, segs, s_seg, s_copy, g_seg, part, total;
    int64_t parts, part_dkv, part_scan;
};
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
    const size_t head = sizeof(float) * (size_t)(p.Hv * p.dk * p.dv);
    L.s_seg = take(head * z.nseg);
    if (back) {
        L.g_seg = take(head * z.nseg);
        const int64_t rows = z.nseg * ((z.seg + kBlockRows - 1) / kBlockRows);
        L.part_dkv = rows;
        L.part_scan = L.part_dkv + z.nseg * (z.seg / 64);
        L.parts = L.part_scan + z.nrank * scan_blocks(p);
        L.part = take(sizeof(float) * (size_t)(L.parts * p.Hv));
    } else {
        L.s_copy = take(head * z.nrank);
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
    a.seg = z.seg;
    a.nrank = z.nrank;
    a.nseg = z.nseg;
    a.count = reinterpret_cast<int32_t*>(base + L.count);
    a.seqs = reinterpret_cast<int32_t*>(base + L.seqs);
    a.first = reinterpret_cast<int32_t*>(base + L.first);
    a.segs = reinterpret_cast<Seg*>(base + L.segs);
    a.s_seg = reinterpret_cast<float*>(base + L.s_seg);
}

template <class K>
hipError_t launch(const char* name, K kernel, dim3 grid, int threads, const Lin& a, hipStream_t st) {
    if (grid.x == 0) return hipSuccess;
    prof_begin(a.p.timer, name, st);
    hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, st, a);
    prof_end(a.p.timer, st);
    return hipGetLastError();
}
unsigned rec_blocks(const Linear& p, int lpr) {
    const int rows = 4 * (64 / lpr) * kLinR;
    return (unsigned)(p.S * p.Hv * ((p.dv + rows - 1) / rows));
}
template <int DT, int LPR>
hipError_t start(const Lin& a, bool chunks, hipStream_t st) {
    const unsigned recs = rec_blocks(a.p, LPR);
    return chunks ? launch("k_lin_first", k_lin_first<DT, LPR>, dim3(recs + 1), kThreads, a, st)
                  : launch("k_lin_rec", k_lin_rec<DT, LPR>, dim3(recs), kThreads, a, st);
}
template <int DT>
hipError_t start_by_row(const Lin& a, bool chunks, hipStream_t st) {
    return a.p.dk > 64 ? start<DT, 32>(a, chunks, st) : a.p.dk > 32 ? start<DT, 16>(a, chunks, st) : start<DT, 8>(a, chunks, st);
}
template <int DT, int DK, int DV>
hipError_t forward_chunks(const Lin& a, hipStream_t st) {
    const Linear& p = a.p;
    hipError_t e = launch("k_lin_add", k_lin_add<DT, DV, DK>, dim3((unsigned)(a.nseg * p.Hv), 1), kThreads, a, st);
    if (e != hipSuccess) return e;
    e = launch("k_lin_scan", k_lin_scan, dim3((unsigned)(a.nrank * p.Hv * scan_blocks(p))), kThreads, a, st);
    if (e != hipSuccess) return e;
    const int64_t nrb = (a.seg + kBlockRows - 1) / kBlockRows;
    return launch("k_lin_out", k_lin_rows<DT, DK, DV, false>, dim3((unsigned)(a.nseg * nrb * p.Hv)), kThreads, a, st);
}
template <int DT, int DK, int DV>
hipError_t backward_chunks(const Lin& a, hipStream_t st) {
    constexpr int IT = DT == GDN_BF16 ? 1 : 1;
    const Linear& p = a.p;
    hipError_t e = launch("k_lin_badd", k_lin_add<DT, DV, DK>, dim3((unsigned)(a.nseg * p.Hv), 2), kThreads, a, st);
    if (e != hipSuccess) return e;
    e = launch("k_lin_bscan", k_lin_bscan, dim3((unsigned)(a.nrank * p.Hv * scan_blocks(p))), kThreads, a, st);
    if (e != hipSuccess) return e;
    const int64_t nrb = (a.seg + kBlockRows - 1) / kBlockRows;
    e = launch("k_lin_dq", k_lin_rows<DT, DV, DK, true>, dim3((unsigned)(a.nseg * nrb * p.Hk)), kThreads, a, st);
    if (e != hipSuccess) return e;
    const int64_t nkb = a.seg / (64 * IT);
    e = launch("k_lin_dkv", k_lin_dkv<DT, DK, DV, IT>, dim3((unsigned)(a.nseg * nkb * p.Hk)), kThreads, a, st);
    if (e != hipSuccess || !a.dalpha) return e;
    return launch("k_lin_dalpha", k_lin_dalpha, dim3((unsigned)p.Hv), 1024, a, st);
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
    return in_chunks(p) ? layout(p, sizes(p, kLinMin), false).total : 0;
}

hipError_t linear_forward(const Linear& p, void* ws, hipStream_t st) {
    Lin a = arguments(p);
    const bool chunks = in_chunks(p);
    a.chunk_min = chunks ? kLinMin : INT64_MAX;
    if (chunks) {
        const LinSizes z = sizes(p, kLinMin);
        const LinLayout L = layout(p, z, false);
        place(a, z, L, static_cast<char*>(ws));
        if (overlap(p)) a.s_copy = reinterpret_cast<float*>(static_cast<char*>(ws) + L.s_copy);
    }
    const bool bf16 = p.dtype == GDN_BF16;
    const hipError_t e = bf16 ? start_by_row<GDN_BF16>(a, chunks, st) : start_by_row<GDN_F32>(a, chunks, st);
    if (e != hipSuccess || !chunks) return e;
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
    a.parts = L.parts;
    a.part_dkv = L.part_dkv;
    a.part_scan = L.part_scan;
    a.dout = b.dout;
    a.ds_out = b.ds_out;
    a.dq = b.dq;
    a.dk = b.dk;
    a.dv = b.dv;
    a.dalpha = b.dalpha;
    a.ds0 = b.ds0;
    const hipError_t e = launch("k_lin_bfirst", k_lin_bfirst, dim3(1 + (unsigned)std::min<int64_t>(std::max<int64_t>(p.N, 1), 1024)), kThreads, a, st);
    if (e != hipSuccess) return e;
    return p.dtype == GDN_BF16 ? backward_by_size<GDN_BF16>(a, st) : backward_by_size<GDN_F32>(a, st);
}

}  // namespace gdn
