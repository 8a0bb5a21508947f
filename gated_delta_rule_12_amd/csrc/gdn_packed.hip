// The gated delta rule over packed ragged sequences with a pool of states
// (gdn_packed_fwd).
//
// Sequence s holds tokens cu[s] .. cu[s + 1] - 1 of [N, heads, features]
// arrays, starts from one slot of a state pool and ends in one; value head h
// reads key head h / (Hv / Hk).  Per token (state rows: value features)
//   predict-then-decay:  S' = S D + beta (v - S k) k^T
//   decay-then-predict:  S' = S D + beta (v - S D k) k^T,   o = scale S' q
// with D = alpha or Diag(alpha) (the recurrence of the Gated DeltaNet
// GPU-parallelisation blog, section 1.2, and of the DeltaNet illustrated
// notes' GDN and KDA paragraphs).
//
// Two forms serve one call, each sequence taking one of them by its length:
//   k_pk_rec, token by token, the state in registers: steps of a generation,
//     drafted tokens, short prompts, and every shape without chunk kernels;
//   the chunk form (scalar gate, bf16, dk = dv = D in {64, 128}, sequences of
//     at least kChunkMin tokens), C = 64 tokens a chunk (notes, WY/UT section):
//       T'    = (I + diag(beta) L)^{-1} diag(beta),  L_tj = e^{g'_t - g_j} k_t.k_j (j < t)
//       Delta = T' (V - diag(gamma') K S^T)
//       O     = scale (diag(gamma) Q S^T + P Delta),  P_tj = e^{g_t - g_j} q_t.k_j (j <= t)
//       S'    = gamma_C S + (diag(gamma_C / gamma) Delta)^T K
//     k_pk_prep forms T' and the gate rows of every chunk at once; k_pk_seg
//     carries a head's state over the chunks of a segment; sequences longer
//     than a segment run as a state pass (every segment but the last, from
//     zero, with the matrix M its start state is multiplied by), the chain of
//     start states (k_pk_chain: S_start(g + 1) = S_end(g) + S_start(g) M(g),
//     the sequence-parallel notes' increment and correction) and the output
//     pass from the true start states.
// Chunks and segments have their places by rule (gdn_packed_common.h).  Slots
// outside the pool read as zero states and are not written.
#include <type_traits>

#include "gdn_internal.h"
#include "gdn_mfma_common.h"
#include "gdn_packed_common.h"
#include "../../include/gdn.h"

namespace gdn {
namespace {

// Sequences of fewer tokens go token by token where there is a choice.
constexpr int kChunkMin = 32;

struct Pk {
    Packed p;
    Offsets at;
    int Hv, group;   // value heads; value heads per key head
    int rec_below;   // k_pk_rec takes sequences of fewer tokens
    int seg_shift;   // a segment holds 2^seg_shift tokens
    int64_t nslot;   // places for chunks
    int64_t nseg;    // places for segments
    float* T;        // [place, head][10 blocks of 16 x 16]: T' (lower blocks, row by row)
    float* G;        // [place, head][kGate]
    float* s_end;    // [place, head][D][D]: end states of the state pass
    float* m_end;    // [place, head][D][D]: M transposed
    float* s_start;  // [place, head][D][D]: start states of the output pass
};

__device__ __forceinline__ const float* state_from(const Packed& p, int64_t s, int64_t h) {
    const int64_t slot = p.slots_in ? (int64_t)p.slots_in[s] : s;
    if (!p.s_in || slot < 0 || slot >= p.n_in) return nullptr;
    return p.s_in + (slot * p.Hv + h) * p.dv * p.dk;
}
__device__ __forceinline__ float* state_to(const Packed& p, int64_t s, int64_t h) {
    const int64_t slot = p.slots_out ? (int64_t)p.slots_out[s] : s;
    if (!p.s_out || slot < 0 || slot >= p.n_out) return nullptr;
    return p.s_out + (slot * p.Hv + h) * p.dv * p.dk;
}

// ---------------------------------------------------------------------------
// token by token
// ---------------------------------------------------------------------------
// LPR lanes hold one row of S, NP pieces of four elements each (piece i of
// lane c at columns 4 (c + LPR i)), R rows a thread; the two dot products are
// summed over the row's lanes by vector-ALU butterflies.  A single token is a
// stream over the state (8 dk dv bytes a head; non-temporal, each byte is
// touched once): k_pk_step.  k_pk_rec stages more of them kStage at a time in
// LDS, the next stage's rows in flight while the current one is worked off.
constexpr int kRecThreads = 256;
constexpr int kStage = 8;
typedef float f32x4v __attribute__((ext_vector_type(4)));

// four consecutive input-typed elements, as loaded and as fp32
template <int DT>
using R4 = std::conditional_t<DT == GDN_BF16, u32x2, f32x4>;
template <int DT>
__device__ __forceinline__ R4<DT> ldr(const void* base, int64_t i) {
    if constexpr (DT == GDN_BF16) return *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(base) + i);
    else return *reinterpret_cast<const f32x4*>(static_cast<const float*>(base) + i);
}
template <int DT>
__device__ __forceinline__ f32x4 cvt(const R4<DT>& u) {
    if constexpr (DT == GDN_BF16)
        return f32x4{__uint_as_float(u[0] << 16), __uint_as_float(u[0] & 0xFFFF0000u), __uint_as_float(u[1] << 16),
                     __uint_as_float(u[1] & 0xFFFF0000u)};
    else return u;
}
template <int DT>
__device__ __forceinline__ f32x4 ld4e(const void* p, int64_t i) {
    return cvt<DT>(ldr<DT>(p, i));
}
__device__ __forceinline__ float dot4e(const f32x4& x, const f32x4& y) {
    return x[0] * y[0] + x[1] * y[1] + x[2] * y[2] + x[3] * y[3];
}
template <int DT>
__device__ __forceinline__ void st_out(void* out, int64_t i, float x) {
    if constexpr (DT == GDN_F32) static_cast<float*>(out)[i] = x;
    else static_cast<uint16_t*>(out)[i] = (uint16_t)pack_bf16(x, 0.f);
}

// S' and o of one token: k, q, g (the gate) in the lane's pieces, v of its rows
template <int LPR, int NP, int R>
__device__ __forceinline__ void rec_token(f32x4 (&S)[R][NP], const f32x4 (&k)[NP], const f32x4 (&q)[NP],
                                          const f32x4 (&g)[NP], const float (&v)[R], float beta, bool dtp, float scale,
                                          float (&o)[R]) {
    float pr[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
        pr[j] = 0.f;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            if (dtp) S[j][i] *= g[i];
            pr[j] += dot4e(S[j][i], k[i]);
        }
    }
#pragma unroll
    for (int j = 0; j < R; ++j) pr[j] = row_sum<LPR>(pr[j]);
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const float e = beta * (v[j] - pr[j]);
        o[j] = 0.f;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            S[j][i] = (dtp ? S[j][i] : S[j][i] * g[i]) + e * k[i];
            o[j] += dot4e(S[j][i], q[i]);
        }
    }
#pragma unroll
    for (int j = 0; j < R; ++j) o[j] = scale * row_sum<LPR>(o[j]);
}

// The workgroup's place: sequence, head, rows; and the state pieces of a thread
struct RecAt {
    int s, h, hk, rb;
    Span sp;
    const float* src;
    float* dst;
};
template <int RB>
__device__ __forceinline__ bool rec_at(const Pk& a, RecAt& x) {
    // workgroups go to the eight XCDs in turn: each XCD takes a run of
    // sequences of its own
    const unsigned nrb = ((unsigned)a.p.dv + RB - 1) / RB, one = nrb * a.Hv, run = 8 * one;
    const unsigned g = blockIdx.x / run, r = blockIdx.x - g * run;
    const unsigned block = (g + 1) * run <= gridDim.x ? g * run + (r % 8) * one + r / 8 : blockIdx.x;
    const unsigned id = block / nrb;
    x.rb = block - id * nrb;
    x.s = id / a.Hv;
    x.h = id - x.s * a.Hv;
    x.hk = x.h / a.group;
    x.sp = span_of(a.at, x.s);
    x.src = state_from(a.p, x.s, x.h);
    x.dst = state_to(a.p, x.s, x.h);
    return x.sp.n < a.rec_below && !(x.sp.n == 0 && x.src == x.dst);
}
template <int LPR, int NP, int R>
__device__ __forceinline__ void rec_load(const Packed& p, const RecAt& x, const int (&row)[R], int c, f32x4 (&S)[R][NP]) {
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int col = 4 * (c + LPR * i);
            S[j][i] = zero4();
            if (x.src && row[j] < (int)p.dv && col < (int)p.dk)
                S[j][i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4v*>(x.src + row[j] * (int)p.dk + col));
        }
}
template <int LPR, int NP, int R>
__device__ __forceinline__ void rec_store(const Packed& p, const RecAt& x, const int (&row)[R], int c, const f32x4 (&S)[R][NP]) {
    if (!x.dst) return;
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int col = 4 * (c + LPR * i);
            if (row[j] < (int)p.dv && col < (int)p.dk)
                __builtin_nontemporal_store((f32x4v)S[j][i], reinterpret_cast<f32x4v*>(x.dst + row[j] * (int)p.dk + col));
        }
}

// Single tokens: read straight from memory, in as few registers and no LDS, so
// that enough workgroups share a compute unit to keep the state's stream
// going (longer sequences are right, one token after the other).
template <int DT, int CH, int LPR, int R>
__global__ __launch_bounds__(kRecThreads) void k_pk_step(Pk a) {
    constexpr int RPW = 64 / LPR, RB = 4 * RPW * R;
    const Packed& p = a.p;
    RecAt x;
    if (!rec_at<RB>(a, x)) return;
    const int dk = (int)p.dk, dv = (int)p.dv;
    const int w = threadIdx.x >> 6, l = threadIdx.x & 63, c = l % LPR;
    const bool dtp = p.order == GDN_DECAY_THEN_PREDICT, on = 4 * c < dk;
    int row[R];
#pragma unroll
    for (int j = 0; j < R; ++j) row[j] = x.rb * RB + (j * 4 + w) * RPW + l / LPR;
    f32x4 S[R][1];
    rec_load<LPR, 1, R>(p, x, row, c, S);
    auto one = [&](int64_t t) {
        f32x4 k[1], q[1], g[1];
        float v[R], o[R];
        k[0] = on ? ld4e<DT>(p.k, t * p.k_stride + x.hk * dk + 4 * c) : zero4();
        q[0] = on ? ld4e<DT>(p.q, t * p.q_stride + x.hk * dk + 4 * c) : zero4();
        if constexpr (CH != 0) {
            g[0] = on ? *reinterpret_cast<const f32x4*>(p.alpha + (t * a.Hv + x.h) * dk + 4 * c) : zero4();
        } else {
            const float al = p.alpha[t * a.Hv + x.h];
            g[0] = f32x4{al, al, al, al};
        }
#pragma unroll
        for (int j = 0; j < R; ++j) v[j] = row[j] < dv ? gdn_ld<DT>(p.v, t * p.v_stride + x.h * dv + row[j]) : 0.f;
        rec_token<LPR, 1, R>(S, k, q, g, v, p.beta[t * a.Hv + x.h], dtp, p.scale, o);
#pragma unroll
        for (int j = 0; j < R; ++j)
            if (c == 0 && row[j] < dv) st_out<DT>(p.out, (t * a.Hv + x.h) * dv + row[j], o[j]);
    };
    if (x.sp.n == 1)
        one(x.sp.begin);
    else
        for (int64_t t = x.sp.begin; t < x.sp.begin + x.sp.n; ++t) one(t);
    rec_store<LPR, 1, R>(p, x, row, c, S);
}

template <int DT, int LPR, int NP, int R, bool CH>
struct RecShared {
    static constexpr int W = 4 * LPR * NP;                 // columns held
    static constexpr int RB = 4 * (64 / LPR) * R;          // rows of a workgroup
    R4<DT> k[2][kStage][W / 4], q[2][kStage][W / 4];
    f32x4 a[CH ? 2 : 1][CH ? kStage : 1][W / 4];
    float v[2][kStage][RB], o[2][kStage][RB];
    float sc[2][kStage][2];  // alpha (scalar gate), beta
};

template <int DT, int CH, int LPR, int NP, int R>
__global__ __launch_bounds__(kRecThreads) void k_pk_rec(Pk a) {
    using Sh = RecShared<DT, LPR, NP, R, CH != 0>;
    constexpr int RPW = 64 / LPR, RB = Sh::RB;
    __shared__ __attribute__((aligned(16))) Sh sh;
    const Packed& p = a.p;
    RecAt x;
    if (!rec_at<RB>(a, x)) return;
    const Span sp = x.sp;
    const int dk = (int)p.dk, dv = (int)p.dv, rb = x.rb, h = x.h, hk = x.hk;
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, c = l % LPR;
    const bool dtp = p.order == GDN_DECAY_THEN_PREDICT;
    int row[R];
#pragma unroll
    for (int j = 0; j < R; ++j) row[j] = rb * RB + (j * 4 + w) * RPW + l / LPR;
    f32x4 S[R][NP];
    rec_load<LPR, NP, R>(p, x, row, c, S);
    if (sp.n > 0) {
        const int pieces = dk / 4;  // of a row
        constexpr int KP = (kStage * Sh::W / 4 + kRecThreads - 1) / kRecThreads;
        constexpr int VP = (kStage * RB + kRecThreads - 1) / kRecThreads;
        R4<DT> kr[KP], qr[KP];
        f32x4 ar[CH ? KP : 1];
        float vr[VP], sr = 0.f;
        auto fetch = [&](int64_t t0) {
            const int m = (int)min<int64_t>(kStage, sp.n - t0);
#pragma unroll
            for (int i = 0; i < KP; ++i) {
                const int e = tid + kRecThreads * i, t = min(e / (Sh::W / 4), m - 1), pc = e % (Sh::W / 4);
                const bool on = pc < pieces;
                const int64_t tok = sp.begin + t0 + t;
                kr[i] = on ? ldr<DT>(p.k, tok * p.k_stride + hk * dk + 4 * pc) : R4<DT>{};
                qr[i] = on ? ldr<DT>(p.q, tok * p.q_stride + hk * dk + 4 * pc) : R4<DT>{};
                if constexpr (CH != 0)
                    ar[i] = on ? *reinterpret_cast<const f32x4*>(p.alpha + (tok * p.Hv + h) * dk + 4 * pc) : zero4();
            }
#pragma unroll
            for (int i = 0; i < VP; ++i) {
                const int e = tid + kRecThreads * i, t = min(e / RB, m - 1), r = rb * RB + e % RB;
                vr[i] = r < dv ? gdn_ld<DT>(p.v, (sp.begin + t0 + t) * p.v_stride + h * dv + r) : 0.f;
            }
            if (tid < 2 * kStage) {
                const int64_t at = (sp.begin + t0 + min(tid >> 1, m - 1)) * p.Hv + h;
                if (tid & 1) sr = p.beta[at];
                else if (!CH) sr = p.alpha[at];
            }
        };
        auto stage = [&](int b) {
#pragma unroll
            for (int i = 0; i < KP; ++i) {
                const int e = tid + kRecThreads * i;
                if (kStage * Sh::W / 4 % kRecThreads == 0 || e < kStage * Sh::W / 4) {
                    (&sh.k[b][0][0])[e] = kr[i];
                    (&sh.q[b][0][0])[e] = qr[i];
                    if constexpr (CH != 0) (&sh.a[b][0][0])[e] = ar[i];
                }
            }
#pragma unroll
            for (int i = 0; i < VP; ++i) {
                const int e = tid + kRecThreads * i;
                if (kStage * RB % kRecThreads == 0 || e < kStage * RB) (&sh.v[b][0][0])[e] = vr[i];
            }
            if (tid < 2 * kStage) (&sh.sc[b][0][0])[tid] = sr;
        };
        fetch(0);
        stage(0);
        __syncthreads();
        int b = 0;
        for (int64_t t0 = 0; t0 < sp.n; t0 += kStage, b ^= 1) {
            const bool more = t0 + kStage < sp.n;
            if (more) fetch(t0 + kStage);
            const int m = (int)min<int64_t>(kStage, sp.n - t0);
            for (int t = 0; t < m; ++t) {
                f32x4 k[NP], q[NP], g[NP];
                float v[R], o[R];
                const float al = sh.sc[b][t][0];
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    k[i] = cvt<DT>(sh.k[b][t][c + LPR * i]);
                    q[i] = cvt<DT>(sh.q[b][t][c + LPR * i]);
                    if constexpr (CH != 0) g[i] = sh.a[b][t][c + LPR * i];
                    else g[i] = f32x4{al, al, al, al};
                }
#pragma unroll
                for (int j = 0; j < R; ++j) v[j] = sh.v[b][t][row[j] - rb * RB];
                rec_token<LPR, NP, R>(S, k, q, g, v, sh.sc[b][t][1], dtp, p.scale, o);
#pragma unroll
                for (int j = 0; j < R; ++j)
                    if (c == 0) sh.o[b][t][row[j] - rb * RB] = o[j];
            }
            if (more) stage(b ^ 1);
            __syncthreads();  // the next stage is in place, this one's outputs are whole
            for (int e = tid; e < m * RB; e += kRecThreads) {
                const int t = e / RB, r = rb * RB + e % RB;
                if (r < dv) st_out<DT>(p.out, ((sp.begin + t0 + t) * p.Hv + h) * dv + r, sh.o[b][t][e % RB]);
            }
        }
    }
    rec_store<LPR, NP, R>(p, x, row, c, S);
}

template <int DT, int CH, int LPR, int NP, int R>
hipError_t launch_rec(const Pk& a, hipStream_t st) {
    constexpr int RB = 4 * (64 / LPR) * R;
    const int64_t blocks = a.p.S * a.p.Hv * ((a.p.dv + RB - 1) / RB);
    hipLaunchKernelGGL((k_pk_rec<DT, CH, LPR, NP, R>), dim3((unsigned)blocks), dim3(kRecThreads), 0, st, a);
    return hipGetLastError();
}
template <int DT, int CH, int LPR, int R>
hipError_t launch_step(const Pk& a, hipStream_t st) {
    constexpr int RB = 4 * (64 / LPR) * R;
    const int64_t blocks = a.p.S * a.p.Hv * ((a.p.dv + RB - 1) / RB);
    hipLaunchKernelGGL((k_pk_step<DT, CH, LPR, R>), dim3((unsigned)blocks), dim3(kRecThreads), 0, st, a);
    return hipGetLastError();
}
template <int DT, int CH>
hipError_t launch_rec_shape(const Pk& a, hipStream_t st) {
    const int64_t pieces = a.p.dk / 4;
    if (std::min(a.p.max_len, a.p.N) <= 1) {
        if (pieces <= 8) return launch_step<DT, CH, 8, 4>(a, st);
        if (pieces <= 16) return launch_step<DT, CH, 16, 4>(a, st);
        return launch_step<DT, CH, 32, 4>(a, st);
    }
    if (pieces <= 8) return launch_rec<DT, CH, 8, 1, 2>(a, st);
    if (pieces <= 16) return launch_rec<DT, CH, 16, 1, 2>(a, st);
    return launch_rec<DT, CH, 16, 2, 2>(a, st);
}

// ---------------------------------------------------------------------------
// chunk form
// ---------------------------------------------------------------------------
// Gate rows of a chunk (floats): gamma, gamma', gamma_C / gamma, the log
// prefix as hi + lo, gamma_C.
constexpr int kGgam = 0, kGgamp = 64, kGtail = 128, kGhi = 192, kGlo = 256, kGlast = 320, kGate = 324;
constexpr int kGatePieces = kGate / 4;
constexpr int kTblk = 10 * 256;  // floats of T' per chunk: lower blocks (m, j), j <= m
constexpr int LDA = C + 4;
__device__ __forceinline__ constexpr int tblk(int m, int j) { return m * (m + 1) / 2 + j; }

// A log gate of a zero gate: low enough that every product over it is zero
// in fp32, finite so that the prefix of the tokens behind it stays exact (it
// is a compensated pair; their ratios cancel it)
constexpr float kLogZero = -256.f;

// x = hi + mid + lo, bf16 each, to the last bit of fp32: both remainders are
// exact (as in split2), so a product with an exact bf16 operand in three
// instructions keeps fp32's accuracy.  (Two terms leave 2^-18 of each
// element, 2e-6 of the state on a long sequence where fp32 arithmetic
// leaves 3e-7.)
__device__ __forceinline__ void split3_2(float a, float b, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    const bf16x2_t m0 = {(__bf16)-1.f, (__bf16)-0.f}, m1 = {(__bf16)-0.f, (__bf16)-1.f};
    hi = pack_bf16(a, b);
    const bf16x2_t h = __builtin_bit_cast(bf16x2_t, hi);
    const float ra = __builtin_amdgcn_fdot2_f32_bf16(h, m0, a, false), rb = __builtin_amdgcn_fdot2_f32_bf16(h, m1, b, false);
    mid = pack_bf16(ra, rb);
    const bf16x2_t m = __builtin_bit_cast(bf16x2_t, mid);
    lo = pack_bf16(__builtin_amdgcn_fdot2_f32_bf16(m, m0, ra, false), __builtin_amdgcn_fdot2_f32_bf16(m, m1, rb, false));
}
struct Split3 {
    u16x4 h, m, l;
};
__device__ __forceinline__ Split3 split3(const f32x4& x) {
    uint32_t h0, m0, l0, h1, m1, l1;
    split3_2(x[0], x[1], h0, m0, l0);
    split3_2(x[2], x[3], h1, m1, l1);
    return {__builtin_bit_cast(u16x4, uint2{h0, h1}), __builtin_bit_cast(u16x4, uint2{m0, m1}),
            __builtin_bit_cast(u16x4, uint2{l0, l1})};
}
// acc += A B over a 16 x 16 x 16 fp32 block (a: row c16, four consecutive
// contraction indices; b: an accumulator tile as it stands)
__device__ __forceinline__ f32x4 blk(const f32x4& a, const f32x4& b, f32x4 acc) {
#pragma unroll
    for (int q = 0; q < 4; ++q) acc = mfma_f32(a[q], b[q], acc);
    return acc;
}

// Per chunk and value head: the gate rows and T'.  One workgroup of four
// waves each; K K^T on bf16 MFMA (exact operands), the inverse in fp32.
template <int D>
__global__ __launch_bounds__(kThreads) void k_pk_prep(Pk a) {
    constexpr int LDK = D + 8, PPR = D / 8, KP = C * PPR / kThreads;
    static_assert(C * LDK * 2 <= C * LDA * 4, "K rows fit the tile");
    __shared__ __attribute__((aligned(16))) float AT[C * LDA];
    __shared__ __attribute__((aligned(16))) float ghi[C], glo[C], gphi[C], gplo[C], gbeta[C];
    const Packed& p = a.p;
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, g4 = l >> 4, c16 = l & 15;
    const int place = blockIdx.x / a.Hv, h = blockIdx.x - place * a.Hv, hk = h / a.group;
    const int64_t s = seq_of_place(a.at, place, 6, l);
    const Span sp = span_of(a.at, s);
    const int64_t c = place - ((sp.begin >> 6) + s);
    if (sp.n < kChunkMin || c < 0 || c * C >= sp.n) return;
    const int64_t t0 = sp.begin + c * C;
    const int nt = (int)min<int64_t>(C, sp.n - c * C);
    const uint16_t* kin = static_cast<const uint16_t*>(p.k) + hk * D;
    uint16_t* Ks = reinterpret_cast<uint16_t*>(AT);
    u32x4 kv[KP];
#pragma unroll
    for (int i = 0; i < KP; ++i) {
        const int e = tid + kThreads * i, t = min(e / PPR, nt - 1), c8 = e % PPR;
        kv[i] = ld_g<u32x4>(kin + (t0 + t) * p.k_stride + c8 * 8);
    }
    if (w == 0) {
        const int64_t r = (t0 + min(l, nt - 1)) * p.Hv + h;
        const float al = p.alpha[r];
        float la = l < nt ? logf(al) : 0.f;
        la = la < kLogZero ? kLogZero : la;
        const Gate g = gate_prefix(la, al, p.beta[r], nt, p.order, l);
        ghi[l] = g.hi;
        glo[l] = g.lo;
        gphi[l] = g.phi;
        gplo[l] = g.plo;
        gbeta[l] = g.beta;
    }
#pragma unroll
    for (int i = 0; i < KP; ++i) {
        const int e = tid + kThreads * i, t = e / PPR, c8 = e % PPR;
        *reinterpret_cast<u32x4*>(&Ks[t * LDK + c8 * 8]) = t < nt ? kv[i] : u32x4{0, 0, 0, 0};
    }
    __syncthreads();
    if (w == 0) {
        float* G = a.G + (int64_t)blockIdx.x * kGate;
        G[kGgam + l] = __expf(ghi[l] + glo[l]);
        G[kGgamp + l] = __expf(gphi[l] + gplo[l]);
        G[kGtail + l] = ratio(ghi[C - 1], glo[C - 1], ghi[l], glo[l]);
        G[kGhi + l] = ghi[l];
        G[kGlo + l] = glo[l];
        if (l < 4) G[kGlast + l] = __expf(ghi[C - 1] + glo[C - 1]);
    }
    auto krow = [&](int m, int k) { return *reinterpret_cast<const u16x8*>(&Ks[(16 * m + c16) * LDK + 32 * k + 8 * g4]); };
    // Gram blocks (m, n), n <= m, dealt 3, 3, 2, 2 over the waves
    f32x4 acc[3];
    int bm[3], bn[3], nbk;
    if (w == 0) { bm[0] = 0; bn[0] = 0; bm[1] = 3; bn[1] = 0; bm[2] = 3; bn[2] = 1; nbk = 3; }
    else if (w == 1) { bm[0] = 1; bn[0] = 0; bm[1] = 1; bn[1] = 1; bm[2] = 3; bn[2] = 2; nbk = 3; }
    else if (w == 2) { bm[0] = 2; bn[0] = 0; bm[1] = 2; bn[1] = 1; bm[2] = 0; bn[2] = 0; nbk = 2; }
    else { bm[0] = 2; bn[0] = 2; bm[1] = 3; bn[1] = 3; bm[2] = 0; bn[2] = 0; nbk = 2; }
#pragma unroll
    for (int q = 0; q < 3; ++q) {
        acc[q] = zero4();
        if (q >= nbk) continue;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) acc[q] = mfma(krow(bm[q], k), krow(bn[q], k), acc[q]);
    }
    __syncthreads();  // the K rows are dead: the tile takes A, as the inverse wants it
#pragma unroll
    for (int q = 0; q < 3; ++q) {
        if (q >= nbk) continue;
        const int m = bm[q], nb = bn[q], j = 16 * nb + c16;
        f32x4 x;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = 16 * m + 4 * g4 + r;
            x[r] = j < t ? gbeta[t] * ratio(gphi[t], gplo[t], ghi[j], glo[j]) * acc[q][r] : 0.f;
        }
        if (nb < m) {
            *reinterpret_cast<f32x4*>(&AT[j * LDA + 16 * m + 4 * g4]) = x;
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) AT[(16 * m + 4 * g4 + r) * LDA + j] = x[r];
        }
    }
    __syncthreads();
    ut_inverse_lds(AT, tid);
    float* T = a.T + (int64_t)blockIdx.x * kTblk;
    for (int e = tid; e < kTblk / 4; e += kThreads) {
        const int b = e >> 6, i = (e & 63) >> 2, j4 = 4 * (e & 3);
        const int m = b >= 6 ? 3 : b >= 3 ? 2 : b >= 1 ? 1 : 0, nb = b - m * (m + 1) / 2;
        const f32x4 x = *reinterpret_cast<const f32x4*>(&AT[(16 * m + i) * LDA + 16 * nb + j4]) *
                        *reinterpret_cast<const f32x4*>(&gbeta[16 * nb + j4]);
        st_g(T + 4 * e, x);
    }
}

// LDS of a segment's workgroup.  K and Q rows are kept with the columns of
// every 32-column block permuted, 16 h + 4 g + r -> 8 g + 4 h + r, so that the
// eight key slots of lane group g in the order two accumulator tiles supply
// them are 16 contiguous bytes.
template <int D, bool OUT>
struct SegShared {
    static constexpr int LDK = D + 8;
    unsigned short K[C * LDK];
    unsigned short V[C * LDK];
    u16x8 KtF[D / 16][2][64];  // K^T as A operands: [key tile][32 tokens][lane]
    f32x4 T[kTblk / 4];
    float G[kGate];
    unsigned short Q[OUT ? C * LDK : 8];
    u16x8 Pf[OUT ? 4 : 1][2][2][64];  // P as A operands, hi and lo
    unsigned short O[OUT ? C * LDK : 8];
};
template <int D>
constexpr int seg_threads() { return 4 * D; }

// One segment of one value head.  Wave w holds value columns 16 w .. of S^T
// for every key (accumulator tiles; they serve as the next product's operand
// as they stand), so nothing but the staged chunk is shared between waves.
// OUT: from the segment's start state, with outputs; the last segment writes
// the end state.  Otherwise the state pass: from zero (segment 0: from the
// sequence's start state, which it also copies for the output pass, so that
// the end state may go where the start state was), beside the same columns
// of M from I (the recurrence with V = 0); end values only.
template <int D, bool OUT>
__global__ __launch_bounds__(seg_threads<D>(), D == 128 ? 2 : 2) void k_pk_seg(Pk a) {
    constexpr int NV = OUT ? 1 : 2;  // states a wave carries: S, M
    constexpr int NW = D / 16, NT = 64 * NW, LDK = SegShared<D, OUT>::LDK;
    constexpr int KS = D / 32, TPW = D / 16, PPR = D / 8, KP = C * PPR / NT;
    constexpr int TP = (kTblk / 4 + NT - 1) / NT;
    static_assert(C * PPR % NT == 0 && kGatePieces <= NT && (2 * TPW) % NW == 0, "staging split");
    __shared__ __attribute__((aligned(16))) SegShared<D, OUT> sh;
    const Packed& p = a.p;
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, g4 = l >> 4, c16 = l & 15;
    const int place = blockIdx.x / a.Hv, h = blockIdx.x - place * a.Hv, hk = h / a.group;
    const int64_t s = seq_of_place(a.at, place, a.seg_shift, l);
    const Span sp = span_of(a.at, s);
    const int64_t base = (sp.begin >> a.seg_shift) + s;  // the sequence's first place
    const int64_t gi = place - base, ng = (sp.n + ((int64_t)1 << a.seg_shift) - 1) >> a.seg_shift;
    if (sp.n < kChunkMin || gi < 0 || gi >= ng || (!OUT && gi == ng - 1)) return;
    const int64_t per = (int64_t)1 << (a.seg_shift - 6);  // chunks of a segment
    const int64_t i_begin = gi * per, i_end = min<int64_t>((sp.n + C - 1) / C, i_begin + per);
    const int64_t cplace = (sp.begin >> 6) + s;  // the sequence's first chunk place
    const uint16_t* kin = static_cast<const uint16_t*>(p.k) + hk * D;
    const uint16_t* qin = static_cast<const uint16_t*>(p.q) + hk * D;
    const uint16_t* vin = static_cast<const uint16_t*>(p.v) + h * D;
    auto in_ws = [&](float* pool, int64_t pl) { return pool + (pl * p.Hv + h) * D * D; };

    const int v = 16 * w + c16;  // this lane's value column
    f32x4 Sacc[NV][TPW];         // [state][key tile]: rows 16 u + 4 g4 + r of column v
    {
        const float* src = OUT && ng > 1 ? in_ws(a.s_start, place) : gi == 0 ? state_from(p, s, h) : nullptr;
#pragma unroll
        for (int u = 0; u < TPW; ++u) {
            const int a0 = 16 * u + 4 * g4;
            Sacc[0][u] = src ? *reinterpret_cast<const f32x4*>(src + (int64_t)v * D + a0) : zero4();
            if constexpr (!OUT) {
                if (gi == 0) *reinterpret_cast<f32x4*>(in_ws(a.s_start, place) + (int64_t)v * D + a0) = Sacc[0][u];
#pragma unroll
                for (int r = 0; r < 4; ++r) Sacc[NV - 1][u][r] = v == a0 + r ? 1.f : 0.f;
            }
        }
    }

    // staging: the next chunk in registers while this one is worked off
    u32x4 kr[KP], vr[KP], qr[OUT ? KP : 1];
    f32x4 tr[TP], gr;
    auto issue = [&](int64_t i, int parts) {  // 1: K, V; 2: Q, T', gate rows
        const int64_t t0 = sp.begin + i * C;
        const int nt = (int)min<int64_t>(C, sp.n - i * C);
#pragma unroll
        for (int k = 0; k < KP; ++k) {
            const int e = tid + NT * k, t = min(e / PPR, nt - 1), c8 = e % PPR;
            if (parts & 1) {
                kr[k] = ld_g<u32x4>(kin + (t0 + t) * p.k_stride + c8 * 8);
                vr[k] = ld_g<u32x4>(vin + (t0 + t) * p.v_stride + c8 * 8);
            }
            if (OUT && (parts & 2)) qr[k] = ld_g<u32x4>(qin + (t0 + t) * p.q_stride + c8 * 8);
        }
        if (parts & 2) {
            const int64_t ch = (cplace + i) * p.Hv + h;
#pragma unroll
            for (int k = 0; k < TP; ++k) tr[k] = ld_g<f32x4>(a.T + ch * kTblk + 4 * min(tid + NT * k, kTblk / 4 - 1));
            gr = ld_g<f32x4>(a.G + ch * kGate + 4 * min(tid, kGatePieces - 1));
        }
    };
    auto store = [&](int64_t i) {
        const int nt = (int)min<int64_t>(C, sp.n - i * C);
        const u32x4 z = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < KP; ++k) {
            const int e = tid + NT * k, t = e / PPR, c8 = e % PPR;
            const bool ok = t < nt;
            *reinterpret_cast<u32x4*>(&sh.V[t * LDK + c8 * 8]) = ok ? vr[k] : z;
            const int p0 = t * LDK + 32 * (c8 >> 2) + 16 * (c8 & 1) + 4 * ((c8 >> 1) & 1);
            const u32x4 kk = ok ? kr[k] : z;
            *reinterpret_cast<u32x2*>(&sh.K[p0]) = u32x2{kk[0], kk[1]};
            *reinterpret_cast<u32x2*>(&sh.K[p0 + 8]) = u32x2{kk[2], kk[3]};
            if (OUT) {
                const u32x4 qq = ok ? qr[k] : z;
                *reinterpret_cast<u32x2*>(&sh.Q[p0]) = u32x2{qq[0], qq[1]};
                *reinterpret_cast<u32x2*>(&sh.Q[p0 + 8]) = u32x2{qq[2], qq[3]};
            }
        }
#pragma unroll
        for (int k = 0; k < TP; ++k)
            if (kTblk / 4 % NT == 0 || tid + NT * k < kTblk / 4) sh.T[tid + NT * k] = tr[k];
        if (tid < kGatePieces) *reinterpret_cast<f32x4*>(&sh.G[4 * tid]) = gr;
    };
    // P blocks (m, c), c <= m, dealt over the waves: rows j of tile c, columns
    // t of tile m, so that two blocks form an A operand as they stand
    auto scores = [&]() {
        for (int bi = w; bi < 10; bi += NW) {
            const int m = bi >= 6 ? 3 : bi >= 3 ? 2 : bi >= 1 ? 1 : 0, c = bi - m * (m + 1) / 2, t = 16 * m + c16;
            f32x4 acc = zero4();
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const u16x8 ka = *reinterpret_cast<const u16x8*>(&sh.K[(16 * c + c16) * LDK + 32 * k + 8 * g4]);
                const u16x8 qb = *reinterpret_cast<const u16x8*>(&sh.Q[t * LDK + 32 * k + 8 * g4]);
                acc = mfma(ka, qb, acc);
            }
            const float th = sh.G[kGhi + t], tl = sh.G[kGlo + t];
            const f32x4 jh = *reinterpret_cast<const f32x4*>(&sh.G[kGhi + 16 * c + 4 * g4]);
            const f32x4 jl = *reinterpret_cast<const f32x4*>(&sh.G[kGlo + 16 * c + 4 * g4]);
            f32x4 pt;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                pt[r] = 16 * c + 4 * g4 + r <= t ? acc[r] * ratio(th, tl, jh[r], jl[r]) : 0.f;
            u16x4 hi, lo;
            split4(pt, hi, lo);
            reinterpret_cast<u16x4*>(&sh.Pf[m][c >> 1][0][l])[c & 1] = hi;
            reinterpret_cast<u16x4*>(&sh.Pf[m][c >> 1][1][l])[c & 1] = lo;
        }
    };
    if constexpr (OUT) {
        // the halves of P's operands above the diagonal, never written again
        if (w == 0) {
            const u16x4 z = u16x4{0, 0, 0, 0};
#pragma unroll
            for (int hl = 0; hl < 2; ++hl) {
                reinterpret_cast<u16x4*>(&sh.Pf[0][0][hl][l])[1] = z;
                reinterpret_cast<u16x4*>(&sh.Pf[2][1][hl][l])[1] = z;
            }
        }
    }
    auto flush = [&](int64_t i) {  // the output tile of chunk i, rows past the end dropped
        const int64_t t0 = sp.begin + i * C;
        const int nt = (int)min<int64_t>(C, sp.n - i * C);
        uint16_t* ob = static_cast<uint16_t*>(p.out) + h * D;
#pragma unroll
        for (int k = 0; k < KP; ++k) {
            const int e = tid + NT * k, t = e / PPR, c8 = e % PPR;
            if (t < nt)
                __builtin_nontemporal_store(*reinterpret_cast<const u32x4*>(&sh.O[t * LDK + 8 * c8]),
                                            reinterpret_cast<u32x4*>(ob + (t0 + t) * p.Hv * D + 8 * c8));
        }
    };
    // an identity operand: lane (column c16) is one where the slot holds key
    // 16 hh + c16 of the 32-key block
    auto idfrag = [&](int hh) {
        u16x8 f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = ((e >> 2) == hh && 4 * g4 + (e & 3) == c16) ? (unsigned short)0x3F80 : (unsigned short)0;
        return f;
    };

    issue(i_begin, 3);
    store(i_begin);
    for (int64_t i = i_begin; i < i_end; ++i) {
        __syncthreads();  // chunk i staged
        const bool more = i + 1 < i_end;
        if (OUT && more) issue(i + 1, 1);
        if constexpr (OUT) scores();
        // K^T as A operands, by exact products with the identity
#pragma unroll
        for (int jj = 0; jj < 2 * TPW / NW; ++jj) {
            const int job = w + NW * jj, tp = job & 1, u = job >> 1;
            u16x4 half[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const u16x8 ka = *reinterpret_cast<const u16x8*>(&sh.K[(16 * (2 * tp + q) + c16) * LDK + 32 * (u >> 1) + 8 * g4]);
                const f32x4 d = mfma(ka, idfrag(u & 1), zero4());
#pragma unroll
                for (int r = 0; r < 4; ++r) half[q][r] = (unsigned short)(__float_as_uint(d[r]) >> 16);
            }
            sh.KtF[u][tp][l] = cat(half[0], half[1]);
        }
        // X = K S^T, S in three terms; Z = Q S^T, S in two (its error, 2^-18,
        // is far below the bf16 rounding of the output)
        f32x4 X[NV][4], Z[OUT ? 4 : 1];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
#pragma unroll
            for (int n = 0; n < NV; ++n) X[n][m] = zero4();
            if constexpr (OUT) Z[m] = zero4();
        }
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            u16x8 bh[NV], bm[NV], bl[NV];
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                const Split3 x = split3(Sacc[n][2 * k]), y = split3(Sacc[n][2 * k + 1]);
                bh[n] = cat(x.h, y.h);
                bm[n] = cat(x.m, y.m);
                bl[n] = cat(x.l, y.l);
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const u16x8 ra = *reinterpret_cast<const u16x8*>(&sh.K[(16 * m + c16) * LDK + 32 * k + 8 * g4]);
#pragma unroll
                for (int n = 0; n < NV; ++n) {
                    X[n][m] = mfma(ra, bl[n], X[n][m]);
                    X[n][m] = mfma(ra, bm[n], X[n][m]);
                    X[n][m] = mfma(ra, bh[n], X[n][m]);
                }
                if constexpr (OUT) {
                    const u16x8 qa = *reinterpret_cast<const u16x8*>(&sh.Q[(16 * m + c16) * LDK + 32 * k + 8 * g4]);
                    Z[m] = mfma(qa, bm[0], Z[m]);
                    Z[m] = mfma(qa, bh[0], Z[m]);
                }
            }
        }
        if (more) issue(i + 1, OUT ? 2 : 3);
        // U = V - diag(gamma') X
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const f32x4 gp = *reinterpret_cast<const f32x4*>(&sh.G[kGgamp + 16 * m + 4 * g4]);
#pragma unroll
            for (int n = 0; n < NV; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float vv = n == 1 ? 0.f : gdn_bf16_to_f32(sh.V[(16 * m + 4 * g4 + r) * LDK + v]);
                    X[n][m][r] = vv - gp[r] * X[n][m][r];
                }
        }
        if constexpr (OUT)
            if (i > i_begin) flush(i - 1);
        // Delta = T' U in fp32; its two terms for the output, and
        // diag(gamma_C / gamma) Delta in three for the state
        u16x4 dh[OUT ? 4 : 1], dl[OUT ? 4 : 1];
        Split3 db[NV][4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            f32x4 d[NV];
#pragma unroll
            for (int n = 0; n < NV; ++n) d[n] = zero4();
#pragma unroll
            for (int j = 0; j <= m; ++j) {
                const f32x4 ta = sh.T[tblk(m, j) * 64 + c16 * 4 + g4];
#pragma unroll
                for (int n = 0; n < NV; ++n) d[n] = blk(ta, X[n][j], d[n]);
            }
            const f32x4 tail = *reinterpret_cast<const f32x4*>(&sh.G[kGtail + 16 * m + 4 * g4]);
            if constexpr (OUT) split4(d[0], dh[m], dl[m]);
#pragma unroll
            for (int n = 0; n < NV; ++n) db[n][m] = split3(tail * d[n]);
        }
        __syncthreads();  // the operands of K^T and P are whole
        const float gC = sh.G[kGlast];
#pragma unroll
        for (int u = 0; u < TPW; ++u) {
            f32x4 acc[NV];
#pragma unroll
            for (int n = 0; n < NV; ++n) acc[n] = gC * Sacc[n][u];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const u16x8 ka = sh.KtF[u][k][l];
#pragma unroll
                for (int n = 0; n < NV; ++n) {
                    acc[n] = mfma(ka, cat(db[n][2 * k].l, db[n][2 * k + 1].l), acc[n]);
                    acc[n] = mfma(ka, cat(db[n][2 * k].m, db[n][2 * k + 1].m), acc[n]);
                    acc[n] = mfma(ka, cat(db[n][2 * k].h, db[n][2 * k + 1].h), acc[n]);
                }
            }
#pragma unroll
            for (int n = 0; n < NV; ++n) Sacc[n][u] = acc[n];
        }
        // O = scale (diag(gamma) Z + P Delta), rounded once to bf16
        if constexpr (OUT) {
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                f32x4 o = zero4();
#pragma unroll
                for (int k = 0; k <= (m >> 1); ++k) {
                    const u16x8 ph = sh.Pf[m][k][0][l], pl = sh.Pf[m][k][1][l];
                    const u16x8 xh = cat(dh[2 * k], dh[2 * k + 1]), xl = cat(dl[2 * k], dl[2 * k + 1]);
                    o = mfma(pl, xh, o);
                    o = mfma(ph, xl, o);
                    o = mfma(ph, xh, o);
                }
                const f32x4 gam = *reinterpret_cast<const f32x4*>(&sh.G[kGgam + 16 * m + 4 * g4]);
                const f32x4 y = p.scale * (gam * Z[m] + o);
                const uint32_t y01 = pack_bf16(y[0], y[1]), y23 = pack_bf16(y[2], y[3]);
                sh.O[(16 * m + 4 * g4 + 0) * LDK + v] = (unsigned short)y01;
                sh.O[(16 * m + 4 * g4 + 1) * LDK + v] = (unsigned short)(y01 >> 16);
                sh.O[(16 * m + 4 * g4 + 2) * LDK + v] = (unsigned short)y23;
                sh.O[(16 * m + 4 * g4 + 3) * LDK + v] = (unsigned short)(y23 >> 16);
            }
        }
        __syncthreads();  // chunk i is worked off, its output tile whole
        if (more) store(i + 1);
    }
    if constexpr (OUT) {
        flush(i_end - 1);
        float* dst = gi == ng - 1 ? state_to(p, s, h) : nullptr;
        if (dst) {
#pragma unroll
            for (int u = 0; u < TPW; ++u)
                *reinterpret_cast<f32x4*>(dst + (int64_t)v * D + 16 * u + 4 * g4) = Sacc[0][u];
        }
    } else {
        float* dst = in_ws(a.s_end, place);
        float* mt = in_ws(a.m_end, place);  // M^T: row key (of the end state), column v
#pragma unroll
        for (int u = 0; u < TPW; ++u) {
            *reinterpret_cast<f32x4*>(dst + (int64_t)v * D + 16 * u + 4 * g4) = Sacc[0][u];
#pragma unroll
            for (int r = 0; r < 4; ++r) mt[(16 * u + 4 * g4 + r) * D + v] = Sacc[NV - 1][u][r];
        }
    }
}

// Start states of a sequence's segments: X <- S_end(g) + X M(g), sixteen rows
// of one head a workgroup (rows are independent), wave w the columns 16 w ..;
// fp32 MFMA, the next three matrices in flight while one multiplies.
template <int D>
__global__ __launch_bounds__(4 * D, 2) void k_pk_chain(Pk a) {
    constexpr int NB = D / 16, LDX = D + 4;
    __shared__ __attribute__((aligned(16))) float X[2][16 * LDX];
    const Packed& p = a.p;
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, g4 = l >> 4, c16 = l & 15;
    const int rt = blockIdx.x % NB;
    const int sh_id = blockIdx.x / NB, s = sh_id / a.Hv, h = sh_id - s * a.Hv;
    const Span sp = span_of(a.at, s);
    const int64_t ng = (sp.n + ((int64_t)1 << a.seg_shift) - 1) >> a.seg_shift;
    if (sp.n < kChunkMin || ng < 2) return;
    const int64_t base = (sp.begin >> a.seg_shift) + s;
    auto at = [&](float* pool, int64_t g) { return pool + ((base + g) * p.Hv + h) * D * D; };
    // rows 4 g4 + r of the sixteen, column 16 w + c16
    const int col = 16 * w + c16;
    auto rows = [&](const float* m) {
        f32x4 x;
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = m[(int64_t)(16 * rt + 4 * g4 + r) * D + col];
        return x;
    };
    f32x4 x = rows(at(a.s_end, 0));
    struct In {
        f32x4 m[NB], add;
    };
    auto fetch = [&](In& in, int64_t g) {
        g = min(g, ng - 1 > 1 ? ng - 2 : (int64_t)0);
        const float* m = at(a.m_end, g) + (int64_t)col * D;
#pragma unroll
        for (int k = 0; k < NB; ++k) in.m[k] = ld_g<f32x4>(m + 16 * k + 4 * g4);
        in.add = rows(at(a.s_end, g));
    };
    // step g: the start state of segment g, then X M(g) + S_end(g)
    auto step = [&](int64_t g, const In& in) {
        float* dst = at(a.s_start, g);
#pragma unroll
        for (int r = 0; r < 4; ++r) dst[(int64_t)(16 * rt + 4 * g4 + r) * D + col] = x[r];
        float* Xs = X[g & 1];
#pragma unroll
        for (int r = 0; r < 4; ++r) Xs[(4 * g4 + r) * LDX + col] = x[r];
        __syncthreads();
        f32x4 acc = in.add, acc2 = zero4();
#pragma unroll
        for (int k = 0; k < NB; k += 2) {
            acc = blk(*reinterpret_cast<const f32x4*>(&Xs[c16 * LDX + 16 * k + 4 * g4]), in.m[k], acc);
            acc2 = blk(*reinterpret_cast<const f32x4*>(&Xs[c16 * LDX + 16 * (k + 1) + 4 * g4]), in.m[k + 1], acc2);
        }
        x = acc + acc2;
    };
    if (ng > 2) {
        // four matrices in flight (each step fetches the one three steps on)
        In in[4];
        fetch(in[0], 1);
        fetch(in[1], 2);
        fetch(in[2], 3);
        for (int64_t g = 1; g < ng - 1; g += 4) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (g + u >= ng - 1) break;
                fetch(in[(u + 3) & 3], g + u + 3);
                step(g + u, in[u]);
            }
        }
    }
    float* dst = at(a.s_start, ng - 1);
#pragma unroll
    for (int r = 0; r < 4; ++r) dst[(int64_t)(16 * rt + 4 * g4 + r) * D + col] = x[r];
}

// Tokens of a segment, as a power of two: as many segments as fill the
// compute units once over all heads, at least kSegMin chunks each.
constexpr int kSegMinShift = 6 + 3;
constexpr int kWhole = 31;  // a sequence's tokens are fewer than 2^31
int seg_shift_for(const Packed& p) {
    const int64_t want = std::max<int64_t>(1, p.N * p.Hv / 256);  // tokens a workgroup
    int sh = kSegMinShift;
    while (((int64_t)1 << sh) < want && sh < 30) ++sh;
    return sh;
}
int64_t longest(const Packed& p) { return std::min(p.N, p.max_len); }

struct PkLayout {
    size_t T, G, s_end, m_end, s_start, total;
};
PkLayout layout(const Packed& p) {
    PkLayout L{};
    if (!packed_chunked(p) || longest(p) < kChunkMin) return L;
    const size_t chunks = (size_t)(p.N / C + p.S) * (size_t)p.Hv;
    size_t off = 0;
    auto take = [&](size_t floats) {
        const size_t at = off;
        off += align256(floats * sizeof(float));
        return at;
    };
    L.T = take(chunks * kTblk);
    L.G = take(chunks * kGate);
    const int sh = seg_shift_for(p);
    if (longest(p) > ((int64_t)1 << sh)) {
        const size_t states = (size_t)((p.N >> sh) + p.S) * (size_t)p.Hv * (size_t)(p.dk * p.dk);
        L.s_end = take(states);
        L.m_end = take(states);
        L.s_start = take(states);
    }
    L.total = off;
    return L;
}

template <int D>
hipError_t launch_chunks(const Pk& a, bool segments, hipStream_t st) {
    const Packed& p = a.p;
    prof_begin(p.timer, "k_pk_prep", st);
    hipLaunchKernelGGL(k_pk_prep<D>, dim3((unsigned)(a.nslot * p.Hv)), dim3(kThreads), 0, st, a);
    prof_end(p.timer, st);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)(a.nseg * p.Hv)), block(seg_threads<D>());
    if (segments) {
        prof_begin(p.timer, "k_pk_state", st);
        hipLaunchKernelGGL((k_pk_seg<D, false>), grid, block, 0, st, a);
        prof_end(p.timer, st);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        prof_begin(p.timer, "k_pk_chain", st);
        hipLaunchKernelGGL(k_pk_chain<D>, dim3((unsigned)(p.S * p.Hv * (D / 16))), dim3(4 * D), 0, st, a);
        prof_end(p.timer, st);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    prof_begin(p.timer, "k_pk_out", st);
    hipLaunchKernelGGL((k_pk_seg<D, true>), grid, block, 0, st, a);
    prof_end(p.timer, st);
    return hipGetLastError();
}

}  // namespace

bool packed_chunked(const Packed& p) {
    return p.dtype == GDN_BF16 && p.gate == GDN_GATE_SCALAR && p.dk == p.dv && (p.dk == 64 || p.dk == 128);
}

size_t packed_workspace(const Packed& p) { return layout(p).total; }

hipError_t packed_forward(const Packed& p, void* ws, hipStream_t st) {
    Pk a{};
    a.p = p;
    a.at = {p.cu, p.N, p.S};
    a.Hv = (int)p.Hv;
    a.group = (int)(p.Hv / p.Hk);
    const PkLayout L = layout(p);
    const bool chunks = L.total > 0;
    a.rec_below = chunks ? kChunkMin : INT32_MAX;
    prof_begin(p.timer, "k_pk_rec", st);
    hipError_t e;
    if (p.dtype == GDN_BF16)
        e = p.gate == GDN_GATE_CHANNEL ? launch_rec_shape<GDN_BF16, 1>(a, st) : launch_rec_shape<GDN_BF16, 0>(a, st);
    else
        e = p.gate == GDN_GATE_CHANNEL ? launch_rec_shape<GDN_F32, 1>(a, st) : launch_rec_shape<GDN_F32, 0>(a, st);
    prof_end(p.timer, st);
    if (e != hipSuccess || !chunks) return e;
    char* base = static_cast<char*>(ws);
    // without segments every sequence is one, whatever its length (max_len
    // is the caller's word, the lengths are the device's)
    const bool segments = longest(p) > ((int64_t)1 << seg_shift_for(p));
    a.seg_shift = segments ? seg_shift_for(p) : kWhole;
    a.nslot = p.N / C + p.S;
    a.nseg = (p.N >> a.seg_shift) + p.S;
    a.T = reinterpret_cast<float*>(base + L.T);
    a.G = reinterpret_cast<float*>(base + L.G);
    a.s_end = reinterpret_cast<float*>(base + L.s_end);
    a.m_end = reinterpret_cast<float*>(base + L.m_end);
    a.s_start = reinterpret_cast<float*>(base + L.s_start);
    return p.dk == 64 ? launch_chunks<64>(a, segments, st) : launch_chunks<128>(a, segments, st);
}

}  // namespace gdn
