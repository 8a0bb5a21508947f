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
//   token by token, the state in registers (k_pk_step, k_pk_rec): steps of a
//     generation, drafted tokens, short prompts, and every shape without chunk
//     kernels;
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
//     the sequence-parallel notes' increment and correction, as a two-level
//     scan where it is long) and the output pass from the true start states.
// Measured (bf16, D = 128): 40 sequences of very different lengths, 16384
// tokens, 16 value heads, 298 us a call (preparation 64, state pass 77, chain
// 18, outputs 148; the bytes alone 47 us); one of 65531, 4 heads, 394 us (47,
// 118, 103, 147; bytes 45 us).  (Calls are timed with inputs that are not in the
// caches; kernels are averages under the profiler, which adds some percent, and
// differ by a microsecond or two from one trace to the next.  Two figures of a
// change, below, are event times of the two builds as they
// were then, not parts of these totals.)
// Chunks have their places by rule (gdn_packed_common.h), segments theirs by
// counts that the preparation's launch makes: only sequences longer than a
// segment have states of segments, so that short ones cost no workspace.
// Slots outside the pool read as zero states and are not written.
#include "gdn_elements.h"
#include "gdn_internal.h"
#include "gdn_mfma_common.h"
#include "gdn_packed_common.h"
#include "../../include/gdn.h"

namespace gdn {
namespace {

// Sequences of fewer tokens go token by token.  Token by token, and in chunks:
// 256 sequences x 16 heads of 128, 24 tokens 385 and 351 us, 32 tokens 508 and
// 359, 64 tokens 932 and 413; 16 sequences, 24 tokens 31 and 38 us, 32 tokens
// 40 and 38; heads of 64, 256 sequences, 32 tokens 166 and 184 us, 48 tokens
// 235 and 188.
constexpr int kChunkMin = 32;
static_assert(kChunkMin == 1 << 5, "a place every 32 tokens serves every sequence in chunks");

struct Pk {
    Packed p;
    Offsets at;
    int Hv, group;   // value heads; value heads per key head
    int64_t rec_below;  // sequences of fewer tokens go token by token
    int seg_shift;   // a segment holds 2^seg_shift tokens
    Places places;   // of the chunks
    int64_t nslot;   // so many of them
    int64_t nseg;    // the most segments, of sequences in chunks
    int64_t nstate;  // the most of sequences of two segments or more
    int64_t nunit;   // the most workgroup-sets of their chains
    int32_t* order;  // sequences by falling length
    int32_t* first;  // [S + 1]: segments before each rank of that order
    int32_t* sfirst; // [S + 1]: ... of sequences of two or more: their places
    int32_t* ufirst; // [S + 1]: chain units before each rank: the blocks' places
    u16x8* T;        // [place, head][kTfrag]: T' as A operands
    float* G;        // [place, head][kGate]
    float* s_end;    // [segment place, head][D][D]: end states of the state pass
    float* m_end;    // [place, head][D][D]: M transposed
    float* s_start;  // [place, head][D][D]: start states of the output pass
    bool two_level;  // long chains of start states run as a two-level scan:
    float* q_blk;    // [block place, head][D][D]: a block of maps as one: addend
    float* p_blk;    // [block place, head][D][D]: and matrix, transposed
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
// touched once): k_pk_step, 256 x 16 states of 128 x 128 in 97 us (bytes: 89).
// k_pk_rec stages more of them kStage at a time in LDS, the next stage's rows
// in flight while the current one is worked off: 48 x 5 tokens, channel gate,
// 29 us (bytes: 18; bound by the states' stream and then by the tokens' sums,
// one behind the other).
constexpr int kRecThreads = 256;
constexpr int kStage = 8;
constexpr int kRecLPR = 16, kRecR = 2;
typedef float f32x4v __attribute__((ext_vector_type(4)));

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
__device__ __forceinline__ bool rec_at(const Pk& a, unsigned blocks, RecAt& x) {
    // each XCD takes whole sequences
    const unsigned nrb = ((unsigned)a.p.dv + RB - 1) / RB, one = nrb * a.Hv;
    const unsigned block = on_one_xcd(blockIdx.x, blocks, one);
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
    if (!rec_at<RB>(a, gridDim.x, x)) return;
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

// the work of the first `blocks` workgroups of a launch
template <int DT, int CH, int LPR, int NP, int R>
__device__ __forceinline__ void rec_block(const Pk& a, unsigned blocks, RecShared<DT, LPR, NP, R, CH != 0>& sh) {
    using Sh = RecShared<DT, LPR, NP, R, CH != 0>;
    constexpr int RPW = 64 / LPR, RB = Sh::RB;
    const Packed& p = a.p;
    RecAt x;
    if (!rec_at<RB>(a, blocks, x)) return;
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
__global__ __launch_bounds__(kRecThreads) void k_pk_rec(Pk a) {
    __shared__ __attribute__((aligned(16))) RecShared<DT, LPR, NP, R, CH != 0> sh;
    rec_block<DT, CH, LPR, NP, R>(a, gridDim.x, sh);
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
    // With few states a token's latency counts, and fewer elements a thread take
    // less of it; with many, the lanes' sums cost more than they hide.  fp32, heads
    // of 128, lanes a row x rows a thread 32 x 1, 16 x 1, 16 x 2: 16 states, 1000
    // tokens 233, 269, 391 us; 256 states, 100 tokens 125, 102, 107 us; 4096, 8
    // tokens 201, 167, 155 us.  Heads of 64, 16 x 1 and 16 x 2: 16 states 231 and
    // 294 us, 1024 of 30 tokens 39 and 43, 4096 of 8 tokens 50 and 46.  (The
    // borders lie somewhere between these; bf16 and channel gates, which were not
    // timed so, take the same.)
    const int64_t states = a.p.S * a.p.Hv;
    if (pieces <= 16) {
        if (states <= 1024)
            return pieces <= 8 ? launch_rec<DT, CH, 8, 1, 1>(a, st) : launch_rec<DT, CH, kRecLPR, 1, 1>(a, st);
        return pieces <= 8 ? launch_rec<DT, CH, 8, 1, kRecR>(a, st) : launch_rec<DT, CH, kRecLPR, 1, kRecR>(a, st);
    }
    if (states <= 32) return launch_rec<DT, CH, 32, 1, 1>(a, st);
    if (states <= 512) return launch_rec<DT, CH, kRecLPR, 2, 1>(a, st);
    return launch_rec<DT, CH, kRecLPR, 2, kRecR>(a, st);
}

// ---------------------------------------------------------------------------
// chunk form
// ---------------------------------------------------------------------------
// Rows of a chunk's factors (floats), t a token: scale gamma_t / xq,
// gamma'_t / xk, gamma_C / (gamma_t xk), the log prefix as hi + lo; then
// gamma_C, 1 / xT, scale / (xq xk), xk, xq (xk, xq, xT: powers of two, below).
constexpr int kGgam = 0, kGgamp = 64, kGtail = 128, kGhi = 192, kGlo = 256, kGlast = 320, kGit = 321, kGip = 322, kGxk = 323,
              kGxq = 324, kGate = 328;
constexpr int kGatePieces = kGate / 4;
// T' of a chunk as A operands of 32 x 32 x 16 products: lower blocks (0, 0),
// (1, 0), (1, 1) of 32 x 32, two steps of 16 columns each, two terms
constexpr int kTfrag = 3 * 2 * 2 * 64;
// ... and of scale P, two terms
constexpr int kPfrag = 3 * 2 * 2 * 64;
constexpr int LDA = C + 4;

typedef float f32x16 __attribute__((ext_vector_type(16)));

// D += A B on a 32 x 32 x 16 bf16 tile: lane l = 32 g + c supplies A[c][8 g ..]
// and B[8 g ..][c]; the accumulator holds D[8 (i / 4) + 4 g + i % 4][c] in
// element i.  Elements 8 j .. 8 j + 7 of an accumulator tile are thus the B
// operand of a step of 16 of its rows as they stand, if the other operand
// takes its columns in that order: 16 j + 4 g + {0 .. 3}, 16 j + 8 + 4 g + {0 .. 3}.
__device__ __forceinline__ f32x16 mfma32(const u16x8& a, const u16x8& b, const f32x16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}
// The same on fp16.
//
// Operands of the state's own products are fp16 in two terms, x = hi + lo to
// 2^-23 of x (bf16 takes three for that, and half as many instructions again),
// with a power of two taken out first, which puts the largest value of a
// column of S, U or Delta, or of a chunk's K, Q or T', between 2^13 and 2^14:
// no scale of the inputs over- or underflows, k and q (bf16) stay exact to
// 2^-38 of the chunk's largest, and a column with an infinity spoils no other.
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ f32x16 mfma32h(const u16x8& a, const u16x8& b, const f32x16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
struct Pow2 {
    float x, inv;  // m x in [2^13, 2^14), NaN for an infinite m; 1 / x
};
__device__ __forceinline__ Pow2 pow2_for(float m) {
    const int e = max(min((int)(__float_as_uint(m) >> 23), 254), 14);
    // (a column with an infinity times NaN: scaled to it, what else the column
    // holds would be zero, finite and wrong)
    return {__builtin_fmaf(m, 0.f, __uint_as_float((uint32_t)(267 - e) << 23)), __uint_as_float((uint32_t)(e - 13) << 23)};
}
constexpr float kInf = __builtin_huge_valf();
__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) x = fmaxf(x, __shfl_xor(x, o, 64));
    return x;
}
__device__ __forceinline__ float max4(const float* x) { return fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])); }
// over the two lanes of a column of a 32 x 32 tile
__device__ __forceinline__ float column_max(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
}
struct Half2 {
    u16x8 h, l;
};
// eight consecutive elements times x, as operands
template <int N>
__device__ __forceinline__ Half2 split_f16(const float (&v)[N], int at, float x) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = v[at + 2 * i], b = v[at + 2 * i + 1];
        h[i] = pack_f16(__builtin_fmaf(a, x, 0.f), __builtin_fmaf(b, x, 0.f));
        asm("" : "+v"(h[i]));  // (taken as packed by what follows, not formed again element by element)
        const f16x2 t = __builtin_bit_cast(f16x2, h[i]);
        l[i] = pack_f16(__builtin_fmaf(a, x, -(float)t[0]), __builtin_fmaf(b, x, -(float)t[1]));
    }
    return {__builtin_bit_cast(u16x8, u32x4{h[0], h[1], h[2], h[3]}), __builtin_bit_cast(u16x8, u32x4{l[0], l[1], l[2], l[3]})};
}
// eight bf16 times x, as fp16
__device__ __forceinline__ u32x4 bf16_to_f16(const u32x4& v, float x) {
    u32x4 y;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        y[i] = pack_f16(__builtin_fmaf(__uint_as_float(v[i] << 16), x, 0.f), __builtin_fmaf(__uint_as_float(v[i] & 0xFFFF0000u), x, 0.f));
    return y;
}
__device__ __forceinline__ float max_abs8(const u32x4& v) {  // of eight bf16
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m = fmaxf(m, fmaxf(fabsf(__uint_as_float(v[i] << 16)), fabsf(__uint_as_float(v[i] & 0xFFFF0000u))));
    return m;
}
__device__ __forceinline__ float finite_max8(float m, const u32x4& v) {  // of m and the finite ones of eight bf16
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float y = fabsf(__uint_as_float(i & 1 ? v[i / 2] & 0xFFFF0000u : v[i / 2] << 16));
        m = y < kInf ? fmaxf(m, y) : m;
    }
    return m;
}
// A log gate of a zero gate: low enough that every product over it is zero
// in fp32, finite so that the prefix of the tokens behind it stays exact (it
// is a compensated pair; their ratios cancel it)
constexpr float kLogZero = -256.f;

struct Split2 {
    u16x8 h, l;
};
template <int N>
__device__ __forceinline__ Split2 split2_8(const float (&x)[N], int at) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) split2(x[at + 2 * i], x[at + 2 * i + 1], h[i], l[i]);
    return {__builtin_bit_cast(u16x8, u32x4{h[0], h[1], h[2], h[3]}), __builtin_bit_cast(u16x8, u32x4{l[0], l[1], l[2], l[3]})};
}

// Segments of a sequence of n tokens, and the workgroup-sets of the chain
// through ng > 1 of them: one, or one a block of maps where it runs as a
// two-level scan (k_pk_chain)
constexpr int kChainShift = 3, kChainLong = 32;  // maps a block; the fewest that go two-level
__device__ __forceinline__ int64_t segments_of(const Pk& a, int64_t n) {
    return (n + ((int64_t)1 << a.seg_shift) - 1) >> a.seg_shift;
}
__device__ __forceinline__ bool in_blocks(const Pk& a, int64_t ng) { return a.two_level && ng - 2 >= kChainLong; }
__device__ __forceinline__ int64_t chain_units(const Pk& a, int64_t ng) {
    return in_blocks(a, ng) ? (ng - 2 + (1 << kChainShift) - 1) >> kChainShift : 1;
}

// Per chunk and value head: the gate rows and T'.  One workgroup of four
// waves each; K K^T on bf16 MFMA (exact operands), the inverse in fp32.  The
// launch's first `recs` workgroups take the short sequences token by token:
// they wait for memory and for their own sums, the chunks keep the compute
// units busy beside them.
template <int D>
__global__ __launch_bounds__(kThreads, 7) void k_pk_prep(Pk a, unsigned recs) {
    constexpr int LDK = D + 8, PPR = D / 8, KP = C * PPR / kThreads;
    static_assert(C * LDK * 2 <= C * LDA * 4, "K rows fit the tile");
    using Rec = RecShared<GDN_BF16, kRecLPR, D / 64, kRecR, false>;
    static_assert(kThreads == kRecThreads && sizeof(Rec) <= C * LDA * 4, "one workgroup serves either");
    __shared__ __attribute__((aligned(16))) float AT[C * LDA];
    __shared__ __attribute__((aligned(16))) float ghi[C], glo[C], gphi[C], gplo[C], gbeta[C], mx[3][4];
    const Packed& p = a.p;
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, g4 = l >> 4, c16 = l & 15;
    if (blockIdx.x == gridDim.x - 1) {  // one workgroup more: the segments' order
        order_sequences(a.at, a.order, reinterpret_cast<int*>(AT), tid, kThreads);
        __syncthreads();
        auto counts = [&](int s, uint32_t(&c)[3]) {
            const int64_t n = span_of(a.at, s).n;
            c[0] = n < kChunkMin ? 0 : (uint32_t)segments_of(a, n);
            c[1] = c[0] > 1 ? c[0] : 0;
            c[2] = c[0] > 1 ? (uint32_t)chain_units(a, c[0]) : 0;
        };
        int32_t* const out[3] = {a.first, a.sfirst, a.ufirst};
        count_ranks<3>((int)p.S, a.order, counts, out, reinterpret_cast<uint32_t*>(AT), tid, kThreads);
        return;
    }
    if (blockIdx.x < recs) {
        rec_block<GDN_BF16, 0, kRecLPR, D / 64, kRecR>(a, recs, *reinterpret_cast<Rec*>(AT));
        return;
    }
    const unsigned id = on_one_xcd(blockIdx.x - recs, gridDim.x - 1 - recs, a.group);
    const int place = id / a.Hv, h = id - place * a.Hv, hk = h / a.group;
    const int64_t s = seq_of_place(a.at, place, a.places, l);
    const Span sp = span_of(a.at, s);
    const int64_t c = place - a.places.first(sp.begin, s);
    if (sp.n < kChunkMin || c < 0 || c * C >= sp.n) return;
    const int64_t t0 = sp.begin + c * C;
    const int nt = (int)min<int64_t>(C, sp.n - c * C);
    const uint16_t* kin = static_cast<const uint16_t*>(p.k) + hk * D;
    uint16_t* Ks = reinterpret_cast<uint16_t*>(AT);
    const uint16_t* qin = static_cast<const uint16_t*>(p.q) + hk * D;
    u32x4 kv[KP];
    float xk = 0.f, xq = 0.f;
#pragma unroll
    for (int i = 0; i < KP; ++i) {
        const int e = tid + kThreads * i, t = min(e / PPR, nt - 1), c8 = e % PPR;
        kv[i] = ld_g<u32x4>(kin + (t0 + t) * p.k_stride + c8 * 8);
        xk = fmaxf(xk, max_abs8(kv[i]));
        xq = fmaxf(xq, max_abs8(ld_g<u32x4>(qin + (t0 + t) * p.q_stride + c8 * 8)));
    }
    if (fmaxf(xk, xq) == kInf) {
        xk = xq = 0.f;
#pragma unroll 1
        for (int e = tid; e < C * PPR; e += kThreads) {
            const int t = min(e / PPR, nt - 1), c8 = e % PPR;
            xk = finite_max8(xk, ld_g<u32x4>(kin + (t0 + t) * p.k_stride + c8 * 8));
            xq = finite_max8(xq, ld_g<u32x4>(qin + (t0 + t) * p.q_stride + c8 * 8));
        }
    }
    xk = wave_max(xk);
    xq = wave_max(xq);
    if (l == 0) {
        mx[0][w] = xk;
        mx[1][w] = xq;
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
    float* const G = a.G + (int64_t)id * kGate;
    if (w == 0) {
        const Pow2 xk = pow2_for(max4(mx[0])), xq = pow2_for(max4(mx[1]));
        G[kGgam + l] = p.scale * __expf(ghi[l] + glo[l]) * xq.inv;
        G[kGgamp + l] = __expf(gphi[l] + gplo[l]) * xk.inv;
        G[kGtail + l] = ratio(ghi[C - 1], glo[C - 1], ghi[l], glo[l]) * xk.inv;
        G[kGhi + l] = ghi[l];
        G[kGlo + l] = glo[l];
        if (l == 0) {
            G[kGlast] = __expf(ghi[C - 1] + glo[C - 1]);
            G[kGip] = p.scale * (xk.inv * xq.inv);
            G[kGxk] = xk.x;
            G[kGxq] = xq.x;
        }
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
    // T' = T diag(beta); blocks above the diagonal (the tile holds A there) zero
    u16x8* T = a.T + (int64_t)id * kTfrag;
    float x[2][8], m = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int e = tid + kThreads * k;
        if (e >= 3 * 2 * 64) continue;
        const int ln = e & 63, st = (e >> 6) & 1, b = e >> 7;
        const int t = 32 * (b > 0) + (ln & 31), j0 = 32 * (b > 1) + 16 * st + 4 * (ln >> 5);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int j = j0 + 8 * hf;
            const f32x4 v = *reinterpret_cast<const f32x4*>(&AT[t * LDA + j]) * *reinterpret_cast<const f32x4*>(&gbeta[j]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                x[k][4 * hf + r] = (j >> 4) > (t >> 4) ? 0.f : v[r];
                const float y = fabsf(x[k][4 * hf + r]);
                m = y < kInf ? fmaxf(m, y) : m;
            }
        }
    }
    m = wave_max(m);
    if (l == 0) mx[2][w] = m;
    __syncthreads();
    const Pow2 xt = pow2_for(max4(mx[2]));
    if (tid == 0) G[kGit] = xt.inv;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int e = tid + kThreads * k;
        if (e >= 3 * 2 * 64) continue;
        const Half2 y = split_f16(x[k], 0, xt.x);
        u16x8* d = T + (e >> 6) * 2 * 64 + (e & 63);
        st_g(d, y.h);
        st_g(d + 64, y.l);
    }
}

// A segment's workgroup in LDS (74 KiB at D = 128 with outputs: two a compute
// unit).  K and Q rows: 16-byte pieces of eight keys in the operands' order,
// keys 16 b + 4 g + {0 .. 3} and + 8 in piece 2 b + g, at piece ^ (row mod
// pieces), so that neither the operands' reads (a row a lane) nor K's columns
// (lds_column4) meet in a bank.  V and the outputs: a wave's own 32 columns of
// 64 rows each, V until it is used and then the outputs.
template <int D, bool OUT>
struct SegShared {
    unsigned short K[C * D];
    unsigned short V[C * D];
    u16x8 T[kTfrag];
    float G[kGate];
    unsigned short Q[OUT ? C * D : 8];
    u16x8 P[OUT ? kPfrag : 1];
};
template <int D>
constexpr int seg_threads() { return 2 * D; }
// x, as if it had just been computed
__device__ __forceinline__ int opaque(int x) {
    asm volatile("" : "+v"(x));
    return x;
}
template <int D>
__device__ __forceinline__ int piece_at(int row, int piece) {
    return row * D + 8 * (piece ^ (row & (D / 8 - 1)));
}

// One segment of one value head.  Bound by the vector ALU (counted at D = 128,
// two workgroups a compute unit: 57 % of the time against 29 % of the matrix
// cores': splits of S, U and Delta into two terms, scaling, gates).  Waves of
// 32 columns read each K and Q operand half as often as waves of 16, and fp16
// pairs take two products a term where bf16 takes three for the same bits: the
// outputs of the batch above 205 -> 158 us.  The next chunk's rows are asked for
// in front of the outputs instead of behind them (158 -> 150 us; 148 -> 138 us
// for the long sequence, where no second workgroup covers the wait); asked for
// in front of Delta: 155 and 135 us.  Wave w holds value columns 32 w .. of S^T
// for every key (accumulator tiles; they serve as the next product's operand
// as they stand), so nothing but the staged chunk and P crosses waves.
// OUT: from the segment's start state, with outputs; the last segment writes
// the end state.  Otherwise the state pass, end values only: S from zero
// (segment 0: from the sequence's start state, which it also copies for the
// output pass, so that the end state may go where the start state was) or, by
// a workgroup of its own, M from I (the recurrence with V = 0).
template <int D, bool OUT>
__global__ __launch_bounds__(seg_threads<D>(), 2) void k_pk_seg(Pk a) {
    constexpr int NT = seg_threads<D>(), KT = D / 32, PPR = D / 8, KP = C * PPR / NT;
    constexpr int GP = (kGatePieces + NT - 1) / NT;
    static_assert(C * PPR % NT == 0, "staging split");
    __shared__ __attribute__((aligned(16))) SegShared<D, OUT> sh;
    const Packed& p = a.p;
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, g = l >> 5, c = l & 31;
    // workgroups that read the same K (and Q) rows: a key head's value heads, S and M
    const unsigned block = on_one_xcd(blockIdx.x, gridDim.x, (OUT ? 1 : 2) * a.group);
    const int place_h = OUT ? block : block >> 1;
    const bool is_m = !OUT && (block & 1);
    const int i_seg = place_h / a.Hv, h = place_h - i_seg * a.Hv, hk = h / a.group;
    const int32_t* const first = OUT ? a.first : a.sfirst;
    if (i_seg >= first[p.S]) return;
    const int64_t rank = rank_holding(first, p.S, i_seg, l), s = a.order[rank];
    const Span sp = span_of(a.at, s);
    const int64_t gi = i_seg - first[rank], ng = segments_of(a, sp.n);
    if (!OUT && (gi == ng - 1 || (is_m && gi == 0))) return;
    const int64_t place = ng > 1 ? a.sfirst[rank] + gi : 0;  // of the segment's states
    // (offsets out of order can hold more segments than N tokens can)
    if (ng > 1 && place - gi + ng > a.nstate) return;
    const int64_t per = (int64_t)1 << (a.seg_shift - 6);       // chunks of a segment
    const int64_t i_begin = gi * per, i_end = min<int64_t>((sp.n + C - 1) / C, i_begin + per);
    const int64_t cplace = a.places.first(sp.begin, s);  // the sequence's first chunk place
    const uint16_t* kin = static_cast<const uint16_t*>(p.k) + hk * D;
    const uint16_t* qin = static_cast<const uint16_t*>(p.q) + hk * D;
    const uint16_t* vin = static_cast<const uint16_t*>(p.v) + h * D + 32 * w;
    auto in_ws = [&](float* pool) { return pool + (place * p.Hv + h) * D * D; };
    const int v = 32 * w + c;  // this lane's value column

    // key tile u, element i: key 32 u + 8 (i / 4) + 4 g + i % 4; times a power of
    // two, 1 / unit (the last update's)
    float S[KT][16], unit = 1.f;
    {
        const float* src = OUT && ng > 1 ? in_ws(a.s_start) : gi == 0 ? state_from(p, s, h) : nullptr;
#pragma unroll
        for (int u = 0; u < KT; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = 32 * u + 8 * i + 4 * g;
                f32x4 x = zero4();
                if (is_m) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) x[r] = v == key + r ? 1.f : 0.f;
                } else if (src) {
                    x = ld_g<f32x4>(src + v * D + key);
                }
                if (!OUT && !is_m && gi == 0) st_g(in_ws(a.s_start) + v * D + key, x);
#pragma unroll
                for (int r = 0; r < 4; ++r) S[u][4 * i + r] = x[r];
            }
    }

    // staging: the next chunk's K and Q in registers from the outputs on,
    // its T' and V straight into LDS once this chunk's are used (addresses: a
    // uniform base and 32 bits a lane)
    u32x4 kr[KP], qr[OUT ? KP : 1];
    float xk, xq;
    f32x4 gr[GP];
    const int t_st = tid / PPR, pc_st = tid % PPR;  // a thread stages rows t_st + 16 k
    constexpr int TS = NT / PPR;
    static_assert(TS == 16, "rows of a staging round keep their place in the swizzle");
    auto at32 = [](const uint16_t* base, uint32_t off) {
        return ld_g<u32x4>(reinterpret_cast<const char*>(base) + off);
    };
    auto issue = [&](int64_t i) {
        const int64_t t0 = sp.begin + i * C;
        const int nt = (int)min<int64_t>(C, sp.n - i * C);
        const uint16_t *kc = kin + t0 * p.k_stride, *qc = qin + t0 * p.q_stride;
#pragma unroll
        for (int k = 0; k < KP; ++k) {
            const uint32_t t = min(t_st + TS * k, nt - 1);
            kr[k] = at32(kc, t * (uint32_t)(2 * p.k_stride) + 16 * pc_st);
            if (OUT) qr[k] = at32(qc, t * (uint32_t)(2 * p.q_stride) + 16 * pc_st);
        }
        const float* gc = a.G + ((cplace + i) * p.Hv + h) * kGate;
        xk = gc[kGxk];
        xq = gc[kGxq];
#pragma unroll
        for (int k = 0; k < GP; ++k) gr[k] = ld_g<f32x4>(gc + 4 * min(tid + NT * k, kGatePieces - 1));
    };
    auto to_lds = [](const void* from, void* to) {  // 16 bytes a lane, to `to` (uniform) + 16 l
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) uint32_t*)from,
                                         (__attribute__((address_space(3))) uint32_t*)to, 16, 0, 0);
    };
    auto fetch_T = [&](int64_t i) {
        const u16x8* tc = a.T + ((cplace + i) * p.Hv + h) * kTfrag;
#pragma unroll
        for (int k = 0; k < kTfrag / NT; ++k) to_lds(tc + NT * k + tid, &sh.T[NT * k + 64 * w]);
    };
    // (rows past the end repeat the last: T' has nothing for them)
    auto fetch_V = [&](int64_t i) {
        const int nt = (int)min<int64_t>(C, sp.n - i * C);
        const uint16_t* vc = vin + (sp.begin + i * C) * p.v_stride;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t t = min((l >> 2) + 16 * k, nt - 1);
            to_lds(reinterpret_cast<const char*>(vc) + (t * (uint32_t)(2 * p.v_stride) + 16 * (l & 3)),
                   &sh.V[w * C * 32 + 512 * k]);
        }
    };
    auto store = [&](int64_t i) {
        const int nt = (int)min<int64_t>(C, sp.n - i * C);
        const u32x4 z = u32x4{0, 0, 0, 0};
        // keys 8 pc .. + 3 and + 4 .. + 7: halves of pieces 2 (pc / 2) and that + 1
        const int p0 = opaque(piece_at<D>(t_st, pc_st & ~1) + 4 * (pc_st & 1)), p1 = p0 ^ 8;
#pragma unroll
        for (int k = 0; k < KP; ++k) {
            const bool ok = t_st + TS * k < nt;
            const u32x4 x = ok ? bf16_to_f16(kr[k], xk) : z;
            *reinterpret_cast<u32x2*>(&sh.K[p0 + TS * D * k]) = u32x2{x[0], x[1]};
            *reinterpret_cast<u32x2*>(&sh.K[p1 + TS * D * k]) = u32x2{x[2], x[3]};
            if (OUT) {
                const u32x4 y = ok ? bf16_to_f16(qr[k], xq) : z;
                *reinterpret_cast<u32x2*>(&sh.Q[p0 + TS * D * k]) = u32x2{y[0], y[1]};
                *reinterpret_cast<u32x2*>(&sh.Q[p1 + TS * D * k]) = u32x2{y[2], y[3]};
            }
        }
#pragma unroll
        for (int k = 0; k < GP; ++k)
            if (tid + NT * k < kGatePieces) *reinterpret_cast<f32x4*>(&sh.G[4 * (tid + NT * k)]) = gr[k];
    };
    auto grow = [&](int row, int m, int i) {  // four gate entries of tokens 32 m + 8 i + 4 g ..
        return *reinterpret_cast<const f32x4*>(&sh.G[row + 32 * m + 8 * i + 4 * g]);
    };
    unsigned short* const Vw = &sh.V[w * C * 32];
    // column c of rows 8 i + 4 g .. + 3 of token tile m of the wave's V
    auto v4 = [&](int m, int i) {
        return lds_column4(&Vw[(32 * m + 8 * i + 4 * g + (l & 15) / 4) * 32 + 16 * ((l >> 4) & 1) + 4 * (l & 3)]);
    };
    // LDS places are formed from one base each where they are used (rows and
    // pieces differ in bits of their own): kept in registers over the loop
    // they would not leave room for the state
    // row 32 m + c of K or Q, keys of step b (16 b ..): base ^ 16 b, + 32 D m
    auto row = [&](const unsigned short* x, int base, int m, int b) {
        return *reinterpret_cast<const u16x8*>(&x[(base ^ (16 * b)) + 32 * D * m]);
    };
    const int row_base = piece_at<D>(c, g);
    // K^T: keys 32 u + c, tokens of step j of tile m, as an A operand.  A lane
    // points at row 4 g + (l % 16) / 4 (and that + 8) of the step, four keys:
    // group l % 4 of 16-key block 2 u + (l / 16) % 2
    const int kc_base = piece_at<D>(4 * g + (l & 15) / 4, 2 * ((l >> 4) & 1) + (l & 1)) + 4 * ((l & 3) >> 1);
    auto kcol = [&](int base, int u, int m, int j) {
        const int at = (base ^ (32 * u)) + (32 * m + 16 * j) * D;
        const int at8 = ((base ^ (32 * u)) ^ (64 & (D - 1))) + (32 * m + 16 * j + 8) * D;
        return cat(lds_column4(&sh.K[at]), lds_column4(&sh.K[at8]));
    };

    issue(i_begin);
    fetch_T(i_begin);
    if (!is_m) fetch_V(i_begin);
    store(i_begin);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    for (int64_t i = i_begin; i < i_end; ++i) {
        __syncthreads();  // chunk i staged
        const int rb = opaque(row_base);
        // scale P^T = K Q^T of the lower blocks, dealt over the waves: rows j,
        // column t, so that eight elements are P's A operand as they stand
        if constexpr (OUT) {
            for (int b = w; b < 3; b += NT / 64) {
                const int jb = b > 1, tb = b > 0;
                f32x16 acc = {};
#pragma unroll
                for (int k = 0; k < D / 16; ++k) acc = mfma32h(row(sh.K, rb, jb, k), row(sh.Q, rb, tb, k), acc);
                const int t = 32 * tb + c;
                const float th = sh.G[kGhi + t], tl = sh.G[kGlo + t], ip = sh.G[kGip];
                float x[16];
#pragma unroll
                for (int i4 = 0; i4 < 4; ++i4) {
                    const f32x4 jh = grow(kGhi, jb, i4), jl = grow(kGlo, jb, i4);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        x[4 * i4 + r] = 32 * jb + 8 * i4 + 4 * g + r <= t ? ip * acc[4 * i4 + r] * ratio(th, tl, jh[r], jl[r]) : 0.f;
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const Split2 y = split2_8(x, 8 * j);
                    sh.P[(b * 2 + j) * 128 + l] = y.h;
                    sh.P[(b * 2 + j) * 128 + 64 + l] = y.l;
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        // X = K S^T
        float m = 0.f;
#pragma unroll
        for (int u = 0; u < KT; ++u)
#pragma unroll
            for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(S[u][e]));
        const float ms = column_max(m);
        const Pow2 xs = pow2_for(ms);
        const float s_inv = xs.inv * unit;
        f32x16 X[2] = {};
#pragma unroll
        for (int b = 0; b < D / 16; ++b) {
            const Half2 y = split_f16(S[b >> 1], 8 * (b & 1), xs.x);
            const u16x8 k0 = row(sh.K, rb, 0, b), k1 = row(sh.K, rb, 1, b);
            X[0] = mfma32h(k0, y.l, X[0]);
            X[1] = mfma32h(k1, y.l, X[1]);
            X[0] = mfma32h(k0, y.h, X[0]);
            X[1] = mfma32h(k1, y.h, X[1]);
        }
        __builtin_amdgcn_sched_barrier(0);
        // U = V - diag(gamma') X (V has arrived in LDS)
        if (OUT) asm volatile("s_waitcnt vmcnt(4)" ::: "memory");  // (all but the last outputs' stores)
        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        float mu = 0.f;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4) {
                const f32x4 gp = s_inv * grow(kGgamp, m, i4);
                u16x4 vv = u16x4{0, 0, 0, 0};
                if (!is_m) vv = v4(m, i4);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    X[m][4 * i4 + r] = gdn_bf16_to_f32(vv[r]) - gp[r] * X[m][4 * i4 + r];
                    mu = fmaxf(mu, fabsf(X[m][4 * i4 + r]));
                }
            }
        const Pow2 xu = pow2_for(column_max(mu));
        __builtin_amdgcn_sched_barrier(0);
        // Delta = T' U
        f32x16 dl[2] = {};
#pragma unroll
        for (int jb = 0; jb < 2; ++jb)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float u[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = X[jb][8 * j + e];
                const Half2 y = split_f16(u, 0, xu.x);
                u16x8 th[2], tl[2];
#pragma unroll
                for (int tb = jb; tb < 2; ++tb) {
                    const u16x8* ta = &sh.T[((tb + jb) * 2 + j) * 128 + l];
                    th[tb] = ta[0], tl[tb] = ta[64];
                }
#pragma unroll
                for (int tb = jb; tb < 2; ++tb) dl[tb] = mfma32h(tl[tb], y.h, dl[tb]);
#pragma unroll
                for (int tb = jb; tb < 2; ++tb) dl[tb] = mfma32h(th[tb], y.l, dl[tb]);
#pragma unroll
                for (int tb = jb; tb < 2; ++tb) dl[tb] = mfma32h(th[tb], y.h, dl[tb]);
            }
        __builtin_amdgcn_sched_barrier(0);
        const float unscale = xu.inv * sh.G[kGit];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = 0; e < 16; ++e) dl[m][e] *= unscale;
        const bool more = i + 1 < i_end;
        __syncthreads();  // T' is used, P whole
        if (more) fetch_T(i + 1);
        if (more) issue(i + 1);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (OUT) {
            // O = diag(scale gamma) Q S^T + scale P Delta, P and Delta in two bf16
            // terms, rounded once to bf16, over V (S is split again: X's phase has
            // no registers for Q S^T)
            f32x16 Z[2] = {};
            const int qb = opaque(row_base);
#pragma unroll
            for (int b = 0; b < D / 16; ++b) {
#pragma unroll
                for (int e = 0; e < 8; ++e) asm volatile("" : "+v"(S[b >> 1][8 * (b & 1) + e]));  // (not X's terms, kept)
                const Half2 y = split_f16(S[b >> 1], 8 * (b & 1), xs.x);
                const u16x8 q0 = row(sh.Q, qb, 0, b), q1 = row(sh.Q, qb, 1, b);
                Z[0] = mfma32h(q0, y.l, Z[0]);
                Z[1] = mfma32h(q1, y.l, Z[1]);
                Z[0] = mfma32h(q0, y.h, Z[0]);
                Z[1] = mfma32h(q1, y.h, Z[1]);
            }
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i4 = 0; i4 < 4; ++i4) {
                    const f32x4 gam = s_inv * grow(kGgam, m, i4);
#pragma unroll
                    for (int r = 0; r < 4; ++r) Z[m][4 * i4 + r] *= gam[r];
                }
#pragma unroll
            for (int jb = 0; jb < 2; ++jb)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = dl[jb][8 * j + e];
                    const Split2 y = split2_8(x, 0);
                    u16x8 ph[2], pl[2];
#pragma unroll
                    for (int m = jb; m < 2; ++m) {
                        const u16x8* pa = &sh.P[((m + jb) * 2 + j) * 128 + l];
                        ph[m] = pa[0], pl[m] = pa[64];
                    }
#pragma unroll
                    for (int m = jb; m < 2; ++m) Z[m] = mfma32(pl[m], y.h, Z[m]);
#pragma unroll
                    for (int m = jb; m < 2; ++m) Z[m] = mfma32(ph[m], y.l, Z[m]);
#pragma unroll
                    for (int m = jb; m < 2; ++m) Z[m] = mfma32(ph[m], y.h, Z[m]);
                }
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i2 = 0; i2 < 8; ++i2) {
                    const uint32_t y = pack_bf16(Z[m][2 * i2], Z[m][2 * i2 + 1]);
                    const int t = 32 * m + 8 * (i2 >> 1) + 4 * g + 2 * (i2 & 1);
                    Vw[t * 32 + c] = (unsigned short)y;
                    Vw[(t + 1) * 32 + c] = (unsigned short)(y >> 16);
                }
        }
        __builtin_amdgcn_sched_barrier(0);
        // S^T <- gamma_C S^T + K^T diag(gamma_C / gamma) Delta, summed in the scale
        // of the larger of the two (the decayed state, not the one before it: a
        // small Delta behind a strong decay keeps its bits)
        float md = 0.f;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4) {
                const f32x4 tail = grow(kGtail, m, i4);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    dl[m][4 * i4 + r] *= tail[r];
                    md = fmaxf(md, fabsf(dl[m][4 * i4 + r]));
                }
            }
        const float g_unit = sh.G[kGlast] * unit;
        const Pow2 xd = pow2_for(fmaxf(column_max(md), ms * g_unit));
        const float gC = ms > 0.f ? g_unit * xd.x : 0.f;  // (a zero state leaves the scale anywhere)
        unit = xd.inv;
        const int kb = opaque(kc_base);
        f32x16 acc[KT];
#pragma unroll
        for (int u = 0; u < KT; ++u)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[u][e] = gC * S[u][e];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = dl[m][8 * j + e];
                const Half2 y = split_f16(x, 0, xd.x);
#pragma unroll
                for (int u = 0; u < KT; u += 2) {
                    const u16x8 k0 = kcol(kb, u, m, j), k1 = kcol(kb, u + 1, m, j);
                    acc[u] = mfma32h(k0, y.l, acc[u]);
                    acc[u + 1] = mfma32h(k1, y.l, acc[u + 1]);
                    acc[u] = mfma32h(k0, y.h, acc[u]);
                    acc[u + 1] = mfma32h(k1, y.h, acc[u + 1]);
                }
            }
#pragma unroll
        for (int u = 0; u < KT; ++u)
#pragma unroll
            for (int e = 0; e < 16; ++e) S[u][e] = acc[u][e];
        // T' has arrived in LDS (and the rows in registers); waited for in front of
        // the output's stores, which the counter counts too
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        // the wave's columns of the output tile, rows past the end dropped; the
        // next V takes their place in LDS, asked for before the stores
        u32x4 o[OUT ? 4 : 1];
        if constexpr (OUT) {
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = *reinterpret_cast<const u32x4*>(&Vw[8 * (l + 64 * k)]);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
        if (more && !is_m) fetch_V(i + 1);
        if constexpr (OUT) {
            __builtin_amdgcn_sched_barrier(0);
            const int nt = (int)min<int64_t>(C, sp.n - i * C);
            uint16_t* ob = static_cast<uint16_t*>(p.out) + (sp.begin + i * C) * p.Hv * D + h * D + 32 * w;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t t = (l >> 2) + 16 * k;
                if ((int)t < nt)
                    __builtin_nontemporal_store(o[k], reinterpret_cast<u32x4*>(reinterpret_cast<char*>(ob) +
                                                                               (t * (uint32_t)(2 * D * a.Hv) + 16 * (l & 3))));
            }
        }
        __syncthreads();  // chunk i is worked off
        if (more) store(i + 1);
    }
#pragma unroll
    for (int u = 0; u < KT; ++u)
#pragma unroll
        for (int e = 0; e < 16; ++e) S[u][e] *= unit;
    float* dst = OUT ? (gi == ng - 1 ? state_to(p, s, h) : nullptr) : is_m ? nullptr : in_ws(a.s_end);
    float* mt = is_m ? in_ws(a.m_end) : nullptr;  // M^T: row key (of the end state), column v
#pragma unroll
    for (int u = 0; u < KT; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int key = 32 * u + 8 * i + 4 * g;
            if (dst) st_g(dst + v * D + key, f32x4{S[u][4 * i], S[u][4 * i + 1], S[u][4 * i + 2], S[u][4 * i + 3]});
            if (mt) {
#pragma unroll
                for (int r = 0; r < 4; ++r) mt[(key + r) * D + v] = S[u][4 * i + r];
            }
        }
}

// Start states of a sequence's segments: X(g + 1) = S_end(g) + X(g) M(g), from
// X(1) = S_end(0).  The maps compose, so a long chain runs as a two-level scan
// (about 3 sqrt of the steps): blocks of 2^kChainShift maps side by side into
// one map each (kCompose: P = M(a) ... M(e - 1) and the addend Q), the blocks'
// start states one after the other (kBlocks), and every block's own from its
// start (kExpand, which alone does the whole of a short chain).
// Sixteen rows of one head a workgroup (rows are independent), wave w the
// columns 16 w ..; fp32 MFMA, the next three matrices in flight while one
// multiplies (a step takes 2.4 us at D = 128: 64 KiB into the compute unit,
// then LDS exchange and products one behind the other).  The two-level scan's
// outer kernels take R = 2 sixteens of rows a workgroup: half the matrices'
// loads, and a round of workgroups instead of two (190 -> 153 us at 127 maps
// of 4 heads).  One level and two: 64 maps, D = 128, 150 and 101 us; at most
// 25 maps, D = 64, 23 and 34 us.
enum { kCompose, kBlocks, kExpand };
// The ranks that may hold chains in blocks: ranks fall by classes of length a
// quarter of an octave wide, so none in front of a sequence of 33 segments has
// fewer than 24.
__host__ __device__ __forceinline__ int64_t block_ranks(const Packed& p, int shift) {
    const int64_t most = p.N >> (shift + 4);
    return p.S < most ? p.S : most;
}
template <int D, int MODE, int R>
__global__ __launch_bounds__(4 * D, 2) void k_pk_chain(Pk a) {
    constexpr int NB = D / 16, LDX = D + 4;
    constexpr int TILES = NB / R, WGS = MODE == kCompose ? 2 * TILES : TILES;  // row tiles of Q (and P)
    __shared__ __attribute__((aligned(16))) float X[2][16 * R * LDX];
    const Packed& p = a.p;
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, g4 = l >> 4, c16 = l & 15;
    // workgroups go to the eight XCDs in turn: those that read the same
    // matrices share one and its L2
    const int j = blockIdx.x / 8, tile = j % WGS, id = (j / WGS) * 8 + blockIdx.x % 8;
    const int rt = tile % TILES * R;
    const bool is_p = MODE == kCompose && tile >= TILES;
    // units (the blocks' chains: sequences by rank, longest first)
    const int64_t unit = id / a.Hv;
    const int h = id - (int)unit * a.Hv;
    if (unit >= (MODE == kBlocks ? block_ranks(p, a.seg_shift) : (int64_t)a.ufirst[p.S])) return;
    const int64_t rank = MODE == kBlocks ? unit : rank_holding(a.ufirst, p.S, (int)unit, l), s = a.order[rank];
    const int64_t ng = segments_of(a, span_of(a.at, s).n);
    const bool two = in_blocks(a, ng);
    if (ng < 2 || (MODE != kExpand && !two)) return;
    const int64_t base = a.sfirst[rank], bbase = a.ufirst[rank], nblk = chain_units(a, ng);
    if (base + ng > a.nstate || bbase + nblk > a.nunit) return;  // (as for the segments)
    const int64_t blk = MODE == kBlocks ? 0 : unit - bbase;
    auto at = [&](float* pool, int64_t g) { return pool + ((base + g) * p.Hv + h) * D * D; };
    auto at_blk = [&](float* pool, int64_t b) { return pool + ((bbase + b) * p.Hv + h) * D * D; };
    // steps g0 .. g1 - 1: maps, or blocks of them
    const int64_t g0 = MODE == kBlocks ? 0 : 1 + (blk << kChainShift);
    const int64_t g1 = MODE == kBlocks ? nblk - 1 : two ? min(ng - 1, g0 + (1 << kChainShift)) : ng - 1;
    const int col = 16 * w + c16;  // rows 4 g4 + r of the sixteen
    struct Rows {
        f32x4 t[R];
    };
    auto rows = [&](const float* m) {
        Rows x;
#pragma unroll
        for (int t = 0; t < R; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) x.t[t][r] = m[(16 * (rt + t) + 4 * g4 + r) * D + col];
        return x;
    };
    auto put = [&](float* m, const Rows& x) {
#pragma unroll
        for (int t = 0; t < R; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) m[(16 * (rt + t) + 4 * g4 + r) * D + col] = x.t[t][r];
    };
    constexpr int AHEAD = 4 - R;
    struct In {
        f32x4 m[NB];
        Rows add;
    };
    const int64_t first = MODE == kCompose ? g0 + 1 : g0;  // (the first map of a block is where P and Q start)
    // (in program order, so that a step waits for its own matrix alone)
    auto fetch = [&](In& in, int64_t g) {
        g = max(min(g, g1 - 1), first);
        const float* m = (MODE == kBlocks ? at_blk(a.p_blk, g) : at(a.m_end, g)) + col * D;
#pragma unroll
        for (int k = 0; k < NB; ++k) in.m[k] = ld_g<f32x4>(m + 16 * k + 4 * g4);
        if (!is_p) in.add = rows(MODE == kBlocks ? at_blk(a.q_blk, g) : at(a.s_end, g));
        else
#pragma unroll
            for (int t = 0; t < R; ++t) in.add.t[t] = zero4();
        __builtin_amdgcn_sched_barrier(0);
    };
    Rows x;
    if (MODE == kCompose) {
        if (!is_p) x = rows(at(a.s_end, g0));
        else
#pragma unroll
            for (int t = 0; t < R; ++t) x.t[t] = ld_g<f32x4>(at(a.m_end, g0) + col * D + 16 * (rt + t) + 4 * g4);
    } else {
        x = MODE == kExpand && blk > 0 ? rows(at(a.s_start, g0)) : rows(at(a.s_end, 0));
        if (MODE == kExpand && blk == 0) put(at(a.s_start, 1), x);
    }
    auto step = [&](int64_t g, const In& in) {
        float* Xs = X[g & 1];
#pragma unroll
        for (int t = 0; t < R; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) Xs[(16 * t + 4 * g4 + r) * LDX + col] = x.t[t][r];
        __syncthreads();
        Rows y;
#pragma unroll
        for (int t = 0; t < R; ++t) {
            f32x4 xa[NB], acc[4] = {in.add.t[t], zero4(), zero4(), zero4()};
#pragma unroll
            for (int k = 0; k < NB; ++k)
                xa[k] = *reinterpret_cast<const f32x4*>(&Xs[(16 * t + c16) * LDX + 16 * k + 4 * g4]);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int k = 0; k < NB; k += 4)
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[e] = mfma_f32(xa[k + e][q], in.m[k + e][q], acc[e]);
            y.t[t] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
        }
        if (g < g1) {
            x = y;
            // (the start of the next segment; of the next block's first)
            if (MODE == kExpand && (g + 1 < g1 || blk == nblk - 1)) put(at(a.s_start, g + 1), x);
            if (MODE == kBlocks) put(at(a.s_start, 1 + ((g + 1) << kChainShift)), x);
        }
    };
    if (first < g1) {
        In in[AHEAD + 1];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) fetch(in[u], first + u);
        for (int64_t g = first; g < g1; g += AHEAD + 1) {
#pragma unroll
            for (int u = 0; u <= AHEAD; ++u) {
                fetch(in[(u + AHEAD) % (AHEAD + 1)], g + u + AHEAD);
                step(g + u, in[u]);
            }
        }
    }
    if (MODE == kCompose) {
        if (!is_p) put(at_blk(a.q_blk, blk), x);
        else
#pragma unroll
            for (int t = 0; t < R; ++t) st_g(at_blk(a.p_blk, blk) + col * D + 16 * (rt + t) + 4 * g4, x.t[t]);
    }
}

// Tokens of a segment, as a power of two: as many segments as there are
// compute units over all heads, at least four chunks each.  Rounded up, so just
// past a power of two there are half as many, each twice as long, and a call
// takes a quarter to two fifths longer (one of 65536 and 65600 tokens, 4 heads:
// 419 and 526 us; of 16384 and 16400, 16 heads: 337 and 469).  Twice as many run
// the output pass two workgroups a compute unit (one of 65531 tokens, 4 heads:
// outputs 113 instead of 139 us), but have twice the matrices to multiply
// through the chain (153 instead of 101 us); mixed batch of 16384, 16 heads:
// state pass, chain and outputs 106, 56, 140 instead of 82, 30, 154 us.
// Heads of 64 have workgroups of two waves, so twice as many, of at least two
// chunks (8 sequences of 2048, 16 heads: 222 us with one a compute unit and
// four chunks, 170 so; 4 of 500, 4 heads: 58 and 44 us; heads of 128, four
// chunks and two: 117 and 135 us for one of 4096, 91 and 80 for 4 of 1000).
constexpr int kWhole = 31;  // a sequence's tokens are fewer than 2^31
int seg_shift_for(const Packed& p) {
    const int64_t want = p.N * p.Hv / (p.dk == 64 ? 512 : 256);  // tokens a workgroup
    int sh = p.dk == 64 ? 7 : 8;
    while (((int64_t)1 << sh) < want && sh < 30) ++sh;
    return sh;
}
int64_t longest(const Packed& p) { return std::min(p.N, p.max_len); }

// whether a sequence may have a chain that is worth two levels
bool two_level(const Packed& p, int shift) { return longest(p) > (int64_t)(kChainLong + 1) << shift; }

// What a batch has at most.  M sequences of more than 2^sh tokens (so M <= N /
// 2^sh) have at most N / 2^sh + M segments together; their chains' units are no
// more than one for each and one for eight segments, nor than N / 2^sh.
struct PkSizes {
    Places places;
    int64_t nslot, nseg, nstate, nunit;
};
PkSizes sizes(const Packed& p, int shift) {
    PkSizes z;
    // (N / 64 + S places, or N / 32 where there are many sequences)
    const int64_t by_seq = p.N / C + p.S, by_32 = p.N / kChunkMin;
    z.places = by_seq <= by_32 ? chunk_places() : Places{5, 0};
    z.nslot = std::min(by_seq, by_32);
    const int64_t whole = p.N >> shift, m = std::min(p.S, whole);
    z.nseg = whole + std::min(p.S, by_32);
    z.nstate = whole + m;
    z.nunit = std::min(whole, m + (z.nstate >> kChainShift));
    return z;
}
// without segments every sequence is one, whatever its length (max_len is the
// caller's word, the lengths are the device's)
int shift_for(const Packed& p) { return longest(p) > (int64_t)1 << seg_shift_for(p) ? seg_shift_for(p) : kWhole; }

struct PkLayout {
    size_t T, G, order, first, s_end, m_end, s_start, q_blk, p_blk, total;
};
PkLayout layout(const Packed& p) {
    PkLayout L{};
    if (!packed_in_chunks(p)) return L;
    const int sh = shift_for(p);
    const PkSizes z = sizes(p, sh);
    const size_t chunks = (size_t)(z.nslot * p.Hv);
    size_t off = 0;
    auto take = [&](size_t floats) {
        const size_t at = off;
        off += align256(floats * sizeof(float));
        return at;
    };
    L.T = take(chunks * kTfrag * 4);
    L.G = take(chunks * kGate);
    L.order = take((size_t)p.S);
    L.first = take(3 * ((size_t)p.S + 1));
    const size_t states = (size_t)(z.nstate * p.Hv * p.dk * p.dk), blocks = (size_t)(z.nunit * p.Hv * p.dk * p.dk);
    L.s_end = take(states);
    L.m_end = take(states);
    L.s_start = take(states);
    if (two_level(p, sh)) {
        L.q_blk = take(blocks);
        L.p_blk = take(blocks);
    }
    L.total = off;
    return L;
}

template <int D>
hipError_t launch_chunks(const Pk& a, hipStream_t st) {
    const Packed& p = a.p;
    prof_begin(p.timer, "k_pk_prep", st);
    const unsigned recs = (unsigned)(p.S * p.Hv * (D / RecShared<GDN_BF16, kRecLPR, D / 64, kRecR, false>::RB));
    hipLaunchKernelGGL(k_pk_prep<D>, dim3(recs + (unsigned)(a.nslot * p.Hv) + 1), dim3(kThreads), 0, st, a, recs);
    prof_end(p.timer, st);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)(a.nseg * p.Hv)), states((unsigned)(2 * a.nstate * p.Hv)), block(seg_threads<D>());
    if (a.nstate > 0) {
        prof_begin(p.timer, "k_pk_state", st);
        hipLaunchKernelGGL((k_pk_seg<D, false>), states, block, 0, st, a);
        prof_end(p.timer, st);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        // eight workgroup-sets at a time, for the eight XCDs
        const int64_t units = a.nunit * p.Hv;
        auto sets = [](int64_t n, int per) { return dim3((unsigned)((n + 7) / 8 * 8 * per)); };
        prof_begin(p.timer, "k_pk_chain", st);
        if (a.two_level) {
            hipLaunchKernelGGL((k_pk_chain<D, kCompose, 2>), sets(units, D / 16), dim3(4 * D), 0, st, a);
            hipLaunchKernelGGL((k_pk_chain<D, kBlocks, 1>), sets(block_ranks(p, a.seg_shift) * p.Hv, D / 16), dim3(4 * D), 0, st, a);
            hipLaunchKernelGGL((k_pk_chain<D, kExpand, 2>), sets(units, D / 32), dim3(4 * D), 0, st, a);
        } else {
            hipLaunchKernelGGL((k_pk_chain<D, kExpand, 1>), sets(units, D / 16), dim3(4 * D), 0, st, a);
        }
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

bool packed_in_chunks(const Packed& p) { return packed_chunked(p) && longest(p) >= kChunkMin; }

size_t packed_workspace(const Packed& p) { return layout(p).total; }

hipError_t packed_forward(const Packed& p, void* ws, hipStream_t st) {
    Pk a{};
    a.p = p;
    a.at = {p.cu, p.N, p.S};
    a.Hv = (int)p.Hv;
    a.group = (int)(p.Hv / p.Hk);
    const PkLayout L = layout(p);
    const bool chunks = L.total > 0;
    a.rec_below = chunks ? kChunkMin : INT64_MAX;  // (a sequence may have INT32_MAX tokens)
    if (!chunks) {
        prof_begin(p.timer, "k_pk_rec", st);
        hipError_t e;
        if (p.dtype == GDN_BF16)
            e = p.gate == GDN_GATE_CHANNEL ? launch_rec_shape<GDN_BF16, 1>(a, st) : launch_rec_shape<GDN_BF16, 0>(a, st);
        else
            e = p.gate == GDN_GATE_CHANNEL ? launch_rec_shape<GDN_F32, 1>(a, st) : launch_rec_shape<GDN_F32, 0>(a, st);
        prof_end(p.timer, st);
        return e;
    }
    char* base = static_cast<char*>(ws);
    a.seg_shift = shift_for(p);
    const PkSizes z = sizes(p, a.seg_shift);
    a.places = z.places;
    a.nslot = z.nslot;
    a.nseg = z.nseg;
    a.nstate = z.nstate;
    a.nunit = z.nunit;
    a.T = reinterpret_cast<u16x8*>(base + L.T);
    a.order = reinterpret_cast<int32_t*>(base + L.order);
    a.first = reinterpret_cast<int32_t*>(base + L.first);
    a.sfirst = a.first + p.S + 1;
    a.ufirst = a.sfirst + p.S + 1;
    a.G = reinterpret_cast<float*>(base + L.G);
    a.s_end = reinterpret_cast<float*>(base + L.s_end);
    a.m_end = reinterpret_cast<float*>(base + L.m_end);
    a.s_start = reinterpret_cast<float*>(base + L.s_start);
    a.two_level = two_level(p, a.seg_shift);
    a.q_blk = reinterpret_cast<float*>(base + L.q_blk);
    a.p_blk = reinterpret_cast<float*>(base + L.p_blk);
    return p.dk == 64 ? launch_chunks<64>(a, st) : launch_chunks<128>(a, st);
}

}  // namespace gdn
