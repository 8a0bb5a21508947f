// Norm of queries and keys over the features of each head, and the rotation of
// feature pairs by the token's position, in one pass, forward and backward
// (gdn_qk_norm_fwd, gdn_qk_norm_backward).
//
// Per row x of d features (one head of one token), weight w:
//   r = 1 / sqrt(mean x^2 + eps),  xhat = x r,  z = xhat w
//   y = R z: each pair (a, b) of the first `rot` features becomes
//       (a cos - b sin, b cos + a sin), the others stay
// and, given dy,
//   g = R^T dy,  dx = r (g w - xhat mean(g w xhat)),  dw = sum over rows of g xhat.
// The pairs are (i, i + rot / 2) or (2 i, 2 i + 1).
//
// A row belongs to LPR lanes of eight features each: two groups of four that hold
// whole pairs (4 p .. and rot / 2 + 4 p .., or 8 p .. and 8 p + 4 ..; behind the
// rotated ones the two halves of the rest), so that the rotation stays within a
// lane and the row's sums are its only exchange.  A group of lanes takes kU
// heads of one token, which share its angles and the weight.  x, dy, y and dx are
// touched once; statistics and sums are fp32.  Memory bounds it: 16384 tokens, 16
// query and 8 key heads of 128, bf16: 201 MB in 35 us (5.7 TB/s; a copy's rate on
// this card is 6.05); backward of 16 and 16 heads 403 MB in 80 us, and 5 for the
// sums of dw.
#include "gdn_elements.h"
#include "gdn_internal.h"
#include "gdn_mfma_common.h"
#include "../../include/gdn.h"

namespace gdn {
namespace {

constexpr int kU = 4;

struct Side {  // q or k
    const char* x;
    const char* dy;
    char* y;       // forward: y; backward: dx (null: not wanted)
    const float* w;
    int64_t xs, gs, ys;  // elements between tokens
    int heads;
    unsigned groups;     // of kU heads
    float* part;         // backward: [blocks][d] addends of dw, or null
    unsigned blocks;
};
struct QkArgs {
    int64_t N, n_pos;
    int d, rot;
    float eps;
    const float* cos;
    const float* sin;
    const int32_t* pos;
    Side side[2];
};

// A lane's place in a row: its two groups of four, and their angles' place (-1:
// not rotated)
struct Lane {
    int a, b, angle;
    bool on;
};
template <bool PAIRS>
__device__ __forceinline__ Lane lane_at(const QkArgs& A, int p) {
    Lane x;
    x.on = 8 * p < A.d;
    if (8 * p < A.rot) {
        x.angle = 4 * p;
        x.a = PAIRS ? 8 * p : 4 * p;
        x.b = PAIRS ? 8 * p + 4 : A.rot / 2 + 4 * p;
    } else {
        const int rest = p - A.rot / 8;
        x.angle = -1;
        x.a = A.rot + 4 * rest;
        x.b = (A.rot + A.d) / 2 + 4 * rest;
    }
    return x;
}
// cos and sin of the lane's four pairs at token t
__device__ __forceinline__ void angles(const QkArgs& A, const Lane& x, int64_t t, f32x4& c, f32x4& s) {
    c = f32x4{1.f, 1.f, 1.f, 1.f};
    s = zero4();
    if (x.on && x.angle >= 0) {
        int64_t at = A.pos ? (int64_t)A.pos[t] : t;
        at = at < 0 ? 0 : at >= A.n_pos ? A.n_pos - 1 : at;
        c = ld_g<f32x4>(A.cos + at * (A.rot / 2) + x.angle);
        s = ld_g<f32x4>(A.sin + at * (A.rot / 2) + x.angle);
    }
}
// the pairs of a lane's eight, turned by the angle
template <bool PAIRS>
__device__ __forceinline__ void turn(f32x4& a, f32x4& b, const f32x4& c, const f32x4& s) {
    if (PAIRS) {
        a = f32x4{a[0] * c[0] - a[1] * s[0], a[1] * c[0] + a[0] * s[0], a[2] * c[1] - a[3] * s[1], a[3] * c[1] + a[2] * s[1]};
        b = f32x4{b[0] * c[2] - b[1] * s[2], b[1] * c[2] + b[0] * s[2], b[2] * c[3] - b[3] * s[3], b[3] * c[3] + b[2] * s[3]};
    } else {
        const f32x4 y = a * c - b * s;
        b = b * c + a * s;
        a = y;
    }
}
template <int DT>
__device__ __forceinline__ R4<DT> load4(const char* row, int at) {
    constexpr int e = DT == GDN_BF16 ? 2 : 4;
    return ld_g<R4<DT>>(row + (int64_t)e * at);
}
template <int DT>
__device__ __forceinline__ void store4(char* row, int at, const f32x4& x) {
    if constexpr (DT == GDN_BF16) st_g(row + 2 * at, u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])});
    else st_g(row + 4 * at, x);
}
__device__ __forceinline__ f32x4 weight4(const float* w, int at, bool on) {
    return w && on ? ld_g<f32x4>(w + at) : f32x4{1.f, 1.f, 1.f, 1.f};
}

template <int DT, int LPR, bool PAIRS>
__global__ __launch_bounds__(kThreads) void k_qk_norm(QkArgs A) {
    constexpr int e = DT == GDN_BF16 ? 2 : 4, GPB = kThreads / LPR;
    const unsigned all = A.side[0].groups + A.side[1].groups;
    const unsigned u = blockIdx.x * GPB + threadIdx.x / LPR;
    const unsigned t = u / all;
    if (t >= A.N) return;
    unsigned gi = u - t * all;
    const bool second = gi >= A.side[0].groups;
    if (second) gi -= A.side[0].groups;
    // (fields of their own: an index that differs between lanes would put the
    // arguments into scratch memory)
    const Side &Q = A.side[0], &K = A.side[1];
    const Lane x = lane_at<PAIRS>(A, threadIdx.x % LPR);
    const int h0 = gi * kU, heads = second ? K.heads : Q.heads;
    const float* w = second ? K.w : Q.w;
    const char* in = (second ? K.x : Q.x) + (int64_t)e * (t * (second ? K.xs : Q.xs) + (int64_t)h0 * A.d);
    char* out = (second ? K.y : Q.y) + (int64_t)e * (t * (second ? K.ys : Q.ys) + (int64_t)h0 * A.d);
    R4<DT> ra[kU], rb[kU];
#pragma unroll
    for (int j = 0; j < kU; ++j) {
        ra[j] = rb[j] = R4<DT>{};
        if (x.on && h0 + j < heads) {
            ra[j] = load4<DT>(in, j * A.d + x.a);
            rb[j] = load4<DT>(in, j * A.d + x.b);
        }
    }
    f32x4 c, s;
    angles(A, x, t, c, s);
    const f32x4 wa = weight4(w, x.a, x.on), wb = weight4(w, x.b, x.on);
#pragma unroll
    for (int j = 0; j < kU; ++j) {
        f32x4 a = cvt<DT>(ra[j]), b = cvt<DT>(rb[j]);
        const float r = rsqrtf(row_sum<LPR>(dot4e(a, a) + dot4e(b, b)) / (float)A.d + A.eps);
        a *= r * wa;
        b *= r * wb;
        turn<PAIRS>(a, b, c, s);
        if (x.on && h0 + j < heads) {
            store4<DT>(out, j * A.d + x.a, a);
            store4<DT>(out, j * A.d + x.b, b);
        }
    }
}

// A block works off every blocks-th set of units of q or of k, and keeps the sums
// of its rows' g xhat in registers on the way.
template <int DT, int LPR, bool PAIRS>
__global__ __launch_bounds__(kThreads) void k_qk_norm_bwd(QkArgs A) {
    constexpr int e = DT == GDN_BF16 ? 2 : 4, GPB = kThreads / LPR;
    __shared__ __attribute__((aligned(16))) float sums[GPB][8 * LPR];
    const bool second = blockIdx.x >= A.side[0].blocks;
    const Side& S = A.side[second];
    const unsigned block = blockIdx.x - (second ? A.side[0].blocks : 0);
    const int grp = threadIdx.x / LPR, p = threadIdx.x % LPR;
    const Lane x = lane_at<PAIRS>(A, p);
    const f32x4 wa = weight4(S.w, x.a, x.on), wb = weight4(S.w, x.b, x.on);
    f32x4 da = zero4(), db = zero4();
    const int64_t units = A.N * S.groups;
    for (int64_t u = (int64_t)block * GPB + grp; u < units; u += (int64_t)S.blocks * GPB) {
        const int64_t t = u / S.groups;
        const int h0 = (int)(u - t * S.groups) * kU;
        const char* in = S.x + (int64_t)e * (t * S.xs + (int64_t)h0 * A.d);
        const char* gin = S.dy + (int64_t)e * (t * S.gs + (int64_t)h0 * A.d);
        R4<DT> ra[kU], rb[kU], ga[kU], gb[kU];
#pragma unroll
        for (int j = 0; j < kU; ++j) {
            ra[j] = rb[j] = ga[j] = gb[j] = R4<DT>{};
            if (x.on && h0 + j < S.heads) {
                ra[j] = load4<DT>(in, j * A.d + x.a);
                rb[j] = load4<DT>(in, j * A.d + x.b);
                ga[j] = load4<DT>(gin, j * A.d + x.a);
                gb[j] = load4<DT>(gin, j * A.d + x.b);
            }
        }
        f32x4 c, s;
        angles(A, x, t, c, s);
#pragma unroll
        for (int j = 0; j < kU; ++j) {
            f32x4 a = cvt<DT>(ra[j]), b = cvt<DT>(rb[j]), fa = cvt<DT>(ga[j]), fb = cvt<DT>(gb[j]);
            turn<PAIRS>(fa, fb, c, -s);
            const float r = rsqrtf(row_sum<LPR>(dot4e(a, a) + dot4e(b, b)) / (float)A.d + A.eps);
            a *= r;
            b *= r;
            const bool row = h0 + j < S.heads;
            if (row) {
                da += fa * a;
                db += fb * b;
            }
            fa *= wa;
            fb *= wb;
            const float m = row_sum<LPR>(dot4e(fa, a) + dot4e(fb, b)) / (float)A.d;
            if (S.y && x.on && row) {
                char* out = S.y + (int64_t)e * (t * S.ys + (int64_t)(h0 + j) * A.d);
                store4<DT>(out, x.a, r * (fa - a * m));
                store4<DT>(out, x.b, r * (fb - b * m));
            }
        }
    }
    if (!S.part) return;
    if (x.on) {
        *reinterpret_cast<f32x4*>(&sums[grp][x.a]) = da;
        *reinterpret_cast<f32x4*>(&sums[grp][x.b]) = db;
    }
    __syncthreads();
    for (int f = threadIdx.x; f < A.d; f += kThreads) {
        float y = 0.f;
        for (int i = 0; i < GPB; ++i) y += sums[i][f];
        S.part[(int64_t)block * A.d + f] = y;
    }
}

// dw: 16 features of q or of k a block, the partial rows in a fixed order
constexpr int kParamThreads = 1024;
__global__ __launch_bounds__(kParamThreads) void k_qk_norm_params(QkArgs A, float* dwq, float* dwk) {
    constexpr int NR = kParamThreads / 16;
    __shared__ float sums[NR][17];
    const int sets = A.d / 16, c = threadIdx.x % 16, f = 16 * (blockIdx.x % sets) + c, r = threadIdx.x / 16;
    const bool second = (int)blockIdx.x >= sets;
    const Side& S = A.side[second];
    float* dw = second ? dwk : dwq;
    if (!dw) return;
    float y = 0.f;
#pragma unroll 8
    for (unsigned b = r; b < S.blocks; b += NR) y += S.part[(int64_t)b * A.d + f];
    sums[r][c] = y;
    for (int o = NR / 2; o > 0; o /= 2) {
        __syncthreads();
        if (r < o) sums[r][c] += sums[r + o][c];
    }
    if (r == 0) dw[f] = sums[0][c];
}

// Lanes a row: d / 8 or the next power of two
int lanes(const QkNorm& p) {
    int n = 2;
    while (8 * n < p.d) n *= 2;
    return n;
}
QkArgs arguments(const QkNorm& p) {
    QkArgs A{};
    A.N = p.N;
    A.n_pos = p.n_pos;
    A.d = (int)p.d;
    A.rot = (int)p.rot;
    A.eps = p.eps;
    A.cos = p.cos;
    A.sin = p.sin;
    A.pos = p.positions;
    auto side = [&](const void* x, const void* dy, void* y, const float* w, int64_t xs, int64_t gs, int64_t ys, int64_t heads) {
        return Side{static_cast<const char*>(x), static_cast<const char*>(dy), static_cast<char*>(y), w, xs, gs, ys, (int)heads,
                    (unsigned)((heads + kU - 1) / kU), nullptr, 0};
    };
    A.side[0] = side(p.q, p.dyq, p.yq, p.wq, p.q_stride, p.gq_stride, p.yq_stride, p.Hq);
    A.side[1] = side(p.k, p.dyk, p.yk, p.wk, p.k_stride, p.gk_stride, p.yk_stride, p.Hk);
    return A;
}
// Blocks of a side in the backward: 1024 of both together, which is four a
// compute unit, shared by their rows
unsigned bwd_blocks(const QkNorm& p, int64_t heads) {
    if (heads == 0 || p.N == 0) return 0;
    const int64_t per = kThreads / lanes(p), units = p.N * ((heads + kU - 1) / kU);
    const int64_t share = std::max<int64_t>(1024 * heads / (p.Hq + p.Hk), 1);
    return (unsigned)std::min((units + per - 1) / per, share);
}

template <int DT, int LPR, bool PAIRS>
void launch_one(bool back, unsigned blocks, const QkArgs& A, hipStream_t st) {
    if (back) hipLaunchKernelGGL((k_qk_norm_bwd<DT, LPR, PAIRS>), dim3(blocks), dim3(kThreads), 0, st, A);
    else hipLaunchKernelGGL((k_qk_norm<DT, LPR, PAIRS>), dim3(blocks), dim3(kThreads), 0, st, A);
}
template <int DT, int LPR>
void launch_style(bool back, bool pairs, unsigned blocks, const QkArgs& A, hipStream_t st) {
    if (pairs) launch_one<DT, LPR, true>(back, blocks, A, st);
    else launch_one<DT, LPR, false>(back, blocks, A, st);
}
template <int DT>
hipError_t launch_row(bool back, const QkNorm& p, unsigned blocks, const QkArgs& A, hipStream_t st) {
    switch (lanes(p)) {
        case 2: launch_style<DT, 2>(back, p.pairs, blocks, A, st); break;
        case 4: launch_style<DT, 4>(back, p.pairs, blocks, A, st); break;
        case 8: launch_style<DT, 8>(back, p.pairs, blocks, A, st); break;
        case 16: launch_style<DT, 16>(back, p.pairs, blocks, A, st); break;
        default: launch_style<DT, 32>(back, p.pairs, blocks, A, st); break;
    }
    return hipGetLastError();
}
hipError_t launch(bool back, const QkNorm& p, unsigned blocks, const QkArgs& A, hipStream_t st) {
    prof_begin(p.timer, back ? "k_qk_norm_bwd" : "k_qk_norm", st);
    const hipError_t e = p.dtype == GDN_BF16 ? launch_row<GDN_BF16>(back, p, blocks, A, st) : launch_row<GDN_F32>(back, p, blocks, A, st);
    prof_end(p.timer, st);
    return e;
}

}  // namespace

int64_t qk_norm_blocks(const QkNorm& p) {
    const int64_t units = p.N * ((p.Hq + kU - 1) / kU + (p.Hk + kU - 1) / kU), per = kThreads / lanes(p);
    return (units + per - 1) / per;
}

hipError_t qk_norm_fwd(const QkNorm& p, hipStream_t st) {
    return launch(false, p, (unsigned)qk_norm_blocks(p), arguments(p), st);
}

size_t qk_norm_workspace(const QkNorm& p) {
    return sizeof(float) * (size_t)p.d * (bwd_blocks(p, p.Hq) + bwd_blocks(p, p.Hk));
}

hipError_t qk_norm_bwd(const QkNorm& p, hipStream_t st) {
    QkArgs A = arguments(p);
    const bool want[2] = {p.yq || p.dwq, p.yk || p.dwk};
    float* dw[2] = {p.dwq, p.dwk};
    float* part = p.part;
    unsigned blocks = 0;
    for (int i = 0; i < 2; ++i) {
        A.side[i].blocks = want[i] ? bwd_blocks(p, i ? p.Hk : p.Hq) : 0;
        if (dw[i]) {
            A.side[i].part = part;
            part += (int64_t)A.side[i].blocks * p.d;
        }
        blocks += A.side[i].blocks;
    }
    if (blocks > 0) {
        const hipError_t e = launch(true, p, blocks, A, st);
        if (e != hipSuccess) return e;
    }
    if (!p.dwq && !p.dwk) return hipSuccess;
    prof_begin(p.timer, "k_qk_norm_params", st);
    hipLaunchKernelGGL(k_qk_norm_params, dim3(2 * (unsigned)p.d / 16), dim3(kParamThreads), 0, st, A, p.dwq, p.dwk);
    prof_end(p.timer, st);
    return hipGetLastError();
}

}  // namespace gdn
