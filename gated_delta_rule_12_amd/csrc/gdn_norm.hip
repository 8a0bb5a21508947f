// Layer norm over the last dimension, forward and backward
// (gdn_layer_norm_fwd, gdn_layer_norm_backward).
//
// Per row x of n elements:
//   mu = mean x,  r = 1 / sqrt(mean (x - mu)^2 + eps),  xhat = (x - mu) r
//   y  = xhat w + b
// and, given dy,
//   g  = dy w,  dx = r (g - mean g - xhat mean(g xhat))
//   dw = sum over rows of dy xhat,  db = sum over rows of dy.
//
// Both directions are one pass over x, dy, y and dx: a row sits in the
// registers of TPR threads (NV vectors of V elements each) between its load and
// its store, and the variance is taken from the centred values, not from a
// difference of sums.  (Workgroups of 1024 threads have 128 registers a thread.
// Backward rows of more than 8192 elements need more and spill: 30 to 65 of
// them in vectors, 94 to 100 element by element, which forward spills 8 to 10.)
// Rows of up
// to 1024 elements (4 a vector) stay within a wave and reduce across lanes on
// the vector ALU; longer rows take a workgroup and one exchange through LDS
// per sum.  All statistics and sums are fp32.
//
// The weight's and bias's gradients: a thread owns the same columns in every
// row it handles, keeps their sums in registers over all its rows, the
// workgroup adds its row groups in LDS and writes one partial row; k_ln_params
// adds the partial rows.  Every sum has a fixed order (no atomics), so
// repeated calls give identical results.
//
// Whole vectors are bound by memory: 262144 x 128 (fp32 in, bf16 out) forward
// 39 us for 203 MB (5.2 TB/s; 31.5 us where the input is still in the last-level
// cache), backward 63 us for 338 MB (5 of them k_ln_params); 16381 x 2048 bf16
// backward 45 us for 201 MB.  Element by element it is the instructions (two
// bytes a load, and four to eight times the threads a row), and beyond 8192
// columns the spills; forward and backward TB/s (the kernels alone, inputs in
// turn from three buffers):
//   262144 x 128 fp32 -> bf16 5.4 and 4.9; x 127 2.7 and 2.6
//   16381 x 2048 bf16 4.8 and 4.7; x 2047 2.8 and 3.0
//   4095 x 8192 bf16 4.7 and 3.7; x 8191 2.6 and 3.3
//   4095 x 12288 bf16 4.4 and 1.9; x 12287 1.9 and 0.8
#include "gdn_internal.h"
#include "../../include/gdn.h"

namespace gdn {
namespace {

struct LnArgs {
    int64_t rows, n;
    float eps;
    const void* x;
    const void* dy;
    const float* w;
    const float* b;
    void* y;        // forward: y; backward: dx
    float* mean;    // written forward, read backward
    float* rstd;
    float* part;    // backward: [2][groups][n] partial sums of dw and db
    int want_params;
};

// V consecutive elements as they lie in memory, kept so until they are used (a
// row in flight takes half the registers in bf16), and as fp32
typedef unsigned int u32x2v __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4v __attribute__((ext_vector_type(4)));
template <int DT, int V>
struct Raw {
    static constexpr int kWords = V == 1 ? 1 : V * (DT == GDN_F32 ? 4 : 2) / 4;
    uint32_t w[kWords];
};
template <int DT, int V>
__device__ __forceinline__ void ld(Raw<DT, V>& r, const void* base, int64_t i) {
    if constexpr (V == 1) {
        if constexpr (DT == GDN_F32) r.w[0] = static_cast<const uint32_t*>(base)[i];
        else r.w[0] = static_cast<const uint16_t*>(base)[i];
    } else {
        const char* p = static_cast<const char*>(base) + i * (DT == GDN_F32 ? 4 : 2);
        if constexpr (Raw<DT, V>::kWords == 2) {
            const u32x2v x = *reinterpret_cast<const u32x2v*>(p);
            r.w[0] = x[0];
            r.w[1] = x[1];
        } else {
            const u32x4v x = *reinterpret_cast<const u32x4v*>(p);
#pragma unroll
            for (int k = 0; k < 4; ++k) r.w[k] = x[k];
        }
    }
}
template <int DT, int V>
__device__ __forceinline__ float el(const Raw<DT, V>& r, int e) {
    if constexpr (DT == GDN_F32) return __uint_as_float(r.w[e]);
    else if constexpr (V == 1) return __uint_as_float(r.w[0] << 16);
    else return __uint_as_float(e & 1 ? r.w[e / 2] & 0xFFFF0000u : r.w[e / 2] << 16);
}
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2v __attribute__((ext_vector_type(2)));
// two fp32 to a bf16 pair, to the nearest, ties to even: the one rounding of
// a bf16 result
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2v{a, b}, bf16x2));
}
template <int DT, int V>
__device__ __forceinline__ void stv(void* base, int64_t i, const float (&f)[V]) {
    if constexpr (DT == GDN_F32) {
        float* p = static_cast<float*>(base) + i;
        if constexpr (V == 1) {
            p[0] = f[0];
        } else {
#pragma unroll
            for (int k = 0; k < V; k += 4) *reinterpret_cast<float4*>(p + k) = make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
        }
    } else {
        uint16_t* p = static_cast<uint16_t*>(base) + i;
        if constexpr (V == 1) p[0] = (uint16_t)pack2(f[0], 0.f);
        else if constexpr (V == 4) *reinterpret_cast<uint2*>(p) = make_uint2(pack2(f[0], f[1]), pack2(f[2], f[3]));
        else *reinterpret_cast<uint4*>(p) = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
    }
}

// Sum over the TPR threads of a row (every thread gets it).  Rows of more
// than a wave exchange their waves' sums through LDS; `red` is the row
// group's (one per workgroup then), and the caller alternates two of them so
// that one barrier a sum is enough.
template <int TPR>
__device__ __forceinline__ float sum_row(float x, float* red) {
    if constexpr (TPR <= 32) {
        return row_sum<TPR>(x);
    } else {
        x = xor32_sum(row_sum<32>(x));
        if constexpr (TPR > 64) {
            if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
            __syncthreads();
            x = 0.f;
#pragma unroll
            for (int i = 0; i < TPR / 64; ++i) x += red[i];
        }
        return x;
    }
}

template <int TPR>
constexpr int ln_threads() { return TPR > 256 ? TPR : 256; }

// A row's vectors of this thread; rows and columns past the end are zero.
template <int DT, int V, int TPR, int NV>
__device__ __forceinline__ void ld_row(Raw<DT, V> (&r)[NV], const void* base, int64_t row, bool on, int n, int c0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = c0 + i * TPR * V;
#pragma unroll
        for (int k = 0; k < Raw<DT, V>::kWords; ++k) r[i].w[k] = 0;
        if (on && c < n) ld<DT, V>(r[i], base, row * n + c);
    }
}
// V entries of a parameter row (w or b), `none` where it is not given
template <int V>
__device__ __forceinline__ void ld_param(float (&f)[V], const float* p, int c, float none) {
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = none;
    if (!p) return;
    if constexpr (V == 1) {
        f[0] = p[c];
    } else {
#pragma unroll
        for (int k = 0; k < V; k += 4) {
            const float4 x = *reinterpret_cast<const float4*>(p + c + k);
            f[k] = x.x;
            f[k + 1] = x.y;
            f[k + 2] = x.z;
            f[k + 3] = x.w;
        }
    }
}

// A workgroup's row groups take rows in steps of the grid, the next row in
// flight while this one is worked off.
template <int XT, int YT, int V, int TPR, int NV>
__global__ __launch_bounds__(ln_threads<TPR>()) void k_ln_fwd(LnArgs a) {
    constexpr int RPB = ln_threads<TPR>() / TPR;
    __shared__ float red[2][16];
    const int n = (int)a.n;
    const int c0 = (threadIdx.x % TPR) * V;
    const float inv_n = 1.f / (float)n;
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    Raw<XT, V> cur[NV], nxt[NV];
    ld_row<XT, V, TPR, NV>(cur, a.x, row, row < a.rows, n, c0);
    // (row - threadIdx.x / TPR is the same for the whole workgroup: so is the loop)
    for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < a.rows; row0 += step, row += step) {
        const bool on = row < a.rows;
        if (row0 + step < a.rows) ld_row<XT, V, TPR, NV>(nxt, a.x, row + step, row + step < a.rows, n, c0);
        float x[NV][V];
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                x[i][e] = el<XT, V>(cur[i], e);
                s += x[i][e];
            }
        const float mean = sum_row<TPR>(s, red[0]) * inv_n;
        float q = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (c0 + i * TPR * V < n) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    x[i][e] -= mean;
                    q += x[i][e] * x[i][e];
                }
            }
        }
        const float rstd = 1.f / __fsqrt_rn(sum_row<TPR>(q, red[1]) * inv_n + a.eps);
        if (on) {
            if (threadIdx.x % TPR == 0) {
                if (a.mean) a.mean[row] = mean;
                if (a.rstd) a.rstd[row] = rstd;
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = c0 + i * TPR * V;
                if (c < n) {
                    float y[V], w[V], b[V];
                    ld_param<V>(w, a.w, c, 1.f);
                    ld_param<V>(b, a.b, c, 0.f);
#pragma unroll
                    for (int e = 0; e < V; ++e) y[e] = x[i][e] * rstd * w[e] + b[e];
                    stv<YT, V>(a.y, row * n + c, y);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) cur[i] = nxt[i];
    }
}

// One workgroup's rows, blockIdx.x RPB + group, in steps of the grid; its
// columns' sums over them to row blockIdx.x of the partial sums.
template <int XT, int YT, int V, int TPR, int NV>
__global__ __launch_bounds__(ln_threads<TPR>()) void k_ln_bwd(LnArgs a) {
    constexpr int NT = ln_threads<TPR>(), RPB = NT / TPR;
    __shared__ float red[4][16];
    __shared__ __attribute__((aligned(16))) float fold[RPB > 1 ? NT * V * NV : 1];
    const int n = (int)a.n;
    const int c0 = (threadIdx.x % TPR) * V;
    const float inv_n = 1.f / (float)n;
    float w[NV][V], sw[NV][V], sb[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = c0 + i * TPR * V;
        ld_param<V>(w[i], c < n ? a.w : nullptr, c, 1.f);
#pragma unroll
        for (int e = 0; e < V; ++e) sw[i][e] = sb[i][e] = 0.f;
    }
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    Raw<XT, V> cx[NV], nx[NV];
    Raw<YT, V> cd[NV], nd[NV];
    float cm = 0.f, cr = 0.f, nm = 0.f, nr = 0.f;
    auto fetch = [&](Raw<XT, V>(&x)[NV], Raw<YT, V>(&d)[NV], float& m, float& r, int64_t at) {
        const bool on = at < a.rows;
        ld_row<XT, V, TPR, NV>(x, a.x, at, on, n, c0);
        ld_row<YT, V, TPR, NV>(d, a.dy, at, on, n, c0);
        m = on ? a.mean[at] : 0.f;
        r = on ? a.rstd[at] : 0.f;
    };
    fetch(cx, cd, cm, cr, row);
    int flip = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < a.rows; row0 += step, row += step, flip ^= 2) {
        const bool on = row < a.rows;
        if (row0 + step < a.rows) fetch(nx, nd, nm, nr, row + step);
        float x[NV][V], g[NV][V];
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            // (a column past the end has dy = 0, and its x is never stored)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float dy = el<YT, V>(cd[i], e), xh = (el<XT, V>(cx[i], e) - cm) * cr;
                sw[i][e] += dy * xh;
                sb[i][e] += dy;
                x[i][e] = xh;
                g[i][e] = dy * w[i][e];
                s1 += g[i][e];
                s2 += g[i][e] * xh;
            }
        }
        const float m1 = sum_row<TPR>(s1, red[flip]) * inv_n;
        const float m2 = sum_row<TPR>(s2, red[flip + 1]) * inv_n;
        if (on && a.y) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = c0 + i * TPR * V;
                if (c < n) {
                    float dx[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) dx[e] = cr * (g[i][e] - m1 - x[i][e] * m2);
                    stv<XT, V>(a.y, row * n + c, dx);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            cx[i] = nx[i];
            cd[i] = nd[i];
        }
        cm = nm;
        cr = nr;
    }
    if (!a.want_params) return;
    float* pw = a.part + (int64_t)blockIdx.x * n;
    float* pb = a.part + ((int64_t)gridDim.x + blockIdx.x) * n;
    if constexpr (RPB == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * TPR * V;
            if (c < n) {
                stv<GDN_F32, V>(pw, c, sw[i]);
                stv<GDN_F32, V>(pb, c, sb[i]);
            }
        }
    } else {
        // row groups added in LDS, column by column (dw, then db)
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < V; ++e)
                    fold[(threadIdx.x / TPR) * (TPR * V * NV) + c0 + i * TPR * V + e] = pass ? sb[i][e] : sw[i][e];
            __syncthreads();
            for (int c = threadIdx.x; c < n; c += NT) {
                float t = 0.f;
#pragma unroll
                for (int r = 0; r < RPB; ++r) t += fold[r * (TPR * V * NV) + c];
                (pass ? pb : pw)[c] = t;
            }
        }
    }
}

// dw (blockIdx.y 0) and db (1) from `groups` partial rows: 16 columns a
// workgroup, 64 threads a column
constexpr int kPc = 16, kPr = 64;
__global__ __launch_bounds__(kPc* kPr) void k_ln_params(const float* part, int groups, int64_t n, float* dw, float* db) {
    __shared__ float red[kPr][kPc + 1];
    float* dst = blockIdx.y ? db : dw;
    if (!dst) return;
    const float* src = part + (blockIdx.y ? (int64_t)groups * n : 0);
    const int tc = threadIdx.x % kPc, tr = threadIdx.x / kPc;
    const int64_t c = (int64_t)blockIdx.x * kPc + tc;
    float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
    if (c < n) {
        int r = tr;
        for (; r + 3 * kPr < groups; r += 4 * kPr) {
            s0 += src[(int64_t)r * n + c];
            s1 += src[(int64_t)(r + kPr) * n + c];
            s2 += src[(int64_t)(r + 2 * kPr) * n + c];
            s3 += src[(int64_t)(r + 3 * kPr) * n + c];
        }
        for (; r < groups; r += kPr) s0 += src[(int64_t)r * n + c];
    }
    red[tr][tc] = (s0 + s1) + (s2 + s3);
    __syncthreads();
    if (tr == 0 && c < n) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kPr; ++i) s += red[i][tc];
        dst[c] = s;
    }
}

// Backward workgroups: enough to fill the device a few times over, no more
// than the rows give work for
constexpr int kMaxGroups = 512;
constexpr int kFwdBlocks = 2048;
int ln_rows_per_block(int tpr) { return tpr > 256 ? 1 : 256 / tpr; }

// Threads a row and vectors a thread: the least that hold the row, at most 32
// elements a thread.
struct LnShape {
    int tpr, nv;
};
constexpr LnShape ln_shape(int64_t n, int v) {
    const int64_t nvec = (n + v - 1) / v;
    if (nvec <= 8) return {8, 1};
    if (nvec <= 16) return {8, 2};
    if (nvec <= 32) return {16, 2};
    if (nvec <= 64) return {32, 2};
    if (nvec <= 128) return {64, 2};
    if (nvec <= 256) return {64, 4};
    if (nvec <= 512) return {256, 2};
    if (nvec <= 1024) return {256, 4};
    if (nvec <= 2048) return v == 8 ? LnShape{1024, 2} : LnShape{256, 8};
    if (nvec <= 4096) return {1024, 4};
    if (nvec <= 8192) return {1024, 8};
    return {1024, 16};
}
// Whether any width takes TPR threads and NV vectors of v elements (the
// shapes change at powers of two of vectors, and the widest row is one)
constexpr bool ln_taken(int v, int tpr, int nv) {
    for (int64_t nvec = 8; nvec * v <= kLayerNormMaxCols; nvec *= 2) {
        const LnShape s = ln_shape(nvec * v, v);
        if (s.tpr == tpr && s.nv == nv) return true;
    }
    return false;
}
int64_t ln_groups(int64_t rows, int tpr) {
    const int64_t rpb = ln_rows_per_block(tpr);
    return std::min<int64_t>((rows + rpb - 1) / rpb, tpr > 256 ? kMaxGroups / 2 : kMaxGroups);
}

template <int XT, int YT, int V, int TPR, int NV>
hipError_t launch(const LnArgs& a, bool bwd, hipStream_t st) {
    if constexpr (!ln_taken(V, TPR, NV)) {
        return hipErrorInvalidValue;  // (never asked for)
    } else {
        const int64_t blocks = (a.rows + ln_rows_per_block(TPR) - 1) / ln_rows_per_block(TPR);
        if (bwd)
            hipLaunchKernelGGL((k_ln_bwd<XT, YT, V, TPR, NV>), dim3((unsigned)ln_groups(a.rows, TPR)), dim3(ln_threads<TPR>()),
                               0, st, a);
        else
            hipLaunchKernelGGL((k_ln_fwd<XT, YT, V, TPR, NV>), dim3((unsigned)std::min<int64_t>(blocks, kFwdBlocks)),
                               dim3(ln_threads<TPR>()), 0, st, a);
        return hipGetLastError();
    }
}

template <int XT, int YT, int V>
hipError_t launch_v(const LnArgs& a, bool bwd, hipStream_t st) {
    const LnShape s = ln_shape(a.n, V);
    switch (s.tpr * 100 + s.nv) {
        case 801: return launch<XT, YT, V, 8, 1>(a, bwd, st);
        case 802: return launch<XT, YT, V, 8, 2>(a, bwd, st);
        case 1602: return launch<XT, YT, V, 16, 2>(a, bwd, st);
        case 3202: return launch<XT, YT, V, 32, 2>(a, bwd, st);
        case 6402: return launch<XT, YT, V, 64, 2>(a, bwd, st);
        case 6404: return launch<XT, YT, V, 64, 4>(a, bwd, st);
        case 25602: return launch<XT, YT, V, 256, 2>(a, bwd, st);
        case 25604: return launch<XT, YT, V, 256, 4>(a, bwd, st);
        case 25608: return launch<XT, YT, V, 256, 8>(a, bwd, st);
        case 102402: return launch<XT, YT, V, 1024, 2>(a, bwd, st);
        case 102404: return launch<XT, YT, V, 1024, 4>(a, bwd, st);
        case 102408: return launch<XT, YT, V, 1024, 8>(a, bwd, st);
        default: return launch<XT, YT, V, 1024, 16>(a, bwd, st);
    }
}

// Vectors a row is moved in: 16 bytes (8 bf16, 4 of a mix or of fp32) where
// rows and pointers are whole vectors, single elements otherwise.
int ln_vector(const LnArgs& a, int xt, int yt) {
    const uintptr_t ptrs = (uintptr_t)a.x | (uintptr_t)a.y | (uintptr_t)a.dy | (uintptr_t)a.w | (uintptr_t)a.b;
    if (ptrs % 16 != 0) return 1;
    if (xt == GDN_BF16 && yt == GDN_BF16 && a.n % 8 == 0) return 8;
    return a.n % 4 == 0 ? 4 : 1;
}

template <int XT, int YT>
hipError_t launch_t(const LnArgs& a, bool bwd, hipStream_t st) {
    const int v = ln_vector(a, XT, YT);
    if constexpr (XT == GDN_BF16 && YT == GDN_BF16)
        if (v == 8) return launch_v<XT, YT, 8>(a, bwd, st);
    return v == 1 ? launch_v<XT, YT, 1>(a, bwd, st) : launch_v<XT, YT, 4>(a, bwd, st);
}

hipError_t launch_any(const LnArgs& a, int xt, int yt, bool bwd, hipStream_t st) {
    if (xt == GDN_BF16) return yt == GDN_BF16 ? launch_t<GDN_BF16, GDN_BF16>(a, bwd, st) : launch_t<GDN_BF16, GDN_F32>(a, bwd, st);
    return yt == GDN_BF16 ? launch_t<GDN_F32, GDN_BF16>(a, bwd, st) : launch_t<GDN_F32, GDN_F32>(a, bwd, st);
}

}  // namespace

size_t layer_norm_workspace(int64_t rows, int64_t n) {
    // the most workgroups any vector width takes for these sizes
    int64_t g = 0;
    for (int v : {1, 4, 8}) g = std::max(g, ln_groups(rows, ln_shape(n, v).tpr));
    return 2 * sizeof(float) * (size_t)g * (size_t)n;
}

hipError_t layer_norm_fwd(const LayerNorm& p, hipStream_t st) {
    if (p.rows == 0) return hipSuccess;
    LnArgs a{};
    a.rows = p.rows; a.n = p.n; a.eps = p.eps;
    a.x = p.x; a.w = p.weight; a.b = p.bias; a.y = p.y; a.mean = p.mean; a.rstd = p.rstd;
    prof_begin(p.timer, "k_ln_fwd", st);
    const hipError_t e = launch_any(a, p.x_dtype, p.y_dtype, false, st);
    prof_end(p.timer, st);
    return e;
}

hipError_t layer_norm_bwd(const LayerNorm& p, hipStream_t st) {
    LnArgs a{};
    a.rows = p.rows; a.n = p.n;
    a.x = p.x; a.dy = p.dy; a.w = p.weight; a.y = p.dx; a.mean = p.mean; a.rstd = p.rstd;
    a.part = p.part;
    a.want_params = p.dweight || p.dbias;
    hipError_t e = hipSuccess;
    int64_t groups = 0;
    if (p.rows > 0) {
        groups = ln_groups(p.rows, ln_shape(p.n, ln_vector(a, p.x_dtype, p.y_dtype)).tpr);
        prof_begin(p.timer, "k_ln_bwd", st);
        e = launch_any(a, p.x_dtype, p.y_dtype, true, st);
        prof_end(p.timer, st);
        if (e != hipSuccess) return e;
    }
    if (a.want_params) {
        prof_begin(p.timer, "k_ln_params", st);
        hipLaunchKernelGGL(k_ln_params, dim3((unsigned)((p.n + kPc - 1) / kPc), 2), dim3(kPc * kPr), 0, st, p.part, (int)groups,
                           p.n, p.dweight, p.dbias);
        prof_end(p.timer, st);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace gdn
