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
// Both directions are one pass over memory: a row sits in the registers of
// TPR threads (NV vectors of V elements each) between its load and its store,
// so x (and dy) are read once and y (dx) is written once, and the variance is
// taken from the centred values, not from a difference of sums.  Rows of up
// to 1024 elements (4 a vector) stay within a wave and reduce across lanes on
// the vector ALU; longer rows take a workgroup and one exchange through LDS
// per sum.  All statistics and sums are fp32.
//
// The weight's and bias's gradients: a thread owns the same columns in every
// row it handles, keeps their sums in registers over all its rows, the
// workgroup adds its row groups in LDS and writes one partial row; k_ln_params
// adds the partial rows.  Every sum has a fixed order (no atomics), so
// repeated calls give identical results.
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

// V consecutive elements as loaded: 4 or 8 move as one or two 16-byte (8-byte)
// pieces, 1 as an element
template <int DT, int V>
struct Vec {
    float f[V];
};
template <int DT, int V>
__device__ __forceinline__ Vec<DT, V> ldv(const void* base, int64_t i) {
    Vec<DT, V> v;
    if constexpr (V == 1) {
        v.f[0] = gdn_ld<DT>(base, i);
    } else if constexpr (DT == GDN_F32) {
#pragma unroll
        for (int k = 0; k < V; k += 4) {
            const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + i + k);
            v.f[k] = x.x;
            v.f[k + 1] = x.y;
            v.f[k + 2] = x.z;
            v.f[k + 3] = x.w;
        }
    } else {
        uint32_t u[V / 2];
        if constexpr (V == 8) {
            const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i);
            u[0] = x.x;
            u[1] = x.y;
            u[2] = x.z;
            u[3] = x.w;
        } else {
            const uint2 x = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + i);
            u[0] = x.x;
            u[1] = x.y;
        }
#pragma unroll
        for (int k = 0; k < V / 2; ++k) {
            v.f[2 * k] = __uint_as_float(u[k] << 16);
            v.f[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
        }
    }
    return v;
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

template <int XT, int YT, int V, int TPR, int NV>
__global__ __launch_bounds__(ln_threads<TPR>()) void k_ln_fwd(LnArgs a) {
    constexpr int RPB = ln_threads<TPR>() / TPR;
    __shared__ float red[2][16];
    const int n = (int)a.n;
    const int c0 = (threadIdx.x % TPR) * V;
    const float inv_n = 1.f / (float)n;
    for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < a.rows; row0 += (int64_t)gridDim.x * RPB) {
        const int64_t row = row0 + threadIdx.x / TPR;
        const bool on = row < a.rows;
        float x[NV][V];
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * TPR * V;
#pragma unroll
            for (int e = 0; e < V; ++e) x[i][e] = 0.f;
            if (on && c < n) {
                const Vec<XT, V> v = ldv<XT, V>(a.x, row * n + c);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    x[i][e] = v.f[e];
                    s += v.f[e];
                }
            }
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
        if (!on) continue;
        if (threadIdx.x % TPR == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * TPR * V;
            if (c < n) {
                float y[V];
                const Vec<GDN_F32, V> w = a.w ? ldv<GDN_F32, V>(a.w, c) : Vec<GDN_F32, V>{};
                const Vec<GDN_F32, V> b = a.b ? ldv<GDN_F32, V>(a.b, c) : Vec<GDN_F32, V>{};
#pragma unroll
                for (int e = 0; e < V; ++e) y[e] = x[i][e] * rstd * (a.w ? w.f[e] : 1.f) + b.f[e];
                stv<YT, V>(a.y, row * n + c, y);
            }
        }
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
        const Vec<GDN_F32, V> v = a.w && c < n ? ldv<GDN_F32, V>(a.w, c) : Vec<GDN_F32, V>{};
#pragma unroll
        for (int e = 0; e < V; ++e) {
            w[i][e] = a.w ? v.f[e] : 1.f;
            sw[i][e] = sb[i][e] = 0.f;
        }
    }
    int flip = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < a.rows; row0 += (int64_t)gridDim.x * RPB, flip ^= 2) {
        const int64_t row = row0 + threadIdx.x / TPR;
        const bool on = row < a.rows;
        float x[NV][V], g[NV][V];
        const float mean = on ? a.mean[row] : 0.f, rstd = on ? a.rstd[row] : 0.f;
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * TPR * V;
#pragma unroll
            for (int e = 0; e < V; ++e) x[i][e] = g[i][e] = 0.f;
            if (on && c < n) {
                const Vec<XT, V> xv = ldv<XT, V>(a.x, row * n + c);
                const Vec<YT, V> dv = ldv<YT, V>(a.dy, row * n + c);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float xh = (xv.f[e] - mean) * rstd;
                    sw[i][e] += dv.f[e] * xh;
                    sb[i][e] += dv.f[e];
                    x[i][e] = xh;
                    g[i][e] = dv.f[e] * w[i][e];
                    s1 += g[i][e];
                    s2 += g[i][e] * xh;
                }
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
                    for (int e = 0; e < V; ++e) dx[e] = rstd * (g[i][e] - m1 - x[i][e] * m2);
                    stv<XT, V>(a.y, row * n + c, dx);
                }
            }
        }
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
// workgroup, 16 threads a column
constexpr int kPc = 16, kPr = 16;
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
constexpr int kMaxGroups = 1024;
int ln_rows_per_block(int tpr) { return tpr > 256 ? 1 : 256 / tpr; }

// Threads a row and vectors a thread: the least that hold the row, at most 32
// elements a thread.
struct LnShape {
    int tpr, nv;
};
LnShape ln_shape(int64_t n, int v) {
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
int64_t ln_groups(int64_t rows, int tpr) {
    const int64_t rpb = ln_rows_per_block(tpr);
    return std::min<int64_t>((rows + rpb - 1) / rpb, tpr > 256 ? kMaxGroups / 4 : kMaxGroups);
}

template <int XT, int YT, int V, int TPR, int NV>
hipError_t launch(const LnArgs& a, bool bwd, hipStream_t st) {
    if constexpr (NV * V > 32) {
        return hipErrorInvalidValue;  // (no shape within kMaxCols asks for it)
    } else {
        const int64_t blocks = (a.rows + ln_rows_per_block(TPR) - 1) / ln_rows_per_block(TPR);
        if (bwd)
            hipLaunchKernelGGL((k_ln_bwd<XT, YT, V, TPR, NV>), dim3((unsigned)ln_groups(a.rows, TPR)), dim3(ln_threads<TPR>()),
                               0, st, a);
        else
            hipLaunchKernelGGL((k_ln_fwd<XT, YT, V, TPR, NV>), dim3((unsigned)std::min<int64_t>(blocks, 1 << 20)),
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
