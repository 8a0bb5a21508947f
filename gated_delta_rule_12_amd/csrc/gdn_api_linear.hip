// C ABI of linear attention with a decay for each head and of the query and key
// norm: argument checks, workspace sizes, dispatch.  Every check runs on the host
// before anything is enqueued.
#include <algorithm>
#include <utility>

#include "gdn_internal.h"
#include "../../include/gdn.h"

namespace gdn {
namespace {

bool aligned(const void* ptr, uintptr_t a) { return (uintptr_t)ptr % a == 0; }
int finish(hipError_t e) { return e == hipSuccess ? GDN_OK : GDN_E_HIP; }

// Memory that a call reads or writes: n rows of `row` bytes, `stride` bytes apart
struct Memory {
    const void* at;
    int64_t row, n = 1, stride = 0;
    uintptr_t begin() const { return (uintptr_t)at; }
    uintptr_t end() const { return begin() + (uintptr_t)((n - 1) * stride + row); }
    bool none() const { return !at || row <= 0 || n <= 0; }
};
// Whether two of them have a byte in common.  Rows of one stride are compared row
// by row (slices of one projection lie between each other); of rows of different
// strides, their whole ranges.
bool meet(Memory a, Memory b) {
    if (a.none() || b.none() || a.end() <= b.begin() || b.end() <= a.begin()) return false;
    for (Memory* m : {&a, &b})
        if (m->n > 1 && m->stride == m->row) *m = Memory{m->at, m->n * m->row};
    if (a.n > 1 && b.n > 1 && a.stride != b.stride) return true;
    if (b.n == 1) std::swap(a, b);
    if (b.n == 1) return true;
    // b's row j and a's row i have one offset for each k = j - i; the smallest at
    // which b's row ends behind the begin of a's
    const int64_t off = (int64_t)(b.begin() - a.begin()), x = -off - b.row, s = b.stride;
    const int64_t k = std::max(x / s - (x % s < 0) + 1, 1 - a.n);
    return k < b.n && off + k * s < a.row;
}
bool dim_ok(int64_t d) { return d >= 16 && d <= 128 && d % 16 == 0; }
// Whether something written meets something read, or another written
template <int W, int R>
bool any_meet(const Memory (&written)[W], const Memory (&read)[R]) {
    for (int i = 0; i < W; ++i) {
        for (const Memory& r : read)
            if (meet(written[i], r)) return true;
        for (int j = 0; j < i; ++j)
            if (meet(written[i], written[j])) return true;
    }
    return false;
}
// All tokens' rows of d elements, and a pool's slots (as many as an index reaches)
template <class P>
Memory tokens_of(const void* at, int64_t d, int64_t stride, const P& p) {
    const int64_t e = p.dtype == GDN_BF16 ? 2 : 4;
    return {at, d * e, p.N, stride * e};
}
Memory pool_of(const void* at, int64_t slots, const Linear& p) {
    return {at, std::min<int64_t>(slots, INT32_MAX) * p.Hv * p.dk * p.dv * 4};
}

// A launch holds fewer than 2^32 threads.  The most a call asks for, for each
// sequence and head: 4 x 256 token by token, 16 x 256 between segments (forward:
// of those alone that have some).  For each segment and head, N Hv / 256 + S Hv of
// them at most: 4 x 256 for the outputs, 8 x 256 for the gradients, twice that in
// fp32.
constexpr int64_t kMaxStates = (int64_t)1 << 21, kMaxChunkStates = (int64_t)1 << 19, kMaxChunkRows = (int64_t)1 << 28;
constexpr int64_t kMaxStride = (int64_t)1 << 23;

int linear_check(const Linear& p, bool chunks, bool back = false) {
    if (p.dtype != GDN_F32 && p.dtype != GDN_BF16) return GDN_E_ARG;
    if (p.N < 0 || p.S < 0 || p.Hk < 0 || p.Hv < 0 || p.dk <= 0 || p.dv <= 0 || p.n_in < 0 || p.n_out < 0 || p.max_len < 0)
        return GDN_E_SHAPE;
    if (p.Hk == 0 ? p.Hv != 0 : p.Hv % p.Hk != 0) return GDN_E_SHAPE;
    // offsets into the sequences are 32-bit integers
    if (p.N > INT32_MAX || p.S > INT32_MAX || p.Hv > 65535) return GDN_E_SHAPE;
    if (!dim_ok(p.dk) || !dim_ok(p.dv)) return GDN_E_UNSUPPORTED;
    if (p.S * p.Hv > kMaxStates) return GDN_E_SHAPE;
    const int half = back && p.dtype == GDN_F32;
    if (chunks && (p.S * p.Hv > kMaxChunkStates >> half || p.N * p.Hv > kMaxChunkRows >> half)) return GDN_E_SHAPE;
    return GDN_OK;
}

Linear linear_sizes(int64_t N, int64_t S, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv, int64_t n_in, int64_t n_out,
                    int64_t max_len, int32_t dtype) {
    Linear p{};
    p.N = N; p.S = S; p.Hk = Hk; p.Hv = Hv; p.dk = dk; p.dv = dv;
    p.n_in = n_in; p.n_out = n_out; p.max_len = max_len;
    p.dtype = dtype;
    return p;
}

// token strides and pointers of q, k, v: whole rows, moved in 16-byte pieces
int linear_inputs(const Linear& p) {
    const int64_t e = p.dtype == GDN_BF16 ? 2 : 4;
    if (p.q_stride < p.Hk * p.dk || p.k_stride < p.Hk * p.dk || p.v_stride < p.Hv * p.dv) return GDN_E_SHAPE;
    if (p.q_stride > kMaxStride || p.k_stride > kMaxStride || p.v_stride > kMaxStride) return GDN_E_SHAPE;
    if ((p.q_stride * e | p.k_stride * e | p.v_stride * e) % 16 != 0) return GDN_E_ARG;
    if (p.N > 0 && (!p.q || !p.k || !p.v)) return GDN_E_ARG;
    if (!p.alpha || !p.cu) return GDN_E_ARG;
    if (!aligned(p.q, 16) || !aligned(p.k, 16) || !aligned(p.v, 16) || !aligned(p.alpha, 4) || !aligned(p.cu, 4) ||
        !aligned(p.slots_in, 4) || !aligned(p.slots_out, 4) || !aligned(p.s_in, 16) || !aligned(p.s_out, 16))
        return GDN_E_ARG;
    // without indices, sequence s has slot s
    if ((p.s_in && !p.slots_in && p.n_in < p.S) || (p.s_out && !p.slots_out && p.n_out < p.S)) return GDN_E_SHAPE;
    return GDN_OK;
}

int linear_common(int64_t N, int64_t S, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv, int64_t n_in, int64_t n_out,
                  int64_t max_len, int32_t dtype, float scale, const void* q, int64_t q_stride, const void* k,
                  int64_t k_stride, const void* v, int64_t v_stride, const float* alpha, const int32_t* cu_seqlens,
                  const float* state_in, const int32_t* slots_in, float* state_out, const int32_t* slots_out, void* out,
                  void* workspace, size_t workspace_bytes, void* stream, gdn_timer* timer) {
    Linear p = linear_sizes(N, S, Hk, Hv, dk, dv, n_in, n_out, max_len, dtype);
    int s = linear_check(p, linear_in_chunks(p));
    if (s != GDN_OK) return s;
    if (S * Hv == 0) return GDN_OK;
    p.scale = scale;
    p.q = q; p.k = k; p.v = v;
    p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride;
    p.alpha = alpha; p.cu = cu_seqlens;
    p.s_in = state_in; p.slots_in = slots_in; p.s_out = state_out; p.slots_out = slots_out;
    p.out = out;
    p.timer = timer;
    if ((s = linear_inputs(p)) != GDN_OK) return s;
    if ((N > 0 && !out) || !aligned(out, 16)) return GDN_E_ARG;
    const size_t need = linear_workspace(p);
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_E_WORKSPACE;
    if (!aligned(workspace, 16)) return GDN_E_ARG;
    // (the pools may be one, or views of one whose slots lie upon each other)
    const int64_t e = dtype == GDN_BF16 ? 2 : 4;
    const Memory from = pool_of(state_in, n_in, p), to = pool_of(state_out, n_out, p);
    const Memory read[] = {tokens_of(q, Hk * dk, q_stride, p), tokens_of(k, Hk * dk, k_stride, p),
                           tokens_of(v, Hv * dv, v_stride, p), {alpha, 4 * Hv}};
    const Memory written[] = {{out, N * Hv * dv * e}, to, {workspace, (int64_t)need}};
    if (any_meet(written, read) || meet(written[0], from) || meet(written[2], from)) return GDN_E_ARG;
    if (meet(from, to) && (int64_t)(from.begin() - to.begin()) % (4 * Hv * dk * dv) != 0) return GDN_E_ARG;
    return finish(linear_forward(p, workspace, static_cast<hipStream_t>(stream)));
}

int linear_bwd_common(int64_t N, int64_t S, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv, int64_t n_in, int32_t dtype,
                      float scale, const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                      int64_t v_stride, const float* alpha, const int32_t* cu_seqlens, const float* state_in,
                      const int32_t* slots_in, const void* grad_out, const float* grad_state_out, void* grad_q, void* grad_k,
                      void* grad_v, float* grad_alpha, float* grad_state0, void* workspace, size_t workspace_bytes,
                      void* stream, gdn_timer* timer) {
    LinearBwd b{};
    Linear& p = b.p;
    p = linear_sizes(N, S, Hk, Hv, dk, dv, n_in, 0, N, dtype);
    int s = linear_check(p, true, true);
    if (s != GDN_OK) return s;
    if (S * Hv == 0) return GDN_OK;
    p.scale = scale;
    p.q = q; p.k = k; p.v = v;
    p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride;
    p.alpha = alpha; p.cu = cu_seqlens;
    p.s_in = state_in; p.slots_in = slots_in;
    p.timer = timer;
    if ((s = linear_inputs(p)) != GDN_OK) return s;
    if (N > 0 && (!grad_out || !grad_q || !grad_k || !grad_v)) return GDN_E_ARG;
    if (!aligned(grad_out, 16) || !aligned(grad_state_out, 16) || !aligned(grad_q, 16) || !aligned(grad_k, 16) ||
        !aligned(grad_v, 16) || !aligned(grad_alpha, 4) || !aligned(grad_state0, 16) || !aligned(workspace, 16))
        return GDN_E_ARG;
    const size_t need = linear_backward_workspace(p);
    if (!workspace || workspace_bytes < need) return GDN_E_WORKSPACE;
    // workgroups write rows and states while others read theirs
    const int64_t e = dtype == GDN_BF16 ? 2 : 4, states = 4 * S * Hv * dk * dv;
    const Memory read[] = {tokens_of(q, Hk * dk, q_stride, p), tokens_of(k, Hk * dk, k_stride, p),
                           tokens_of(v, Hv * dv, v_stride, p), {grad_out, N * Hv * dv * e}, {grad_state_out, states},
                           pool_of(state_in, n_in, p), {alpha, 4 * Hv}};
    const Memory written[] = {{grad_q, N * Hk * dk * e}, {grad_k, N * Hk * dk * e}, {grad_v, N * Hv * dv * e},
                              {grad_alpha, 4 * Hv}, {grad_state0, states}, {workspace, (int64_t)need}};
    if (any_meet(written, read)) return GDN_E_ARG;
    b.dout = grad_out; b.ds_out = grad_state_out;
    b.dq = grad_q; b.dk = grad_k; b.dv = grad_v; b.dalpha = grad_alpha; b.ds0 = grad_state0;
    return finish(linear_backward(b, workspace, static_cast<hipStream_t>(stream)));
}

int qk_check(const QkNorm& p, int32_t rotation) {
    if (p.dtype != GDN_F32 && p.dtype != GDN_BF16) return GDN_E_ARG;
    if (rotation != GDN_ROTATE_HALVES && rotation != GDN_ROTATE_PAIRS) return GDN_E_ARG;
    if (p.N < 0 || p.Hq < 0 || p.Hk < 0 || p.d <= 0 || p.rot < 0 || p.rot > p.d || p.n_pos < 0) return GDN_E_SHAPE;
    if (p.N > INT32_MAX || p.n_pos > INT32_MAX || p.Hq > 65535 || p.Hk > 65535) return GDN_E_SHAPE;
    if (p.d > 256 || p.d % 16 != 0 || p.rot % 16 != 0) return GDN_E_UNSUPPORTED;
    if (qk_norm_blocks(p) >= (int64_t)1 << 24) return GDN_E_SHAPE;
    return GDN_OK;
}
// One of q and k: rows of x and of y (and dy), if it has heads
int qk_side(const QkNorm& p, int64_t heads, const void* x, int64_t xs, const void* y, int64_t ys) {
    const int64_t e = p.dtype == GDN_BF16 ? 2 : 4;
    if (heads == 0 || p.N == 0) return GDN_OK;
    if (xs < heads * p.d || ys < heads * p.d || xs > kMaxStride || ys > kMaxStride) return GDN_E_SHAPE;
    if (!x || !y || !aligned(x, 16) || !aligned(y, 16) || (xs | ys) * e % 16 != 0) return GDN_E_ARG;
    return GDN_OK;
}
int qk_tables(const QkNorm& p) {
    if (!aligned(p.wq, 16) || !aligned(p.wk, 16) || !aligned(p.cos, 16) || !aligned(p.sin, 16) || !aligned(p.positions, 4))
        return GDN_E_ARG;
    if (p.rot == 0 || p.N == 0) return GDN_OK;
    if (!p.cos || !p.sin) return GDN_E_ARG;
    return p.n_pos > 0 ? GDN_OK : GDN_E_SHAPE;
}
// What of q's or k's rows the rows at y may lie upon: nothing of them, or each row
// upon its own (in place)
bool same_rows(const Memory& x, const Memory& y) { return x.at == y.at && x.row == y.row && (x.n == 1 || x.stride == y.stride); }
bool qk_meet(const Memory& y, const Memory& x) { return !same_rows(x, y) && meet(x, y); }
QkNorm qk_sizes(int64_t N, int64_t Hq, int64_t Hk, int64_t d, int64_t rot, int64_t n_pos, int32_t dtype, int32_t rotation) {
    QkNorm p{};
    p.N = N; p.Hq = Hq; p.Hk = Hk; p.d = d; p.rot = rot; p.n_pos = n_pos;
    p.dtype = dtype;
    p.pairs = rotation == GDN_ROTATE_PAIRS;
    return p;
}

int qk_fwd_common(int64_t N, int64_t Hq, int64_t Hk, int64_t d, int64_t rot, int64_t n_pos, int32_t dtype, int32_t rotation,
                  float eps, const void* q, int64_t q_stride, const void* k, int64_t k_stride, const float* weight_q,
                  const float* weight_k, const float* cos, const float* sin, const int32_t* positions, void* q_out,
                  int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream, gdn_timer* timer) {
    QkNorm p = qk_sizes(N, Hq, Hk, d, rot, n_pos, dtype, rotation);
    int s = qk_check(p, rotation);
    if (s != GDN_OK) return s;
    p.eps = eps;
    p.q = q; p.k = k; p.q_stride = q_stride; p.k_stride = k_stride;
    p.wq = weight_q; p.wk = weight_k; p.cos = cos; p.sin = sin; p.positions = positions;
    p.yq = q_out; p.yk = k_out; p.yq_stride = q_out_stride; p.yk_stride = k_out_stride;
    p.timer = timer;
    if ((s = qk_side(p, Hq, q, q_stride, q_out, q_out_stride)) != GDN_OK) return s;
    if ((s = qk_side(p, Hk, k, k_stride, k_out, k_out_stride)) != GDN_OK) return s;
    if ((s = qk_tables(p)) != GDN_OK) return s;
    if (N * (Hq + Hk) == 0) return GDN_OK;
    const Memory read[] = {{weight_q, 4 * d}, {weight_k, 4 * d}, {cos, 2 * rot * n_pos}, {sin, 2 * rot * n_pos}, {positions, 4 * N}};
    const Memory xq = tokens_of(q, Hq * d, q_stride, p), xk = tokens_of(k, Hk * d, k_stride, p);
    const Memory written[] = {tokens_of(q_out, Hq * d, q_out_stride, p), tokens_of(k_out, Hk * d, k_out_stride, p)};
    if (any_meet(written, read) || qk_meet(written[0], xq) || meet(written[0], xk) || meet(written[1], xq) || qk_meet(written[1], xk))
        return GDN_E_ARG;
    return finish(qk_norm_fwd(p, static_cast<hipStream_t>(stream)));
}

int qk_bwd_common(int64_t N, int64_t Hq, int64_t Hk, int64_t d, int64_t rot, int64_t n_pos, int32_t dtype, int32_t rotation,
                  float eps, const void* grad_q_out, int64_t gq_stride, const void* grad_k_out, int64_t gk_stride,
                  const void* q, int64_t q_stride, const void* k, int64_t k_stride, const float* weight_q,
                  const float* weight_k, const float* cos, const float* sin, const int32_t* positions, void* grad_q,
                  void* grad_k, float* grad_weight_q, float* grad_weight_k, void* workspace, size_t workspace_bytes,
                  void* stream, gdn_timer* timer) {
    QkNorm p = qk_sizes(N, Hq, Hk, d, rot, n_pos, dtype, rotation);
    int s = qk_check(p, rotation);
    if (s != GDN_OK) return s;
    p.eps = eps;
    p.q = q; p.k = k; p.q_stride = q_stride; p.k_stride = k_stride;
    p.dyq = grad_q_out; p.dyk = grad_k_out; p.gq_stride = gq_stride; p.gk_stride = gk_stride;
    p.wq = weight_q; p.wk = weight_k; p.cos = cos; p.sin = sin; p.positions = positions;
    p.yq = grad_q; p.yk = grad_k; p.yq_stride = Hq * d; p.yk_stride = Hk * d;
    p.dwq = grad_weight_q; p.dwk = grad_weight_k;
    p.timer = timer;
    if ((grad_q || grad_weight_q) && (s = qk_side(p, Hq, q, q_stride, grad_q_out, gq_stride)) != GDN_OK) return s;
    if ((grad_k || grad_weight_k) && (s = qk_side(p, Hk, k, k_stride, grad_k_out, gk_stride)) != GDN_OK) return s;
    if ((s = qk_tables(p)) != GDN_OK) return s;
    if (!aligned(grad_q, 16) || !aligned(grad_k, 16) || !aligned(grad_weight_q, 4) || !aligned(grad_weight_k, 4)) return GDN_E_ARG;
    const size_t need = grad_weight_q || grad_weight_k ? qk_norm_workspace(p) : 0;
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return GDN_E_WORKSPACE;
        if (!aligned(workspace, 16)) return GDN_E_ARG;
    }
    // (the weights' gradients are written behind everything else)
    const Memory none{nullptr, 0};
    const Memory xq = grad_q || grad_weight_q ? tokens_of(q, Hq * d, q_stride, p) : none,
                 xk = grad_k || grad_weight_k ? tokens_of(k, Hk * d, k_stride, p) : none,
                 gq = xq.at ? tokens_of(grad_q_out, Hq * d, gq_stride, p) : none,
                 gk = xk.at ? tokens_of(grad_k_out, Hk * d, gk_stride, p) : none;
    const Memory read[] = {{weight_q, 4 * d}, {weight_k, 4 * d}, {cos, 2 * rot * n_pos}, {sin, 2 * rot * n_pos}, {positions, 4 * N}};
    const Memory yq = tokens_of(grad_q, Hq * d, Hq * d, p), yk = tokens_of(grad_k, Hk * d, Hk * d, p), ws{workspace, (int64_t)need};
    const Memory first[] = {yq, yk, ws}, all[] = {{grad_weight_q, 4 * d}, {grad_weight_k, 4 * d}, yq, yk, ws};
    if (any_meet(first, read) || any_meet(all, {none}) || any_meet({ws}, {xq, xk, gq, gk}) || any_meet({yq}, {xk, gk}) ||
        any_meet({yk}, {xq, gq}) || qk_meet(yq, xq) || qk_meet(yq, gq) || qk_meet(yk, xk) || qk_meet(yk, gk))
        return GDN_E_ARG;
    p.part = static_cast<float*>(workspace);
    return finish(qk_norm_bwd(p, static_cast<hipStream_t>(stream)));
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_linear_fwd(int64_t N, int64_t S, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv, int64_t n_in, int64_t n_out,
                   int64_t max_len, int32_t dtype, float scale, const void* q, int64_t q_stride, const void* k,
                   int64_t k_stride, const void* v, int64_t v_stride, const float* alpha, const int32_t* cu_seqlens,
                   const float* state_in, const int32_t* slots_in, float* state_out, const int32_t* slots_out, void* out,
                   void* workspace, size_t workspace_bytes, void* stream) {
    return linear_common(N, S, Hk, Hv, dk, dv, n_in, n_out, max_len, dtype, scale, q, q_stride, k, k_stride, v, v_stride, alpha,
                         cu_seqlens, state_in, slots_in, state_out, slots_out, out, workspace, workspace_bytes, stream, nullptr);
}

int gdn_linear_fwd_timed(int64_t N, int64_t S, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv, int64_t n_in, int64_t n_out,
                         int64_t max_len, int32_t dtype, float scale, const void* q, int64_t q_stride, const void* k,
                         int64_t k_stride, const void* v, int64_t v_stride, const float* alpha, const int32_t* cu_seqlens,
                         const float* state_in, const int32_t* slots_in, float* state_out, const int32_t* slots_out,
                         void* out, void* workspace, size_t workspace_bytes, void* stream, gdn_timer* timer) {
    return linear_common(N, S, Hk, Hv, dk, dv, n_in, n_out, max_len, dtype, scale, q, q_stride, k, k_stride, v, v_stride, alpha,
                         cu_seqlens, state_in, slots_in, state_out, slots_out, out, workspace, workspace_bytes, stream, timer);
}

size_t gdn_linear_workspace_bytes(int64_t N, int64_t S, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv, int64_t max_len,
                                  int32_t dtype) {
    const Linear p = linear_sizes(N, S, Hk, Hv, dk, dv, 0, 0, max_len, dtype);
    return linear_check(p, linear_in_chunks(p)) != GDN_OK || S * Hv == 0 ? 0 : linear_workspace(p);
}

int gdn_linear_backward(int64_t N, int64_t S, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv, int64_t n_in, int32_t dtype,
                        float scale, const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                        int64_t v_stride, const float* alpha, const int32_t* cu_seqlens, const float* state_in,
                        const int32_t* slots_in, const void* grad_out, const float* grad_state_out, void* grad_q,
                        void* grad_k, void* grad_v, float* grad_alpha, float* grad_state0, void* workspace,
                        size_t workspace_bytes, void* stream) {
    return linear_bwd_common(N, S, Hk, Hv, dk, dv, n_in, dtype, scale, q, q_stride, k, k_stride, v, v_stride, alpha, cu_seqlens,
                             state_in, slots_in, grad_out, grad_state_out, grad_q, grad_k, grad_v, grad_alpha, grad_state0,
                             workspace, workspace_bytes, stream, nullptr);
}

int gdn_linear_backward_timed(int64_t N, int64_t S, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv, int64_t n_in,
                              int32_t dtype, float scale, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                              const void* v, int64_t v_stride, const float* alpha, const int32_t* cu_seqlens,
                              const float* state_in, const int32_t* slots_in, const void* grad_out,
                              const float* grad_state_out, void* grad_q, void* grad_k, void* grad_v, float* grad_alpha,
                              float* grad_state0, void* workspace, size_t workspace_bytes, void* stream, gdn_timer* timer) {
    return linear_bwd_common(N, S, Hk, Hv, dk, dv, n_in, dtype, scale, q, q_stride, k, k_stride, v, v_stride, alpha, cu_seqlens,
                             state_in, slots_in, grad_out, grad_state_out, grad_q, grad_k, grad_v, grad_alpha, grad_state0,
                             workspace, workspace_bytes, stream, timer);
}

size_t gdn_linear_backward_workspace_bytes(int64_t N, int64_t S, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv, int32_t dtype) {
    const Linear p = linear_sizes(N, S, Hk, Hv, dk, dv, 0, 0, N, dtype);
    return linear_check(p, true, true) != GDN_OK || S * Hv == 0 ? 0 : linear_backward_workspace(p);
}

int gdn_qk_norm_fwd(int64_t N, int64_t Hq, int64_t Hk, int64_t d, int64_t rot, int64_t n_pos, int32_t dtype, int32_t rotation,
                    float eps, const void* q, int64_t q_stride, const void* k, int64_t k_stride, const float* weight_q,
                    const float* weight_k, const float* cos, const float* sin, const int32_t* positions, void* q_out,
                    int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream) {
    return qk_fwd_common(N, Hq, Hk, d, rot, n_pos, dtype, rotation, eps, q, q_stride, k, k_stride, weight_q, weight_k, cos, sin,
                         positions, q_out, q_out_stride, k_out, k_out_stride, stream, nullptr);
}

int gdn_qk_norm_fwd_timed(int64_t N, int64_t Hq, int64_t Hk, int64_t d, int64_t rot, int64_t n_pos, int32_t dtype,
                          int32_t rotation, float eps, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                          const float* weight_q, const float* weight_k, const float* cos, const float* sin,
                          const int32_t* positions, void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                          void* stream, gdn_timer* timer) {
    return qk_fwd_common(N, Hq, Hk, d, rot, n_pos, dtype, rotation, eps, q, q_stride, k, k_stride, weight_q, weight_k, cos, sin,
                         positions, q_out, q_out_stride, k_out, k_out_stride, stream, timer);
}

int gdn_qk_norm_backward(int64_t N, int64_t Hq, int64_t Hk, int64_t d, int64_t rot, int64_t n_pos, int32_t dtype,
                         int32_t rotation, float eps, const void* grad_q_out, int64_t gq_stride, const void* grad_k_out,
                         int64_t gk_stride, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                         const float* weight_q, const float* weight_k, const float* cos, const float* sin,
                         const int32_t* positions, void* grad_q, void* grad_k, float* grad_weight_q, float* grad_weight_k,
                         void* workspace, size_t workspace_bytes, void* stream) {
    return qk_bwd_common(N, Hq, Hk, d, rot, n_pos, dtype, rotation, eps, grad_q_out, gq_stride, grad_k_out, gk_stride, q, q_stride,
                         k, k_stride, weight_q, weight_k, cos, sin, positions, grad_q, grad_k, grad_weight_q, grad_weight_k,
                         workspace, workspace_bytes, stream, nullptr);
}

int gdn_qk_norm_backward_timed(int64_t N, int64_t Hq, int64_t Hk, int64_t d, int64_t rot, int64_t n_pos, int32_t dtype,
                               int32_t rotation, float eps, const void* grad_q_out, int64_t gq_stride,
                               const void* grad_k_out, int64_t gk_stride, const void* q, int64_t q_stride, const void* k,
                               int64_t k_stride, const float* weight_q, const float* weight_k, const float* cos,
                               const float* sin, const int32_t* positions, void* grad_q, void* grad_k,
                               float* grad_weight_q, float* grad_weight_k, void* workspace, size_t workspace_bytes,
                               void* stream, gdn_timer* timer) {
    return qk_bwd_common(N, Hq, Hk, d, rot, n_pos, dtype, rotation, eps, grad_q_out, gq_stride, grad_k_out, gk_stride, q, q_stride,
                         k, k_stride, weight_q, weight_k, cos, sin, positions, grad_q, grad_k, grad_weight_q, grad_weight_k,
                         workspace, workspace_bytes, stream, timer);
}

size_t gdn_qk_norm_workspace_bytes(int64_t N, int64_t Hq, int64_t Hk, int64_t d) {
    const QkNorm p = qk_sizes(N, Hq, Hk, d, 0, 0, GDN_F32, GDN_ROTATE_HALVES);
    return qk_check(p, GDN_ROTATE_HALVES) != GDN_OK ? 0 : qk_norm_workspace(p);
}

}  // extern "C"
