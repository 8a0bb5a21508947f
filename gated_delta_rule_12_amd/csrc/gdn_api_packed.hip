// C ABI of the packed gated delta rule and of layer norm: argument checks,
// workspace sizes, dispatch.  Every check runs on the host before anything is
// enqueued.
#include "gdn_internal.h"
#include "../../include/gdn.h"

namespace gdn {
namespace {

bool aligned(const void* ptr, uintptr_t a) { return (uintptr_t)ptr % a == 0; }
int finish(hipError_t e) { return e == hipSuccess ? GDN_OK : GDN_E_HIP; }
bool dim_ok(int64_t d) { return d >= 16 && d <= 128 && d % 16 == 0; }
// A launch holds fewer than 2^32 threads.  The most a call asks for: 4 x 256 a
// sequence and head token by token; 8 x 512 a sequence and head and, beside
// those, 8 x 512 a head and 2048 tokens or 256 a head and 64 tokens in chunks.
constexpr int64_t kMaxStates = (int64_t)1 << 21, kMaxChunkStates = (int64_t)1 << 19, kMaxChunkRows = (int64_t)1 << 28;
constexpr int64_t kMaxStride = (int64_t)1 << 23;

int packed_check(const Packed& p) {
    if (p.dtype != GDN_F32 && p.dtype != GDN_BF16) return GDN_E_ARG;
    if (p.gate != GDN_GATE_SCALAR && p.gate != GDN_GATE_CHANNEL) return GDN_E_ARG;
    if (p.order != GDN_PREDICT_THEN_DECAY && p.order != GDN_DECAY_THEN_PREDICT) return GDN_E_ARG;
    if (p.N < 0 || p.S < 0 || p.Hk < 0 || p.Hv < 0 || p.dk <= 0 || p.dv <= 0 || p.n_in < 0 || p.n_out < 0 || p.max_len < 0)
        return GDN_E_SHAPE;
    if (p.Hk == 0 ? p.Hv != 0 : p.Hv % p.Hk != 0) return GDN_E_SHAPE;
    // offsets into the sequences are 32-bit integers
    if (p.N > INT32_MAX || p.S > INT32_MAX || p.Hv > 65535) return GDN_E_SHAPE;
    if (!dim_ok(p.dk) || !dim_ok(p.dv)) return GDN_E_UNSUPPORTED;
    if (p.S * p.Hv > kMaxStates) return GDN_E_SHAPE;
    return GDN_OK;
}
int chunk_check(const Packed& p) {
    return p.S * p.Hv > kMaxChunkStates || p.N * p.Hv > kMaxChunkRows ? GDN_E_SHAPE : GDN_OK;
}
int packed_fwd_check(const Packed& p) {
    const int s = packed_check(p);
    return s == GDN_OK && packed_in_chunks(p) ? chunk_check(p) : s;
}
int packed_bwd_check(const Packed& p) {
    const int s = packed_check(p);
    if (s != GDN_OK) return s;
    return chunked_backward_supported(p.dk, p.dv, p.gate) ? chunk_check(p) : GDN_E_UNSUPPORTED;
}

Packed packed_sizes(int64_t N, int64_t S, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv, int64_t n_in,
                    int64_t n_out, int64_t max_len, int32_t dtype, int32_t gate, int32_t order) {
    Packed p{};
    p.N = N; p.S = S; p.Hk = Hk; p.Hv = Hv; p.dk = dk; p.dv = dv;
    p.n_in = n_in; p.n_out = n_out; p.max_len = max_len;
    p.dtype = dtype; p.gate = gate; p.order = order;
    return p;
}

// token strides and pointers of q, k, v: whole rows, moved in 16-byte pieces
int packed_inputs(const Packed& p) {
    const int64_t e = p.dtype == GDN_BF16 ? 2 : 4;
    if (p.q_stride < p.Hk * p.dk || p.k_stride < p.Hk * p.dk || p.v_stride < p.Hv * p.dv) return GDN_E_SHAPE;
    // (a chunk's rows are addressed with 32-bit offsets)
    if (p.q_stride > kMaxStride || p.k_stride > kMaxStride || p.v_stride > kMaxStride) return GDN_E_SHAPE;
    if ((p.q_stride * e | p.k_stride * e | p.v_stride * e) % 16 != 0) return GDN_E_ARG;
    if (p.N > 0 && (!p.q || !p.k || !p.v || !p.alpha || !p.beta)) return GDN_E_ARG;
    if (!p.cu) return GDN_E_ARG;
    if (!aligned(p.q, 16) || !aligned(p.k, 16) || !aligned(p.v, 16) || !aligned(p.beta, 4) || !aligned(p.cu, 4) ||
        !aligned(p.alpha, p.gate == GDN_GATE_CHANNEL ? 16 : 4) || !aligned(p.slots_in, 4) || !aligned(p.slots_out, 4) ||
        !aligned(p.s_in, 16) || !aligned(p.s_out, 16))
        return GDN_E_ARG;
    // without indices, sequence s has slot s
    if ((p.s_in && !p.slots_in && p.n_in < p.S) || (p.s_out && !p.slots_out && p.n_out < p.S)) return GDN_E_SHAPE;
    return GDN_OK;
}

int packed_common(int64_t N, int64_t S, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv, int64_t n_in,
                  int64_t n_out, int64_t max_len, int32_t dtype, int32_t gate, int32_t order, float scale, const void* q, int64_t q_stride,
                  const void* k, int64_t k_stride, const void* v, int64_t v_stride, const float* alpha, const float* beta,
                  const int32_t* cu_seqlens, const float* state_in, const int32_t* slots_in, float* state_out,
                  const int32_t* slots_out, void* out, void* workspace, size_t workspace_bytes, void* stream,
                  gdn_timer* timer) {
    Packed p = packed_sizes(N, S, Hk, Hv, dk, dv, n_in, n_out, max_len, dtype, gate, order);
    int s = packed_fwd_check(p);
    if (s != GDN_OK) return s;
    if (S * Hv == 0) return GDN_OK;
    p.scale = scale;
    p.q = q; p.k = k; p.v = v;
    p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride;
    p.alpha = alpha; p.beta = beta; p.cu = cu_seqlens;
    p.s_in = state_in; p.slots_in = slots_in; p.s_out = state_out; p.slots_out = slots_out;
    p.out = out;
    p.timer = timer;
    if ((s = packed_inputs(p)) != GDN_OK) return s;
    if ((N > 0 && !out) || !aligned(out, 16)) return GDN_E_ARG;
    const size_t need = packed_workspace(p);
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_E_WORKSPACE;
    if (!aligned(workspace, 16)) return GDN_E_ARG;
    return finish(packed_forward(p, workspace, static_cast<hipStream_t>(stream)));
}

int packed_bwd_common(int64_t N, int64_t S, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv, int64_t n_in, int32_t dtype,
                      int32_t gate, int32_t order, float scale, const void* q, int64_t q_stride, const void* k,
                      int64_t k_stride, const void* v, int64_t v_stride, const float* alpha, const float* beta,
                      const int32_t* cu_seqlens, const float* state_in, const int32_t* slots_in, const void* grad_out,
                      const float* grad_state_out, float* grad_q, float* grad_k, float* grad_v, float* grad_alpha,
                      float* grad_beta, float* grad_state0, void* workspace, size_t workspace_bytes, void* stream,
                      gdn_timer* timer) {
    PackedBwd b{};
    Packed& p = b.p;
    p = packed_sizes(N, S, Hk, Hv, dk, dv, n_in, 0, N, dtype, gate, order);
    int s = packed_bwd_check(p);
    if (s != GDN_OK) return s;
    if (S * Hv == 0) return GDN_OK;
    p.scale = scale;
    p.q = q; p.k = k; p.v = v;
    p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride;
    p.alpha = alpha; p.beta = beta; p.cu = cu_seqlens;
    p.s_in = state_in; p.slots_in = slots_in;
    p.timer = timer;
    if ((s = packed_inputs(p)) != GDN_OK) return s;
    if (N > 0 && (!grad_out || !grad_q || !grad_k || !grad_v || !grad_alpha || !grad_beta)) return GDN_E_ARG;
    if (!aligned(grad_out, 16) || !aligned(grad_state_out, 16) || !aligned(grad_q, 16) || !aligned(grad_k, 16) ||
        !aligned(grad_v, 16) || !aligned(grad_alpha, 4) || !aligned(grad_beta, 4) || !aligned(grad_state0, 16) ||
        !aligned(workspace, 16))
        return GDN_E_ARG;
    const size_t need = packed_backward_workspace(p);
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_E_WORKSPACE;
    b.dout = grad_out; b.ds_out = grad_state_out;
    b.dq = grad_q; b.dk = grad_k; b.dv = grad_v; b.dalpha = grad_alpha; b.dbeta = grad_beta; b.ds0 = grad_state0;
    return finish(packed_backward(b, workspace, static_cast<hipStream_t>(stream)));
}

int norm_check(int64_t rows, int64_t n, int32_t x_dtype, int32_t y_dtype) {
    if ((x_dtype != GDN_F32 && x_dtype != GDN_BF16) || (y_dtype != GDN_F32 && y_dtype != GDN_BF16)) return GDN_E_ARG;
    if (rows < 0 || n <= 0 || rows > ((int64_t)1 << 40)) return GDN_E_SHAPE;
    if (n > kLayerNormMaxCols) return GDN_E_UNSUPPORTED;
    return GDN_OK;
}
bool elem_aligned(const void* ptr, int32_t dtype) { return aligned(ptr, dtype == GDN_BF16 ? 2 : 4); }

int norm_fwd_common(int64_t rows, int64_t n, int32_t x_dtype, int32_t y_dtype, float eps, const void* x,
                    const float* weight, const float* bias, void* y, float* mean, float* rstd, void* stream,
                    gdn_timer* timer) {
    const int s = norm_check(rows, n, x_dtype, y_dtype);
    if (s != GDN_OK) return s;
    if (rows == 0) return GDN_OK;
    if (!x || !y) return GDN_E_ARG;
    if (!elem_aligned(x, x_dtype) || !elem_aligned(y, y_dtype) || !aligned(weight, 4) || !aligned(bias, 4) ||
        !aligned(mean, 4) || !aligned(rstd, 4))
        return GDN_E_ARG;
    LayerNorm p{};
    p.rows = rows; p.n = n; p.x_dtype = x_dtype; p.y_dtype = y_dtype; p.eps = eps;
    p.x = x; p.weight = weight; p.bias = bias; p.y = y; p.mean = mean; p.rstd = rstd;
    p.timer = timer;
    return finish(layer_norm_fwd(p, static_cast<hipStream_t>(stream)));
}

int norm_bwd_common(int64_t rows, int64_t n, int32_t x_dtype, int32_t y_dtype, const void* grad_y, const void* x,
                    const float* weight, const float* mean, const float* rstd, void* grad_x, float* grad_weight,
                    float* grad_bias, void* workspace, size_t workspace_bytes, void* stream, gdn_timer* timer) {
    const int s = norm_check(rows, n, x_dtype, y_dtype);
    if (s != GDN_OK) return s;
    if (!grad_x && !grad_weight && !grad_bias) return GDN_OK;
    if (rows > 0 && (!grad_y || !x || !mean || !rstd)) return GDN_E_ARG;
    if (!elem_aligned(x, x_dtype) || !elem_aligned(grad_x, x_dtype) || !elem_aligned(grad_y, y_dtype) ||
        !aligned(weight, 4) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(grad_weight, 4) || !aligned(grad_bias, 4))
        return GDN_E_ARG;
    if (rows > 0 && (grad_weight || grad_bias)) {
        if (!workspace || workspace_bytes < layer_norm_workspace(rows, n)) return GDN_E_WORKSPACE;
        if (!aligned(workspace, 16)) return GDN_E_ARG;
    }
    LayerNorm p{};
    p.rows = rows; p.n = n; p.x_dtype = x_dtype; p.y_dtype = y_dtype;
    p.x = x; p.dy = grad_y; p.weight = weight; p.dx = grad_x;
    p.mean = const_cast<float*>(mean); p.rstd = const_cast<float*>(rstd);
    p.dweight = grad_weight; p.dbias = grad_bias;
    p.part = static_cast<float*>(workspace);
    p.timer = timer;
    return finish(layer_norm_bwd(p, static_cast<hipStream_t>(stream)));
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_packed_fwd(int64_t N, int64_t S, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv, int64_t n_in,
                   int64_t n_out, int64_t max_len, int32_t dtype, int32_t gate, int32_t order, float scale, const void* q,
                   int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride, const float* alpha,
                   const float* beta, const int32_t* cu_seqlens, const float* state_in, const int32_t* slots_in,
                   float* state_out, const int32_t* slots_out, void* out, void* workspace, size_t workspace_bytes,
                   void* stream) {
    return packed_common(N, S, Hk, Hv, dk, dv, n_in, n_out, max_len, dtype, gate, order, scale, q, q_stride, k, k_stride, v,
                         v_stride, alpha, beta, cu_seqlens, state_in, slots_in, state_out, slots_out, out, workspace,
                         workspace_bytes, stream, nullptr);
}

int gdn_packed_fwd_timed(int64_t N, int64_t S, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv, int64_t n_in,
                         int64_t n_out, int64_t max_len, int32_t dtype, int32_t gate, int32_t order, float scale, const void* q,
                         int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                         const float* alpha, const float* beta, const int32_t* cu_seqlens, const float* state_in,
                         const int32_t* slots_in, float* state_out, const int32_t* slots_out, void* out, void* workspace,
                         size_t workspace_bytes, void* stream, gdn_timer* timer) {
    return packed_common(N, S, Hk, Hv, dk, dv, n_in, n_out, max_len, dtype, gate, order, scale, q, q_stride, k, k_stride, v,
                         v_stride, alpha, beta, cu_seqlens, state_in, slots_in, state_out, slots_out, out, workspace,
                         workspace_bytes, stream, timer);
}

size_t gdn_packed_workspace_bytes(int64_t N, int64_t S, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv, int64_t max_len,
                                  int32_t dtype, int32_t gate) {
    const Packed p = packed_sizes(N, S, Hk, Hv, dk, dv, 0, 0, max_len, dtype, gate, GDN_PREDICT_THEN_DECAY);
    return packed_fwd_check(p) != GDN_OK || S * Hv == 0 ? 0 : packed_workspace(p);
}

int gdn_packed_path(int64_t dk, int64_t dv, int32_t dtype, int32_t gate) {
    const Packed p = packed_sizes(0, 0, 1, 1, dk, dv, 0, 0, 0, dtype, gate, GDN_PREDICT_THEN_DECAY);
    const int s = packed_check(p);
    if (s != GDN_OK) return s;
    return packed_chunked(p) ? GDN_PATH_MFMA : GDN_PATH_VALU;
}

int gdn_packed_backward(int64_t N, int64_t S, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv, int64_t n_in,
                        int32_t dtype, int32_t gate, int32_t order, float scale, const void* q, int64_t q_stride,
                        const void* k, int64_t k_stride, const void* v, int64_t v_stride, const float* alpha,
                        const float* beta, const int32_t* cu_seqlens, const float* state_in, const int32_t* slots_in,
                        const void* grad_out, const float* grad_state_out, float* grad_q, float* grad_k, float* grad_v,
                        float* grad_alpha, float* grad_beta, float* grad_state0, void* workspace, size_t workspace_bytes,
                        void* stream) {
    return packed_bwd_common(N, S, Hk, Hv, dk, dv, n_in, dtype, gate, order, scale, q, q_stride, k, k_stride, v, v_stride,
                             alpha, beta, cu_seqlens, state_in, slots_in, grad_out, grad_state_out, grad_q, grad_k, grad_v,
                             grad_alpha, grad_beta, grad_state0, workspace, workspace_bytes, stream, nullptr);
}

int gdn_packed_backward_timed(int64_t N, int64_t S, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv, int64_t n_in,
                        int32_t dtype, int32_t gate, int32_t order, float scale, const void* q, int64_t q_stride,
                        const void* k, int64_t k_stride, const void* v, int64_t v_stride, const float* alpha,
                        const float* beta, const int32_t* cu_seqlens, const float* state_in, const int32_t* slots_in,
                        const void* grad_out, const float* grad_state_out, float* grad_q, float* grad_k, float* grad_v,
                        float* grad_alpha, float* grad_beta, float* grad_state0, void* workspace, size_t workspace_bytes,
                        void* stream, gdn_timer* timer) {
    return packed_bwd_common(N, S, Hk, Hv, dk, dv, n_in, dtype, gate, order, scale, q, q_stride, k, k_stride, v, v_stride,
                             alpha, beta, cu_seqlens, state_in, slots_in, grad_out, grad_state_out, grad_q, grad_k, grad_v,
                             grad_alpha, grad_beta, grad_state0, workspace, workspace_bytes, stream, timer);
}

size_t gdn_packed_backward_workspace_bytes(int64_t N, int64_t S, int64_t Hk, int64_t Hv, int64_t dk, int64_t dv,
                                           int32_t dtype, int32_t gate) {
    const Packed p = packed_sizes(N, S, Hk, Hv, dk, dv, 0, 0, N, dtype, gate, GDN_PREDICT_THEN_DECAY);
    return packed_bwd_check(p) != GDN_OK ? 0 : packed_backward_workspace(p);
}

int gdn_layer_norm_fwd(int64_t rows, int64_t n, int32_t x_dtype, int32_t y_dtype, float eps, const void* x,
                       const float* weight, const float* bias, void* y, float* mean, float* rstd, void* stream) {
    return norm_fwd_common(rows, n, x_dtype, y_dtype, eps, x, weight, bias, y, mean, rstd, stream, nullptr);
}

int gdn_layer_norm_fwd_timed(int64_t rows, int64_t n, int32_t x_dtype, int32_t y_dtype, float eps, const void* x,
                             const float* weight, const float* bias, void* y, float* mean, float* rstd, void* stream,
                             gdn_timer* timer) {
    return norm_fwd_common(rows, n, x_dtype, y_dtype, eps, x, weight, bias, y, mean, rstd, stream, timer);
}

int gdn_layer_norm_backward(int64_t rows, int64_t n, int32_t x_dtype, int32_t y_dtype, const void* grad_y, const void* x,
                            const float* weight, const float* mean, const float* rstd, void* grad_x, float* grad_weight,
                            float* grad_bias, void* workspace, size_t workspace_bytes, void* stream) {
    return norm_bwd_common(rows, n, x_dtype, y_dtype, grad_y, x, weight, mean, rstd, grad_x, grad_weight, grad_bias,
                           workspace, workspace_bytes, stream, nullptr);
}

int gdn_layer_norm_backward_timed(int64_t rows, int64_t n, int32_t x_dtype, int32_t y_dtype, const void* grad_y,
                                  const void* x, const float* weight, const float* mean, const float* rstd, void* grad_x,
                                  float* grad_weight, float* grad_bias, void* workspace, size_t workspace_bytes,
                                  void* stream, gdn_timer* timer) {
    return norm_bwd_common(rows, n, x_dtype, y_dtype, grad_y, x, weight, mean, rstd, grad_x, grad_weight, grad_bias,
                           workspace, workspace_bytes, stream, timer);
}

size_t gdn_layer_norm_workspace_bytes(int64_t rows, int64_t n) {
    return norm_check(rows, n, GDN_F32, GDN_F32) != GDN_OK ? 0 : layer_norm_workspace(rows, n);
}

}  // extern "C"
