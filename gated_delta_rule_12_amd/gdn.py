"""Thin Python binding of libgdn.so (include/gdn.h).

Argument marshalling only: every step of the forward pass runs in the HIP
kernels of libgdn.so.  PyTorch supplies device memory and the stream.  There
is no fallback: if the library is missing or no GPU is present, calls raise.

Low-level names mirror the C ABI (gdn_chunk_fwd, gdn_recurrent_ref,
gdn_seqpar_fwd, gdn_decode_step, ...); chunk_fwd / seqpar_fwd / recurrent_ref /
decode_step are the same calls taking torch tensors and allocating the
outputs and the workspace.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libgdn.so")

GDN_F32, GDN_BF16 = 0, 1
GDN_GATE_SCALAR, GDN_GATE_CHANNEL = 0, 1
GDN_PREDICT_THEN_DECAY, GDN_DECAY_THEN_PREDICT = 0, 1
GDN_OK, GDN_E_ARG, GDN_E_SHAPE, GDN_E_UNSUPPORTED, GDN_E_WORKSPACE, GDN_E_HIP = 0, -1, -2, -3, -4, -5
GDN_E_SCRATCH = -6
GDN_NOALLOC_SCRATCH_BYTES = 128 << 20
GDN_PATH_VALU, GDN_PATH_MFMA = 0, 1
GDN_ROTATE_HALVES, GDN_ROTATE_PAIRS = 0, 1
GDN_BWD_TOKEN, GDN_BWD_CHUNKED = 0, 1

# every symbol include/gdn.h declares
EXPORTS = ("gdn_chunk_fwd", "gdn_recurrent_ref", "gdn_seqpar_fwd", "gdn_decode_step",
           "gdn_decode_step_raw", "gdn_backward", "gdn_backward_workspace_bytes",
           "gdn_workspace_bytes",
           "gdn_validate", "gdn_chunk_path", "gdn_chunk_segments", "gdn_seqpar_segments",
           "gdn_status_str", "gdn_abi_version",
           "gdn_timer_create", "gdn_timer_destroy", "gdn_timer_read", "gdn_chunk_fwd_timed",
           "gdn_seqpar_fwd_timed", "gdn_decode_step_timed", "gdn_backward_timed",
           "gdn_chunk_fwd_noalloc", "gdn_chunk_fwd_raw", "gdn_chunk_fwd_raw_timed",
           "gdn_raw_workspace_bytes", "gdn_backward_path",
           "gdn_packed_fwd", "gdn_packed_fwd_timed", "gdn_packed_workspace_bytes", "gdn_packed_path",
           "gdn_packed_backward", "gdn_packed_backward_timed", "gdn_packed_backward_workspace_bytes",
           "gdn_layer_norm_fwd", "gdn_layer_norm_fwd_timed", "gdn_layer_norm_backward",
           "gdn_layer_norm_backward_timed", "gdn_layer_norm_workspace_bytes",
           "gdn_linear_fwd", "gdn_linear_fwd_timed", "gdn_linear_workspace_bytes",
           "gdn_linear_backward", "gdn_linear_backward_timed", "gdn_linear_backward_workspace_bytes",
           "gdn_qk_norm_fwd", "gdn_qk_norm_fwd_timed", "gdn_qk_norm_backward", "gdn_qk_norm_backward_timed",
           "gdn_qk_norm_workspace_bytes")

_lib = None


class GdnError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_str(status)} ({status})")
        self.status = status


def lib():
    """Load libgdn.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    L = ctypes.CDLL(LIB_PATH)
    i64, i32, f32, vp, sz = (ctypes.c_int64, ctypes.c_int32, ctypes.c_float,
                             ctypes.c_void_p, ctypes.c_size_t)
    shape = [i64, i64, i64, i64, i64]
    tens = [vp] * 8
    L.gdn_chunk_fwd.argtypes = shape + [i32, i32, i32, i32, f32] + tens + [vp, sz, vp]
    L.gdn_chunk_fwd.restype = ctypes.c_int
    L.gdn_chunk_fwd_raw.argtypes = shape + [i32, i32, i32, i32, f32] + tens + [vp, sz, vp]
    L.gdn_chunk_fwd_raw.restype = ctypes.c_int
    L.gdn_raw_workspace_bytes.argtypes = shape + [i32, i32, i32]
    L.gdn_raw_workspace_bytes.restype = sz
    L.gdn_chunk_fwd_noalloc.argtypes = shape + [i32, i32, i32, i32, f32] + tens + [vp]
    L.gdn_chunk_fwd_noalloc.restype = ctypes.c_int
    L.gdn_seqpar_fwd.argtypes = shape + [i32, i32, i32, i32, f32, i32] + tens + [vp, sz, vp]
    L.gdn_seqpar_fwd.restype = ctypes.c_int
    L.gdn_recurrent_ref.argtypes = shape + [i32, i32, i32, f32] + tens + [vp]
    L.gdn_recurrent_ref.restype = ctypes.c_int
    L.gdn_decode_step.argtypes = [i64] * 4 + [i32, i32, i32, f32] + tens + [vp]
    L.gdn_decode_step.restype = ctypes.c_int
    L.gdn_decode_step_raw.argtypes = [i64] * 4 + [i32, i32, i32, f32] + tens + [vp]
    L.gdn_decode_step_raw.restype = ctypes.c_int
    L.gdn_backward.argtypes = shape + [i32, i32, i32, f32] + [vp] * 14 + [vp, sz, vp]
    L.gdn_backward.restype = ctypes.c_int
    L.gdn_backward_workspace_bytes.argtypes = shape + [i32]
    L.gdn_backward_workspace_bytes.restype = sz
    L.gdn_workspace_bytes.argtypes = shape + [i32, i32, i32, i32]
    L.gdn_workspace_bytes.restype = sz
    L.gdn_validate.argtypes = shape + [i32, i32, i32, i32, i32]
    L.gdn_validate.restype = ctypes.c_int
    L.gdn_chunk_path.argtypes = [i64, i64, i32, i32, i32]
    L.gdn_chunk_path.restype = ctypes.c_int
    L.gdn_backward_path.argtypes = [i64, i64, i32]
    L.gdn_backward_path.restype = ctypes.c_int
    L.gdn_chunk_segments.argtypes = shape + [i32, i32, i32]
    L.gdn_chunk_segments.restype = ctypes.c_int
    L.gdn_seqpar_segments.argtypes = shape + [i32, i32, i32, i32]
    L.gdn_seqpar_segments.restype = ctypes.c_int
    L.gdn_status_str.argtypes = [ctypes.c_int]
    L.gdn_status_str.restype = ctypes.c_char_p
    L.gdn_abi_version.argtypes = []
    L.gdn_abi_version.restype = ctypes.c_int
    L.gdn_timer_create.argtypes = [ctypes.POINTER(vp)]
    L.gdn_timer_create.restype = ctypes.c_int
    L.gdn_timer_destroy.argtypes = [vp]
    L.gdn_timer_destroy.restype = ctypes.c_int
    L.gdn_timer_read.argtypes = [vp, ctypes.c_int, ctypes.c_char_p, sz,
                                 ctypes.POINTER(ctypes.c_double), ctypes.POINTER(i64)]
    L.gdn_timer_read.restype = ctypes.c_int
    L.gdn_packed_fwd.argtypes = ([i64] * 9 + [i32, i32, i32, f32] + [vp, i64] * 3 + [vp] * 8 + [vp, sz, vp])
    L.gdn_packed_fwd.restype = ctypes.c_int
    L.gdn_packed_workspace_bytes.argtypes = [i64] * 7 + [i32, i32]
    L.gdn_packed_workspace_bytes.restype = sz
    L.gdn_packed_path.argtypes = [i64, i64, i32, i32]
    L.gdn_packed_path.restype = ctypes.c_int
    L.gdn_packed_backward.argtypes = ([i64] * 7 + [i32, i32, i32, f32] + [vp, i64] * 3 + [vp] * 13 + [vp, sz, vp])
    L.gdn_packed_backward.restype = ctypes.c_int
    L.gdn_packed_backward_workspace_bytes.argtypes = [i64] * 6 + [i32, i32]
    L.gdn_packed_backward_workspace_bytes.restype = sz
    L.gdn_layer_norm_fwd.argtypes = [i64, i64, i32, i32, f32] + [vp] * 7
    L.gdn_layer_norm_fwd.restype = ctypes.c_int
    L.gdn_layer_norm_backward.argtypes = [i64, i64, i32, i32] + [vp] * 9 + [sz, vp]
    L.gdn_layer_norm_backward.restype = ctypes.c_int
    L.gdn_layer_norm_workspace_bytes.argtypes = [i64, i64]
    L.gdn_layer_norm_workspace_bytes.restype = sz
    L.gdn_linear_fwd.argtypes = [i64] * 9 + [i32, f32] + [vp, i64] * 3 + [vp] * 7 + [vp, sz, vp]
    L.gdn_linear_fwd.restype = ctypes.c_int
    L.gdn_linear_workspace_bytes.argtypes = [i64] * 7 + [i32]
    L.gdn_linear_workspace_bytes.restype = sz
    L.gdn_linear_backward.argtypes = [i64] * 7 + [i32, f32] + [vp, i64] * 3 + [vp] * 11 + [vp, sz, vp]
    L.gdn_linear_backward.restype = ctypes.c_int
    L.gdn_linear_backward_workspace_bytes.argtypes = [i64] * 6 + [i32]
    L.gdn_linear_backward_workspace_bytes.restype = sz
    L.gdn_qk_norm_fwd.argtypes = [i64] * 6 + [i32, i32, f32] + [vp, i64] * 2 + [vp] * 5 + [vp, i64] * 2 + [vp]
    L.gdn_qk_norm_fwd.restype = ctypes.c_int
    L.gdn_qk_norm_backward.argtypes = [i64] * 6 + [i32, i32, f32] + [vp, i64] * 4 + [vp] * 9 + [vp, sz, vp]
    L.gdn_qk_norm_backward.restype = ctypes.c_int
    L.gdn_qk_norm_workspace_bytes.argtypes = [i64] * 4
    L.gdn_qk_norm_workspace_bytes.restype = sz
    # the *_timed variants: the same arguments plus the timer
    for name in ("gdn_chunk_fwd", "gdn_chunk_fwd_raw", "gdn_seqpar_fwd", "gdn_decode_step",
                 "gdn_backward", "gdn_packed_fwd", "gdn_packed_backward", "gdn_layer_norm_fwd", "gdn_layer_norm_backward",
                 "gdn_linear_fwd", "gdn_linear_backward", "gdn_qk_norm_fwd", "gdn_qk_norm_backward"):
        f = getattr(L, name + "_timed")
        f.argtypes = getattr(L, name).argtypes + [vp]
        f.restype = ctypes.c_int
    _lib = L
    return L


# ---- raw C ABI ---------------------------------------------------------------

def gdn_chunk_fwd(*args):
    return lib().gdn_chunk_fwd(*args)


def gdn_seqpar_fwd(*args):
    return lib().gdn_seqpar_fwd(*args)


def gdn_recurrent_ref(*args):
    return lib().gdn_recurrent_ref(*args)


def gdn_decode_step(*args):
    return lib().gdn_decode_step(*args)


def gdn_decode_step_raw(*args):
    return lib().gdn_decode_step_raw(*args)


def gdn_backward(*args):
    return lib().gdn_backward(*args)


def gdn_backward_workspace_bytes(B, T, H, dk, dv, gate=GDN_GATE_SCALAR) -> int:
    return int(lib().gdn_backward_workspace_bytes(B, T, H, dk, dv, gate))


def gdn_workspace_bytes(B, T, H, dk, dv, chunk, dtype, gate, n_segments=1) -> int:
    return int(lib().gdn_workspace_bytes(B, T, H, dk, dv, chunk, dtype, gate, n_segments))


def gdn_validate(B, T, H, dk, dv, chunk, dtype, gate, order, n_segments=1) -> int:
    return int(lib().gdn_validate(B, T, H, dk, dv, chunk, dtype, gate, order, n_segments))


def gdn_chunk_path(dk, dv, chunk, dtype, gate) -> int:
    return int(lib().gdn_chunk_path(dk, dv, chunk, dtype, gate))


def gdn_backward_path(dk, dv, gate) -> int:
    return int(lib().gdn_backward_path(dk, dv, gate))


def gdn_chunk_segments(B, T, H, dk, dv, chunk, dtype, gate) -> int:
    return int(lib().gdn_chunk_segments(B, T, H, dk, dv, chunk, dtype, gate))


def gdn_seqpar_segments(B, T, H, dk, dv, chunk, dtype, gate, n_segments) -> int:
    return int(lib().gdn_seqpar_segments(B, T, H, dk, dv, chunk, dtype, gate, n_segments))


def gdn_packed_workspace_bytes(N, S, Hk, Hv, dk, dv, max_len, dtype, gate) -> int:
    return int(lib().gdn_packed_workspace_bytes(N, S, Hk, Hv, dk, dv, max_len, dtype, gate))


def gdn_linear_workspace_bytes(N, S, Hk, Hv, dk, dv, max_len, dtype) -> int:
    return int(lib().gdn_linear_workspace_bytes(N, S, Hk, Hv, dk, dv, max_len, dtype))


def gdn_linear_backward_workspace_bytes(N, S, Hk, Hv, dk, dv, dtype) -> int:
    return int(lib().gdn_linear_backward_workspace_bytes(N, S, Hk, Hv, dk, dv, dtype))


def gdn_qk_norm_workspace_bytes(N, Hq, Hk, d) -> int:
    return int(lib().gdn_qk_norm_workspace_bytes(N, Hq, Hk, d))


def gdn_packed_path(dk, dv, dtype, gate) -> int:
    return int(lib().gdn_packed_path(dk, dv, dtype, gate))


def gdn_packed_backward_workspace_bytes(N, S, Hk, Hv, dk, dv, dtype, gate) -> int:
    return int(lib().gdn_packed_backward_workspace_bytes(N, S, Hk, Hv, dk, dv, dtype, gate))


def gdn_layer_norm_workspace_bytes(rows, n) -> int:
    return int(lib().gdn_layer_norm_workspace_bytes(rows, n))


def gdn_status_str(status: int) -> str:
    return lib().gdn_status_str(int(status)).decode()


status_str = gdn_status_str


def gdn_abi_version() -> int:
    return int(lib().gdn_abi_version())


class Timer:
    """A caller-owned per-kernel timer (gdn_timer_create / gdn_timer_read /
    gdn_timer_destroy).  Pass it as timer= to the torch-level helpers; they
    then call the *_timed entry points, which bracket each kernel with HIP
    events on the launch stream."""

    def __init__(self):
        h = ctypes.c_void_p()
        rc = lib().gdn_timer_create(ctypes.byref(h))
        if rc != GDN_OK:
            raise GdnError(rc, "gdn_timer_create")
        self.handle = h

    def read(self):
        """Every kernel timed so far: {name: (total ms, launches)}."""
        res = {}
        buf = ctypes.create_string_buffer(128)
        i = 0
        while True:
            ms, cnt = ctypes.c_double(), ctypes.c_int64()
            if lib().gdn_timer_read(self.handle, i, buf, 128, ctypes.byref(ms),
                                    ctypes.byref(cnt)) != GDN_OK:
                break
            res[buf.value.decode()] = (ms.value, cnt.value)
            i += 1
        return res

    def close(self):
        if self.handle is not None:
            lib().gdn_timer_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _call(name, args, timer):
    """The entry point `name`, or its *_timed variant with the timer."""
    if timer is None:
        return getattr(lib(), name)(*args)
    return getattr(lib(), name + "_timed")(*args, timer.handle)


# ---- torch-level helpers -------------------------------------------------------

def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype_code(t):
    import torch
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    if t.dtype == torch.float32:
        return GDN_F32
    raise TypeError(f"q/k/v must be bfloat16 or float32, got {t.dtype}")


def _check(q, k, v, alpha, beta, state0):
    import torch
    if q.dim() != 4 or k.shape != q.shape or v.dim() != 4 or v.shape[:3] != q.shape[:3]:
        raise ValueError("q, k must be [B,T,H,dk] and v [B,T,H,dv]")
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k, v must share a dtype")
    tensors = [q, k, v, alpha, beta] + ([state0] if state0 is not None else [])
    for t in tensors:
        if not t.is_cuda:
            raise ValueError("all tensors must be on the GPU")
        if not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")
    for t in tensors[3:]:
        if t.dtype != torch.float32:
            raise TypeError("alpha, beta, state0 must be float32")
    B, T, H, dk = q.shape
    dv = v.shape[3]
    if alpha.shape == (B, T, H):
        gate = GDN_GATE_SCALAR
    elif alpha.shape == (B, T, H, dk):
        gate = GDN_GATE_CHANNEL
    else:
        raise ValueError("alpha must be [B,T,H] or [B,T,H,dk]")
    if beta.shape != (B, T, H):
        raise ValueError("beta must be [B,T,H]")
    if state0 is not None and state0.shape != (B, H, dv, dk):
        raise ValueError("state0 must be [B,H,dv,dk]")
    return B, T, H, dk, dv, gate


def _stream():
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def workspace_for(q, v, alpha, chunk=64, n_segments=None):
    import torch
    B, T, H, dk = q.shape
    gate = GDN_GATE_SCALAR if alpha.dim() == 3 else GDN_GATE_CHANNEL
    n = gdn_workspace_bytes(B, T, H, dk, v.shape[3], chunk, _dtype_code(q), gate,
                            1 if n_segments is None else n_segments)
    return torch.empty(max(n, 1), dtype=torch.uint8, device=q.device)


def chunk_fwd(q, k, v, alpha, beta, state0=None, *, chunk=64,
              order=GDN_PREDICT_THEN_DECAY, scale=1.0, n_segments=None,
              out=None, state_out=None, workspace=None, timer=None):
    """Chunkwise forward: gdn_chunk_fwd (the library's schedule) when
    n_segments is None, else gdn_seqpar_fwd with that many segments (1: a
    single stream).  timer: a Timer (the *_timed entry point) or None.
    Returns (out [B,T,H,dv] fp32, final state [B,H,dv,dk] fp32)."""
    import torch
    B, T, H, dk, dv, gate = _check(q, k, v, alpha, beta, state0)
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=torch.float32, device=q.device)
    if state_out is None:
        state_out = torch.empty((B, H, dv, dk), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = workspace_for(q, v, alpha, chunk, n_segments)
    args = [B, T, H, dk, dv, chunk, _dtype_code(q), gate, order, scale]
    tens = [_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(state0),
            _ptr(out), _ptr(state_out)]
    tail = [_ptr(workspace), workspace.numel(), _stream()]
    if n_segments is None:
        where = "gdn_chunk_fwd"
        rc = _call(where, [*args, *tens, *tail], timer)
    else:
        where = "gdn_seqpar_fwd"
        rc = _call(where, [*args, n_segments, *tens, *tail], timer)
    if rc != GDN_OK:
        raise GdnError(rc, where)
    return out, state_out


def chunk_fwd_raw(q, k, v, alpha_logit, beta_logit, state0=None, *, chunk=64,
                  order=GDN_PREDICT_THEN_DECAY, scale=1.0, out=None, state_out=None,
                  workspace=None, timer=None):
    """gdn_chunk_fwd_raw: the forward on raw projections q, k (L2-normalised
    in the kernels) and gate / beta logits (through a sigmoid in the
    kernels); timer: a Timer (gdn_chunk_fwd_raw_timed) or None.
    Returns (out [B,T,H,dv] fp32, final state [B,H,dv,dk])."""
    import torch
    B, T, H, dk, dv, gate = _check(q, k, v, alpha_logit, beta_logit, state0)
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=torch.float32, device=q.device)
    if state_out is None:
        state_out = torch.empty((B, H, dv, dk), dtype=torch.float32, device=q.device)
    if workspace is None:
        n = int(lib().gdn_raw_workspace_bytes(B, T, H, dk, dv, chunk, _dtype_code(q), gate))
        workspace = torch.empty(max(n, 1), dtype=torch.uint8, device=q.device)
    rc = _call("gdn_chunk_fwd_raw",
               [B, T, H, dk, dv, chunk, _dtype_code(q), gate, order, scale,
                _ptr(q), _ptr(k), _ptr(v), _ptr(alpha_logit), _ptr(beta_logit),
                _ptr(state0), _ptr(out), _ptr(state_out), _ptr(workspace),
                workspace.numel(), _stream()], timer)
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_chunk_fwd_raw")
    return out, state_out


def chunk_fwd_noalloc(q, k, v, alpha, beta, state0=None, *, chunk=64,
                      order=GDN_PREDICT_THEN_DECAY, scale=1.0, out=None, state_out=None):
    """gdn_chunk_fwd_noalloc: the forward with the library's static device
    scratch as its workspace (the call itself allocates nothing; out and
    state_out are allocated here when not given)."""
    import torch
    B, T, H, dk, dv, gate = _check(q, k, v, alpha, beta, state0)
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=torch.float32, device=q.device)
    if state_out is None:
        state_out = torch.empty((B, H, dv, dk), dtype=torch.float32, device=q.device)
    rc = lib().gdn_chunk_fwd_noalloc(B, T, H, dk, dv, chunk, _dtype_code(q), gate, order, scale,
                                     _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                     _ptr(state0), _ptr(out), _ptr(state_out), _stream())
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_chunk_fwd_noalloc")
    return out, state_out


def seqpar_fwd(q, k, v, alpha, beta, state0=None, *, n_segments=8, **kw):
    return chunk_fwd(q, k, v, alpha, beta, state0, n_segments=n_segments, **kw)


def recurrent_ref(q, k, v, alpha, beta, state0=None, *, order=GDN_PREDICT_THEN_DECAY,
                  scale=1.0, out=None, state_out=None):
    import torch
    B, T, H, dk, dv, gate = _check(q, k, v, alpha, beta, state0)
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=torch.float32, device=q.device)
    if state_out is None:
        state_out = torch.empty((B, H, dv, dk), dtype=torch.float32, device=q.device)
    rc = gdn_recurrent_ref(B, T, H, dk, dv, _dtype_code(q), gate, order, scale,
                           _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(state0),
                           _ptr(out), _ptr(state_out), _stream())
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_recurrent_ref")
    return out, state_out


def backward(q, k, v, alpha, beta, state0, grad_out, grad_state_out=None, *,
             order=GDN_PREDICT_THEN_DECAY, scale=1.0, want_grad_state0=True, workspace=None,
             timer=None):
    """Gradients through the forward pass: gdn_backward.
    grad_out [B,T,H,dv] fp32 = dL/d out; grad_state_out [B,H,dv,dk] fp32 =
    dL/d S_T or None (zero).  Returns (dq, dk, dv, dalpha, dbeta, dstate0),
    fp32, shaped like q, k, v, alpha, beta and the state (dstate0 None when
    not wanted)."""
    import torch
    B, T, H, dk, dv, gate = _check(q, k, v, alpha, beta, state0)
    for t in (grad_out, grad_state_out):
        if t is not None and (not t.is_cuda or not t.is_contiguous() or t.dtype != torch.float32):
            raise ValueError("gradients must be contiguous float32 GPU tensors")
    if grad_out.shape != (B, T, H, dv):
        raise ValueError("grad_out must be [B,T,H,dv]")
    if grad_state_out is not None and grad_state_out.shape != (B, H, dv, dk):
        raise ValueError("grad_state_out must be [B,H,dv,dk]")
    dev = q.device
    f32 = torch.float32
    dq = torch.empty((B, T, H, dk), dtype=f32, device=dev)
    dkk = torch.empty((B, T, H, dk), dtype=f32, device=dev)
    dvv = torch.empty((B, T, H, dv), dtype=f32, device=dev)
    dal = torch.empty(alpha.shape, dtype=f32, device=dev)
    dbe = torch.empty((B, T, H), dtype=f32, device=dev)
    ds0 = torch.empty((B, H, dv, dk), dtype=f32, device=dev) if want_grad_state0 else None
    if workspace is None:
        n = gdn_backward_workspace_bytes(B, T, H, dk, dv, gate)
        workspace = torch.empty(max(n, 1), dtype=torch.uint8, device=dev)
    rc = _call("gdn_backward",
               [B, T, H, dk, dv, _dtype_code(q), gate, order, scale,
                _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(state0),
                _ptr(grad_out), _ptr(grad_state_out), _ptr(dq), _ptr(dkk), _ptr(dvv),
                _ptr(dal), _ptr(dbe), _ptr(ds0), _ptr(workspace), workspace.numel(),
                _stream()], timer)
    if rc != GDN_OK:
        raise GdnError(rc, "gdn_backward")
    return dq, dkk, dvv, dal, dbe, ds0


def decode_step(q, k, v, alpha, beta, state=None, *, order=GDN_PREDICT_THEN_DECAY,
                scale=1.0, out=None, state_out=None, inplace=False, raw=False, timer=None):
    """One token on a persistent state: gdn_decode_step.
    q, k [B,H,dk], v [B,H,dv] (bf16 or fp32), alpha [B,H] or [B,H,dk], beta
    [B,H] fp32, state [B,H,dv,dk] fp32 or None (zero).  inplace=True writes the
    new state over `state`.  raw=True calls gdn_decode_step_raw: q, k are raw
    projections (L2-normalised in the kernel) and alpha, beta are logits
    (passed through a sigmoid in the kernel).
    Returns (out [B,H,dv] fp32, new state)."""
    import torch
    if q.dim() != 3 or k.shape != q.shape or v.dim() != 3 or v.shape[:2] != q.shape[:2]:
        raise ValueError("q, k must be [B,H,dk] and v [B,H,dv]")
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k, v must share a dtype")
    B, H, dk = q.shape
    dv = v.shape[2]
    tensors = [q, k, v, alpha, beta] + ([state] if state is not None else [])
    for t in tensors:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("all tensors must be contiguous and on the GPU")
    for t in tensors[3:]:
        if t.dtype != torch.float32:
            raise TypeError("alpha, beta, state must be float32")
    if alpha.shape == (B, H):
        gate = GDN_GATE_SCALAR
    elif alpha.shape == (B, H, dk):
        gate = GDN_GATE_CHANNEL
    else:
        raise ValueError("alpha must be [B,H] or [B,H,dk]")
    if beta.shape != (B, H):
        raise ValueError("beta must be [B,H]")
    if state is not None and state.shape != (B, H, dv, dk):
        raise ValueError("state must be [B,H,dv,dk]")
    if inplace:
        if state is None:
            raise ValueError("inplace needs a state")
        state_out = state
    if out is None:
        out = torch.empty((B, H, dv), dtype=torch.float32, device=q.device)
    if state_out is None:
        state_out = torch.empty((B, H, dv, dk), dtype=torch.float32, device=q.device)
    if raw and timer is not None:
        raise ValueError("the raw decode step has no timed variant")
    name = "gdn_decode_step_raw" if raw else "gdn_decode_step"
    rc = _call(name, [B, H, dk, dv, _dtype_code(q), gate, order, scale,
                      _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(state),
                      _ptr(out), _ptr(state_out), _stream()], timer)
    if rc != GDN_OK:
        raise GdnError(rc, name)
    return out, state_out


# ---- packed ragged sequences over a pool of states ------------------------------

def _enqueue(where, args, device, timer):
    """Entry point `where` (or its *_timed variant) on the current stream of
    GPU `device`; raises GdnError."""
    import torch
    C = torch._C
    fn = getattr(_lib or lib(), where if timer is None else where + "_timed")
    tail = () if timer is None else (timer.handle,)
    if C._cuda_getDevice() == device:
        rc = fn(*args, C._cuda_getCurrentRawStream(device), *tail)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, C._cuda_getCurrentRawStream(device), *tail)
    if rc != GDN_OK:
        raise GdnError(rc, where)


def _addr(t):
    return None if t is None else t.data_ptr()


def _on(t, device, dtype, what):
    """t (a tensor or None) is contiguous, of dtype and on GPU `device`."""
    if t is not None:
        if t.dtype != dtype:
            raise TypeError(f"{what} must be {dtype}")
        if t.get_device() != device:
            raise ValueError(f"{what} must be on the GPU of q")
        if not t.is_contiguous():
            raise ValueError(f"{what} must be contiguous")


def _heads_contiguous(tensors):
    """[N,H,d] tensors whose tokens are contiguous rows, at any stride."""
    for t in tensors:
        if not t.is_contiguous() and (t.stride(2) != 1 or (t.stride(1) != t.shape[2] and t.shape[1] > 1)):
            raise ValueError("the heads and features of a token of q, k, v must be contiguous")


def _packed_check(q, k, v, alpha, beta, cu_seqlens, pools, slots):
    import torch
    f32, i32 = torch.float32, torch.int32
    shape = q.shape
    if len(shape) != 3 or k.shape != shape or v.dim() != 3 or v.shape[0] != shape[0]:
        raise ValueError("q, k must be [N,Hk,dk] and v [N,Hv,dv]")
    N, Hk, dk = shape
    _, Hv, dv = v.shape
    dt = q.dtype
    if k.dtype != dt or v.dtype != dt:
        raise TypeError("q, k, v must share a dtype")
    _heads_contiguous((q, k, v))
    if alpha.shape == (N, Hv):
        gate = GDN_GATE_SCALAR
    elif alpha.shape == (N, Hv, dk):
        gate = GDN_GATE_CHANNEL
    else:
        raise ValueError("alpha must be [N,Hv] or [N,Hv,dk]")
    if beta.shape != (N, Hv):
        raise ValueError("beta must be [N,Hv]")
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must be [S+1]")
    S = cu_seqlens.shape[0] - 1
    for t, i in zip(pools, slots):
        if t is not None:
            pool = t.shape
            if len(pool) != 4 or pool[1:] != (Hv, dv, dk):
                raise ValueError("state pools must be [slots,Hv,dv,dk]")
            # (an empty tensor has no address, which would stand for no pool)
            if pool[0] == 0 and i is None and S * Hv:
                raise GdnError(GDN_E_SHAPE, "an empty state pool without slots")
    for t in slots:
        if t is not None and t.shape != (S,):
            raise ValueError("slots must be [S]")
    dev = q.get_device()
    _on(alpha, dev, f32, "alpha")
    _on(beta, dev, f32, "beta")
    _on(cu_seqlens, dev, i32, "cu_seqlens")
    for t in pools:
        _on(t, dev, f32, "a state pool")
    for t in slots:
        _on(t, dev, i32, "slots")
    if dev < 0 or k.get_device() != dev or v.get_device() != dev:
        raise ValueError("q, k, v must be on one GPU")
    return N, S, Hk, Hv, dk, dv, gate, dev


def _token_stride(t):
    """Elements between tokens; a lone token's stride says nothing."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2]


def _token_strides(q, k, v):
    return _token_stride(q), _token_stride(k), _token_stride(v)


def packed_workspace_for(q, v, alpha, cu_seqlens, max_len=None):
    """A workspace for packed_fwd on tensors like these."""
    import torch
    N, Hk, dk = q.shape
    gate = GDN_GATE_SCALAR if alpha.dim() == 2 else GDN_GATE_CHANNEL
    n = gdn_packed_workspace_bytes(N, cu_seqlens.shape[0] - 1, Hk, v.shape[1], dk, v.shape[2],
                                   N if max_len is None else max_len, _dtype_code(q), gate)
    return torch.empty(max(n, 1), dtype=torch.uint8, device=q.device)


def packed_fwd(q, k, v, alpha, beta, cu_seqlens, state_in=None, slots_in=None, state_out=None,
               slots_out=None, *, max_len=None, order=GDN_PREDICT_THEN_DECAY, scale=1.0, out=None,
               workspace=None, timer=None):
    """Packed ragged sequences with a pool of states: gdn_packed_fwd.
    q, k [N,Hk,dk], v [N,Hv,dv] (bf16 or fp32; slices of a wider projection
    along the heads are taken as they are), alpha [N,Hv] or [N,Hv,dk], beta
    [N,Hv], cu_seqlens [S+1] int32; state pools [slots,Hv,dv,dk], slots [S]
    int32 (-1: a zero start state, an end state not written; None: sequence s
    has slot s).  state_out None: a new pool [S,Hv,dv,dk], in the sequences'
    order.  max_len: a bound on the lengths (it picks kernels; None: N).
    Returns (out [N,Hv,dv] of q's dtype, state_out)."""
    import torch
    if state_out is None and slots_out is not None:
        raise ValueError("slots_out needs state_out")
    N, S, Hk, Hv, dk, dv, gate, dev = _packed_check(q, k, v, alpha, beta, cu_seqlens,
                                                    (state_in, state_out), (slots_in, slots_out))
    if state_out is None:
        state_out = q.new_empty((S, Hv, dv, dk), dtype=torch.float32)
    if out is None:
        out = q.new_empty((N, Hv, dv))
    else:
        if out.shape != (N, Hv, dv):
            raise ValueError("out must be [N,Hv,dv]")
        _on(out, dev, q.dtype, "out")
    if max_len is None:
        max_len = N
    code = _dtype_code(q)
    _on(workspace, dev, torch.uint8, "workspace")
    if workspace is None:
        n = lib().gdn_packed_workspace_bytes(N, S, Hk, Hv, dk, dv, max_len, code, gate)
        if n:
            workspace = q.new_empty((n,), dtype=torch.uint8)
    sq, sk, sv = _token_strides(q, k, v)
    args = (N, S, Hk, Hv, dk, dv, 0 if state_in is None else state_in.shape[0], state_out.shape[0], max_len, code, gate, order, scale,
            _addr(q), sq, _addr(k), sk, _addr(v), sv, _addr(alpha), _addr(beta), _addr(cu_seqlens),
            _addr(state_in), _addr(slots_in), _addr(state_out), _addr(slots_out), _addr(out),
            _addr(workspace), 0 if workspace is None else workspace.numel())
    _enqueue("gdn_packed_fwd", args, dev, timer)
    return out, state_out


def packed_backward(q, k, v, alpha, beta, cu_seqlens, state_in, slots_in, grad_out, grad_state_out=None, *,
                    order=GDN_PREDICT_THEN_DECAY, scale=1.0, want_grad_state0=True, workspace=None, timer=None):
    """Gradients through packed_fwd: gdn_packed_backward (scalar gate, dk = dv in
    {64, 128}).  grad_out [N,Hv,dv] of q's dtype = dL/d out; grad_state_out
    [S,Hv,dv,dk] fp32 = dL/d of the end states, in the sequences' order, or
    None (zero).  Returns (dq, dk, dv, dalpha, dbeta, dstate0), fp32, shaped
    like q, k, v, alpha, beta and the sequences' states [S,Hv,dv,dk] (None when
    not wanted); rows outside every sequence are zero."""
    import torch
    N, S, Hk, Hv, dk, dv, gate, dev = _packed_check(q, k, v, alpha, beta, cu_seqlens, (state_in,), (slots_in,))
    f32 = torch.float32
    if grad_out.shape != (N, Hv, dv):
        raise ValueError("grad_out must be [N,Hv,dv]")
    _on(grad_out, dev, q.dtype, "grad_out")
    if grad_state_out is not None and grad_state_out.shape != (S, Hv, dv, dk):
        raise ValueError("grad_state_out must be [S,Hv,dv,dk]")
    _on(grad_state_out, dev, f32, "grad_state_out")
    # (without sequences the entry point enqueues nothing, and every row is outside them)
    new = q.new_empty if S * Hv else q.new_zeros
    grads = [new(t.shape, dtype=f32) for t in (q, k, v, alpha, beta)]
    ds0 = q.new_empty((S, Hv, dv, dk), dtype=f32) if want_grad_state0 else None
    code = _dtype_code(q)
    _on(workspace, dev, torch.uint8, "workspace")
    if workspace is None:
        n = lib().gdn_packed_backward_workspace_bytes(N, S, Hk, Hv, dk, dv, code, gate)
        if n:
            workspace = q.new_empty((n,), dtype=torch.uint8)
    sq, sk, sv = _token_strides(q, k, v)
    args = (N, S, Hk, Hv, dk, dv, 0 if state_in is None else state_in.shape[0], code, gate, order, scale,
            _addr(q), sq, _addr(k), sk, _addr(v), sv, _addr(alpha), _addr(beta), _addr(cu_seqlens),
            _addr(state_in), _addr(slots_in), _addr(grad_out), _addr(grad_state_out), *map(_addr, grads), _addr(ds0),
            _addr(workspace), 0 if workspace is None else workspace.numel())
    _enqueue("gdn_packed_backward", args, dev, timer)
    return (*grads, ds0)


# ---- linear attention with a decay for each head ---------------------------------

def _linear_check(q, k, v, alpha, cu_seqlens, pools, slots):
    import torch
    f32, i32 = torch.float32, torch.int32
    shape = q.shape
    if len(shape) != 3 or k.shape != shape or v.dim() != 3 or v.shape[0] != shape[0]:
        raise ValueError("q, k must be [N,Hk,dk] and v [N,Hv,dv]")
    N, Hk, dk = shape
    _, Hv, dv = v.shape
    dt = q.dtype
    if k.dtype != dt or v.dtype != dt:
        raise TypeError("q, k, v must share a dtype")
    _heads_contiguous((q, k, v))
    if alpha.shape != (Hv,):
        raise ValueError("alpha must be [Hv]")
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must be [S+1]")
    S = cu_seqlens.shape[0] - 1
    for t, i in zip(pools, slots):
        if t is not None:
            pool = t.shape
            if len(pool) != 4 or pool[1:] != (Hv, dv, dk):
                raise ValueError("state pools must be [slots,Hv,dv,dk]")
            # (an empty tensor has no address, which would stand for no pool)
            if pool[0] == 0 and i is None and S * Hv:
                raise GdnError(GDN_E_SHAPE, "an empty state pool without slots")
    for t in slots:
        if t is not None and t.shape != (S,):
            raise ValueError("slots must be [S]")
    dev = q.get_device()
    _on(alpha, dev, f32, "alpha")
    _on(cu_seqlens, dev, i32, "cu_seqlens")
    for t in pools:
        _on(t, dev, f32, "a state pool")
    for t in slots:
        _on(t, dev, i32, "slots")
    if dev < 0 or k.get_device() != dev or v.get_device() != dev:
        raise ValueError("q, k, v must be on one GPU")
    return N, S, Hk, Hv, dk, dv, dev


def linear_workspace_for(q, v, cu_seqlens, max_len=None):
    """A workspace for linear_fwd on tensors like these."""
    import torch
    N, Hk, dk = q.shape
    n = gdn_linear_workspace_bytes(N, cu_seqlens.shape[0] - 1, Hk, v.shape[1], dk, v.shape[2],
                                   N if max_len is None else max_len, _dtype_code(q))
    return torch.empty(max(n, 1), dtype=torch.uint8, device=q.device)


def linear_fwd(q, k, v, alpha, cu_seqlens, state_in=None, slots_in=None, state_out=None, slots_out=None, *,
               max_len=None, scale=1.0, out=None, workspace=None, timer=None):
    """Linear attention with a decay for each head over packed ragged sequences:
    gdn_linear_fwd, S_t = alpha S_{t-1} + v_t k_t^T and o_t = scale S_t q_t.
    q, k [N,Hk,dk], v [N,Hv,dv] (bf16 or fp32; slices of a wider projection
    along the heads are taken as they are), alpha [Hv] fp32; cu_seqlens, the
    state pools, slots and max_len as for packed_fwd (state_out None: a new pool
    [S,Hv,dv,dk], in the sequences' order; state_in: in place).  out and the
    workspace may not share memory with anything else.
    Returns (out [N,Hv,dv] of q's dtype, state_out)."""
    import torch
    if state_out is None and slots_out is not None:
        raise ValueError("slots_out needs state_out")
    N, S, Hk, Hv, dk, dv, dev = _linear_check(q, k, v, alpha, cu_seqlens, (state_in, state_out), (slots_in, slots_out))
    if state_out is None:
        state_out = q.new_empty((S, Hv, dv, dk), dtype=torch.float32)
    if out is None:
        out = q.new_empty((N, Hv, dv))
    else:
        if out.shape != (N, Hv, dv):
            raise ValueError("out must be [N,Hv,dv]")
        _on(out, dev, q.dtype, "out")
    if max_len is None:
        max_len = N
    code = _dtype_code(q)
    _on(workspace, dev, torch.uint8, "workspace")
    if workspace is None:
        n = lib().gdn_linear_workspace_bytes(N, S, Hk, Hv, dk, dv, max_len, code)
        if n:
            workspace = q.new_empty((n,), dtype=torch.uint8)
    sq, sk, sv = _token_strides(q, k, v)
    args = (N, S, Hk, Hv, dk, dv, 0 if state_in is None else state_in.shape[0], state_out.shape[0], max_len, code, scale,
            _addr(q), sq, _addr(k), sk, _addr(v), sv, _addr(alpha), _addr(cu_seqlens), _addr(state_in), _addr(slots_in),
            _addr(state_out), _addr(slots_out), _addr(out), _addr(workspace), 0 if workspace is None else workspace.numel())
    _enqueue("gdn_linear_fwd", args, dev, timer)
    return out, state_out


def linear_backward(q, k, v, alpha, cu_seqlens, state_in, slots_in, grad_out, grad_state_out=None, *, scale=1.0,
                    want_grad_alpha=True, want_grad_state0=True, workspace=None, timer=None):
    """Gradients through linear_fwd: gdn_linear_backward.  grad_out [N,Hv,dv] of
    q's dtype = dL/d out; grad_state_out [S,Hv,dv,dk] fp32 = dL/d of the end
    states, in the sequences' order, or None (zero).  Returns (dq, dk, dv of q's
    dtype, dalpha [Hv] and dstate0 [S,Hv,dv,dk] fp32 or None where not wanted);
    rows outside every sequence are zero."""
    import torch
    N, S, Hk, Hv, dk, dv, dev = _linear_check(q, k, v, alpha, cu_seqlens, (state_in,), (slots_in,))
    f32 = torch.float32
    if grad_out.shape != (N, Hv, dv):
        raise ValueError("grad_out must be [N,Hv,dv]")
    _on(grad_out, dev, q.dtype, "grad_out")
    if grad_state_out is not None and grad_state_out.shape != (S, Hv, dv, dk):
        raise ValueError("grad_state_out must be [S,Hv,dv,dk]")
    _on(grad_state_out, dev, f32, "grad_state_out")
    # (without sequences the entry point enqueues nothing, and every row is outside them)
    new = q.new_empty if S * Hv else q.new_zeros
    grads = [new(t.shape) for t in (q, k, v)]
    da = new((Hv,), dtype=f32) if want_grad_alpha else None
    ds0 = q.new_empty((S, Hv, dv, dk), dtype=f32) if want_grad_state0 else None
    code = _dtype_code(q)
    _on(workspace, dev, torch.uint8, "workspace")
    if workspace is None:
        n = lib().gdn_linear_backward_workspace_bytes(N, S, Hk, Hv, dk, dv, code)
        if n:
            workspace = q.new_empty((n,), dtype=torch.uint8)
    sq, sk, sv = _token_strides(q, k, v)
    args = (N, S, Hk, Hv, dk, dv, 0 if state_in is None else state_in.shape[0], code, scale, _addr(q), sq, _addr(k), sk,
            _addr(v), sv, _addr(alpha), _addr(cu_seqlens), _addr(state_in), _addr(slots_in), _addr(grad_out),
            _addr(grad_state_out), *map(_addr, grads), _addr(da), _addr(ds0), _addr(workspace),
            0 if workspace is None else workspace.numel())
    _enqueue("gdn_linear_backward", args, dev, timer)
    return (*grads, da, ds0)


# ---- norm of queries and keys with the position's rotation -----------------------

def _qk_check(q, k, weights, cos, sin, positions):
    import torch
    f32 = torch.float32
    if q.dim() != 3 or k.dim() != 3 or k.shape[0] != q.shape[0] or k.shape[2] != q.shape[2]:
        raise ValueError("q must be [N,Hq,d] and k [N,Hk,d]")
    N, Hq, d = q.shape
    if k.dtype != q.dtype:
        raise TypeError("q, k must share a dtype")
    _heads_contiguous((q, k))
    dev = q.get_device()
    if dev < 0 or k.get_device() != dev:
        raise ValueError("q, k must be on one GPU")
    for t in weights:
        if t is not None and t.shape != (d,):
            raise ValueError("the weights must be [d]")
        _on(t, dev, f32, "the weights")
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin go together")
    n_pos = rot = 0
    if cos is not None:
        if cos.dim() != 2 or sin.shape != cos.shape:
            raise ValueError("cos and sin must be [n_pos,rot/2]")
        n_pos, rot = cos.shape[0], 2 * cos.shape[1]
        _on(cos, dev, f32, "cos and sin")
        _on(sin, dev, f32, "cos and sin")
    if positions is not None and positions.shape != (N,):
        raise ValueError("positions must be [N]")
    _on(positions, dev, torch.int32, "positions")
    return N, Hq, k.shape[1], d, rot, n_pos, dev


def qk_norm_fwd(q, k, weight_q=None, weight_k=None, cos=None, sin=None, positions=None, *, eps=1e-6, interleaved=False,
                q_out=None, k_out=None, timer=None):
    """RMS norm of queries and keys over each head's features and the rotation of
    feature pairs by the token's position, in one pass: gdn_qk_norm_fwd.
    q [N,Hq,d], k [N,Hk,d] (bf16 or fp32; slices of a wider projection along the
    heads are taken as they are), weights [d] fp32 or None (ones), cos and sin
    [n_pos,rot/2] fp32 or None (no rotation), positions [N] int32 or None (token t
    is at position t).  Features i and i + rot/2 turn together, interleaved: 2i
    and 2i + 1.  q_out, k_out: where to (None: new tensors; q and k themselves:
    in place; no other memory of q, k or each other).  Returns (q_out, k_out)."""
    N, Hq, Hk, d, rot, n_pos, dev = _qk_check(q, k, (weight_q, weight_k), cos, sin, positions)
    outs = []
    for x, y in ((q, q_out), (k, k_out)):
        if y is None:
            y = x.new_empty(x.shape)
        elif y.shape != x.shape or y.dtype != x.dtype or y.get_device() != dev:
            raise ValueError("q_out and k_out must be as q and k")
        else:
            _heads_contiguous((y,))
        outs.append(y)
    sq, sk, so, sp = (_token_stride(t) for t in (q, k, *outs))
    args = (N, Hq, Hk, d, rot, n_pos, _dtype_code(q), int(interleaved), eps, _addr(q), sq, _addr(k), sk, _addr(weight_q),
            _addr(weight_k), _addr(cos), _addr(sin), _addr(positions), _addr(outs[0]), so, _addr(outs[1]), sp)
    _enqueue("gdn_qk_norm_fwd", args, dev, timer)
    return tuple(outs)


def qk_norm_backward(grad_q_out, grad_k_out, q, k, weight_q=None, weight_k=None, cos=None, sin=None, positions=None, *,
                     eps=1e-6, interleaved=False, want_x=True, want_weights=True, workspace=None, timer=None):
    """Gradients of qk_norm_fwd: gdn_qk_norm_backward.  Returns (grad_q, grad_k of
    q's dtype, grad_weight_q, grad_weight_k [d] fp32), None where not wanted."""
    import torch
    N, Hq, Hk, d, rot, n_pos, dev = _qk_check(q, k, (weight_q, weight_k), cos, sin, positions)
    for g, x in ((grad_q_out, q), (grad_k_out, k)):
        if g.shape != x.shape or g.dtype != x.dtype or g.get_device() != dev:
            raise ValueError("the incoming gradients must be as q and k")
    _heads_contiguous((grad_q_out, grad_k_out))
    dq, dk = (x.new_empty(x.shape) if want_x else None for x in (q, k))
    dwq, dwk = (q.new_empty((d,), dtype=torch.float32) if want_weights else None for _ in range(2))
    _on(workspace, dev, torch.uint8, "workspace")
    if workspace is None and want_weights:
        workspace = q.new_empty((lib().gdn_qk_norm_workspace_bytes(N, Hq, Hk, d),), dtype=torch.uint8)
    gq, gk, sq, sk = (_token_stride(t) for t in (grad_q_out, grad_k_out, q, k))
    args = (N, Hq, Hk, d, rot, n_pos, _dtype_code(q), int(interleaved), eps, _addr(grad_q_out), gq, _addr(grad_k_out), gk,
            _addr(q), sq, _addr(k), sk, _addr(weight_q), _addr(weight_k), _addr(cos), _addr(sin), _addr(positions),
            _addr(dq), _addr(dk), _addr(dwq), _addr(dwk), _addr(workspace), 0 if workspace is None else workspace.numel())
    _enqueue("gdn_qk_norm_backward", args, dev, timer)
    return dq, dk, dwq, dwk


# ---- layer norm -------------------------------------------------------------------

def _norm_code(dtype):
    import torch
    if dtype == torch.bfloat16:
        return GDN_BF16
    if dtype == torch.float32:
        return GDN_F32
    raise TypeError(f"layer norm takes bfloat16 or float32, got {dtype}")


def _norm_check(x, params, stats):
    import torch
    dev = x.get_device()
    if x.dim() < 1 or dev < 0 or not x.is_contiguous():
        raise ValueError("x must be contiguous and on the GPU")
    n = x.shape[-1]
    if n == 0:
        raise ValueError("rows must hold at least one element")
    rows = x.numel() // n
    for t in params:
        if t is not None:
            if t.shape != (n,):
                raise ValueError("weight and bias must be [n]")
            _on(t, dev, torch.float32, "weight and bias")
    for t in stats:
        if t.numel() != rows:
            raise ValueError("mean and rstd must hold one value a row")
        _on(t, dev, torch.float32, "mean and rstd")
    return rows, n, dev


def layer_norm_fwd(x, weight=None, bias=None, *, eps=1e-5, out_dtype=None, out=None, timer=None):
    """Layer norm over the last dimension: gdn_layer_norm_fwd.  x bf16 or fp32,
    weight and bias [n] fp32 or None; out_dtype: bf16 or fp32 (None: x's).
    Returns (y, mean, rstd), the statistics fp32 and shaped as x without its
    last dimension."""
    import torch
    rows, n, dev = _norm_check(x, (weight, bias), ())
    shape = x.shape
    if out is None:
        out = x.new_empty(shape, dtype=out_dtype or x.dtype)
    else:
        if out.shape != shape:
            raise ValueError("out must be shaped as x")
        _on(out, dev, out_dtype or out.dtype, "out")
    mean = x.new_empty(shape[:-1], dtype=torch.float32)
    rstd = x.new_empty(shape[:-1], dtype=torch.float32)
    _enqueue("gdn_layer_norm_fwd", (rows, n, _norm_code(x.dtype), _norm_code(out.dtype), eps, x.data_ptr(),
                                    _addr(weight), _addr(bias), out.data_ptr(), mean.data_ptr(), rstd.data_ptr()),
             dev, timer)
    return out, mean, rstd


def layer_norm_backward(grad_y, x, weight, mean, rstd, *, want_x=True, want_weight=True, want_bias=True,
                        workspace=None, timer=None):
    """Gradients of layer_norm_fwd: gdn_layer_norm_backward.  Returns (grad_x of
    x's dtype, grad_weight [n], grad_bias [n] fp32), None where not wanted."""
    import torch
    rows, n, dev = _norm_check(x, (weight,), (mean, rstd))
    if grad_y.shape != x.shape:
        raise ValueError("grad_y must be shaped as x")
    _on(grad_y, dev, grad_y.dtype, "grad_y")
    f32 = torch.float32
    dx = x.new_empty(x.shape) if want_x else None
    dw = x.new_empty((n,), dtype=f32) if want_weight else None
    db = x.new_empty((n,), dtype=f32) if want_bias else None
    _on(workspace, dev, torch.uint8, "workspace")
    if workspace is None and (want_weight or want_bias):
        workspace = x.new_empty((lib().gdn_layer_norm_workspace_bytes(rows, n),), dtype=torch.uint8)
    _enqueue("gdn_layer_norm_backward", (rows, n, _norm_code(x.dtype), _norm_code(grad_y.dtype), grad_y.data_ptr(),
                                         x.data_ptr(), _addr(weight), mean.data_ptr(), rstd.data_ptr(), _addr(dx),
                                         _addr(dw), _addr(db), _addr(workspace),
                                         0 if workspace is None else workspace.numel()), dev, timer)
    return dx, dw, db
