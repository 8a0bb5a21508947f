"""Host-side checks of the packed rule's and layer norm's entry points: sizes,
paths and refusals, which come before any device is touched (no GPU needed)."""
import ctypes

import pytest

from gated_delta_rule_12_amd import gdn

F = ctypes.c_void_p(0x10000)  # never dereferenced: every call below is refused first
NUL = ctypes.c_void_p(0)
OK, ARG, SHAPE, UNSUP, WS = gdn.GDN_OK, gdn.GDN_E_ARG, gdn.GDN_E_SHAPE, gdn.GDN_E_UNSUPPORTED, gdn.GDN_E_WORKSPACE


def fwd(N=100, S=2, Hk=2, Hv=4, dk=64, dv=64, n_in=2, n_out=2, max_len=1, dtype=1, gate=0, order=0, q=F, sq=None, k=F,
        sk=None, v=F, sv=None, alpha=F, beta=F, cu=F, s_in=F, slots_in=NUL, s_out=F, slots_out=NUL, out=F, ws=NUL, wsb=0):
    sq = Hk * dk if sq is None else sq
    sk = Hk * dk if sk is None else sk
    sv = Hv * dv if sv is None else sv
    return gdn.lib().gdn_packed_fwd(N, S, Hk, Hv, dk, dv, n_in, n_out, max_len, dtype, gate, order, 1.0, q, sq, k, sk, v, sv,
                                    alpha, beta, cu, s_in, slots_in, s_out, slots_out, out, ws, wsb, NUL)


ODD = ctypes.c_void_p(0x10002)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), ARG), (dict(gate=3), ARG), (dict(order=-1), ARG),
    (dict(N=-1), SHAPE), (dict(S=-1), SHAPE), (dict(Hk=3), SHAPE), (dict(Hk=0), SHAPE), (dict(dk=0), SHAPE),
    (dict(max_len=-1), SHAPE), (dict(n_in=-1), SHAPE), (dict(N=2**31), SHAPE), (dict(S=2**31), SHAPE),
    (dict(S=2**25, Hv=8, n_in=2**25, n_out=2**25), SHAPE),     # more workgroups than a grid holds
    (dict(dk=72), UNSUP), (dict(dv=144), UNSUP), (dict(dk=8), UNSUP),
    (dict(S=2**18, Hv=16, n_in=2**18, n_out=2**18), SHAPE),
    (dict(S=2**16, Hv=16, n_in=2**16, n_out=2**16, max_len=64, dk=64, dv=64, sv=1024), SHAPE),  # fewer with chunk kernels
    (dict(N=2**25, Hv=16, max_len=2**25, dk=64, dv=64, sv=1024), SHAPE),
    (dict(sq=127), SHAPE), (dict(sv=255), SHAPE), (dict(sk=2**31), SHAPE),
    (dict(sq=2**23 + 8), SHAPE), (dict(sk=2**23 + 8), SHAPE), (dict(sv=2**23 + 8), SHAPE),  # 32-bit offsets in a chunk
    (dict(sq=132), ARG), (dict(sk=129), ARG), (dict(sv=258, dtype=0), ARG),   # strides of whole 16-byte pieces
    (dict(q=NUL), ARG), (dict(k=NUL), ARG), (dict(v=NUL), ARG), (dict(alpha=NUL), ARG), (dict(beta=NUL), ARG),
    (dict(cu=NUL), ARG), (dict(out=NUL), ARG),
    (dict(q=ODD), ARG), (dict(k=ODD), ARG), (dict(v=ODD), ARG), (dict(out=ODD), ARG), (dict(s_in=ODD), ARG),
    (dict(s_out=ODD), ARG), (dict(cu=ODD), ARG), (dict(slots_in=ODD), ARG), (dict(beta=ODD), ARG),
    (dict(alpha=ctypes.c_void_p(0x10004), gate=1), ARG),
    (dict(n_in=1), SHAPE), (dict(n_out=1), SHAPE),             # a pool without indices holds every sequence
    (dict(max_len=100), WS), (dict(max_len=100, ws=F, wsb=16), WS),
    (dict(S=0), OK), (dict(Hk=0, Hv=0), OK),                   # nothing to do
])
def test_packed_refusals(kw, want):
    assert fwd(**kw) == want


def test_packed_workspace_and_path():
    ws = gdn.gdn_packed_workspace_bytes
    assert gdn.gdn_packed_path(128, 128, 1, 0) == gdn.GDN_PATH_MFMA
    assert gdn.gdn_packed_path(64, 64, 1, 0) == gdn.GDN_PATH_MFMA
    for a in ((64, 128, 1, 0), (128, 128, 0, 0), (128, 128, 1, 1), (32, 32, 1, 0)):
        assert gdn.gdn_packed_path(*a) == gdn.GDN_PATH_VALU
    assert gdn.gdn_packed_path(60, 64, 1, 0) == UNSUP and gdn.gdn_packed_path(64, 64, 5, 0) == ARG
    # single tokens, and shapes without chunk kernels, need none
    assert ws(256, 256, 16, 16, 128, 128, 1, 1, 0) == 0
    assert ws(5000, 3, 4, 4, 128, 128, 5000, 0, 0) == 0
    assert ws(5000, 3, 4, 4, 128, 128, 5000, 1, 1) == 0
    assert ws(5000, 3, 4, 3, 128, 128, 5000, 1, 0) == 0      # refused
    small, large = ws(5000, 3, 4, 4, 128, 128, 400, 1, 0), ws(5000, 3, 4, 4, 128, 128, 5000, 1, 0)
    one = ws(5000, 3, 4, 4, 128, 128, 100, 1, 0)  # a segment each: no states of segments
    assert 0 < one < small <= large and large % 256 == 0


def norm_fwd(rows=4, n=64, xt=0, yt=1, x=F, w=F, b=F, y=F, m=F, r=F):
    return gdn.lib().gdn_layer_norm_fwd(rows, n, xt, yt, 1e-5, x, w, b, y, m, r, NUL)


def norm_bwd(rows=4, n=64, xt=0, yt=1, dy=F, x=F, w=F, m=F, r=F, dx=F, dw=F, db=F, ws=F, wsb=1 << 30):
    return gdn.lib().gdn_layer_norm_backward(rows, n, xt, yt, dy, x, w, m, r, dx, dw, db, ws, wsb, NUL)


@pytest.mark.parametrize("kw,want", [
    (dict(xt=2), ARG), (dict(yt=-1), ARG), (dict(rows=-1), SHAPE), (dict(n=0), SHAPE), (dict(n=16385), UNSUP),
    (dict(x=NUL), ARG), (dict(y=NUL), ARG), (dict(x=ODD), ARG), (dict(w=ODD), ARG), (dict(b=ODD), ARG), (dict(m=ODD), ARG),
    (dict(y=ctypes.c_void_p(0x10001)), ARG), (dict(rows=0), OK),
])
def test_norm_forward_refusals(kw, want):
    assert norm_fwd(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(xt=2), ARG), (dict(yt=7), ARG), (dict(rows=-1), SHAPE), (dict(n=-3), SHAPE), (dict(n=20000), UNSUP),
    (dict(dy=NUL), ARG), (dict(x=NUL), ARG), (dict(m=NUL), ARG), (dict(r=NUL), ARG), (dict(dx=ODD), ARG), (dict(dw=ODD), ARG),
    (dict(ws=NUL), WS), (dict(wsb=100), WS), (dict(ws=ctypes.c_void_p(0x10008)), ARG),
    (dict(dx=NUL, dw=NUL, db=NUL), OK),
])
def test_norm_backward_refusals(kw, want):
    assert norm_bwd(**kw) == want


def test_norm_workspace():
    ws = gdn.gdn_layer_norm_workspace_bytes
    assert ws(10, 0) == 0 and ws(10, 16385) == 0 and ws(-1, 64) == 0
    assert ws(1, 64) >= 8 * 64
    assert ws(1 << 20, 128) <= 2 * 4 * 1024 * 128


def test_binding_refuses_before_the_library():
    """Shapes, types, devices and strides are checked in the binding."""
    import torch
    z = torch.zeros
    q, v = z(10, 2, 64, dtype=torch.bfloat16), z(10, 4, 64, dtype=torch.bfloat16)
    a, cu = z(10, 4), torch.tensor([0, 4, 10], dtype=torch.int32)
    pool = z(2, 4, 64, 64)
    with pytest.raises(ValueError, match="GPU"):
        gdn.packed_fwd(q, q, v, a, a, cu, pool)
    for bad in (dict(q=z(10, 128)), dict(k=q[:9]), dict(v=v[:9]), dict(alpha=z(10, 3)), dict(beta=z(9, 4)), dict(cu=z(0)),
                dict(cu=cu[None]), dict(pool=z(2, 4, 64)), dict(pool=z(2, 4, 32, 64)), dict(q=q.transpose(1, 2)),
                dict(q=z(10, 2, 128, dtype=torch.bfloat16)[:, :, ::2])):
        x = dict(q=q, k=q, v=v, alpha=a, beta=a, cu=cu, pool=pool)
        x.update(bad)
        if "q" in bad and "k" not in bad:
            x["k"] = bad["q"]
        with pytest.raises(ValueError):
            gdn.packed_fwd(*x.values())
    with pytest.raises(TypeError):
        gdn.packed_fwd(q, q, v.float(), a, a, cu, pool)
    with pytest.raises(TypeError):
        gdn.packed_fwd(q, q, v, a, a, cu.long(), pool)
    with pytest.raises(TypeError):
        gdn.packed_fwd(q, q, v, a.double(), a, cu, pool)
    with pytest.raises(ValueError, match="slots"):
        gdn.packed_fwd(q, q, v, a, a, cu, pool, cu)
    with pytest.raises(ValueError, match="state_out"):
        gdn.packed_fwd(q, q, v, a, a, cu, pool, None, None, cu[:2])
    with pytest.raises(ValueError):
        gdn.layer_norm_fwd(z(4, 64))
    with pytest.raises(ValueError):
        gdn.layer_norm_backward(z(4, 64), z(4, 64), None, z(4), z(4))


def bwd(N=100, S=2, Hk=2, Hv=4, dk=64, dv=64, n_in=2, dtype=1, gate=0, order=0, q=F, k=F, v=F, sq=128, sk=128, sv=256, alpha=F,
        beta=F, cu=F, s_in=F, slots_in=NUL, g=F, gs=F, dq=F, dkk=F, dvv=F, da=F, db=F, ds=F, ws=F, wsb=1 << 40):
    return gdn.lib().gdn_packed_backward(N, S, Hk, Hv, dk, dv, n_in, dtype, gate, order, 1.0, q, sq, k, sk, v, sv, alpha, beta,
                                         cu, s_in, slots_in, g, gs, dq, dkk, dvv, da, db, ds, ws, wsb, NUL)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), ARG), (dict(gate=2), ARG), (dict(order=2), ARG), (dict(N=-1), SHAPE), (dict(Hk=3), SHAPE),
    (dict(gate=1), UNSUP), (dict(dk=128), UNSUP), (dict(dk=32, dv=32), UNSUP), (dict(dk=60), UNSUP),
    (dict(sq=100), SHAPE), (dict(sq=129), ARG), (dict(n_in=1), SHAPE), (dict(sv=2**23 + 8), SHAPE),
    (dict(S=2**18, n_in=2**18), SHAPE), (dict(N=2**27), SHAPE),
    (dict(q=NUL), ARG), (dict(cu=NUL), ARG), (dict(g=NUL), ARG), (dict(dq=NUL), ARG), (dict(dkk=NUL), ARG), (dict(dvv=NUL), ARG),
    (dict(da=NUL), ARG), (dict(db=NUL), ARG), (dict(g=ODD), ARG), (dict(dq=ctypes.c_void_p(0x10004)), ARG), (dict(da=ODD), ARG),
    (dict(ds=ctypes.c_void_p(0x10008)), ARG), (dict(gs=ODD), ARG), (dict(ws=NUL), WS), (dict(wsb=1000), WS), (dict(ws=ODD), ARG),
    (dict(S=0), OK),
])
def test_packed_backward_refusals(kw, want):
    assert bwd(**kw) == want


def test_packed_backward_workspace():
    ws = gdn.gdn_packed_backward_workspace_bytes
    assert ws(100, 2, 2, 4, 32, 32, 1, 0) == 0 and ws(100, 2, 2, 4, 64, 64, 1, 1) == 0 and ws(0, 0, 2, 4, 64, 64, 1, 0) == 0
    one, shared = ws(1000, 2, 4, 4, 64, 64, 1, 0), ws(1000, 2, 2, 4, 64, 64, 1, 0)
    assert shared == one + 2 * (1000 * 4 * 64 * 4)
    assert ws(1 << 20, 1, 64, 64, 128, 128, 1, 0) <= (8 << 30) + (1 << 20)  # heads in groups


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,Hv", [(1024, 32), (5120, 16), (16384, 16), (65531, 4), (4096, 1)])
def test_packed_workspace_does_not_grow_with_short_sequences(N, Hv, d):
    """Sequences that no chunk kernel or segment serves need offsets and counts
    alone: at most three times the workspace of one sequence of N tokens (chunks of
    32 to 64 tokens, segments more than half full) and 20 bytes a sequence."""
    ws = gdn.gdn_packed_workspace_bytes
    one = ws(N, 1, Hv, Hv, d, d, N, 1, 0)
    for S in (2, 40, N // 8, N, 2**19 // Hv):
        assert 0 < ws(N, S, Hv, Hv, d, d, N, 1, 0) <= 3 * one + 20 * S + 4096, S


def test_packed_workspace_of_a_server_step():
    """Single tokens beside a prompt, and alone with no bound on their lengths given."""
    ws = gdn.gdn_packed_workspace_bytes
    assert ws(1024, 1024, 32, 32, 128, 128, 1024, 1, 0) < 64 << 20
    assert ws(5120, 1025, 16, 16, 128, 128, 4096, 1, 0) < 256 << 20


def test_an_empty_pool_without_slots_is_refused():
    """A pool of no slots holds no sequence; it is not the same as no pool."""
    import torch
    z = torch.zeros
    q, v, a = z(10, 2, 64, dtype=torch.bfloat16), z(10, 4, 64, dtype=torch.bfloat16), z(10, 4)
    cu, none = torch.tensor([0, 4, 10], dtype=torch.int32), z(0, 4, 64, 64)
    for call in (lambda: gdn.packed_fwd(q, q, v, a, a, cu, none), lambda: gdn.packed_fwd(q, q, v, a, a, cu, None, None, none),
                 lambda: gdn.packed_backward(q, q, v, a, a, cu, none, None, v)):
        with pytest.raises(gdn.GdnError) as e:
            call()
        assert e.value.status == SHAPE
