"""Host-side checks of the entry points of linear attention and of the query and
key norm: sizes and refusals, which come before any device is touched (no GPU
needed)."""
import ctypes

import pytest

from gated_delta_rule_12_amd import gdn

F = ctypes.c_void_p(0x10000)  # never dereferenced: every call below is refused first
NUL = ctypes.c_void_p(0)
ODD, HALF = ctypes.c_void_p(0x10002), ctypes.c_void_p(0x10008)
FAR = ctypes.c_void_p(1 << 40)
STATES = 4 * 2 * 4 * 64 * 64  # bytes of two sequences' states of four heads of 64
OK, ARG, SHAPE, UNSUP, WS = gdn.GDN_OK, gdn.GDN_E_ARG, gdn.GDN_E_SHAPE, gdn.GDN_E_UNSUPPORTED, gdn.GDN_E_WORKSPACE


def fwd(N=100, S=2, Hk=2, Hv=4, dk=64, dv=64, n_in=2, n_out=2, max_len=1, dtype=1, q=F, sq=None, k=F, sk=None, v=F, sv=None,
        alpha=F, cu=F, s_in=F, slots_in=NUL, s_out=F, slots_out=NUL, out=F, ws=NUL, wsb=0):
    sq = Hk * dk if sq is None else sq
    sk = Hk * dk if sk is None else sk
    sv = Hv * dv if sv is None else sv
    return gdn.lib().gdn_linear_fwd(N, S, Hk, Hv, dk, dv, n_in, n_out, max_len, dtype, 1.0, q, sq, k, sk, v, sv, alpha, cu,
                                    s_in, slots_in, s_out, slots_out, out, ws, wsb, NUL)


def bwd(N=100, S=2, Hk=2, Hv=4, dk=64, dv=64, n_in=2, dtype=1, q=F, sq=None, k=F, sk=None, v=F, sv=None, alpha=F, cu=F,
        s_in=F, slots_in=NUL, go=F, gs=F, dq=F, dkk=F, dvv=F, da=F, ds=FAR, ws=F, wsb=1 << 40):
    sq = Hk * dk if sq is None else sq
    sk = Hk * dk if sk is None else sk
    sv = Hv * dv if sv is None else sv
    return gdn.lib().gdn_linear_backward(N, S, Hk, Hv, dk, dv, n_in, dtype, 1.0, q, sq, k, sk, v, sv, alpha, cu, s_in,
                                         slots_in, go, gs, dq, dkk, dvv, da, ds, ws, wsb, NUL)


BOTH = [
    (dict(dtype=2), ARG), (dict(dtype=-1), ARG),
    (dict(N=-1), SHAPE), (dict(S=-1), SHAPE), (dict(Hk=3), SHAPE), (dict(Hk=0), SHAPE), (dict(dk=0), SHAPE),
    (dict(n_in=-1), SHAPE), (dict(N=2**31), SHAPE), (dict(S=2**31), SHAPE), (dict(Hk=1, Hv=65536), SHAPE),
    (dict(dk=72), UNSUP), (dict(dv=144), UNSUP), (dict(dk=8), UNSUP),
    (dict(sq=127), SHAPE), (dict(sv=255), SHAPE), (dict(sk=2**31), SHAPE),
    (dict(sq=2**23 + 8), SHAPE), (dict(sk=2**23 + 8), SHAPE), (dict(sv=2**23 + 8), SHAPE),
    (dict(sq=132), ARG), (dict(sk=129), ARG), (dict(sv=258, dtype=0), ARG),   # strides of whole 16-byte pieces
    (dict(q=NUL), ARG), (dict(k=NUL), ARG), (dict(v=NUL), ARG), (dict(alpha=NUL), ARG), (dict(cu=NUL), ARG),
    (dict(q=ODD), ARG), (dict(k=HALF), ARG), (dict(v=ODD), ARG), (dict(s_in=HALF), ARG), (dict(cu=ODD), ARG),
    (dict(alpha=ODD), ARG), (dict(slots_in=ODD), ARG),
    (dict(n_in=1), SHAPE),                                     # a pool without indices holds every sequence
    (dict(S=0), OK), (dict(Hk=0, Hv=0), OK),                   # nothing to do
]


@pytest.mark.parametrize("kw,want", BOTH + [
    (dict(max_len=-1), SHAPE), (dict(n_out=-1), SHAPE), (dict(n_out=1), SHAPE),
    (dict(out=NUL), ARG), (dict(out=HALF), ARG), (dict(s_out=ODD), ARG), (dict(slots_out=ODD), ARG),
    (dict(S=2**25, Hv=8, n_in=2**25, n_out=2**25), SHAPE),     # more workgroups than a grid holds
    (dict(S=2**18, Hv=16, n_in=2**18, n_out=2**18), SHAPE),
    (dict(S=2**16, Hv=16, n_in=2**16, n_out=2**16, max_len=64), SHAPE),  # fewer with segments
    (dict(N=2**25, Hv=16, max_len=2**25), SHAPE),
    (dict(max_len=100), WS), (dict(max_len=100, ws=F, wsb=16), WS), (dict(max_len=100, ws=HALF, wsb=1 << 40), ARG),
])
def test_linear_refusals(kw, want):
    assert fwd(**kw) == want


@pytest.mark.parametrize("kw,want", BOTH + [
    (dict(go=NUL), ARG), (dict(dq=NUL), ARG), (dict(dkk=NUL), ARG), (dict(dvv=NUL), ARG),
    (dict(go=HALF), ARG), (dict(gs=HALF), ARG), (dict(dq=HALF), ARG), (dict(dkk=ODD), ARG), (dict(dvv=HALF), ARG),
    (dict(da=ODD), ARG), (dict(ds=HALF), ARG), (dict(ws=HALF), ARG), (dict(ws=NUL), WS), (dict(wsb=16), WS),
    (dict(S=2**16, Hv=16, n_in=2**16), SHAPE), (dict(N=2**25, Hv=16), SHAPE),
    (dict(ds=F), ARG), (dict(ds=ctypes.c_void_p(0x10000 + STATES - 16)), ARG),  # grad_state_out's memory
    (dict(gs=FAR), ARG), (dict(ds=ctypes.c_void_p(0x10000 + STATES), wsb=16), WS),
])
def test_linear_backward_refusals(kw, want):
    assert bwd(**kw) == want


# Buffers apart from each other (names as in fwd and bwd), and others within them
APART = {n: (i + 1) << 36 for i, n in enumerate(("q", "k", "v", "alpha", "cu", "s_in", "s_out", "out", "go", "gs", "dq", "dkk",
                                                 "dvv", "da", "ds", "ws", "gq", "gk", "wq", "wk", "cos", "sin", "pos", "qo",
                                                 "ko", "dwq", "dwk"))}


def at(name, offset=0):
    return ctypes.c_void_p(APART[name] + offset)


def apart(f, over, **kw):
    """f with buffers of their own, but those of `over`, {name: (name, offset)}"""
    names = f.__code__.co_varnames[:f.__code__.co_argcount]
    args = {n: at(n) for n in names if n in APART}
    args.update({n: at(*x) for n, x in over.items()})
    return f(**{**args, **kw})


ROW = 2 * 64 * 2  # bytes of a token's keys


@pytest.mark.parametrize("over", [
    {"ds": ("s_in", 0)}, {"ds": ("s_in", STATES - 16)}, {"s_in": ("ds", STATES - 16)},  # start states are read behind it
    {"dq": ("q", 0)}, {"dkk": ("q", 0)}, {"dkk": ("k", 0)}, {"dvv": ("v", 0)}, {"dvv": ("go", 0)}, {"dq": ("go", 0)},
    {"dvv": ("k", 100 * ROW - 16)}, {"go": ("dvv", 200 * ROW - 16)}, {"dq": ("v", 16)},
    {"dkk": ("dq", 100 * ROW - 16)}, {"dvv": ("dkk", 0)}, {"ds": ("gs", STATES // 2)}, {"ds": ("dq", 0)},
    {"da": ("alpha", 0)}, {"da": ("alpha", 12)}, {"da": ("ds", 16)}, {"ws": ("q", 0)}, {"ws": ("ds", 256)}, {"gs": ("ws", 16)},
])
def test_linear_backward_refuses_shared_memory(over):
    assert apart(bwd, over) == ARG
    assert apart(bwd, over, wsb=16) == WS  # the last of the checks


SHARED = [
    {"out": ("v", 0)}, {"out": ("q", 0)}, {"out": ("k", 100 * ROW - 16)}, {"v": ("out", 200 * ROW - 16)},
    {"out": ("s_in", STATES - 16)}, {"out": ("s_out", 0)}, {"s_out": ("v", 16)}, {"s_out": ("alpha", 0)},
    {"s_out": ("s_in", 16)}, {"s_in": ("s_out", STATES - 16)},  # pools, but not slot upon slot
]


@pytest.mark.parametrize("max_len,over", [(n, over) for n in (1, 100) for over in SHARED] + [
    (100, over) for over in ({"ws": ("s_in", 0)}, {"ws": ("s_out", 0)}, {"ws": ("k", 0)}, {"out": ("ws", 256)})])
def test_linear_refuses_shared_memory(max_len, over):
    assert apart(fwd, over, max_len=max_len, wsb=1 << 40) == ARG


def test_linear_workspace():
    ws = gdn.gdn_linear_workspace_bytes
    assert ws(256, 256, 16, 16, 128, 128, 1, 1) == 0 and ws(31, 1, 1, 1, 64, 64, 1000, 0) == 0  # token by token
    assert ws(1000, 3, 2, 3, 64, 64, 1000, 1) == 0 and ws(1000, 3, 2, 4, 60, 64, 1000, 1) == 0  # refused
    state = 4 * 16 * 128 * 128
    one = ws(4096, 1, 16, 16, 128, 128, 4096, 1)
    assert 17 * state < one < 19 * state and one % 256 == 0
    # short sequences take no places for states
    assert ws(4096 + 1000, 1001, 16, 16, 128, 128, 4096, 1) < 400 * state
    assert ws(2**31 - 1, 1, 1, 1, 16, 16, 2**31 - 1, 1) == 0  # over the limit of rows
    back = gdn.gdn_linear_backward_workspace_bytes
    assert back(4096, 1, 16, 16, 128, 128, 1) > 2 * 17 * state and back(4096, 0, 16, 16, 128, 128, 1) == 0
    assert back(4096, 1, 16, 16, 120, 128, 1) == 0
    # few tokens: the sums of a key head's value heads in parts, 32 MiB of them at most
    assert 0 < back(1500, 2, 1, 16, 128, 128, 1) - back(1500, 2, 16, 16, 128, 128, 1) <= 2**25
    assert back(20000, 2, 1, 16, 128, 128, 1) == back(20000, 2, 16, 16, 128, 128, 1)
    # gradients in fp32 have twice the workgroups
    assert back(2**23, 1, 16, 16, 16, 16, 0) > 0 and back(2**23 + 1, 1, 16, 16, 16, 16, 0) == 0
    assert back(2**14, 2**14, 16, 16, 16, 16, 0) > 0 and back(2**15, 2**14 + 1, 16, 16, 16, 16, 0) == 0
    assert back(2**24, 1, 16, 16, 16, 16, 1) > 0


def qk(N=10, Hq=4, Hk=2, d=64, rot=32, n_pos=100, dtype=1, rotation=0, eps=1e-6, q=F, sq=None, k=F, sk=None, wq=F, wk=F, cos=F,
       sin=F, pos=F, qo=F, so=None, ko=F, sp=None):
    sq, so = (Hq * d if s is None else s for s in (sq, so))
    sk, sp = (Hk * d if s is None else s for s in (sk, sp))
    return gdn.lib().gdn_qk_norm_fwd(N, Hq, Hk, d, rot, n_pos, dtype, rotation, eps, q, sq, k, sk, wq, wk, cos, sin, pos, qo,
                                     so, ko, sp, NUL)


def qk_bwd(N=10, Hq=4, Hk=2, d=64, rot=32, n_pos=100, dtype=1, rotation=0, eps=1e-6, gq=F, sgq=None, gk=F, sgk=None, q=F,
           sq=None, k=F, sk=None, wq=F, wk=F, cos=F, sin=F, pos=F, dq=F, dkk=F, dwq=F, dwk=F, ws=F, wsb=1 << 40):
    sq, sgq = (Hq * d if s is None else s for s in (sq, sgq))
    sk, sgk = (Hk * d if s is None else s for s in (sk, sgk))
    return gdn.lib().gdn_qk_norm_backward(N, Hq, Hk, d, rot, n_pos, dtype, rotation, eps, gq, sgq, gk, sgk, q, sq, k, sk, wq,
                                          wk, cos, sin, pos, dq, dkk, dwq, dwk, ws, wsb, NUL)


NORM = [
    (dict(dtype=2), ARG), (dict(rotation=2), ARG), (dict(rotation=-1), ARG),
    (dict(N=-1), SHAPE), (dict(Hq=-1), SHAPE), (dict(Hk=-1), SHAPE), (dict(d=0), SHAPE), (dict(rot=-16), SHAPE),
    (dict(rot=80), SHAPE), (dict(n_pos=-1), SHAPE), (dict(n_pos=0), SHAPE), (dict(N=2**31), SHAPE), (dict(n_pos=2**31), SHAPE),
    (dict(Hq=65536), SHAPE), (dict(N=2**30, Hq=128, d=256), SHAPE),
    (dict(d=72), UNSUP), (dict(d=272), UNSUP), (dict(rot=24), UNSUP),
    (dict(sq=255), SHAPE), (dict(sk=127), SHAPE), (dict(sq=2**23 + 8), SHAPE),
    (dict(sq=260), ARG), (dict(sk=130, dtype=0), ARG),
    (dict(q=NUL), ARG), (dict(k=NUL), ARG), (dict(cos=NUL), ARG), (dict(sin=NUL), ARG),
    (dict(q=HALF), ARG), (dict(k=HALF), ARG), (dict(wq=HALF), ARG), (dict(wk=ODD), ARG), (dict(cos=HALF), ARG),
    (dict(sin=ODD), ARG), (dict(pos=ODD), ARG),
]


@pytest.mark.parametrize("kw,want", NORM + [
    (dict(qo=NUL), ARG), (dict(ko=NUL), ARG), (dict(qo=HALF), ARG), (dict(so=255), SHAPE), (dict(sp=132), ARG),
    (dict(N=0), OK), (dict(Hq=0, Hk=0), OK), (dict(N=0, q=NUL, k=NUL, qo=NUL, ko=NUL, cos=NUL, sin=NUL), OK),
])
def test_qk_norm_refusals(kw, want):
    assert qk(**kw) == want


@pytest.mark.parametrize("kw,want", NORM + [
    (dict(gq=NUL), ARG), (dict(gk=NUL), ARG), (dict(gq=HALF), ARG), (dict(sgq=255), SHAPE), (dict(sgk=132), ARG),
    (dict(dq=HALF), ARG), (dict(dkk=ODD), ARG), (dict(dwq=ODD), ARG), (dict(dwk=ODD), ARG),
    (dict(ws=NUL), WS), (dict(wsb=16), WS), (dict(ws=HALF), ARG),
    (dict(dq=NUL, dkk=NUL, dwq=NUL, dwk=NUL, q=NUL, k=NUL, gq=NUL, gk=NUL), OK),  # nothing wanted
])
def test_qk_norm_backward_refusals(kw, want):
    assert qk_bwd(**kw) == want


QROW, KROW = 4 * 64 * 2, 2 * 64 * 2  # bytes of a token's queries and keys


@pytest.mark.parametrize("over,kw", [
    ({"qo": ("k", 0), "ko": ("q", 0)}, {}),                                 # swapped
    ({"qo": ("k", 0)}, {}), ({"ko": ("q", 16)}, {}),
    ({"qo": ("q", QROW)}, {}), ({"q": ("qo", 9 * QROW)}, {}), ({"ko": ("k", 9 * KROW)}, {}),  # by whole tokens
    ({"qo": ("q", 16)}, {}), ({"qo": ("q", 0)}, dict(so=512)), ({"ko": ("k", 0)}, dict(sk=512)),  # one stride of two
    ({"qo": ("ko", 10 * KROW - 16)}, {}), ({"qo": ("ko", 0)}, {}),
    # in one projection of 512 elements a token: q's columns 0 .., k's 256 ..
    ({"k": ("q", 512), "qo": ("q", 0), "ko": ("q", 512 - 16)}, dict(sq=512, sk=512, so=512, sp=512)),
    ({"k": ("q", 512), "qo": ("q", 0), "ko": ("q", 512 + 1024)}, dict(sq=512, sk=512, so=512, sp=512)),
    ({"qo": ("wk", 0)}, {}), ({"ko": ("cos", 100 * 64 - 16)}, {}), ({"ko": ("pos", 32)}, {}),
])
def test_qk_norm_refuses_shared_memory(over, kw):
    assert apart(qk, over, **kw) == ARG


@pytest.mark.parametrize("over,kw", [
    ({"dq": ("k", 0)}, {}), ({"dq": ("gk", 0)}, {}), ({"dkk": ("gq", 0)}, {}), ({"dkk": ("q", 16)}, {}),
    ({"dq": ("q", QROW)}, {}), ({"dq": ("gq", 16)}, {}), ({"dkk": ("gk", 9 * KROW)}, {}),
    ({"dq": ("q", 0)}, dict(sq=512)), ({"dq": ("gq", 0)}, dict(sgq=512)), ({"dkk": ("gk", 0)}, dict(sgk=512)),
    ({"dq": ("dkk", 0)}, {}), ({"dwq": ("dwk", 0)}, {}), ({"dwq": ("dq", 16)}, {}), ({"dwk": ("ws", 0)}, {}),
    ({"ws": ("q", 0)}, {}), ({"ws": ("gk", 0)}, {}), ({"ws": ("wq", 0)}, {}), ({"ws": ("dq", 0)}, {}),
    ({"dq": ("sin", 0)}, {}), ({"dkk": ("wk", 0)}, {}),
])
def test_qk_norm_backward_refuses_shared_memory(over, kw):
    assert apart(qk_bwd, over, **kw) == ARG
    assert apart(qk_bwd, over, **{**kw, "wsb": 16}) == WS  # the last of the checks


def test_qk_norm_workspace():
    ws = gdn.gdn_qk_norm_workspace_bytes
    assert ws(1, 4, 2, 64) == 2 * 64 * 4 and ws(0, 4, 2, 64) == 0 and ws(10, 4, 2, 60) == 0
    assert 0 < ws(10**6, 16, 16, 128) <= 1024 * 128 * 4 and ws(1000, 65535, 0, 16) > 0 and ws(10**6, 65535, 0, 16) == 0
