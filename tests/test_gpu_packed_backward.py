"""gdn_packed_backward against the oracle's backward (fp64 chain rule through the
token loop) over every sequence, and against differences of its forward.

Tolerance, as for gdn_backward: fp32 throughout (unit roundoff 2^-24) with
sums of at most 128 terms (7.6e-6 of their terms' sizes at worst), so 1e-5 of a
gradient's largest value per sequence and head.
"""
from __future__ import annotations

import numpy as np
import pytest

from gated_delta_rule_12_amd import gdn
from packed_case import Packed

pytestmark = pytest.mark.gpu
PTD, DTP = gdn.GDN_PREDICT_THEN_DECAY, gdn.GDN_DECAY_THEN_PREDICT
TOL = 1e-5
NAMES = ("dq", "dk", "dv", "dalpha", "dbeta", "dstate0")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn.lib()


def tensors(c):
    return {n: c.cuda(n) for n in ("q", "k", "v", "alpha", "beta", "cu", "pool", "slots_in", "dout", "dstate")}


def run(c, t=None, with_state=True, with_grad_state=True, **kw):
    import torch
    t = t or tensors(c)
    print(f"case {c.lengths} hk={c.hk} hv={c.hv} d={c.dk} {c.dtype} order={c.order}", flush=True)
    got = gdn.packed_backward(t["q"], t["k"], t["v"], t["alpha"], t["beta"], t["cu"], t["pool"] if with_state else None,
                              t["slots_in"] if with_state else None, t["dout"], t["dstate"] if with_grad_state else None,
                              order=c.order, scale=c.scale, **kw)
    torch.cuda.synchronize()
    return got


def check(c, got):
    ref = c.backward()
    for name, x, r in zip(NAMES, got, ref):
        if x is None:
            continue
        x = x.double().cpu().numpy()
        assert x.shape == r.shape and np.isfinite(x).all(), name
        if name == "dstate0":
            e = np.abs(x - r).max(axis=(2, 3)) / np.maximum(np.abs(r).max(axis=(2, 3)), 1e-30)
            worst = e.max()
        else:
            worst = 0.0
            for s, n in enumerate(c.lengths):
                a = int(c.a["cu"][s])
                if n:
                    xs, rs = x[a:a + n], r[a:a + n]
                    ax = (0, 2) if rs.ndim == 3 else (0,)
                    top = np.abs(rs).max(axis=ax)  # zero: dalpha of a lone token on a zero state
                    worst = max(worst, (np.abs(xs - rs).max(axis=ax) / np.where(top > 0, top, 1.0)).max())
            last = int(c.a["cu"][-1])
            assert (x[last:] == 0).all(), name
        print(f"  {name}: err {worst:.2e}", flush=True)
        assert worst <= TOL, (name, worst)


CASES = [
    Packed((1,), 1, 1, 64, 64),
    Packed((1, 2, 63), 1, 2, 64, 64, slots=1, tail=3),
    Packed((64, 65, 128), 2, 2, 64, 64, order=DTP),
    Packed((150, 0, 7, 0), 1, 3, 128, 128, slots=2),
    Packed((300, 1, 90), 2, 4, 128, 128, order=DTP, fresh=(1,), scale=0.125, tail=70),
    Packed((129, 200), 2, 2, 128, 128, dtype="f32", slots=1),
    Packed((40, 100), 1, 4, 64, 64, dtype="f32", order=DTP),
    Packed((700, 20), 1, 2, 128, 128, alpha_mean=6.0),
    Packed((200, 64), 1, 2, 64, 64, alpha_mean=-4.0),
    Packed((90, 100, 80, 70), 4, 16, 128, 128),   # a chain workgroup of two state slices
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_gradients(i):
    c = CASES[i]
    c.seed = 200 + i
    c.make()
    check(c, run(c))


def test_without_states():
    c = Packed((100, 65), 1, 2, 64, 64, seed=31).make()
    c.a["slots_in"][:] = -1
    c.a["dstate"][:] = 0
    got = run(c, with_state=False, with_grad_state=False, want_grad_state0=False)
    assert got[5] is None
    check(c, got)


def test_against_differences():
    """Central differences of the oracle's forward, a sample of every input."""
    c = Packed((20, 70, 3), 1, 2, 64, 64, dtype="f32", seed=32, slots=1).make()
    got = [x.double().cpu().numpy() for x in run(c)]
    n = sum(c.lengths)

    def loss():
        o, e = c.forward()
        return float((o[:n] * c.a["dout"][:n]).sum() + (e * c.a["dstate"]).sum())
    r = np.random.Generator(np.random.PCG64(1))
    for name, x in (("q", got[0]), ("k", got[1]), ("v", got[2]), ("alpha", got[3]), ("beta", got[4])):
        a = c.a[name] = c.a[name].astype(np.float64)
        for _ in range(6):
            i = tuple(int(r.integers(0, m)) for m in a.shape)
            old, h = a[i], 1e-5
            a[i] = old + h
            up = loss()
            a[i] = old - h
            down = loss()
            a[i] = old
            # the loss is about 1e2 with 64-bit roundings of 1e-14 of that, and
            # its third derivatives times h^2 about 1e-8
            assert abs((up - down) / (2 * h) - x[i]) <= 2e-5 * np.abs(x).max() + 1e-6, (name, i)


def test_tokens_in_front_have_zero_gradients():
    c = Packed((70, 100, 30), 1, 2, 64, 64, seed=33).make()
    t = tensors(c)
    t.update(cu=t["cu"][1:], slots_in=t["slots_in"][1:], dstate=t["dstate"][1:].contiguous())
    got = run(c, t)
    for x in got[:5]:
        assert (x[:70] == 0).all()
    c.lengths, c.a["cu"] = c.lengths[1:], c.a["cu"][1:]
    c.a["slots_in"], c.a["dstate"] = c.a["slots_in"][1:], c.a["dstate"][1:]
    c.forward = None
    ref = [np.zeros(c.a[n].shape) for n in ("q", "k", "v", "alpha", "beta")]
    import oracle
    for s in range(2):
        a, b = int(c.a["cu"][s]), int(c.a["cu"][s + 1])
        rep = lambda x: np.repeat(x[a:b], 2, axis=1)[None]  # noqa: E731
        r = oracle.backward(rep(c.a["q"]), rep(c.a["k"]), c.a["v"][a:b][None], c.a["alpha"][a:b][None], c.a["beta"][a:b][None],
                            c.a["pool"][c.a["slots_in"][s]][None], c.a["dout"][a:b][None], c.a["dstate"][s][None])
        for dst, val in zip(ref, (r[0][0].sum(1, keepdims=True), r[1][0].sum(1, keepdims=True), r[2][0], r[3][0], r[4][0])):
            dst[a:b] = val
    for x, r in zip(got, ref):
        assert np.abs(x.double().cpu().numpy() - r).max() <= TOL * np.abs(r).max()


def test_slices_of_one_projection():
    import torch
    c = Packed((100, 7, 1), 2, 4, 64, 64, seed=34).make()
    t = tensors(c)
    whole = run(c, t)
    N = t["q"].shape[0]
    row = torch.cat([t["q"].reshape(N, -1), t["k"].reshape(N, -1), t["v"].reshape(N, -1), t["v"].new_zeros(N, 8)], 1)
    t.update(q=row[:, :128].view(N, 2, 64), k=row[:, 128:256].view(N, 2, 64), v=row[:, 256:512].view(N, 4, 64))
    for x, y in zip(run(c, t), whole):
        assert torch.equal(x, y)


@pytest.mark.parametrize("d", [64, 128])
def test_far_tokens(d):
    """Token strides up to the limit: elements past 2^31, bytes past 2^32."""
    import torch
    c = Packed((270, 31), 1, 2, d, d, seed=36).make()
    far = torch.empty((301, 2**23), dtype=torch.bfloat16, device="cuda")
    far[:, :d], far[:, d:2 * d] = c.cuda("q")[:, 0], c.cuda("k")[:, 0]
    far[:, -2 * d:] = c.cuda("v").view(301, 2 * d)
    t = tensors(c)
    t.update(q=far[:, :d].view(301, 1, d), k=far[:, d:2 * d].view(301, 1, d), v=far[:, -2 * d:].view(301, 2, d))
    check(c, run(c, t))


def test_bad_offsets_stay_in_bounds():
    """Falling, negative and far offsets and slots (the values are not defined)."""
    import torch
    c = Packed((100, 70, 30), 1, 2, 64, 64, seed=35).make()
    t = tensors(c)
    N = t["q"].shape[0]
    L = gdn.lib()
    for cu in ([0, 150, 90, 200], [-5, 100, 10**6, 200], [200, 100, 0, -1], [0, 0, 0, 2**31 - 1]):
        cut = torch.tensor(cu, dtype=torch.int32).cuda()
        slots = torch.tensor([10**9, -7, 2], dtype=torch.int32).cuda()
        guards = [torch.full((n + 512,), 7.0, device="cuda") for n in (N * 64, N * 64, N * 128, N * 2, N * 2, 3 * 2 * 64 * 64)]
        n = gdn.gdn_packed_backward_workspace_bytes(N, 3, 1, 2, 64, 64, 1, 0)
        ws = torch.empty(n + 1024, dtype=torch.uint8, device="cuda").fill_(7)
        rc = L.gdn_packed_backward(N, 3, 1, 2, 64, 64, 3, 1, 0, 0, 1.0, t["q"].data_ptr(), 64, t["k"].data_ptr(), 64,
                                   t["v"].data_ptr(), 128, t["alpha"].data_ptr(), t["beta"].data_ptr(), cut.data_ptr(),
                                   t["pool"].data_ptr(), slots.data_ptr(), t["dout"].data_ptr(), t["dstate"].data_ptr(),
                                   *[g[256:].data_ptr() for g in guards], ws.data_ptr(), n,
                                   torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert rc == gdn.GDN_OK
        for g in guards:
            assert (g[:256] == 7.0).all() and (g[-256:] == 7.0).all()
        assert (ws[n:] == 7).all()


def test_head_groups_of_a_large_batch():
    """More chunks and heads than one launch's records hold: the same results
    as half of the heads at a time (a launch of their own)."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    N, hk, hv, d = 9000, 32, 128, 128
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q, k = (torch.nn.functional.normalize(rnd(N, hk, d), dim=-1).bfloat16() for _ in range(2))
    v, dout = rnd(N, hv, d).bfloat16(), rnd(N, hv, d).bfloat16()
    al, be = torch.sigmoid(2 + 0.5 * rnd(N, hv)), torch.sigmoid(rnd(N, hv))
    cu = torch.tensor([0, 700, 701, 5000, 9000], dtype=torch.int32).cuda()
    per = gdn.gdn_packed_backward_workspace_bytes(N, 4, 1, 4, d, d, 1, 0) - 2 * 4 * N * 4 * d - 8192
    assert per * hk > 8 << 30
    whole = gdn.packed_backward(q, k, v, al, be, cu, None, None, dout)
    torch.cuda.synchronize()
    for half in range(2):
        a, b = slice(16 * half, 16 * half + 16), slice(64 * half, 64 * half + 64)
        part = gdn.packed_backward(q[:, a].contiguous(), k[:, a].contiguous(), v[:, b].contiguous(), al[:, b].contiguous(),
                                   be[:, b].contiguous(), cu, None, None, dout[:, b].contiguous())
        torch.cuda.synchronize()
        for x, y, h in zip(whole, part, (a, a, b, b, b, b)):
            assert torch.equal(x[:, h], y)


def test_repeats_are_identical_and_graphs_replay():
    import torch
    c = Packed((1, 300, 70), 2, 4, 64, 64, seed=36).make()
    t = tensors(c)
    ws = torch.empty(gdn.gdn_packed_backward_workspace_bytes(371, 3, 2, 4, 64, 64, 1, 0), dtype=torch.uint8, device="cuda")
    first = run(c, t, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gdn.packed_backward(t["q"], t["k"], t["v"], t["alpha"], t["beta"], t["cu"], t["pool"], t["slots_in"], t["dout"],
                            t["dstate"], workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = gdn.packed_backward(t["q"], t["k"], t["v"], t["alpha"], t["beta"], t["cu"], t["pool"], t["slots_in"], t["dout"],
                                  t["dstate"], workspace=ws)
    for _ in range(3):
        for x in got:
            x.zero_()
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, first))
        again = run(c, t)
        assert all(torch.equal(x, y) for x, y in zip(again, first))


def test_a_training_step_of_a_block():
    """norm -> packed rule -> heads' norm and back, against the same chain of
    64-bit definitions on the values the kernels hand on."""
    import torch
    c = Packed((90, 40, 1), 2, 4, 64, 64, dtype="f32", seed=37, fresh=(0, 1, 2)).make()
    t = tensors(c)
    N = t["q"].shape[0]
    x = torch.randn(N, 512, generator=torch.Generator().manual_seed(1)).cuda()
    w0, w1 = torch.rand(512).cuda() + 0.5, torch.rand(64).cuda() + 0.5
    # the block's input norm gives the rule's q, k, v rows
    y, m0, r0 = gdn.layer_norm_fwd(x, w0)
    q, k, v = (y[:, a:b].unflatten(1, (-1, 64)) for a, b in ((0, 128), (128, 256), (256, 512)))
    q, k = (z * 0.1 for z in (q, k))
    out, _ = gdn.packed_fwd(q, k, v, t["alpha"], t["beta"], t["cu"])
    z, m1, r1 = gdn.layer_norm_fwd(out, w1)
    dz = t["dout"]
    dout, dw1, db1 = gdn.layer_norm_backward(dz, out, w1, m1, r1)
    dq, dk, dv, da, db, _ = gdn.packed_backward(q, k, v, t["alpha"], t["beta"], t["cu"], None, None, dout)
    dy = torch.cat([0.1 * dq.flatten(1), 0.1 * dk.flatten(1), dv.flatten(1)], 1)
    dx, dw0, db0 = gdn.layer_norm_backward(dy, x, w0, m0, r0)
    torch.cuda.synchronize()

    X, W0, W1 = (p.double().cpu().requires_grad_() for p in (x, w0, w1))
    A, B = (t[n].double().cpu().requires_grad_() for n in ("alpha", "beta"))

    def norm(u, w):
        u = u - u.mean(-1, keepdim=True)
        return u * (u.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * w
    Y = norm(X, W0)
    Q, K, V = (Y[:, a:b].unflatten(1, (-1, 64)) for a, b in ((0, 128), (128, 256), (256, 512)))
    Q, K = (0.1 * u.repeat_interleave(2, 1) for u in (Q, K))
    outs = []
    for s in range(3):
        S = torch.zeros(4, 64, 64, dtype=torch.float64)
        for i in range(int(c.a["cu"][s]), int(c.a["cu"][s + 1])):
            e = B[i][:, None] * (V[i] - (S @ K[i][..., None])[..., 0])
            S = A[i][:, None, None] * S + e[..., None] * K[i][:, None, :]
            outs.append((S @ Q[i][..., None])[..., 0])
    (norm(torch.stack(outs), W1) * dz.double().cpu()).sum().backward()
    # fp32 all the way: each of the six kernels adds its 1e-5
    for got, ref in ((dx, X.grad), (dw0, W0.grad), (dw1, W1.grad), (da, A.grad), (db, B.grad)):
        assert (got.double().cpu() - ref).abs().max() <= 6e-5 * ref.abs().max()


@pytest.mark.parametrize("d", [64, 128])
def test_without_sequences_every_row_is_zero(d):
    """cu_seqlens of one entry: no sequence, so every row is outside them."""
    import torch
    c = Packed((70,), 1, 2, d, d, seed=51).make()
    t = tensors(c)
    t.update(cu=t["cu"][:1], slots_in=t["slots_in"][:0], dstate=t["dstate"][:0])
    # (memory that the gradients may get back is not zero)
    dirty = [torch.full((70, 2, d), 7.0, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    del dirty
    got = run(c, t)
    for name, x in zip(NAMES[:5], got):
        assert (x == 0).all(), name
    assert got[5].shape == (0, 2, d, d)
    # no value heads: q and k have gradients of zero all the same
    dq, dkk, dvv, *_ = gdn.packed_backward(t["q"], t["k"], t["v"][:, :0], t["alpha"][:, :0].contiguous(),
                                           t["beta"][:, :0].contiguous(), c.cuda("cu"), None, None,
                                           t["dout"][:, :0].contiguous())
    torch.cuda.synchronize()
    assert (dq == 0).all() and (dkk == 0).all() and dvv.shape == (70, 0, d)


@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "bf16"), (128, "f32")])
def test_non_finite_values_stay_where_they_are(d, dtype):
    """Rows outside the sequences are not read, and what is not finite in one
    sequence leaves the others' gradients as they are, bit for bit."""
    import torch
    c = Packed((70, 1, 130, 33), 1, 2, d, d, dtype=dtype, seed=52, tail=70).make()
    t = tensors(c)
    t.update(cu=t["cu"][1:], slots_in=t["slots_in"][1:], dstate=t["dstate"][1:].contiguous())
    first = run(c, t)
    for n in ("q", "k", "v", "alpha", "beta", "dout"):
        t[n][:70], t[n][234:] = np.nan, np.inf
    for x, y in zip(first, run(c, t)):
        assert torch.equal(x, y)
    t["v"][71 + 65, 1, 3], t["dout"][71 + 100, 0, 2] = np.inf, np.nan  # the second of three sequences
    for name, x, y in zip(NAMES, first, run(c, t)):
        if name == "dstate0":
            assert torch.equal(x[0], y[0]) and torch.equal(x[2], y[2]) and not torch.isfinite(y[1]).all()
        else:
            assert torch.equal(x[:71], y[:71]) and torch.equal(x[201:], y[201:]) and not torch.isfinite(y[71:201]).all(), name
