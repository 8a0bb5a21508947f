"""gdn_qk_norm_fwd and gdn_qk_norm_backward against 64-bit formulas.

Tolerances, derived before the first run.  With u = 2^-24: a row's sum of d
squares is off by at most d u of itself (all its terms are positive), half of
which reaches r; the hardware's reciprocal square root adds 2 u, products and the
rotation's sum 4 u of the sizes of its two terms:
    |error| <= (d / 2 + 8) u size,   size = |z_a cos| + |z_b sin|,
and 2^-8 |value| where it is rounded to bf16.  Backward: each sum over a row is
off by d u of the sum of its terms' sizes; dx is formed from terms of sizes r |g
w| and r |xhat| mean |g w xhat|:
    |error| <= (2 d + 16) u (r |g| |w| + r |xhat| mean(|g| |w| |xhat|)),
with |g| the rotation's size as above; weights' gradients, sums over R rows
whose partial sums are at most R long:
    |error| <= (R + d + 16) u sum |g xhat|.
"""
from __future__ import annotations

import numpy as np
import pytest

from gated_delta_rule_12_amd import gdn
from linear_case import Linear, qk_norm, qk_norm_backward, rotate, rounded

pytestmark = pytest.mark.gpu
U = 2.0**-24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn.lib()


class Case:
    def __init__(self, N, hq, hk, d, rot, dtype="bf16", interleaved=False, n_pos=50, weights=True, positions=True, eps=1e-6,
                 fused=False, seed=0):
        self.__dict__.update(locals())
        r = np.random.Generator(np.random.PCG64(seed))
        scale = np.exp(r.uniform(-3, 3, (N, 1, 1)))
        self.x = [rounded(scale * r.standard_normal((N, h, d)), dtype) for h in (hq, hk)]
        self.dy = [rounded(r.standard_normal((N, h, d)), dtype) for h in (hq, hk)]
        self.w = [(1 + 0.3 * r.standard_normal(d)).astype(np.float32) if weights else None for _ in range(2)]
        angle = r.uniform(-50, 50, (n_pos, rot // 2))
        self.cos, self.sin = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
        self.pos = r.integers(0, n_pos, N).astype(np.int32) if positions else None
        at = self.pos if positions else np.minimum(np.arange(N), n_pos - 1)
        self.table = (self.cos[at].astype(np.float64), self.sin[at].astype(np.float64)) if rot else (None, None)

    def up(self, x, low=False):
        import torch
        if x is None:
            return None
        t = torch.from_numpy(x).cuda()
        return t.to(torch.bfloat16) if low and self.dtype == "bf16" else t

    def args(self):
        import torch
        q, k = (self.up(x, True) for x in self.x)
        if self.fused:
            both = torch.cat([q, k, k], 1)
            q, k = both[:, :self.hq], both[:, self.hq:self.hq + self.hk]
        rot = [self.up(x) if self.rot else None for x in (self.cos, self.sin)]
        return [q, k, *(self.up(w) for w in self.w), *rot, self.up(self.pos)]

    def kw(self):
        return dict(eps=self.eps, interleaved=self.interleaved)

    def forward(self):
        """[(values, sizes)] of q and k"""
        out = []
        for x, w in zip(self.x, self.w):
            w = np.ones(self.d) if w is None else w.astype(np.float64)
            y = qk_norm(x.astype(np.float64), w, *self.table, self.eps, self.interleaved)
            z = np.abs(qk_norm(x.astype(np.float64), w, None, None, self.eps, False))
            out.append((y, self.turned(z)))
        return out

    def turned(self, z):
        """sizes of z's pairs behind a rotation"""
        if not self.rot:
            return z
        c, s = (np.abs(t)[:, None] for t in self.table)
        return np.maximum(rotate(z, c, s, self.interleaved), rotate(z, c, -s, self.interleaved))

    def backward(self):
        """[(dx, its size, dw, its size)] of q and k"""
        out = []
        for x, dy, w in zip(self.x, self.dy, self.w):
            w = np.ones(self.d) if w is None else w.astype(np.float64)
            x, dy = x.astype(np.float64), dy.astype(np.float64)
            dx, dw = qk_norm_backward(dy, x, w, *self.table, self.eps, self.interleaved)
            g = self.turned(np.abs(dy))
            r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + self.eps)
            xh = np.abs(x * r)
            gw = g * np.abs(w)
            out.append((dx, r * gw + r * xh * (gw * xh).mean(-1, keepdims=True), dw, (g * xh).sum((0, 1))))
        return out


def near(got, ref, lim, dtype):
    got = got.float().cpu().numpy()
    lim = lim + (2.0**-8 * np.abs(ref) if dtype == "bf16" else 0)
    bad = np.abs(got - ref) > lim
    assert got.shape == ref.shape and not bad.any(), (int(bad.sum()), float(np.abs(got - ref).max(initial=0)))


def check(c, **kw):
    import torch
    print(f"case N={c.N} hq={c.hq} hk={c.hk} d={c.d} rot={c.rot} {c.dtype} interleaved={c.interleaved}", flush=True)
    a = c.args()
    outs = gdn.qk_norm_fwd(*a, **c.kw(), **kw)
    grads = gdn.qk_norm_backward(*(c.up(x, True) for x in c.dy), *a, **c.kw())
    torch.cuda.synchronize()
    for y, (ref, size) in zip(outs, c.forward()):
        near(y, ref, (c.d / 2 + 8) * U * size, c.dtype)
    for i, (dx, size, dw, dwsize) in enumerate(c.backward()):
        near(grads[i], dx, (2 * c.d + 16) * U * size, c.dtype)
        near(grads[2 + i], dw, (c.N * (c.hq, c.hk)[i] + c.d + 16) * U * dwsize, "f32")
    return outs, grads


CASES = [
    Case(1, 1, 1, 128, 128), Case(1, 16, 4, 128, 64, interleaved=True), Case(7, 5, 3, 64, 32), Case(33, 3, 9, 96, 96),
    Case(300, 8, 2, 128, 128, n_pos=1000), Case(17, 4, 4, 16, 16), Case(17, 4, 4, 16, 0), Case(40, 2, 6, 32, 16, interleaved=True),
    Case(65, 6, 1, 48, 32), Case(29, 7, 2, 112, 112, interleaved=True), Case(12, 3, 3, 256, 128), Case(9, 2, 2, 240, 240),
    Case(5, 3, 1, 128, 128, dtype="f32"), Case(130, 9, 5, 64, 48, dtype="f32", interleaved=True), Case(77, 4, 4, 80, 16, dtype="f32"),
    Case(21, 1, 2, 256, 256, dtype="f32"), Case(50, 16, 16, 16, 16, dtype="f32", interleaved=True),
    Case(60, 4, 2, 64, 64, fused=True), Case(60, 4, 2, 128, 32, dtype="f32", fused=True, weights=False),
    Case(70, 2, 2, 64, 64, positions=False, n_pos=50), Case(8, 2, 0, 64, 64), Case(8, 0, 2, 64, 64),
    Case(5000, 4, 3, 64, 64), Case(2000, 16, 16, 128, 128, dtype="f32"),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_forward_and_backward(i):
    check(CASES[i])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("N,hq,hk,d", [(9000, 16, 16, 128), (4001, 31, 5, 48)])
def test_gradients_of_more_rows_than_workgroups_hold(N, hq, hk, d, interleaved, dtype):
    """Workgroups that take several rounds, the last of them in part.  A weight's
    gradient is a chain of a lane's rows, of a workgroup's groups of lanes and, in 64
    chains joined by a tree, of the workgroups: each addition off by u of sums that
    are at most the sum of sizes, each term by (d / 2 + 8) u of itself.  One
    workgroup adds some twenty times that."""
    import torch
    c = Case(N, hq, hk, d, 32, dtype=dtype, interleaved=interleaved, n_pos=1000, seed=17)
    got = gdn.qk_norm_backward(*(c.up(x, True) for x in c.dy), *c.args(), **c.kw())
    torch.cuda.synchronize()
    per = 256 // (1 << (d // 8 - 1).bit_length())  # groups of four heads that a workgroup takes a round
    for i, (dx, size, dw, dwsize) in enumerate(c.backward()):
        h = (hq, hk)[i]
        units = N * -(-h // 4)
        blocks = min(-(-units // per), 1024 * h // (hq + hk))
        rounds = -(-units // (per * blocks))
        assert rounds > 1 and units % (per * blocks) != 0
        near(got[i], dx, (2 * d + 16) * U * size, dtype)
        near(got[2 + i], dw, (4 * rounds + per + -(-blocks // 64) + 6 + d / 2 + 8) * U * dwsize, "f32")


def test_in_place_and_into_slices():
    import torch
    for dtype in ("bf16", "f32"):
        c = Case(90, 4, 2, 64, 32, dtype=dtype, fused=True, seed=3)
        a = c.args()
        want = [x.clone() for x in gdn.qk_norm_fwd(*a, **c.kw())]
        rest = a[0]._base[:, 6:].clone()
        got = gdn.qk_norm_fwd(*a, **c.kw(), q_out=a[0], k_out=a[1])
        torch.cuda.synchronize()
        assert got[0] is a[0] and torch.equal(a[0], want[0]) and torch.equal(a[1], want[1])
        assert torch.equal(a[0]._base[:, 6:], rest)  # the rest of the projection


def test_into_other_slices_of_the_same_projection():
    """Results between the inputs' rows are no memory of theirs; swapped or shifted
    by a token they are, and refused."""
    import torch
    c = Case(90, 4, 2, 64, 32, seed=16)
    a = c.args()
    want = gdn.qk_norm_fwd(*a, **c.kw())
    wide = torch.full((91, 14, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    wide[:90, :4], wide[:90, 7:9] = a[0], a[1]
    q, k, yk, yq = wide[:90, :4], wide[:90, 7:9], wide[:90, 4:6], wide[:90, 9:13]
    gdn.qk_norm_fwd(q, k, *a[2:], **c.kw(), q_out=yq, k_out=yk)
    torch.cuda.synchronize()
    assert torch.equal(yq, want[0]) and torch.equal(yk, want[1]) and torch.equal(q, a[0]) and torch.equal(k, a[1])
    assert (wide[:, 6] == 3).all() and (wide[:, 13] == 3).all() and (wide[90] == 3).all()
    for out in (dict(q_out=wide[1:, :4]), dict(q_out=wide[:90, 6:10]), dict(k_out=wide[:90, 3:5]), dict(q_out=yq, k_out=wide[:90, 12:])):
        with pytest.raises(gdn.GdnError):
            gdn.qk_norm_fwd(q, k, *a[2:], **c.kw(), **out)


def test_gradients_into_their_own_buffers():
    """grad_q, grad_k over the incoming gradients (raw entry point)."""
    import ctypes

    import torch
    c = Case(90, 4, 2, 64, 32, seed=4)
    a, dy = c.args(), [c.up(x, True) for x in c.dy]
    want = gdn.qk_norm_backward(*dy, *a, **c.kw())
    ws = torch.empty(gdn.gdn_qk_norm_workspace_bytes(90, 4, 2, 64), dtype=torch.uint8, device="cuda")
    dw = [torch.empty(64, device="cuda") for _ in range(2)]
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    rc = gdn.lib().gdn_qk_norm_backward(90, 4, 2, 64, 32, 50, 1, 0, 1e-6, p(dy[0]), 256, p(dy[1]), 128, p(a[0]), 256, p(a[1]), 128,
                                        *map(p, a[2:]), p(dy[0]), p(dy[1]), *map(p, dw), p(ws), ws.numel(),
                                        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert rc == 0
    for x, y in zip((*dy, *dw), want):
        assert torch.equal(x, y)


def test_positions_outside_the_table_are_clamped():
    import torch
    c = Case(6, 2, 1, 64, 64, n_pos=10, seed=5)
    a = c.args()
    a[6] = torch.tensor([-1, -2**31, 0, 9, 10, 2**31 - 1], dtype=torch.int32, device="cuda")
    got = gdn.qk_norm_fwd(*a, **c.kw())
    a[6] = torch.tensor([0, 0, 0, 9, 9, 9], dtype=torch.int32, device="cuda")
    want = gdn.qk_norm_fwd(*a, **c.kw())
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_parts_of_the_gradients():
    import torch
    c = Case(300, 4, 2, 64, 32, seed=6)
    a, dy = c.args(), [c.up(x, True) for x in c.dy]
    want = gdn.qk_norm_backward(*dy, *a, **c.kw())
    x = gdn.qk_norm_backward(*dy, *a, **c.kw(), want_weights=False)
    w = gdn.qk_norm_backward(*dy, *a, **c.kw(), want_x=False)
    torch.cuda.synchronize()
    assert x[2] is x[3] is w[0] is w[1] is None
    for i in range(2):
        assert torch.equal(x[i], want[i]) and torch.equal(w[2 + i], want[2 + i])


def test_bad_and_constant_rows_stay_rows():
    import torch
    c = Case(9, 3, 2, 64, 32, seed=7)
    a, dy = c.args(), [c.up(x, True) for x in c.dy]
    first = gdn.qk_norm_fwd(*a, **c.kw()) + gdn.qk_norm_backward(*dy, *a, **c.kw())
    a[0][4, 1, 5], a[0][5, 0, 40], a[0][6, 2] = float("nan"), float("inf"), 0.0
    again = gdn.qk_norm_fwd(*a, **c.kw()) + gdn.qk_norm_backward(*dy, *a, **c.kw())
    torch.cuda.synchronize()
    keep = torch.ones(9, 3, dtype=torch.bool, device="cuda")
    keep[4, 1] = keep[5, 0] = keep[6, 2] = False
    for i in (0, 2):
        assert torch.equal(first[i][keep], again[i][keep])
        assert torch.isfinite(again[i][6, 2]).all()
    assert (again[0][6, 2] == 0).all() and torch.isnan(again[0][4, 1]).all() and torch.isnan(again[2][4, 1]).all()
    assert torch.equal(first[1], again[1]) and torch.equal(first[3], again[3]) and torch.equal(first[5], again[5])


def test_against_differences():
    import torch
    c = Case(20, 3, 2, 64, 48, dtype="f32", seed=8)
    a, dy = c.args(), [c.up(x, True).double() for x in c.dy]
    got = gdn.qk_norm_backward(*(g.float() for g in dy), *a, **c.kw())
    loss = lambda a: sum(float((y.double() * g).sum()) for y, g in zip(gdn.qk_norm_fwd(*a, **c.kw()), dy))  # noqa: E731
    r = torch.Generator(device="cuda").manual_seed(9)
    for i, g in enumerate(got):
        e = torch.randn(a[i].shape, generator=r, device="cuda")
        if i < 2:
            e = e * a[i].square().mean(-1, keepdim=True).sqrt()  # steps of the rows' own sizes
        up, down = ([x if j != i else x + s * 2.0**-8 * e for j, x in enumerate(a)] for s in (1, -1))
        want = (loss(up) - loss(down)) * 2.0**7
        have, size = float((g.double() * e).sum()), float((g.double() * e).square().sum().sqrt())
        # third derivatives of a row times 2^-16, and 1e4 fp32 roundings
        assert abs(want - have) <= 1e-3 * (abs(have) + 10 * size), (i, want, have, size)


def test_repeats_are_identical_and_graphs_replay():
    import torch
    c = Case(3000, 8, 4, 128, 64, seed=10)
    a, dy = c.args(), [c.up(x, True) for x in c.dy]
    call = lambda: gdn.qk_norm_fwd(*a, **c.kw()) + gdn.qk_norm_backward(*dy, *a, **c.kw())  # noqa: E731
    first = [x.clone() for x in call()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call()
    for i in range(3):
        for x in got:
            x.fill_(3.0)
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, first):
            assert torch.equal(x, y)
        for x, y in zip(call(), first):
            assert torch.equal(x, y)


def test_large_offsets():
    """Rows past 2^31 elements."""
    import torch
    N, h, d = 2**31 // (2 * 2048) + 3, 2, 64  # tokens 4096 elements apart: a slice of a wide projection
    wide = torch.zeros((N, 64, d), dtype=torch.bfloat16, device="cuda")
    c = Case(3, h, h, d, d, n_pos=N, seed=11, positions=False)
    c.pos = np.array([N - 3, N - 2, N - 1], np.int32)
    c.table = (c.cos[c.pos].astype(np.float64), c.sin[c.pos].astype(np.float64))
    a = c.args()
    wide[-3:, 60:62], wide[-3:, 62:] = a[0], a[1]
    q, k = wide[:, 60:62], wide[:, 62:]
    out = gdn.qk_norm_fwd(q, k, *a[2:6], None, **c.kw(), q_out=q, k_out=k)
    torch.cuda.synchronize()
    for y, (ref, size) in zip(out, c.forward()):
        near(y[-3:], ref, (d / 2 + 8) * U * size, "bf16")


def test_timer_names_the_kernels():
    import torch
    c = Case(30, 2, 2, 64, 64, seed=12)
    a, tm = c.args(), gdn.Timer()
    gdn.qk_norm_fwd(*a, **c.kw(), timer=tm)
    gdn.qk_norm_backward(*(c.up(x, True) for x in c.dy), *a, **c.kw(), timer=tm)
    torch.cuda.synchronize()
    assert set(tm.read()) == {"k_qk_norm", "k_qk_norm_bwd", "k_qk_norm_params"}


def test_binding_refuses():
    import torch
    c = Case(9, 2, 2, 64, 64, seed=13)
    a = c.args()

    def bad(i, x, err):
        with pytest.raises(err):
            gdn.qk_norm_fwd(*a[:i], x, *a[i + 1:])
    bad(0, a[0].float(), TypeError)
    bad(0, a[0][:8], ValueError)
    bad(1, a[1][:, :, ::2], ValueError)
    bad(1, a[1].cpu(), ValueError)
    bad(2, a[2][:32], ValueError)
    bad(2, a[2].double(), TypeError)
    bad(4, None, ValueError)
    bad(4, a[4][:, :16], ValueError)
    bad(5, a[5].cpu(), ValueError)
    bad(6, a[6][:3], ValueError)
    bad(6, a[6].long(), TypeError)
    with pytest.raises(gdn.GdnError):
        gdn.qk_norm_fwd(*a[:4], a[4][:, :12].contiguous(), a[5][:, :12].contiguous(), a[6])
    with pytest.raises(ValueError):
        gdn.qk_norm_fwd(*a, q_out=a[0][:5])
    with pytest.raises(ValueError):
        gdn.qk_norm_backward(a[0].float(), a[1], *a)


def test_a_block_in_prompts_steps_and_training():
    """Projection, norm and rotation, linear attention: a prompt, then single
    tokens from the states it left, against both references in a row; and the
    gradients of the whole chain against theirs, by the sums of sizes."""
    import torch
    n, h, d, eps = 400, 2, 64, 1e-6
    N = n + 40
    c = Case(N, h, h, d, 32, n_pos=500, seed=14, dtype="f32")
    c.pos = np.arange(7, 7 + N, dtype=np.int32)
    c.table = (c.cos[c.pos].astype(np.float64), c.sin[c.pos].astype(np.float64))
    a = c.args()
    (qn, _), (kn, _) = c.forward()
    lin = Linear((N,), h, h, d, d, dtype="f32", scale=d**-0.5, fresh=(0,), seed=15).make()
    lin.a["q"], lin.a["k"] = qn, kn
    ref, ends = lin.forward()
    v, alpha = lin.cuda("v"), lin.cuda("alpha")
    pool = torch.full((3, h, d, d), 5.0, device="cuda")
    slot, none = (torch.tensor([x], dtype=torch.int32, device="cuda") for x in (1, -1))
    got = []
    for lo, hi in [(0, n)] + [(t, t + 1) for t in range(n, N)]:
        q, k = gdn.qk_norm_fwd(a[0][lo:hi], a[1][lo:hi], *a[2:6], a[6][lo:hi], eps=eps)
        cu = torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda")
        got.append(gdn.linear_fwd(q, k, v[lo:hi], alpha, cu, pool, none if lo == 0 else slot, pool, slot, max_len=hi - lo,
                                  scale=lin.scale)[0])
    torch.cuda.synchronize()
    # fp32 throughout: q and k each off by (d / 2 + 8) u of themselves, then as linear attention's
    size, esize = lin.forward(size=True)
    tol = (2 * (d / 2 + 8) + N + 4 * d) * U + 2.0**-16
    assert (np.abs(torch.cat(got).cpu().numpy() - ref) <= 2 * tol * size).all()
    assert (np.abs(pool[1].cpu().numpy() - ends[0]) <= 2 * tol * esize[0]).all()
    assert (pool[0] == 5).all() and (pool[2] == 5).all()

    q, k = gdn.qk_norm_fwd(*a, eps=eps)
    cu = torch.tensor([0, N], dtype=torch.int32, device="cuda")
    g = gdn.linear_backward(q, k, v, alpha, cu, None, None, lin.cuda("dout"), scale=lin.scale)
    dq, dk, dwq, dwk = gdn.qk_norm_backward(g[0], g[1], *a, eps=eps)
    torch.cuda.synchronize()
    lin.a["dstate"][:] = 0
    r, rs = lin.backward(), lin.backward(size=True)
    for i, (got_x, got_w) in enumerate(((dq, dwq), (dk, dwk))):
        c.dy = [r[0], r[1]]
        dx, _, dw, _ = c.backward()[i]
        c.dy = [rs[0], rs[1]]
        _, sx, _, sw = c.backward()[i]
        assert (np.abs(got_x.cpu().numpy() - dx) <= 4 * tol * sx).all()
        assert (np.abs(got_w.cpu().numpy() - dw) <= 4 * (tol + N * h * U) * sw).all()
