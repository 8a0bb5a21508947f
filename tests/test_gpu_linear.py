"""gdn_linear_fwd and gdn_linear_backward against 64-bit token loops.

Tolerances, derived before the first run, in the size of a result: the same sum
with every term by its absolute value.  Each factor of a term carries at most one
split into two bf16 terms (2^-17 of the factor; bf16 only) and one power of the
decay (an exponent x log2 a rounded to 2^-24 of itself: at most 126 2^-24 < 2^-17
relative to a power that is not zero), scores are sums of dk (dv) products, and
a result a sum of as many terms as the sequence has tokens, and dk (dv) of its
state, each addition off by 2^-24:
    |error| <= (2 2^-17 + (n + 2 dk + 2 dv) 2^-24) size,
with 2^-8 |value| more where it is rounded to bf16.  That is the worst case;
roundings in no common direction add up by the square root of their number, 256
of 2^-25 in a segment and one a segment behind it, so the root mean square of
states' and fp32 results' errors is held to 2^-20 of that of the values.
"""
from __future__ import annotations

import numpy as np
import pytest

from gated_delta_rule_12_amd import gdn
from linear_case import Linear

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn.lib()


def rms(x):
    return float(np.sqrt(np.mean(np.square(x)))) if x.size else 0.0


def near(c, got, ref, size, dtype):
    lim = (2.0**-16 + (max(c.lengths) + 2 * c.dk + 2 * c.dv) * 2.0**-24) * size
    if dtype == "bf16":
        lim = lim + 2.0**-8 * np.abs(ref)
    err = np.abs(got - ref)
    worst = float((err / np.maximum(lim, 1e-300))[err > 0].max(initial=0.0))
    assert (err <= lim).all(), (int((err > lim).sum()), worst, float(np.abs(ref).max()))
    if dtype == "f32":
        assert rms(err) <= 2.0**-20 * rms(ref), (rms(err), rms(ref))


NAMES = ("q", "k", "v", "alpha", "cu", "pool", "slots_in", "slots_out")


def run(c, max_len=None, inplace=False, tensors=None, **kw):
    import torch
    t = {n: c.cuda(n) for n in NAMES}
    t.update(tensors or {})
    pool_out = t["pool"] if inplace else torch.full_like(t["pool"], 7.0)
    out = torch.full((c.a["q"].shape[0], c.hv, c.dv), 7.0, dtype=t["q"].dtype, device="cuda")
    print(f"case {c.lengths[:12]} hk={c.hk} hv={c.hv} dk={c.dk} dv={c.dv} {c.dtype}", flush=True)
    gdn.linear_fwd(t["q"], t["k"], t["v"], t["alpha"], t["cu"], t["pool"], t["slots_in"], pool_out,
                   t["slots_in"] if inplace else t["slots_out"], max_len=max_len, scale=c.scale, out=out, **kw)
    torch.cuda.synchronize()
    return out.float().cpu().numpy(), pool_out.cpu().numpy()


def check(c, out, pool, inplace=False):
    (ref, ends), (size, esize) = c.forward(), c.forward(size=True)
    n = sum(c.lengths)
    near(c, out[:n], ref[:n], size[:n], c.dtype)
    assert (out[n:] == 7.0).all()  # rows behind the last sequence
    slots = c.a["slots_in"] if inplace else c.a["slots_out"]
    used = slots >= 0
    near(c, pool[slots[used]], ends[used], esize[used], "f32")
    rest = np.setdiff1d(np.arange(len(pool)), slots)
    assert (pool[rest] == (c.a["pool"][rest] if inplace else 7.0)).all()  # slots nobody wrote


CASES = [
    # token by token: single tokens, drafted tokens, every row layout
    Linear((1,), 1, 1, 128, 128),
    Linear((1, 3, 2, 5, 16, 31), 1, 4, 64, 64, slots=2, tail=3),
    Linear((2, 0, 7, 1), 2, 2, 32, 128, dtype="f32", slots=1, fresh=(2,)),
    Linear((30, 1, 9), 1, 3, 96, 48, slots=2),
    Linear((4, 12), 2, 2, 16, 16, dtype="f32"),
    # one segment: borders of blocks of 16, 32, 64 and 128 rows, beside short and empty ones
    Linear((32, 33, 63), 1, 1, 64, 64),
    Linear((64, 65, 127), 1, 2, 128, 128, slots=1),
    Linear((0, 128, 1, 0, 129, 31, 0), 2, 4, 128, 128, slots=2, tail=5, fresh=(1,)),
    Linear((200, 255, 256), 1, 3, 64, 128, scale=0.3),
    Linear((40, 100), 2, 2, 128, 64, dtype="f32", slots=1),
    Linear((77, 191), 1, 2, 64, 64, dtype="f32"),
    # several segments, other sizes than whole tiles
    Linear((257, 512, 5, 700), 1, 2, 128, 128, slots=1),
    Linear((1100, 30, 513), 2, 4, 48, 96, slots=1, fresh=(0,)),
    Linear((300, 1000), 1, 2, 80, 112, dtype="f32", scale=-2.0),
    Linear((385, 641), 2, 2, 16, 128),
    Linear((385, 641), 1, 2, 112, 32, dtype="f32"),
    # decays: none, strong, almost none, all at once, next to one
    Linear((300, 40), 1, 4, 64, 64, alpha=(1.0, 0.0, 1e-3, 1e-30), slots=1),
    Linear((300, 40), 2, 4, 64, 64, dtype="f32", alpha=(1.0, 0.0, 0.05, 1 - 2.0**-24)),
    Linear((20, 3), 2, 4, 64, 64, alpha=(1.0, 0.0, 1e-3, 0.5)),
    # a long chain of segments
    Linear((5000, 1, 2600), 1, 1, 64, 64, alpha=(1 - 2.0**-12,)),
    # chains beside short sequences, 8 and 16 segments in flight
    Linear((1300, 2600) + (1,) * 15, 1, 1, 128, 128, alpha=(1 - 2.0**-9,)),
    Linear((8500,) + (2,) * 16, 1, 1, 128, 128, alpha=(1 - 2.0**-11,)),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_forward(i):
    c = CASES[i]
    c.seed = 100 + i
    c.make()
    check(c, *run(c))


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("i,lengths,hk,hv,dk,dv", [(0, (300, 33, 513, 2), 1, 2, 128, 64), (1, (257, 40), 2, 4, 112, 48),
                                                   (2, (31, 32, 256, 1000), 1, 3, 80, 16)])
def test_keys_wider_than_values(i, lengths, hk, hv, dk, dv, inplace):
    c = Linear(lengths, hk, hv, dk, dv, slots=1, seed=50 + i).make()
    check(c, *run(c, inplace=inplace), inplace=inplace)


@pytest.mark.parametrize("lengths,dk,dv", [((1, 1, 1), 128, 128), ((3, 90, 1200, 256), 128, 128), ((5, 600, 33), 48, 96)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place(lengths, dk, dv, dtype):
    c = Linear(lengths, 2, 4, dk, dv, dtype=dtype, slots=2, fresh=(1,), seed=7).make()
    c.a["slots_in"][1] = np.setdiff1d(np.arange(len(lengths) + 2), c.a["slots_in"])[0]
    out, pool = run(c, inplace=True)
    check(c, out, pool, inplace=True)


def test_overlapping_pools():
    """In place through two views of one pool whose slots are named differently."""
    import torch
    c = Linear((300, 70, 5), 1, 2, 64, 64, seed=6).make()
    both = torch.full((6, 2, 64, 64), 7.0, device="cuda")
    both[1:4] = c.cuda("pool")
    c.a["slots_in"] = c.a["slots_out"] = np.array([0, 1, 2], np.int32)
    here = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    out, end = gdn.linear_fwd(*(c.cuda(n) for n in ("q", "k", "v", "alpha", "cu")), both[1:], None, both[:5], here)
    torch.cuda.synchronize()
    assert (both[0] == 7.0).all() and (both[4:] == 7.0).all()
    check(c, out.float().cpu().numpy(), both[1:4].cpu().numpy())


@pytest.mark.parametrize("max_len", [0, 1, 31, 32, 200, 100000])
def test_any_max_len_gives_the_same_results(max_len):
    c = Linear((1, 700, 65, 33), 2, 4, 64, 64, seed=8).make()
    check(c, *run(c, max_len=max_len))


def test_without_states():
    import torch
    c = Linear((40, 300, 2), 1, 2, 64, 64, fresh=(0, 1, 2), seed=9).make()
    out, end = gdn.linear_fwd(*(c.cuda(n) for n in ("q", "k", "v", "alpha", "cu")))
    c.a["slots_out"] = np.arange(3, dtype=np.int32)
    check(c, out.float().cpu().numpy(), end.cpu().numpy())
    # end states not wanted: the slots are all outside
    none = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    pool = torch.full_like(end, 7.0)
    again, _ = gdn.linear_fwd(*(c.cuda(n) for n in ("q", "k", "v", "alpha", "cu")), None, None, pool, none)
    torch.cuda.synchronize()
    assert torch.equal(out, again) and (pool == 7.0).all()


@pytest.mark.parametrize("lengths", [(3, 1, 2), (90, 700, 2, 256)])
def test_end_states_not_wanted(lengths):
    """state_out NULL, which the entry point takes and the binding does not pass on."""
    import ctypes

    import torch
    c = Linear(lengths, 1, 2, 64, 64, seed=52, slots=1).make()
    t = {n: c.cuda(n) for n in NAMES}
    want, _ = run(c)
    N, S = sum(lengths), len(lengths)
    out = torch.full((N, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    n = gdn.gdn_linear_workspace_bytes(N, S, 1, 2, 64, 64, max(lengths), 1)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    p = lambda x: ctypes.c_void_p(x.data_ptr())  # noqa: E731
    rc = gdn.lib().gdn_linear_fwd(N, S, 1, 2, 64, 64, S + 1, 0, max(lengths), 1, 1.0, p(t["q"]), 64, p(t["k"]), 64, p(t["v"]), 128,
                                  p(t["alpha"]), p(t["cu"]), p(t["pool"]), p(t["slots_in"]), None, None, p(out), p(ws), n,
                                  ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert rc == 0 and np.array_equal(out.float().cpu().numpy(), want)


def test_slices_of_one_projection():
    import torch
    c = Linear((90, 300, 3), 2, 4, 64, 64, seed=10).make()
    both = torch.cat([c.cuda("q"), c.cuda("k"), c.cuda("v")], 1)
    t = {"q": both[:, :2], "k": both[:, 2:4], "v": both[:, 4:]}
    check(c, *run(c, tensors=t))


def test_two_sequences_start_from_one_slot():
    c = Linear((90, 5, 300), 1, 2, 64, 64, seed=11, slots=1).make()
    c.a["slots_in"][:] = 2
    check(c, *run(c))


def test_prompt_then_steps_equal_one_prompt():
    """A prompt, then drafted and single tokens from the pool: the whole sequence
    at once, up to rounding."""
    import torch
    c = Linear((600, 450), 1, 2, 128, 128, seed=15, slots=2).make()
    t = {n: c.cuda(n) for n in ("q", "k", "v", "alpha", "pool", "slots_in")}
    pool = t["pool"].clone()
    got = torch.empty((1050, 2, 128), dtype=torch.bfloat16, device="cuda")
    at = [0, 600]
    for take in ((500, 380), (5, 1), (1, 1), (70, 64), (23, 3), (1, 1)):
        idx = torch.cat([torch.arange(a, a + n) for a, n in zip(at, take)]).cuda()
        cu = torch.tensor([0, take[0], sum(take)], dtype=torch.int32).cuda()
        got[idx], _ = gdn.linear_fwd(*(t[n][idx] for n in ("q", "k", "v")), t["alpha"], cu, pool, t["slots_in"], pool,
                                     t["slots_in"], max_len=max(take))
        at = [a + n for a, n in zip(at, take)]
    assert at == [600, 1050]
    torch.cuda.synchronize()
    (ref, ends), (size, esize) = c.forward(), c.forward(size=True)
    near(c, got.float().cpu().numpy(), ref, size, "bf16")
    near(c, pool.cpu().numpy()[c.a["slots_in"]], ends, esize, "f32")


def guarded(n, dtype, fill, rim=4096):
    """n elements within a filled buffer, and a check that nothing around them changed."""
    import torch
    whole = torch.full((n + 2 * rim,), fill, dtype=dtype, device="cuda")
    return whole[rim:rim + n], lambda: bool((whole[:rim] == fill).all() and (whole[-rim:] == fill).all())


@pytest.mark.parametrize("lengths,dk,dv,hv,dtype", [
    ((1,) * 90 + (33,), 64, 64, 2, "bf16"),
    ((1,) * 60 + (700,) + (2, 0, 31) * 30 + (32, 1300), 128, 128, 4, "bf16"),
    ((40, 33, 64, 31) * 12 + (1,) * 150 + (900, 257, 129), 48, 64, 4, "f32"),
])
def test_exact_workspace(lengths, dk, dv, hv, dtype):
    """Within a workspace of the size that is asked for, whatever it held before."""
    import torch
    c = Linear(lengths, 1, hv, dk, dv, dtype=dtype, seed=43, slots=1).make()
    n = gdn.gdn_linear_workspace_bytes(sum(lengths), len(lengths), 1, hv, dk, dv, sum(lengths), int(dtype == "bf16"))
    for fill in (0xA5, 0xFF):
        ws, untouched = guarded(n, torch.uint8, fill)
        check(c, *run(c, workspace=ws))
        assert untouched()


def test_many_ranks():
    """More sequences in segments than the plan's search holds in LDS."""
    lengths = (33, 1) * 2100 + (300,)
    c = Linear(lengths, 1, 1, 16, 16, seed=12).make()
    check(c, *run(c))


@pytest.mark.parametrize("S", [3, 40])
def test_bad_offsets_and_slots_write_nothing_else(S):
    """Offsets and slots of any value: nothing outside the outputs, the pool and
    the workspace, and no slot that the call does not name; forward and backward."""
    import torch
    N, hv, d = 3000, 2, 64
    r = np.random.Generator(np.random.PCG64(44))
    c = Linear((N,), 1, hv, d, d, seed=44).make()
    t = {n: c.cuda(n) for n in ("q", "k", "v", "alpha", "pool", "dout")}
    state = hv * d * d
    for cu in ([0, N] * S, [N, 0] * S, [0] * (2 * S) + [2**31 - 1], [-2**31] + [2**31 - 1] * (2 * S),
               list(r.integers(-10, N + 10, 2 * S))):
        cu = cu[:S + 1]
        slots = r.choice([-1, -2**31, 2**31 - 1, S + 2, 5], S)
        slots[0] = 1
        pool, pool_whole = guarded((S + 2) * state, torch.float32, 7.0)
        out, out_whole = guarded(N * hv * d, torch.bfloat16, 7.0)
        ws, ws_whole = guarded(gdn.gdn_linear_workspace_bytes(N, S, 1, hv, d, d, N, 1), torch.uint8, 0xA5)
        print("offsets", cu[:6], "slots", slots[:6], flush=True)
        cu, slots = (torch.tensor(np.array(x), dtype=torch.int32).cuda() for x in (cu, slots))
        gdn.linear_fwd(t["q"], t["k"], t["v"], t["alpha"], cu, t["pool"], slots, pool.view(S + 2, hv, d, d), slots,
                       out=out.view(N, hv, d), workspace=ws)
        torch.cuda.synchronize()
        assert pool_whole() and out_whole() and ws_whole()
        rest = [s for s in range(S + 2) if s not in (1, 5)]
        assert (pool.view(S + 2, -1)[rest] == 7.0).all()
        ws, ws_whole = guarded(gdn.gdn_linear_backward_workspace_bytes(N, S, 1, hv, d, d, 1), torch.uint8, 0xA5)
        gdn.linear_backward(t["q"], t["k"], t["v"], t["alpha"], cu, t["pool"], slots, t["dout"], workspace=ws)
        torch.cuda.synchronize()
        assert ws_whole()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_non_finite_rows_outside_the_sequences(dtype):
    """Rows in front of the first and behind the last sequence are not read."""
    import torch
    c = Linear((70, 1, 500, 33), 1, 2, 64, 64, dtype=dtype, seed=45, tail=70).make()
    t = {n: c.cuda(n) for n in ("q", "k", "v", "alpha", "cu", "pool", "slots_in", "dout", "dstate")}
    call = lambda: (gdn.linear_fwd(t["q"], t["k"], t["v"], t["alpha"], t["cu"][1:], t["pool"], t["slots_in"][1:]) +  # noqa: E731
                    gdn.linear_backward(t["q"], t["k"], t["v"], t["alpha"], t["cu"][1:], t["pool"], t["slots_in"][1:],
                                        t["dout"], t["dstate"][1:]))
    first = call()
    for n in ("q", "k", "v", "dout"):
        t[n][:70], t[n][604:] = np.nan, np.inf
    again = call()
    torch.cuda.synchronize()
    for i, (x, y) in enumerate(zip(first, again)):
        rows = slice(70, 604) if i in (0, 2, 3, 4) else slice(None)
        assert torch.equal(x[rows], y[rows])
        if i in (2, 3, 4):
            assert (y[:70] == 0).all() and (y[604:] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [np.inf, np.nan])
@pytest.mark.parametrize("what", ["v", "q", "k", "pool"])
def test_non_finite_inputs_propagate(what, value, dtype):
    """One infinity or NaN: what the formula makes non-finite is so, and every
    other value is right; beyond the formula one in v reaches, within its feature,
    at most the 31 tokens in front of its own."""
    c = Linear((40, 700, 33), 1, 2, 64, 64, dtype=dtype, seed=41).make()
    t = 40 + 300
    free = np.zeros((773, 2, 64), bool)
    if what == "v":
        c.a["v"][t, 1, 5] = value
        free[t - 31:t, 1, 5] = True
    elif what == "pool":
        c.a["pool"][c.a["slots_in"][1], 1, 5, 7] = value
    else:
        c.a[what][t, 0, 5] = value
    out, pool = run(c)
    with np.errstate(invalid="ignore"):
        (ref, ends), (size, esize) = c.forward(), c.forward(size=True)
    bad = ~np.isfinite(ref)
    assert bad.any() and not np.isfinite(out[bad]).any()
    assert np.isfinite(out[~bad & ~free]).all()
    ok = ~bad & np.isfinite(out)
    near(c, out[ok], ref[ok], size[ok], dtype)
    got = pool[c.a["slots_out"]]
    bad = ~np.isfinite(ends)
    assert not np.isfinite(got[bad]).any() and np.isfinite(got[~bad]).all()
    near(c, got[~bad], ends[~bad], esize[~bad], "f32")


@pytest.mark.parametrize("value", [np.inf, np.nan])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,da", [((64, 64), True), ((128, 128), False), ((80, 48), False), ((64, 128), False), ((128, 64), True)])
def test_non_finite_states_leave_the_features_beside_theirs(d, da, dtype, value):
    """One infinity or NaN in a start state or in the gradient of an end state, at
    an even and at an odd key feature: dq (dk) is non-finite in that feature alone,
    dv in its value feature, with or without dalpha."""
    for n, i, at in (("pool", 24, 1), ("pool", 25, 1), ("dstate", 24, 2), ("dstate", 25, 2), ("dstate", 12, 0)):
        c = Linear((300, 40, 33), 1, 2, *d, dtype=dtype, seed=48).make()
        c.a[n][c.a["slots_in"][at] if n == "pool" else at, 1, 5, i] = value
        got = grads_of(c, want_grad_alpha=da)
        with np.errstate(invalid="ignore"):
            want, sizes = c.backward(), c.backward(size=True)
        for name, x, ref, size in zip(("dq", "dk", "dv", "dalpha", "dstate0"), got, want, sizes):
            if x is None:
                continue
            fine = np.isfinite(ref)
            wrong = np.argwhere(np.isfinite(x) != fine)
            assert not len(wrong), (n, name, len(wrong), wrong[0], wrong[-1])
            if name != "dalpha":
                near(c, x[fine], ref[fine], size[fine], "f32" if name == "dstate0" else dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [np.inf, np.nan])
@pytest.mark.parametrize("what", ["q", "k", "v", "dout"])
@pytest.mark.parametrize("d,at", [((64, 64), (0, 300)), ((128, 128), (31, 511)), ((64, 128), (143, 440)), ((80, 48), (255, 256)),
                                  ((128, 64), (17, 699))])
def test_non_finite_inputs_reach_no_token_that_does_not_see_them(d, at, what, value, dtype):
    """Infinities or NaN at two tokens of one sequence: outputs, states and gradients
    are non-finite where the formula is, and right everywhere else, in front of
    those tokens (dk, dv: behind them) as well."""
    c = Linear((40, 700, 33), 1, 2, *d, dtype=dtype, seed=46).make()
    for i, t in enumerate(at):
        if what in ("v", "dout"):
            c.a[what][40 + t, 1, 5 + 20 * i] = value
        else:
            c.a[what][40 + t, 0, 5 + 20 * i] = -value
    out, pool = run(c)
    got = [out, pool[c.a["slots_out"]], *grads_of(c)]
    with np.errstate(invalid="ignore"):
        want = [*c.forward(), *c.backward()]
        sizes = [*c.forward(size=True), *c.backward(size=True)]
    for name, x, ref, size in zip(("out", "states", "dq", "dk", "dv", "dalpha", "dstate0"), got, want, sizes):
        fine = np.isfinite(ref)
        wrong = np.argwhere(np.isfinite(x) != fine)
        assert not len(wrong), (name, len(wrong), wrong[0], wrong[-1])
        if name == "dalpha":
            lim = (2.0**-16 + (max(c.lengths) + 2 * c.dk + 2 * c.dv) * 2.0**-24) * size
            assert (np.abs(x - ref) <= lim)[fine].all()
        else:
            near(c, x[fine], ref[fine], size[fine], "f32" if name in ("states", "dstate0") else dtype)


@pytest.mark.parametrize("dk", [16, 48, 80, 112])
def test_infinite_states_of_single_tokens(dk):
    """Token by token an infinity stays what the formula makes of it, in the last
    features of head sizes that are no power of two as well."""
    c = Linear((1, 3), 1, 2, dk, 16, dtype="f32", seed=47).make()
    c.a["pool"][:, :, 3, dk - 1] = np.inf
    out, pool = run(c, max_len=3)
    (ref, ends), (size, _) = c.forward(), c.forward(size=True)
    assert np.isinf(ref[:, :, 3]).all() and np.array_equal(out[:, :, 3], ref[:, :, 3])
    rest = np.arange(16) != 3
    near(c, out[:, :, rest], ref[:, :, rest], size[:, :, rest], "f32")
    assert np.array_equal(np.isinf(pool[c.a["slots_out"]]), np.isinf(ends))


@pytest.mark.parametrize("back", [False, True])
def test_repeats_are_identical_and_graphs_replay(back):
    import torch
    c = Linear((1, 600, 70, 1100), 2, 4, 128, 128, seed=14).make()
    t = {n: c.cuda(n) for n in (*NAMES, "dout", "dstate")}
    args = [t[n] for n in ("q", "k", "v", "alpha", "cu")]
    if back:
        ws = torch.empty(gdn.gdn_linear_backward_workspace_bytes(1771, 4, 2, 4, 128, 128, 1), dtype=torch.uint8, device="cuda")
        call = lambda ws=ws: gdn.linear_backward(*args, t["pool"], t["slots_in"], t["dout"], t["dstate"], workspace=ws)  # noqa: E731
    else:
        ws = gdn.linear_workspace_for(t["q"], t["v"], t["cu"])
        call = lambda ws=ws: gdn.linear_fwd(*args, t["pool"], t["slots_in"], workspace=ws)  # noqa: E731
    first = call()
    torch.cuda.synchronize()
    first = [x.clone() for x in first]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call()
    for i in range(4):
        # other lengths under the same graph, then the first ones again
        cu = torch.tensor([0, 600, 601, 700, 1771], dtype=torch.int32) if i == 1 else torch.from_numpy(c.a["cu"])
        t["cu"].copy_(cu)
        for x in got:
            x.fill_(3.0)
        ws.fill_(255)  # nothing in the workspace is taken over from an earlier call
        g.replay()
        torch.cuda.synchronize()
        want = call(torch.full_like(ws, 0)) if i == 1 else first
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)


def test_other_stream_and_two_calls_at_once():
    import torch
    cs = [Linear((700, 90), 1, 2, 128, 128, seed=16).make(), Linear((64, 1000), 1, 2, 128, 128, seed=17).make()]
    ts = [{n: c.cuda(n) for n in (*NAMES, "dout", "dstate")} for c in cs]

    def call(t):
        args = [t[n] for n in ("q", "k", "v", "alpha", "cu", "pool", "slots_in")]
        return gdn.linear_fwd(*args) + gdn.linear_backward(*args, t["dout"], t["dstate"])
    alone = [call(t) for t in ts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ts]
    for _ in range(4):
        both = []
        for t, s in zip(ts, streams):
            with torch.cuda.stream(s):
                both.append(call(t))
        torch.cuda.synchronize()
        for x, y in zip(alone, both):
            for a, b in zip(x, y):
                assert torch.equal(a, b)


def test_large_offsets():
    """A pool whose last state lies past 2^31 elements, tokens past 2^31 bytes."""
    import torch
    d, hv = 128, 16
    slots = 2**31 // (hv * d * d) + 8
    c = Linear((70, 1), 1, hv, d, d, seed=18).make()
    t = {n: c.cuda(n) for n in ("q", "k", "v", "alpha", "cu")}
    pool = torch.empty((slots, hv, d, d), device="cuda")
    at = torch.tensor([slots - 1, slots - 2], dtype=torch.int32).cuda()
    pool[slots - 1], pool[slots - 2] = c.cuda("pool")[0], c.cuda("pool")[1]
    c.a["slots_in"] = np.array([0, 1], np.int32)
    N = 2**30 // (hv * d) + 200
    v = torch.zeros((N, hv, d), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((N, 1, d), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros_like(q)
    q[-71:], k[-71:], v[-71:] = t["q"], t["k"], t["v"]
    cu = (t["cu"] + (N - 71)).to(torch.int32)
    out, _ = gdn.linear_fwd(q, k, v, t["alpha"], cu, pool, at, pool, at, max_len=70)
    torch.cuda.synchronize()
    (ref, ends), (size, esize) = c.forward(), c.forward(size=True)
    near(c, out[-71:].float().cpu().numpy(), ref, size, "bf16")
    near(c, pool[[slots - 1, slots - 2]].cpu().numpy(), ends, esize, "f32")


def test_timer_names_the_kernels():
    import torch
    c = Linear((600, 3), 1, 2, 128, 128, seed=19).make()
    tm = gdn.Timer()
    args = [c.cuda(n) for n in ("q", "k", "v", "alpha", "cu", "pool")]
    gdn.linear_fwd(*args, timer=tm)
    gdn.linear_backward(*args, None, c.cuda("dout"), timer=tm)
    torch.cuda.synchronize()
    assert set(tm.read()) == {"k_lin_plan", "k_lin_add", "k_lin_scan", "k_lin_out", "k_lin_bfirst", "k_lin_badd",
                              "k_lin_bscan", "k_lin_grads", "k_lin_join"}


# ---- gradients -------------------------------------------------------------------

GRADS = [
    Linear((1,), 1, 1, 64, 64),
    Linear((3, 0, 40, 16), 1, 2, 64, 64, tail=4, slots=1),
    Linear((64, 65, 127), 1, 1, 128, 128, fresh=(1,)),
    Linear((128, 1, 200, 257), 2, 4, 128, 128, scale=0.3, slots=1),
    Linear((300, 520, 31), 1, 4, 64, 64),
    Linear((600, 90), 2, 2, 48, 96, dtype="f32"),
    Linear((513, 5), 1, 2, 128, 128, dtype="f32", scale=-0.5),
    Linear((260, 33), 1, 3, 112, 16),
    Linear((130, 256), 1, 1, 64, 128),
    Linear((130, 300), 1, 2, 128, 64, dtype="f32", fresh=(0,)),
    Linear((300, 40), 1, 4, 64, 64, alpha=(1.0, 0.0, 1e-3, 0.5)),
    Linear((300, 40), 2, 4, 64, 64, dtype="f32", alpha=(1.0, 0.0, 1e-3, 0.5)),
    Linear((3000,), 1, 1, 64, 64, alpha=(1 - 2.0**-10,)),
    # a key head's value heads in one sum, in two uneven ones, in one each
    Linear((3, 1, 0, 2) * 50, 1, 6, 32, 64, tail=2),
    Linear((3, 17) * 20, 1, 5, 64, 32, dtype="f32", tail=1),
    Linear((1, 200, 5), 2, 16, 16, 48, tail=3),
    # chains beside short sequences, 8 and 16 segments in flight
    Linear((1300, 2600) + (1,) * 15, 1, 1, 128, 128, alpha=(1 - 2.0**-9,)),
    Linear((8500,) + (2,) * 16, 1, 1, 128, 128, alpha=(1 - 2.0**-11,)),
]


def grads_of(c, **kw):
    import torch
    print(f"grad case {c.lengths} hk={c.hk} hv={c.hv} dk={c.dk} dv={c.dv} {c.dtype}", flush=True)
    got = gdn.linear_backward(*(c.cuda(n) for n in ("q", "k", "v", "alpha", "cu", "pool", "slots_in", "dout", "dstate")),
                              scale=c.scale, **kw)
    torch.cuda.synchronize()
    return [None if x is None else x.float().cpu().numpy() for x in got]


@pytest.mark.parametrize("i", range(len(GRADS)))
def test_gradients(i):
    c = GRADS[i]
    c.seed = 300 + i
    c.make()
    got = grads_of(c)
    for name, x, ref, size in zip(("dq", "dk", "dv", "dalpha", "dstate0"), got, c.backward(), c.backward(size=True)):
        print(name, flush=True)
        if name == "dalpha":
            # (a sum of terms of both signs: no bound on the root mean square)
            lim = (2.0**-16 + (max(c.lengths) + 2 * c.dk + 2 * c.dv) * 2.0**-24) * size
            assert (np.abs(x - ref) <= lim).all(), (x, ref, size)
        else:
            near(c, x, ref, size, "f32" if name == "dstate0" else c.dtype)


@pytest.mark.parametrize("lengths", [(139,), (40, 300, 700)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_of_decays_are_sums_in_fp32(lengths, dtype):
    """Over heads of one decay, whose gradients are sums of like terms of either
    sign, errors stand to the values as a term's error to a term: of 2^-24 each
    where every factor is held in fp32, added up by the square root of their number
    (256 in a segment, then one a segment): the root mean square is held to 2^-20
    of the values', where factors of 16 bits leave 2^-18 and more."""
    c = Linear(lengths, 16, 32, 128, 128, dtype=dtype, alpha=(0.98,), scale=128**-0.5, seed=24).make()
    got, ref = grads_of(c)[3], c.backward()[3]
    assert rms(got - ref) <= 2.0**-20 * rms(ref), (rms(got - ref), rms(ref))


def test_gradients_without_states():
    c = Linear((90, 300, 0), 1, 2, 64, 64, fresh=(0, 1, 2), seed=21).make()
    c.a["dstate"][:] = 0
    import torch
    for start in (c.cuda("pool"), None):
        for da, ds in ((True, True), (False, True), (True, False), (False, False)):
            got = gdn.linear_backward(*(c.cuda(n) for n in ("q", "k", "v", "alpha", "cu")), start,
                                      c.cuda("slots_in") if start is not None else None, c.cuda("dout"),
                                      want_grad_alpha=da, want_grad_state0=ds)
            torch.cuda.synchronize()
            assert (got[3] is None) == (not da) and (got[4] is None) == (not ds)
            for x, ref, size in list(zip(got, c.backward(), c.backward(size=True)))[:3]:
                near(c, x.float().cpu().numpy(), ref, size, "bf16")
            if da:
                ref, size = c.backward()[3], c.backward(size=True)[3]
                assert (np.abs(got[3].cpu().numpy() - ref) <= 2.0**-15 * size).all()
            if ds:
                near(c, got[4].cpu().numpy(), c.backward()[4], c.backward(size=True)[4], "f32")


def test_gradients_against_differences():
    """d L along a direction, L formed from the forward's fp32 results."""
    import torch
    c = Linear((90, 300, 5), 1, 2, 64, 64, dtype="f32", alpha=(0.9, 0.97), seed=22).make()
    t = {n: c.cuda(n) for n in (*NAMES, "dout", "dstate")}
    got = gdn.linear_backward(t["q"], t["k"], t["v"], t["alpha"], t["cu"], t["pool"], t["slots_in"], t["dout"], t["dstate"])

    def loss(x):
        out, end = gdn.linear_fwd(x["q"], x["k"], x["v"], x["alpha"], t["cu"], x["pool"], t["slots_in"])
        return float((out.double() * t["dout"].double()).sum() + (end.double() * t["dstate"].double()).sum())
    r = torch.Generator(device="cuda").manual_seed(5)
    for n, g, h in zip(("q", "k", "v", "alpha", "pool"), got, (2.0**-8, 2.0**-8, 2.0**-5, 2.0**-10, 2.0**-5)):
        e = torch.randn(t[n].shape, generator=r, device="cuda")
        if n == "pool":
            g = torch.zeros_like(t["pool"]).index_copy(0, t["slots_in"].long(), g)
        up, down = ({**t, n: t[n] + s * h * e} for s in (1, -1))
        want = (loss(up) - loss(down)) / (2 * h)
        have = float((g.double() * e.double()).sum())
        # linear in all but alpha (there h^2 of the third derivative); a loss is a sum of 1e5 fp32 roundings of 1e-7
        scale = float((g.double() ** 2).sum().sqrt())
        assert abs(want - have) <= 2e-3 * scale + 1e-3 * abs(want), (n, want, have, scale)


def test_gradients_of_slices_and_tokens_in_front():
    import torch
    c = Linear((90, 300, 3), 2, 4, 64, 64, seed=23).make()
    both = torch.cat([c.cuda("q"), c.cuda("k"), c.cuda("v")], 1)
    rest = [c.cuda(n) for n in ("alpha", "cu", "pool", "slots_in", "dout", "dstate")]
    want = gdn.linear_backward(c.cuda("q"), c.cuda("k"), c.cuda("v"), *rest)
    got = gdn.linear_backward(both[:, :2], both[:, 2:4], both[:, 4:], *rest)
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def test_without_sequences_every_row_is_zero():
    import torch
    z = lambda *s, dt=torch.bfloat16: torch.ones(*s, dtype=dt, device="cuda")  # noqa: E731
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = gdn.linear_backward(z(5, 1, 64), z(5, 1, 64), z(5, 2, 64), z(2, dt=torch.float32), cu, None, None, z(5, 2, 64))
    torch.cuda.synchronize()
    assert all((x == 0).all() for x in got[:4]) and got[4].shape == (0, 2, 64, 64)
    # sequences, but no tokens: the state's gradient passes through
    G = torch.randn(3, 2, 64, 64, device="cuda")
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    got = gdn.linear_backward(z(0, 1, 64), z(0, 1, 64), z(0, 2, 64), z(2, dt=torch.float32), cu, None, None, z(0, 2, 64), G)
    out, end = gdn.linear_fwd(z(0, 1, 64), z(0, 1, 64), z(0, 2, 64), z(2, dt=torch.float32), cu, G, None)
    torch.cuda.synchronize()
    assert torch.equal(got[4], G) and (got[3] == 0).all() and torch.equal(end, G) and out.shape == (0, 2, 64)


def test_binding_refuses():
    import torch
    c = Linear((40, 3), 1, 2, 64, 64, seed=24).make()
    t = [c.cuda(n) for n in ("q", "k", "v", "alpha", "cu", "pool", "slots_in")]

    def bad(i, x, err):
        with pytest.raises(err):
            gdn.linear_fwd(*t[:i], x, *t[i + 1:])
        with pytest.raises(err):
            gdn.linear_backward(*t[:i], x, *t[i + 1:], c.cuda("dout"))
    bad(0, t[0].float(), TypeError)
    bad(0, t[0][:, :, :48], ValueError)
    bad(2, t[2].transpose(1, 2), ValueError)
    bad(3, t[3].double(), TypeError)
    bad(3, t[3][:1], ValueError)
    bad(3, t[3].cpu(), ValueError)
    bad(4, t[4].long(), TypeError)
    bad(5, t[5][:, :1], ValueError)
    bad(6, t[6][:1], ValueError)
    with pytest.raises(ValueError):
        gdn.linear_fwd(*t, None, t[6])
    with pytest.raises(gdn.GdnError):
        gdn.linear_fwd(*t, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(gdn.GdnError):
        gdn.linear_fwd(*t[:5], t[5][:0], None)
    with pytest.raises(TypeError):
        gdn.linear_backward(*t, c.cuda("dout").float())
