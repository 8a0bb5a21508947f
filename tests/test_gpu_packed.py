"""gdn_packed_fwd against the oracle's fp64 token loop over every sequence.

Tolerances, derived before the first run.  bf16 outputs: one rounding of at
most 2^-8 of the value (half a step), plus the kernel's own error, fp32
sums of at most 128 terms and two-term bf16 splits (2^-17 of the largest
value): 2^-8 |o| + 2^-14 max |o| leaves a factor of eight on the latter.
States and fp32 outputs: fp32 throughout (operands split into terms that keep
them to 2^-23 of their column's largest), a 128-term sum is off by at most 128
2^-24 = 7.6e-6 of its terms' sizes, and gates below one keep a token's error from
growing: 1e-5 of the largest value, the library's bound for fp32.
"""
from __future__ import annotations

import numpy as np
import pytest

from gated_delta_rule_12_amd import gdn
from packed_case import Packed

pytestmark = pytest.mark.gpu
PTD, DTP = gdn.GDN_PREDICT_THEN_DECAY, gdn.GDN_DECAY_THEN_PREDICT


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn.lib()


def out_ok(o, ref, dtype):
    top = np.abs(ref).max() if ref.size else 0.0
    lim = 2.0**-8 * np.abs(ref) + 2.0**-14 * top if dtype == "bf16" else 1e-5 * top
    bad = np.abs(o - ref) > lim
    assert not bad.any(), (int(bad.sum()), float(np.abs(o - ref).max()), float(top))


def state_ok(s, ref):
    top = np.abs(ref).max(axis=(-1, -2), keepdims=True)
    err = np.abs(s - ref).max(axis=(-1, -2), keepdims=True) / np.where(top > 0, top, 1.0)
    assert err.max() <= 1e-5, float(err.max())


def run(c, max_len=None, inplace=False, tensors=None, **kw):
    import torch
    c.make()
    t = {n: c.cuda(n) for n in ("q", "k", "v", "alpha", "beta", "cu", "pool", "slots_in", "slots_out")}
    t.update(tensors or {})
    pool_out = t["pool"] if inplace else torch.full_like(t["pool"], 7.0)
    out = torch.full((c.a["q"].shape[0], c.hv, c.dv), 7.0, dtype=t["q"].dtype, device="cuda")
    print(f"case {c.lengths} hk={c.hk} hv={c.hv} dk={c.dk} dv={c.dv} {c.dtype} {c.gate} order={c.order}", flush=True)
    gdn.packed_fwd(t["q"], t["k"], t["v"], t["alpha"], t["beta"], t["cu"], t["pool"], t["slots_in"], pool_out,
                   t["slots_in"] if inplace else t["slots_out"], max_len=max_len, order=c.order, scale=c.scale, out=out, **kw)
    torch.cuda.synchronize()
    return out.float().cpu().numpy(), pool_out.cpu().numpy()


def check(c, out, pool, inplace=False):
    ref, ends = c.forward()
    n = sum(c.lengths)
    out_ok(out[:n], ref[:n], c.dtype)
    assert (out[n:] == 7.0).all()  # rows behind the last sequence
    slots = c.a["slots_in"] if inplace else c.a["slots_out"]
    used = slots >= 0
    state_ok(pool[slots[used]], ends[used])
    rest = np.setdiff1d(np.arange(len(pool)), slots)
    assert (pool[rest] == (c.a["pool"][rest] if inplace else 7.0)).all()  # slots nobody wrote


CASES = [
    # single tokens, drafted tokens, a stage of the token loop and one more
    Packed((1,), 1, 1, 128, 128),
    Packed((1, 1, 1, 1, 1), 2, 4, 128, 128, slots=3),
    Packed((1, 3, 2, 5, 16, 17), 1, 4, 64, 64, slots=2, tail=3),
    Packed((2, 33, 1, 7), 2, 2, 128, 128, gate="channel", order=DTP, slots=1),
    # shapes without chunk kernels, long and short, both types and gates
    Packed((5, 130, 1), 1, 2, 48, 16, slots=1),
    Packed((70, 3), 2, 2, 16, 128, dtype="f32", order=DTP),
    Packed((40, 1, 90), 1, 3, 96, 128, dtype="f32", gate="channel", slots=2),
    Packed((100, 37), 2, 4, 128, 128, dtype="f32"),
    Packed((19, 64), 1, 1, 128, 128, gate="channel"),
    # chunk form: one chunk, borders, tails, beside short ones and empty ones
    Packed((64,), 1, 1, 64, 64),
    Packed((65, 64, 63), 1, 2, 64, 64, slots=1),
    Packed((0, 200, 1, 0, 128, 66, 0), 2, 4, 128, 128, slots=2, tail=5),
    Packed((129, 1, 300), 1, 3, 128, 128, order=DTP, fresh=(0, 2), slots=1),
    Packed((191, 250), 4, 4, 64, 64, order=DTP, scale=0.125),
    # segments
    Packed((1100, 30, 513), 1, 2, 128, 128, slots=1),
    Packed((512, 511, 1537), 2, 2, 64, 64, order=DTP, fresh=(2,)),
    Packed((2600,), 1, 1, 128, 128, alpha_mean=6.0),   # long memory
    Packed((900, 700), 1, 2, 128, 128, alpha_mean=-4.0),  # strong decay
    # many segments: the chain of start states in two levels, and in one beside it
    Packed((9000, 1300, 7, 4700), 1, 1, 64, 64, slots=1, alpha_mean=5.0),
    Packed((5377, 6144), 1, 2, 128, 128, order=DTP, alpha_mean=5.0),
    Packed((4000, 9100), 1, 1, 128, 128, slots=1, alpha_mean=5.0),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_forward(i):
    c = CASES[i]
    c.seed = 100 + i
    check(c, *run(c))


@pytest.mark.parametrize("dtype,gate", [("f32", "scalar"), ("bf16", "channel"), ("f32", "channel")])
@pytest.mark.parametrize("dk,dv", [(32, 32), (64, 48), (128, 128)])
@pytest.mark.parametrize("S,hv", [(3, 2), (20, 4), (140, 4), (300, 4)])
def test_token_form_over_few_and_many_states(S, hv, dk, dv, dtype, gate):
    """The token-by-token kernels by number of states: 1 to 12 tokens each."""
    lengths = tuple(1 + (7 * s) % 12 for s in range(S))
    c = Packed(lengths, 2, hv, dk, dv, dtype=dtype, gate=gate, order=S % 2, seed=37)
    check(c, *run(c))


@pytest.mark.parametrize("lengths,d", [((1, 1, 1), 128), ((3, 90, 1200), 128), ((5, 600), 64)])
def test_in_place(lengths, d):
    c = Packed(lengths, 2, 4, d, d, slots=2, seed=7)
    out, pool = run(c, inplace=True)
    check(c, out, pool, inplace=True)


@pytest.mark.parametrize("max_len", [0, 1, 64, 200, 100000])
def test_any_max_len_gives_the_same_results(max_len):
    c = Packed((1, 700, 65, 1300), 2, 4, 64, 64, seed=8)
    check(c, *run(c, max_len=max_len))


def test_zero_gates_reset_the_state():
    """alpha = 0 inside, at the start and at the end of a chunk; a whole row of zeros."""
    for order in (PTD, DTP):
        c = Packed((300, 20), 1, 2, 128, 128, order=order, seed=9)
        make = c.make

        def with_zeros():
            make()
            for t in (0, 5, 63, 64, 127, 200, 201, 299, 300, 310):
                c.a["alpha"][t] = 0.0
            return c
        c.make = with_zeros
        check(c, *run(c))


@pytest.mark.parametrize("q,k,v,state", [(40, 0, 0, 0), (-60, 0, 0, 0), (0, -20, 0, 0), (0, -45, 0, -45), (0, 0, 60, 60),
                                         (0, 0, -80, -80), (20, -30, -10, 35), (0, 0, 0, 40), (0, 0, 40, 0), (-30, 1, 30, 30)])
@pytest.mark.parametrize("d", [64, 128])
def test_any_scale(d, q, k, v, state):
    """Inputs and states times powers of two: as near to the exact results as
    without (every scale a factor of the results, which are compared by their
    largest; two times the keys with a quarter of beta keeps the state bounded)."""
    c = Packed((70, 700, 3), 1, 2, d, d, seed=31)
    make = c.make

    def scaled():
        make()
        for n, e in (("q", q), ("k", k), ("v", v), ("pool", state)):
            c.a[n] = (c.a[n] * np.float32(2.0**e)).astype(np.float32)
        if k > 0:
            c.a["beta"] /= np.float32(4.0**k)
        return c
    c.make = scaled
    check(c, *run(c))


def test_tokens_and_features_of_different_sizes():
    """Value features over twelve decades, tokens that grow over a chunk border,
    one chunk of zeros: held to each feature's own largest value."""
    c = Packed((400, 90), 1, 2, 128, 128, seed=32, fresh=(0, 1))
    make = c.make

    def sized():
        make()
        c.a["v"] *= (2.0 ** np.linspace(-20, 20, 128).round()).astype(np.float32)
        c.a["v"][64:128] = 0
        c.a["v"][192:256] *= 2.0**12
        c.a["q"][256:320] = 0
        c.a["k"][320:330] = 0
        return c
    c.make = sized
    out, pool = run(c)
    ref, ends = c.forward()
    for lo, hi in ((0, 400), (400, 490)):
        top = np.abs(ref[lo:hi]).max(0)
        assert (np.abs(out[lo:hi] - ref[lo:hi]) <= 2.0**-8 * np.abs(ref[lo:hi]) + 2.0**-14 * top).all()
    got = pool[c.a["slots_out"]]
    assert (np.abs(got - ends) <= 1e-5 * np.abs(ends).max(-1, keepdims=True)).all()


@pytest.mark.parametrize("size", [1.0, 2.0**40, 2.0**100, 0.0])
def test_a_large_state_is_forgotten(size):
    """A gate of zero takes a state of any size away; values follow chunks later."""
    c = Packed((330, 50), 1, 2, 64, 64, seed=33)
    make = c.make

    def forgetful():
        make()
        c.a["pool"] *= np.float32(size)
        c.a["alpha"][[0, 330]] = 0.0
        c.a["v"][:200] = 0
        c.a["k"][0] = c.a["k"][330] = 0  # the first prediction would still read the state
        c.a["q"][[0, 330]] = 0
        return c
    c.make = forgetful
    check(c, *run(c))


def test_nan_stays_in_its_sequence():
    """A NaN or an infinity in v reaches its value feature's later tokens and
    those of its chunk of 64 (the chunk's products take them together), no
    other feature, head or sequence."""
    c = Packed((200, 30, 130, 1), 1, 2, 128, 128, seed=10)
    make = c.make

    def with_nan():
        make()
        c.a["v"][210, 0, 3] = np.nan   # second sequence, head 0, value feature 3
        c.a["v"][231 + 50, 1, 7] = np.inf  # third, head 1, value feature 7
        return c
    c.make = with_nan
    out, pool = run(c)
    c.make = make
    c.make()
    c.seed = 10
    ref, ends = c.forward()
    hit = np.zeros(out.shape, bool)
    hit[210:230, 0, 3] = hit[281:360, 1, 7] = True
    assert not np.isfinite(out[hit]).any()
    hit[230:281, 1, 7] = True  # the chunk that the infinity is in
    assert np.isfinite(out[~hit]).all()
    out_ok(out[~hit], ref[~hit], "bf16")


def test_slices_of_one_projection():
    """q, k, v as views of a wider row."""
    import torch
    c = Packed((100, 7, 1), 2, 4, 64, 64, seed=11).make()
    q, k, v = c.cuda("q"), c.cuda("k"), c.cuda("v")
    N = q.shape[0]
    row = torch.cat([q.reshape(N, -1), k.reshape(N, -1), v.reshape(N, -1), v.new_zeros(N, 8)], 1)
    parts = {"q": row[:, :128].view(N, 2, 64), "k": row[:, 128:256].view(N, 2, 64), "v": row[:, 256:512].view(N, 4, 64)}
    assert parts["q"].stride(0) == 520
    check(c, *run(c, tensors=parts))


@pytest.mark.parametrize("d,gate", [(64, "scalar"), (128, "scalar"), (128, "channel")])
def test_far_tokens(d, gate):
    """Token strides up to the limit: elements past 2^31, bytes past 2^32 (in
    chunks, rows of one chunk a gigabyte apart)."""
    import torch
    c = Packed((270, 30, 1), 1, 2, d, d, gate=gate, seed=34).make()
    far = torch.empty((301, 2**23), dtype=torch.bfloat16, device="cuda")
    far[:, :d], far[:, d:2 * d] = c.cuda("q")[:, 0], c.cuda("k")[:, 0]
    far[:, -2 * d:] = c.cuda("v").view(301, 2 * d)
    check(c, *run(c, tensors={"q": far[:, :d].view(301, 1, d), "k": far[:, d:2 * d].view(301, 1, d),
                              "v": far[:, -2 * d:].view(301, 2, d)}))


def test_two_sequences_start_from_one_slot():
    c = Packed((70, 70, 3), 1, 2, 64, 64, seed=12, slots=1)
    make = c.make

    def shared():
        make()
        c.a["slots_in"][:] = c.a["slots_in"][0]
        return c
    c.make = shared
    check(c, *run(c))


@pytest.mark.parametrize("front", [1, 70, 700])
def test_tokens_in_front_of_the_first_sequence(front):
    """cu_seqlens need not begin at 0: rows in front are left as they were."""
    import torch
    c = Packed((front, 600, 3, 90), 1, 2, 64, 64, seed=20).make()
    t = {n: c.cuda(n) for n in ("q", "k", "v", "alpha", "beta", "cu", "pool", "slots_in", "slots_out")}
    out = torch.full((t["q"].shape[0], 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    pool = torch.full_like(t["pool"], 7.0)
    gdn.packed_fwd(t["q"], t["k"], t["v"], t["alpha"], t["beta"], t["cu"][1:], t["pool"], t["slots_in"][1:], pool,
                   t["slots_out"][1:], out=out)
    torch.cuda.synchronize()
    ref, ends = c.forward()
    o = out.float().cpu().numpy()
    assert (o[:front] == 7.0).all()
    out_ok(o[front:], ref[front:], "bf16")
    state_ok(pool.cpu().numpy()[c.a["slots_out"][1:]], ends[1:])
    assert (pool[int(c.a["slots_out"][0])] == 7.0).all()


def test_bad_offsets_and_slots_stay_in_bounds():
    """Falling, negative and far offsets and slots write nothing but the tokens
    and slots of the call (the values themselves are not defined)."""
    import torch
    c = Packed((100, 70, 30), 1, 2, 64, 64, seed=13).make()
    t = {n: c.cuda(n) for n in ("q", "k", "v", "alpha", "beta", "pool")}
    guard = torch.full((c.a["q"].shape[0] + 128, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    for cu in ([0, 150, 90, 200], [-5, 100, 10**6, 200], [200, 100, 0, -1], [0, 0, 0, 2**31 - 1]):
        for slots in ([0, 1, 2], [-7, 10**9, 2]):
            out = guard[64:-64]
            gdn.packed_fwd(t["q"], t["k"], t["v"], t["alpha"], t["beta"], torch.tensor(cu, dtype=torch.int32).cuda(), t["pool"],
                           torch.tensor(slots, dtype=torch.int32).cuda(), torch.zeros_like(t["pool"]),
                           torch.tensor(slots, dtype=torch.int32).cuda(), out=out)
            torch.cuda.synchronize()
            assert (guard[:64] == 7.0).all() and (guard[-64:] == 7.0).all()


def test_repeats_are_identical_and_graphs_replay():
    import torch
    c = Packed((1, 600, 70, 1100), 2, 4, 128, 128, seed=14).make()
    t = {n: c.cuda(n) for n in ("q", "k", "v", "alpha", "beta", "cu", "pool", "slots_in", "slots_out")}
    out = torch.empty((t["q"].shape[0], 4, 128), dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros_like(t["pool"])
    ws = gdn.packed_workspace_for(t["q"], t["v"], t["alpha"], t["cu"])
    call = lambda: gdn.packed_fwd(t["q"], t["k"], t["v"], t["alpha"], t["beta"], t["cu"], t["pool"], t["slots_in"],  # noqa: E731
                                  pool, t["slots_out"], out=out, workspace=ws)
    call()
    torch.cuda.synchronize()
    first = (out.clone(), pool.clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for i in range(4):
        # other lengths under the same graph, then the first ones again
        cu = torch.tensor([0, 600, 601, 700, 1771], dtype=torch.int32) if i == 1 else torch.from_numpy(c.a["cu"])
        t["cu"].copy_(cu)
        out.zero_()
        pool.zero_()
        ws.fill_(255)  # nothing in the workspace is taken over from an earlier call
        g.replay()
        torch.cuda.synchronize()
        if i == 1:
            again, pool2 = torch.empty_like(out), torch.zeros_like(pool)
            gdn.packed_fwd(t["q"], t["k"], t["v"], t["alpha"], t["beta"], t["cu"], t["pool"], t["slots_in"], pool2,
                           t["slots_out"], out=again)
            torch.cuda.synchronize()
            assert torch.equal(out, again) and torch.equal(pool, pool2)
        else:
            assert torch.equal(out, first[0]) and torch.equal(pool, first[1])


def test_prompt_then_steps_equal_one_prompt():
    """A prompt, then drafted and single tokens from the pool: the whole
    sequence at once, up to rounding."""
    import torch
    c = Packed((600, 450), 1, 2, 128, 128, seed=15, slots=2).make()
    t = {n: c.cuda(n) for n in ("q", "k", "v", "alpha", "beta", "pool", "slots_in")}
    ref, ends = c.forward()
    pool = t["pool"].clone()
    got = torch.empty((1050, 2, 128), dtype=torch.bfloat16, device="cuda")
    at = [0, 600]
    for take in ((500, 380), (5, 1), (1, 1), (70, 64), (23, 3), (1, 1)):
        idx = torch.cat([torch.arange(a, a + n) for a, n in zip(at, take)]).cuda()
        cu = torch.tensor([0, take[0], sum(take)], dtype=torch.int32).cuda()
        o, _ = gdn.packed_fwd(*(t[n][idx] for n in ("q", "k", "v", "alpha", "beta")), cu, pool, t["slots_in"], pool,
                              t["slots_in"], max_len=max(take))
        got[idx] = o
        at = [a + n for a, n in zip(at, take)]
    assert at == [600, 1050]
    torch.cuda.synchronize()
    out_ok(got.float().cpu().numpy(), ref, "bf16")
    state_ok(pool.cpu().numpy()[c.a["slots_in"]], ends)


def test_other_stream_and_two_calls_at_once():
    import torch
    cs = [Packed((700, 90), 1, 2, 128, 128, seed=16).make(), Packed((64, 1000), 1, 2, 128, 128, seed=17).make()]
    ts = [{n: c.cuda(n) for n in ("q", "k", "v", "alpha", "beta", "cu", "pool", "slots_in")} for c in cs]
    args = lambda t: [t[n] for n in ("q", "k", "v", "alpha", "beta", "cu", "pool", "slots_in")]  # noqa: E731
    alone = [gdn.packed_fwd(*args(t)) for t in ts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ts]
    both = []
    for _ in range(4):
        both = []
        for t, s in zip(ts, streams):
            with torch.cuda.stream(s):
                both.append(gdn.packed_fwd(*args(t)))
    torch.cuda.synchronize()
    for x, y in zip(alone, both):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_large_offsets():
    """A pool whose last state lies past 2^31 elements, tokens past 2^31 bytes."""
    import torch
    d, hv = 128, 16
    slots = 2**31 // (hv * d * d) + 8
    c = Packed((70, 1), 1, hv, d, d, seed=18).make()
    t = {n: c.cuda(n) for n in ("q", "k", "v", "alpha", "beta", "cu")}
    pool = torch.empty((slots, hv, d, d), device="cuda")
    at = torch.tensor([slots - 1, slots - 2], dtype=torch.int32).cuda()
    pool[slots - 1], pool[slots - 2] = t["alpha"].new_tensor(c.a["pool"][0]), t["alpha"].new_tensor(c.a["pool"][1])
    c.a["slots_in"] = np.array([0, 1], np.int32)
    # the sequences at the end of a long row of tokens
    N = 2**30 // (hv * d) + 200
    big = torch.zeros((N, hv, d), dtype=torch.bfloat16, device="cuda")
    big[-71:] = t["v"]
    q = torch.zeros((N, 1, d), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros_like(q)
    q[-71:], k[-71:] = t["q"], t["k"]
    al, be = torch.ones((N, hv), device="cuda"), torch.zeros((N, hv), device="cuda")
    al[-71:], be[-71:] = t["alpha"], t["beta"]
    cu = (t["cu"] + (N - 71)).to(torch.int32)
    out, _ = gdn.packed_fwd(q, k, big, al, be, cu, pool, at, pool, at, max_len=70)
    torch.cuda.synchronize()
    ref, ends = c.forward()
    out_ok(out[-71:].float().cpu().numpy(), ref, "bf16")
    state_ok(pool[[slots - 1, slots - 2]].cpu().numpy(), ends)


def test_timer_names_the_kernels():
    import torch
    c = Packed((600, 3), 1, 2, 128, 128, seed=19).make()
    tm = gdn.Timer()
    o, _ = gdn.packed_fwd(*(c.cuda(n) for n in ("q", "k", "v", "alpha", "beta", "cu", "pool")), timer=tm)
    torch.cuda.synchronize()
    assert set(tm.read()) == {"k_pk_prep", "k_pk_state", "k_pk_chain", "k_pk_out"}


@pytest.mark.parametrize("d,order", [(64, PTD), (128, DTP)])
@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("what", ["v", "q", "k", "alpha", "beta", "pool"])
def test_non_finite_inputs_propagate(what, value, d, order):
    """One infinity or NaN: what the formulas make non-finite is so, and every
    finite output is the right one.  Beyond the formulas it may reach (as NaN)
    the tokens of its own chunk of 64: in v those of its value feature, in a gate
    or beta of its head, in k of every head that reads it; in q nothing but its
    own token."""
    c = Packed((40, 700, 33), 1, 2, d, d, order=order, seed=41)
    c.make()
    t, lo = 40 + 300, 40 + 256   # the token, its chunk's first
    free = np.zeros((773, 2, d), bool)
    if what == "v":
        c.a["v"][t, 1, 5] = value
        free[lo:lo + 64, 1, 5] = True
    elif what == "q":
        c.a["q"][t, 0, 5] = value
    elif what == "k":
        c.a["k"][t, 0, 5] = value
        free[lo:lo + 64] = True
    elif what == "pool":
        c.a["pool"][c.a["slots_in"][1], 1, 5, 7] = value
    else:
        c.a[what][t, 1] = value
        free[lo:lo + 64, 1] = True
    c.make = lambda: c
    out, pool = run(c)
    ref, ends = c.forward()
    bad = ~np.isfinite(ref)
    assert bad.any() and not np.isfinite(out[bad]).any()
    assert np.isfinite(out[~bad & ~free]).all()
    ok = ~bad & np.isfinite(out)
    out_ok(out[ok], ref[ok], "bf16")
    got = pool[c.a["slots_out"]]
    bad = ~np.isfinite(ends)
    assert not np.isfinite(got[bad]).any() and np.isfinite(got[~bad]).all()
    assert (np.abs(got - ends)[~bad] <= 1e-5 * np.abs(ends[~bad]).max()).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["scalar", "channel"])
@pytest.mark.parametrize("dk,dv", [(32, 32), (48, 16), (96, 128), (64, 64), (128, 128), (16, 112)])
def test_single_tokens(dk, dv, gate, dtype):
    """A step of one token a sequence in every type, gate and row layout, in both
    orders, into another pool and in place; an empty sequence among them."""
    lengths = (1, 1, 0, 1, 1, 1, 1)
    for order in (PTD, DTP):
        c = Packed(lengths, 2, 6, dk, dv, dtype=dtype, gate=gate, order=order, slots=2, fresh=(3,), tail=2, seed=42)
        check(c, *run(c, max_len=1))
        c.fresh = ()
        out, pool = run(c, max_len=1, inplace=True)
        check(c, out, pool, inplace=True)


def guarded(n, dtype, fill, rim=4096):
    """n elements within a filled buffer, and a check that nothing around them changed."""
    import torch
    whole = torch.full((n + 2 * rim,), fill, dtype=dtype, device="cuda")
    return whole[rim:rim + n], lambda: bool((whole[:rim] == fill).all() and (whole[-rim:] == fill).all())


@pytest.mark.parametrize("lengths,d,hv", [
    ((1,) * 90 + (33,), 64, 2),                                            # single tokens and one chunk
    ((1,) * 60 + (700,) + (2, 0, 31) * 30 + (32, 1300), 128, 4),           # two prompts of several segments
    ((40, 33, 64, 31) * 12 + (1,) * 150 + (900, 257, 129), 64, 4),
    ((3,) * 300 + (6000,) + (1,) * 100 + (40, 300), 64, 1),                # a chain in two levels, one in one
    ((3,) * 100 + (10000,) + (1,) * 300 + (400, 9000), 128, 1),
])
def test_many_short_sequences_beside_prompts(lengths, d, hv):
    """Sequences without chunks or segments have no places in the workspace."""
    import torch
    c = Packed(lengths, 1, hv, d, d, seed=43, slots=1, alpha_mean=5.0).make()
    n = gdn.gdn_packed_workspace_bytes(sum(lengths), len(lengths), 1, hv, d, d, sum(lengths), gdn.GDN_BF16, 0)
    ws, untouched = guarded(n, torch.uint8, 0xA5)
    check(c, *run(c, workspace=ws))
    assert untouched()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("S", [3, 40])
def test_bad_offsets_and_slots_write_nothing_else(S, d):
    """Offsets and slots of any value: nothing outside the outputs, the pool and
    the workspace, and no slot that the call does not name."""
    import torch
    N, hv = 3000, 2
    r = np.random.Generator(np.random.PCG64(44))
    c = Packed((N,), 1, hv, d, d, seed=44).make()
    t = {n: c.cuda(n) for n in ("q", "k", "v", "alpha", "beta")}
    state = hv * d * d
    for cu in ([0, N] * S, [N, 0] * S, [0] * (2 * S) + [2**31 - 1], [-2**31] + [2**31 - 1] * (2 * S),
               list(r.integers(-10, N + 10, 2 * S))):
        cu = cu[:S + 1]
        slots = r.choice([-1, -2**31, 2**31 - 1, S + 2, 5], S)
        slots[0] = 1
        pool, pool_whole = guarded((S + 2) * state, torch.float32, 7.0)
        out, out_whole = guarded(N * hv * d, torch.bfloat16, 7.0)
        n = gdn.gdn_packed_workspace_bytes(N, S, 1, hv, d, d, N, gdn.GDN_BF16, 0)
        ws, ws_whole = guarded(n, torch.uint8, 0xA5)
        print("offsets", cu[:6], "slots", slots[:6], flush=True)
        cu, slots = (torch.tensor(np.array(x), dtype=torch.int32).cuda() for x in (cu, slots))
        gdn.packed_fwd(t["q"], t["k"], t["v"], t["alpha"], t["beta"], cu, c.cuda("pool"), slots, pool.view(S + 2, hv, d, d),
                       slots, out=out.view(N, hv, d), workspace=ws)
        torch.cuda.synchronize()
        assert pool_whole() and out_whole() and ws_whole()
        rest = [s for s in range(S + 2) if s not in (1, 5)]
        assert (pool.view(S + 2, -1)[rest] == 7.0).all()


@pytest.mark.parametrize("d", [64, 128])
def test_non_finite_rows_outside_the_sequences(d):
    """Rows in front of the first and behind the last sequence are not read."""
    import torch
    c = Packed((70, 1, 500, 33), 1, 2, d, d, seed=45, tail=70).make()
    t = {n: c.cuda(n) for n in ("q", "k", "v", "alpha", "beta", "cu", "pool", "slots_in")}
    call = lambda: gdn.packed_fwd(t["q"], t["k"], t["v"], t["alpha"], t["beta"], t["cu"][1:], t["pool"],  # noqa: E731
                                  t["slots_in"][1:])
    out, pool = call()
    for n in ("q", "k", "v", "alpha", "beta"):
        t[n][:70], t[n][604:] = np.nan, np.inf
    again, pool2 = call()
    torch.cuda.synchronize()
    assert torch.equal(out[70:604], again[70:604]) and torch.equal(pool, pool2)
