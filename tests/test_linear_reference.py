"""The references of the linear attention and query and key norm tests pinned: by
hand-computed values, by finite differences and by reverse mode in 64 bits."""
import numpy as np
import pytest
import torch

from linear_case import Linear, linear_tokens, linear_tokens_backward, qk_norm, qk_norm_backward


def test_two_tokens_by_hand():
    q = k = np.array([[1.0, 0.0], [1.0, 1.0]])
    v = np.array([[2.0], [4.0]])
    out, S = linear_tokens(q, k, v, 0.5, np.array([[8.0, 16.0]]), 1.0)
    # S_1 = (4, 8) + (2, 0), o_1 = 6; S_2 = (3, 4) + (4, 4), o_2 = 15
    assert out[:, 0].tolist() == [6.0, 15.0] and S.tolist() == [[7.0, 8.0]]


def test_zero_and_unit_decay():
    r = np.random.default_rng(0)
    q, k, v = (r.standard_normal((6, 3)) for _ in range(3))
    S = r.standard_normal((3, 3))
    out, end = linear_tokens(q, k, v, 0.0, S, 2.0)
    assert np.allclose(out, 2 * (q * k).sum(1, keepdims=True) * v) and np.allclose(end, np.outer(v[5], k[5]))
    out, end = linear_tokens(q, k, v, 1.0, S, 1.0)
    assert np.allclose(end, S + v.T @ k) and np.allclose(out[5], end @ q[5])


def test_pairs_of_tokens():
    """The sum over pairs that defines the layer, against the recurrence."""
    r = np.random.default_rng(1)
    n, a = 20, 0.9
    q, k, v = (r.standard_normal((n, 4)) for _ in range(3))
    S = r.standard_normal((4, 4))
    d = np.subtract.outer(np.arange(n), np.arange(n))
    D = np.where(d >= 0, a ** np.maximum(d, 0), 0)
    out, _ = linear_tokens(q, k, v, a, S, 1.0)
    assert np.allclose(out, (D * (q @ k.T)) @ v + a ** (np.arange(n) + 1)[:, None] * (q @ S.T))


@pytest.mark.parametrize("alpha", [0.8, 1.0, 0.0])
def test_gradients_by_reverse_mode_and_differences(alpha):
    r = np.random.default_rng(2)
    n, dk, dv, scale = 7, 3, 2, 0.5
    x = [r.standard_normal(s) for s in ((n, dk), (n, dk), (n, dv))] + [np.float64(alpha), r.standard_normal((dv, dk))]
    do, G = r.standard_normal((n, dv)), r.standard_normal((dv, dk))
    got = linear_tokens_backward(*x[:5], scale, do, G)
    t = [torch.tensor(y, requires_grad=True) for y in x]
    S, loss = t[4], 0.0
    for i in range(n):
        S = t[3] * S + t[2][i][:, None] * t[1][i][None]
        loss = loss + scale * ((S @ t[0][i]) * torch.tensor(do[i])).sum()
    (loss + (S * torch.tensor(G)).sum()).backward()
    for y, z in zip(got, t):
        assert np.allclose(y, z.grad.numpy(), rtol=1e-12, atol=1e-12)

    def f(x):
        o, S = linear_tokens(*x, scale)
        return (o * do).sum() + (S * G).sum()
    for i, g in enumerate(got):
        e = r.standard_normal(np.shape(x[i]))
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + 1e-6 * e, x[i] - 1e-6 * e
        assert abs((f(up) - f(down)) / 2e-6 - (g * e).sum()) < 1e-6 * max(1.0, np.abs(g).sum())


def test_sizes_bound_the_results():
    c = Linear((5, 0, 9), 1, 2, 16, 32, scale=-2.0, slots=1, tail=2, seed=3).make()
    for small, large in ((c.forward(), c.forward(size=True)), (c.backward(), c.backward(size=True))):
        for x, y in zip(small, large):
            assert (np.abs(x[~np.isnan(x)]) <= y[~np.isnan(y)] * (1 + 1e-12)).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_and_rotation(interleaved):
    r = np.random.default_rng(4)
    # a quarter turn of the pair of unequal features moves each to the other's place
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])
    cos, sin = np.array([[0.0]]), np.array([[1.0]])
    y = qk_norm(x, np.ones(4), cos, sin, 0.0, interleaved)
    assert np.allclose(y, np.array([[[-4.0, 3.0, 0.0, 0.0]]]) * 2 / 5)
    x, dy, w = r.standard_normal((5, 2, 8)), r.standard_normal((5, 2, 8)), r.standard_normal(8)
    angle = r.standard_normal((5, 3))
    dx, dw = qk_norm_backward(dy, x, w, np.cos(angle), np.sin(angle), 1e-3, interleaved)
    f = lambda x, w: (qk_norm(x, w, np.cos(angle), np.sin(angle), 1e-3, interleaved) * dy).sum()  # noqa: E731
    for _ in range(3):
        ex, ew = r.standard_normal(x.shape), r.standard_normal(8)
        assert abs((f(x + 1e-6 * ex, w) - f(x - 1e-6 * ex, w)) / 2e-6 - (dx * ex).sum()) < 1e-7
        assert abs((f(x, w + 1e-6 * ew) - f(x, w - 1e-6 * ew)) / 2e-6 - (dw * ew).sum()) < 1e-7
