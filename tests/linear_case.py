"""Packed inputs of linear attention and of the query and key norm for their
tests, and their references in 64 bits: token loops, one sequence at a time."""
from __future__ import annotations

from dataclasses import dataclass, field

import numpy as np


def rounded(x, dtype):
    """fp64 -> fp32, or to the nearest bf16 (as fp32)."""
    x = np.asarray(x, np.float64).astype(np.float32)
    if dtype == "bf16":
        u = x.view(np.uint32)
        x = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return x


def linear_tokens(q, k, v, alpha, S, scale):
    """One sequence, one value head: S_t = alpha S_{t-1} + v_t k_t^T, o_t = scale S_t q_t.
    Returns (out [n,dv], end state)."""
    out = np.zeros((len(q), v.shape[1]))
    S = S.astype(np.float64)
    for t in range(len(q)):
        S = alpha * S + np.outer(v[t], k[t])
        out[t] = scale * (S @ q[t])
    return out, S


def linear_tokens_backward(q, k, v, alpha, S, scale, dout, G):
    """The chain rule through linear_tokens, token by token from the last:
    (dq, dk, dv, dalpha, dS0); G is the gradient of the end state."""
    states = [S.astype(np.float64)]
    for t in range(len(q)):
        states.append(alpha * states[-1] + np.outer(v[t], k[t]))
    dq, dk, dv, da = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape), 0.0
    G = G.astype(np.float64)
    for t in range(len(q) - 1, -1, -1):
        dq[t] = scale * (states[t + 1].T @ dout[t])
        G = G + scale * np.outer(dout[t], q[t])
        dv[t], dk[t] = G @ k[t], G.T @ v[t]
        da += (G * states[t]).sum()
        G = alpha * G
    return dq, dk, dv, da, G


@dataclass
class Linear:
    lengths: tuple
    hk: int = 2
    hv: int = 4
    dk: int = 64
    dv: int = 64
    dtype: str = "bf16"
    scale: float = 1.0
    alpha: tuple = ()         # decays of the heads, in turn; (): between 0.7 and 0.999
    slots: int = 0            # slots of the pool beyond one a sequence
    fresh: tuple = ()         # sequences that start from a zero state
    tail: int = 0             # rows behind the last sequence
    seed: int = 0
    a: dict = field(default_factory=dict)

    def make(self):
        """The arrays, in the values that are uploaded."""
        r = np.random.Generator(np.random.PCG64(self.seed))
        N, S = sum(self.lengths) + self.tail, len(self.lengths)
        a = self.a
        a["q"] = rounded(r.standard_normal((N, self.hk, self.dk)) / np.sqrt(self.dk), self.dtype)
        a["k"] = rounded(r.standard_normal((N, self.hk, self.dk)) / np.sqrt(self.dk), self.dtype)
        a["v"] = rounded(r.standard_normal((N, self.hv, self.dv)), self.dtype)
        al = self.alpha or tuple(1.0 - 2.0 ** -e for e in np.linspace(1.7, 10.0, self.hv))
        a["alpha"] = np.array([al[h % len(al)] for h in range(self.hv)], np.float32)
        a["cu"] = np.concatenate([[0], np.cumsum(self.lengths)]).astype(np.int32)
        P = S + self.slots
        a["pool"] = (0.3 * r.standard_normal((P, self.hv, self.dv, self.dk))).astype(np.float32)
        a["slots_in"] = r.permutation(P)[:S].astype(np.int32)
        a["slots_in"][list(self.fresh)] = -1
        a["slots_out"] = r.permutation(P)[:S].astype(np.int32)
        a["dout"] = rounded(r.standard_normal((N, self.hv, self.dv)), self.dtype)
        a["dstate"] = r.standard_normal((S, self.hv, self.dv, self.dk)).astype(np.float32)
        return self

    def cuda(self, name):
        import torch
        x = torch.from_numpy(self.a[name]).cuda()
        return x.to(torch.bfloat16) if self.dtype == "bf16" and name in ("q", "k", "v", "dout") else x

    def _each(self, size):
        """(sequence, its tokens, value head, key head, the head's inputs); size:
        all of them by their absolute values, so that results bound the sums of
        their terms' sizes."""
        f = (lambda x: np.abs(x.astype(np.float64))) if size else (lambda x: x.astype(np.float64))
        a = self.a
        for s, n in enumerate(self.lengths):
            t = slice(int(a["cu"][s]), int(a["cu"][s]) + n)
            for h in range(self.hv):
                hk = h // (self.hv // self.hk)
                S = a["pool"][a["slots_in"][s], h] if a["slots_in"][s] >= 0 else np.zeros((self.dv, self.dk))
                yield s, t, h, hk, (f(a["q"][t, hk]), f(a["k"][t, hk]), f(a["v"][t, h]), float(a["alpha"][h]), f(S),
                                    abs(self.scale) if size else self.scale)

    def forward(self, size=False):
        """(out [N,hv,dv] with NaN outside the sequences, end states [S,hv,dv,dk])"""
        out = np.full((sum(self.lengths) + self.tail, self.hv, self.dv), np.nan)
        ends = np.zeros((len(self.lengths), self.hv, self.dv, self.dk))
        for s, t, h, _, x in self._each(size):
            out[t, h], ends[s, h] = linear_tokens(*x)
        return out, ends

    def backward(self, size=False):
        """(dq, dk, dv, dalpha, dstate0), zero outside the sequences"""
        a = self.a
        f = np.abs if size else (lambda x: x)
        dq, dk, dv = (np.zeros(a[n].shape) for n in "qkv")
        da, ds = np.zeros(self.hv), np.zeros(a["dstate"].shape)
        for s, t, h, hk, x in self._each(size):
            r = linear_tokens_backward(*x, f(a["dout"][t, h].astype(np.float64)), f(a["dstate"][s, h].astype(np.float64)))
            dq[t, hk] += r[0]
            dk[t, hk] += r[1]
            dv[t, h] = r[2]
            da[h] += r[3]
            ds[s, h] = r[4]
        return dq, dk, dv, da, ds


def rotate(y, cos, sin, interleaved):
    """Pairs of y's first 2 * cos.shape[-1] features turned; cos, sin [N,1,rot/2]."""
    r = cos.shape[-1]
    z = y.copy()
    first = 2 * np.arange(r) if interleaved else np.arange(r)
    second = first + (1 if interleaved else r)
    z[..., first] = y[..., first] * cos - y[..., second] * sin
    z[..., second] = y[..., second] * cos + y[..., first] * sin
    return z


def qk_norm(x, w, cos, sin, eps, interleaved):
    """x [N,H,d] fp64 -> normed, weighted and rotated (cos None: not)."""
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return y if cos is None else rotate(y, cos[:, None], sin[:, None], interleaved)


def qk_norm_backward(dy, x, w, cos, sin, eps, interleaved):
    """(dx, dw), dw summed over tokens and heads"""
    g = dy if cos is None else rotate(dy, cos[:, None], -sin[:, None], interleaved)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xhat = x * r
    return r * (g * w - xhat * (g * w * xhat).mean(-1, keepdims=True)), (g * xhat).sum((0, 1))
