"""Packed ragged inputs for the packed tests, and their reference: the oracle's
fp64 token loop, one sequence at a time."""
from __future__ import annotations

from dataclasses import dataclass, field

import numpy as np

import oracle


@dataclass
class Packed:
    lengths: tuple
    hk: int = 2
    hv: int = 4
    dk: int = 64
    dv: int = 64
    dtype: str = "bf16"
    gate: str = "scalar"
    order: int = 0
    scale: float = 1.0
    alpha_mean: float = 2.0
    slots: int = 0            # slots of the pool beyond one a sequence
    fresh: tuple = ()         # sequences that start from a zero state
    tail: int = 0             # rows behind the last sequence
    seed: int = 0
    a: dict = field(default_factory=dict)

    def make(self):
        """The arrays, in the values that are uploaded (fp32, exactly bf16 where the case is)."""
        r = np.random.Generator(np.random.PCG64(self.seed))
        N, S = sum(self.lengths) + self.tail, len(self.lengths)

        def rounded(x):
            x = x.astype(np.float32)
            if self.dtype == "bf16":
                u = x.view(np.uint32)
                x = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
            return x

        def unit(*shape):
            x = r.standard_normal(shape)
            return rounded(x / np.sqrt((x * x).sum(-1, keepdims=True)))

        a = self.a
        a["q"], a["k"] = unit(N, self.hk, self.dk), unit(N, self.hk, self.dk)
        a["v"] = rounded(r.standard_normal((N, self.hv, self.dv)))
        g = (N, self.hv, self.dk) if self.gate == "channel" else (N, self.hv)
        a["alpha"] = (1 / (1 + np.exp(-(self.alpha_mean + 0.5 * r.standard_normal(g))))).astype(np.float32)
        a["beta"] = (1 / (1 + np.exp(-r.standard_normal((N, self.hv))))).astype(np.float32)
        a["cu"] = np.concatenate([[0], np.cumsum(self.lengths)]).astype(np.int32)
        P = S + self.slots
        a["pool"] = (0.3 * r.standard_normal((P, self.hv, self.dv, self.dk))).astype(np.float32)
        a["slots_in"] = r.permutation(P)[:S].astype(np.int32)
        a["slots_in"][list(self.fresh)] = -1
        a["slots_out"] = r.permutation(P)[:S].astype(np.int32)
        a["dout"] = rounded(r.standard_normal((N, self.hv, self.dv)))
        a["dstate"] = r.standard_normal((S, self.hv, self.dv, self.dk)).astype(np.float32)
        return self

    def cuda(self, name):
        import torch
        x = torch.from_numpy(self.a[name]).cuda()
        return x.to(torch.bfloat16) if self.dtype == "bf16" and name in ("q", "k", "v", "dout") else x

    def _sequences(self):
        a, G = self.a, self.hv // self.hk
        for s, n in enumerate(self.lengths):
            t = slice(int(a["cu"][s]), int(a["cu"][s]) + n)
            start = None if a["slots_in"][s] < 0 else a["pool"][a["slots_in"][s]][None]
            rep = lambda x: np.repeat(x, G, axis=1)[None]  # noqa: E731
            yield s, t, (rep(a["q"][t]), rep(a["k"][t]), a["v"][t][None], a["alpha"][t][None], a["beta"][t][None], start)

    def _kw(self):
        return {"gate": oracle.GATE_SCALAR if self.gate == "scalar" else oracle.GATE_CHANNEL, "order": self.order,
                "scale": self.scale}

    def forward(self):
        """(out [N,Hv,dv] with NaN outside the sequences, end states [S,Hv,dv,dk])"""
        out = np.full((sum(self.lengths) + self.tail, self.hv, self.dv), np.nan)
        ends = np.zeros((len(self.lengths), self.hv, self.dv, self.dk))
        for s, t, x in self._sequences():
            if t.stop > t.start:
                o, e = oracle.forward(*x, **self._kw())
                out[t], ends[s] = o[0], e[0]
            elif x[5] is not None:
                ends[s] = x[5][0]
        return out, ends

    def backward(self):
        """(dq, dk, dv, dalpha, dbeta, dstate0), zero outside the sequences"""
        a, G = self.a, self.hv // self.hk
        g = [np.zeros(a[n].shape) for n in ("q", "k", "v", "alpha", "beta")]
        ds = a["dstate"].astype(np.float64).copy()
        for s, t, x in self._sequences():
            if t.stop == t.start:
                continue
            r = oracle.backward(*x, a["dout"][t][None], a["dstate"][s][None], **self._kw())
            shared = lambda y: y[0].reshape(-1, self.hk, G, self.dk).sum(2)  # noqa: E731
            for dst, val in zip(g, (shared(r[0]), shared(r[1]), r[2][0], r[3][0], r[4][0])):
                dst[t] = val
            ds[s] = r[5][0]
        return (*g, ds)
