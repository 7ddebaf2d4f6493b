"""Attention over head groups and its gradient in 64 bits, and how far a kernel that
rounds where the ABI says may be from them (tests only; shares no code with the library)."""
from __future__ import annotations

import math

import torch


def half_step(dtype):
    """Largest relative error of one rounding to ``dtype``."""
    return torch.finfo(dtype).eps / 2


def least(dtype):
    """Largest absolute error of a rounding to ``dtype`` below its normal range: half of fp16's smallest step; bf16
    has fp32's range, whose values below 2^-126 may be flushed to zero."""
    return {torch.float16: 2.0 ** -25}.get(dtype, 2.0 ** -126)


class Reference:
    """Forward and gradients of one call, float64, with the sums that bound the errors.

    q, k, v (and dout): lists of P tensors [B, S, h, D].  Everything is kept as [B, H, ...].
    """

    def __init__(self, q, k, v, dout=None, *, scale=None, softcap=0.0, slopes=None, causal=False, prefix=None,
                 q_docs=None, k_docs=None, clean=False):
        self.dtype, self.P = q[0].dtype, len(q)
        wide = lambda ts: torch.cat([t.double() for t in ts], 2).transpose(1, 2)  # noqa: E731
        q, k, v = wide(q), wide(k), wide(v)
        B, H, Sq, D = q.shape
        Hkv, Sk = k.shape[1:3]
        self.share = H // Hkv
        self.scale = D ** -0.5 if scale is None else scale
        see = torch.ones((B, Sq, Sk), dtype=torch.bool, device=q.device)
        pos = torch.arange(Sq, device=q.device) + Sk - Sq
        keys = torch.arange(Sk, device=q.device)
        if causal:
            see &= (keys[None] <= pos[:, None])[None] | (
                (keys[None, None] < prefix[:, None, None]) if prefix is not None else torch.zeros_like(see))
        if q_docs is not None:
            see &= (q_docs[:, :, None] == k_docs[:, None, :]) & (q_docs >= 0)[:, :, None]
        self.see = see[:, None]
        if clean:  # what padding tokens hold must not matter: leave it out of the products
            q = torch.where((q_docs >= 0)[:, None, :, None], q, 0.0)
            k = torch.where((k_docs >= 0)[:, None, :, None], k, 0.0)
            v = torch.where((k_docs >= 0)[:, None, :, None], v, 0.0)
        kk, vv = k.repeat_interleave(self.share, 1), v.repeat_interleave(self.share, 1)
        x = q @ kk.transpose(-1, -2) * self.scale
        t = torch.tanh(x / softcap) if softcap else None
        z = softcap * t if softcap else x
        if slopes is not None:
            z = z - slopes.double()[:, None, None] * (pos[:, None] - keys[None]).abs()
        z = torch.where(self.see, z, -math.inf)
        self.lse = torch.logsumexp(z, -1)
        base = torch.where(self.lse == -math.inf, 0.0, self.lse)
        w = torch.where(self.see, torch.exp(z - base[..., None]), 0.0)
        self.out = w @ vv
        u, tiny = half_step(self.dtype), least(self.dtype)
        # A score's error: the product of Q and K is summed on the tensor cores in at most 8 + 8 steps that drop bits
        # below 2^-23 of the running sum (<= |q|.|k|): 2^-19; the cap's tanh and the bias in fp32: 2^-21 of their size.
        size = (q.abs() @ kk.abs().transpose(-1, -2)) * abs(self.scale)
        far = (slopes.double()[:, None, None] * (pos[:, None] - keys[None]).abs()) if slopes is not None else 0.0
        score = 2.0 ** -19 * size + 2.0 ** -21 * (softcap + far)
        self.score = torch.where(self.see, score, 0.0)
        worst = self.score.amax(-1) if Sk else torch.zeros_like(self.lse)
        # the row's sum: n fp32 terms in any order are off by at most (n - 1) 2^-24 of the sum of their sizes, each
        # term by the exponential's 2 units and its argument's rounding: 32 * 2^-24
        sums = (max(Sq, Sk) + 64) * 2.0 ** -24
        self.lse_tol = worst + sums + 2.0 ** -23 * base.abs()
        # a weight: rounded to the I/O type once; its score's and its row sum's errors
        dw = w * (u + 2 * worst[..., None] + sums) + tiny
        self.out_tol = u * self.out.abs() + dw @ vv.abs() + tiny
        if dout is None:
            return
        g = wide(dout)
        if clean:
            g = torch.where((q_docs >= 0)[:, None, :, None], g, 0.0)
        dp = g @ vv.transpose(-1, -2)
        delta = (g * self.out).sum(-1, keepdim=True)
        bend = 1 - t.square() if softcap else torch.ones_like(z)
        dx = w * (dp - delta) * bend
        join = lambda y: y.unflatten(1, (Hkv, self.share)).sum(2)  # noqa: E731
        self.dq, self.dk, self.dv = self.scale * dx @ kk, join(self.scale * dx.transpose(-1, -2) @ q), join(w.transpose(-1, -2) @ g)
        # dP - delta: the product's error as a score's; delta from the rounded output; bend: 2^-20 absolute
        inner = 2.0 ** -19 * (g.abs() @ vv.abs().transpose(-1, -2)) + (g.abs() * (self.out_tol + 2.0 ** -19 * self.out.abs())).sum(-1, keepdim=True)
        ddx = dx.abs() * (u + 2 * worst[..., None] + 2 * sums + 2.0 ** -18) + w * inner * bend + w * (dp - delta).abs() * 2.0 ** -20 + tiny * (1 + (dp - delta).abs())
        ddx = torch.where(self.see, ddx, 0.0)
        dw = torch.where(self.see, dw, 0.0)
        s = abs(self.scale)
        self.dq_tol = u * self.dq.abs() + s * (ddx @ kk.abs()) + tiny
        self.dk_tol = u * self.dk.abs() + join(s * ddx.transpose(-1, -2) @ q.abs()) + tiny
        self.dv_tol = u * self.dv.abs() + join(dw.transpose(-1, -2) @ g.abs()) + tiny

    def check(self, name, groups):
        """Every element of P tensors [B, S, h, D] (lse: [B, h, S]) within its bound."""
        if name == "lse":
            got = torch.cat([t.double() for t in groups], 1)
            empty = self.lse == -math.inf
            assert torch.equal(got == -math.inf, empty), "rows that see nothing"
            off = torch.where(empty, 0.0, (got - self.lse).abs())
        else:
            got = torch.cat([t.double() for t in groups], 2).transpose(1, 2)
            off = (got - getattr(self, name)).abs()
        tol = getattr(self, name + "_tol")
        bad = ~(off <= tol)
        assert not bool(bad.any()), (name, int(bad.sum()), float(off.nan_to_num(9e9).max()), float((off / tol.clamp(min=1e-30)).nan_to_num(9e9).max()))
