"""Gradients of the attention in 64 bits with bounds that leave out the rounding of the forward pass's output (tests
only; shares no code with the library)."""
from __future__ import annotations

import math

import torch

from attention_util import half_step, least


class Gradients:
    """dQ and dK of one call, float64 [B, H, S, D], and how far a kernel may be from them whose sum of P dP is its own.

    One batch of heads without sharing.  ``flush``: largest absolute error of a rounded dx besides half a step.
    """

    def __init__(self, q, k, v, dout, out, *, softcap=0.0, slopes=None, causal=False, docs=None, scale=None, flush=None):
        dtype, D = q[0].dtype, q[0].shape[-1]
        q, k, v, g, o = (torch.cat([t.double() for t in ts], 2).transpose(1, 2) for ts in (q, k, v, dout, out))
        Sq, Sk = q.shape[2], k.shape[2]
        scale = D ** -0.5 if scale is None else scale
        pos, keys = torch.arange(Sq, device=q.device) + Sk - Sq, torch.arange(Sk, device=q.device)
        x = q @ k.transpose(-1, -2) * scale
        t = torch.tanh(x / softcap) if softcap else None
        z = softcap * t if softcap else x.clone()
        far = slopes.double()[:, None, None] * (pos[:, None] - keys).abs() if slopes is not None else torch.zeros_like(z)
        z -= far
        see = torch.ones((Sq, Sk), dtype=torch.bool, device=q.device)
        if causal:
            see = keys <= pos[:, None]
        see = see.expand(z.shape[0], 1, Sq, Sk)
        if docs is not None:
            see = see & (docs[:, :, None] == docs[:, None, :])[:, None]
        w = torch.where(see, z, -math.inf).softmax(-1)
        dp = g @ v.transpose(-1, -2)
        inner = dp - (w * dp).sum(-1, keepdim=True)
        bend = 1 - t.square() if softcap else 1.0
        dx = w * inner * bend
        self.dq, self.dk = scale * dx @ k, scale * dx.transpose(-1, -2) @ q
        u, tiny = half_step(dtype), least(dtype)
        flush = tiny if flush is None else flush
        # scores: products summed in steps that drop bits below 2^-23 of the running sum (<= |q|.|k|): 2^-19; cap
        # and bias in fp32: 2^-21 of their size.  Of the weights that matters as much again, and their sum's error.
        score = 2.0 ** -19 * (q.abs() @ k.abs().transpose(-1, -2)) * abs(scale) + 2.0 ** -21 * (softcap + far)
        weight = 2 * torch.where(see, score, 0.0).amax(-1, keepdim=True) + (max(Sq, Sk) + 64) * 2.0 ** -24
        product = 2.0 ** -19 * (g.abs() @ v.abs().transpose(-1, -2))
        # what dO . O lacks of delta: half a step of O; the kernel's sum of it: its terms' errors, Sk additions of fp32
        e = (g * (o - w @ v)).sum(-1, keepdim=True).abs() + 2.0 ** -19 * (g.abs() * o.abs()).sum(-1, keepdim=True)
        size = inner.abs() + e
        delta = (w * ((weight + Sk * 2.0 ** -24) * size + product)).sum(-1, keepdim=True)
        # dx is rounded before e P is taken from it, e P once
        ddx = w * bend * ((u + weight + 2.0 ** -18) * (size + e) + product + delta) + w * size * 2.0 ** -20 + flush
        ddx = torch.where(see, ddx, 0.0) * abs(scale)
        self.dq_tol = u * self.dq.abs() + ddx @ k.abs() + tiny
        self.dk_tol = u * self.dk.abs() + ddx.transpose(-1, -2) @ q.abs() + tiny

    def check(self, name, groups, factor=1.0):
        got = torch.cat([t.double() for t in groups], 2).transpose(1, 2) * factor
        off, tol = (got - getattr(self, name)).abs(), getattr(self, name + "_tol")
        bad = ~(off <= tol)
        worst = (off / tol).nan_to_num(9e9)
        where = [int(i) for i in torch.unravel_index(worst.argmax(), worst.shape)]
        assert not bool(bad.any()), (name, int(bad.sum()), where, float(worst.max()))
