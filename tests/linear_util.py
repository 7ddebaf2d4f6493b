"""Linear attention in 64 bits, pair by pair, with bounds for a kernel that works in chunks (tests only; shares no code
with the library).

Sizes: with absolute values everywhere, A_i = |scale| (sum_j w_ij (|q_i| . |k_j|) |v_j| + w_i |q_i| |state|).  A kernel rounds
to the I/O type (half a step u, relative) the weights (q . k) w of a chunk or the state's entries -- either way u A at
most, and u |o| for the result.  Everything else is fp32: decays within 2^-20 of themselves where they count (an exponent x has
an error of 2^-24 x, and 2^-24 x e^-x < 2^-24), sums and the products' dropped bits 2^-17 of A together, and a state's
keys kept to 2^-17.  So |error| <= u |o| + (u + 2^-15) A.  A state is off by 2^-15 of its own size with absolute values.

That is the worst case, every rounding in the same direction.  Roundings of random inputs are independent: the norm
of the error is then at most sqrt(2) u of the result's norm -- one rounding of the terms and one of the result, each u / sqrt(3)
on the average and u at most -- and 2^-18 of a state's.
"""
from __future__ import annotations

import torch


def wide(groups):
    """P views [B, S, h, D] as float64 [B, H, S, D]."""
    return torch.cat([g.double() for g in groups], 2).transpose(1, 2)


def weights(decay, n, reverse=False):
    """[H, n, n]: e^(-decay (i - j)) where j <= i (reverse: e^(-decay (j - i)) where j >= i)."""
    i = torch.arange(n, device=decay.device, dtype=torch.float64)
    gone = (i[None] - i[:, None]) if reverse else (i[:, None] - i[None])
    return torch.where(gone >= 0, torch.exp(-decay.double()[:, None, None] * gone.clamp(min=0)), 0.0)


def power(decay, n):
    return torch.exp(-decay.double()[:, None] * n)


def recurrence(q, k, v, decay, scale, start=None, start_scale=None, reverse=False):
    """(out, its size A, last state, its size) of [B, H, S, D] in 64 bits.  ``start`` enters with start_scale in place of scale;
    reverse: rows see themselves and later ones, and the state starts behind the last."""
    start_scale = scale if start_scale is None else start_scale
    n = q.shape[2]
    w = weights(decay, n, reverse)
    i = torch.arange(n, device=q.device, dtype=torch.float64)
    age = power(decay, n - 1 - i if reverse else i + 1)[..., None]  # of the start, at each row
    left = power(decay, i + 1 if reverse else n - 1 - i)[..., None]  # of each row, in the last state
    whole = torch.exp(-decay.double() * n)[:, None, None]

    def both(a, b, c, s, f, f0):
        out = f * ((a @ b.transpose(-1, -2)) * w) @ c
        last = (b * left).transpose(-1, -2) @ c
        if s is not None:
            out = out + f0 * (a * age) @ s
            last = last * (f / f0 if reverse and f0 else 1.0) + whole * s
        elif reverse:
            last = last * (f / start_scale if start_scale else 1.0)
        return out, last

    out, last = both(q, k, v, start, scale, start_scale)
    size, last_size = both(q.abs(), k.abs(), v.abs(), None if start is None else start.abs(), abs(scale), abs(start_scale))
    return out, size, last, last_size


def check_rows(name, groups, want, size, dtype, norm=True):
    """P tensors [B, S, h, D] against float64 [B, H, S, D]."""
    got = wide(groups)
    u = torch.finfo(dtype).eps / 2
    off = (got - want).abs()
    tol = u * want.abs() + (u + 2.0 ** -15) * size + torch.finfo(dtype).tiny * torch.finfo(dtype).eps
    beyond = want.abs() + tol >= torch.finfo(dtype).max  # may be infinite of the same sign
    off = torch.where(beyond & (got == want.sign() * float("inf")), 0.0, off)
    assert bool((off <= tol).all()), (name, float((off / tol).nan_to_num(9e9).max()))
    if norm and want.numel() >= 4096:
        assert float(off.norm()) <= (2 ** 0.5 * u + 2.0 ** -18) * float(want.norm()), (name, float(off.norm() / want.norm()) / u)


def check_state(name, got, want, size, norm=True):
    off = (got.double() - want).abs()
    assert bool((off <= 2.0 ** -15 * size + 2.0 ** -126).all()), (name, float((off / size).nan_to_num(9e9).max()))
    if norm and float(want.norm()):
        assert float(off.norm()) <= 2.0 ** -18 * float(want.norm()), (name, float(off.norm() / want.norm()))
