"""The paged cache in 64 bits, sequence by sequence (tests only; shares no code with the library)."""
from __future__ import annotations

import math

import torch

E4M3 = torch.float8_e4m3fn


def rotated(x, weight, rope, cos_sin, at, eps=1e-6):
    """Rows [T, h, D] normalised and rotated at positions ``at``, float64, and the size of what each element sums."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * weight.double()
    if rope is None:
        return x, x.abs()
    D = x.shape[-1]
    cos, sin = (t[:, None] for t in cos_sin.double()[at].unbind(-1))
    i = torch.arange(D // 2, device=x.device)
    a, b = (i, i + D // 2) if rope == "neox" else (2 * i, 2 * i + 1)
    y, size = torch.empty_like(x), torch.empty_like(x)
    y[..., a], y[..., b] = x[..., a] * cos - x[..., b] * sin, x[..., a] * sin + x[..., b] * cos
    size[..., a] = (x[..., a] * cos).abs() + (x[..., b] * sin).abs()
    size[..., b] = (x[..., a] * sin).abs() + (x[..., b] * cos).abs()
    return y, size


def values(codes, scale):
    return codes.float().double() * scale.double()[..., None, None]


def table(rows, D, theta=10000.0):
    angle = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * theta ** (
        -torch.arange(D // 2, device="cuda", dtype=torch.float64) * 2 / D)
    return torch.stack([angle.cos(), angle.sin()], -1).float()


def check_half(before, after, page_table, lens, starts, new, size):
    """One half (codes, scales) of a cache after an append of float64 rows ``new`` [T, Hkv, D] (exact up to 2^-20 size)."""
    (c0, s0), (c1, s1) = before, after
    page = c0.shape[2]
    touched = torch.zeros(c0.shape[:1], dtype=torch.bool)
    for n, length in enumerate(lens):
        lo, row = length - (starts[n + 1] - starts[n]), starts[n]
        while lo < length:
            hi = min(length, (lo // page + 1) * page)
            where, off, rows = page_table[n][lo // page], lo % page, hi - lo
            touched[where] = True
            x, err = new[row:row + rows].transpose(0, 1), 2.0 ** -20 * size[row:row + rows].transpose(0, 1)
            s = s1[where].double()
            assert bool((torch.exp2(torch.round(torch.log2(s))) == s).all()), "a power of two"
            finite = torch.where(x.isfinite(), x.abs(), 0.0)
            most, slack = finite.amax((1, 2)), err.nan_to_num(0, 0, 0).amax((1, 2))
            floor = s0[where].double() if off else torch.full_like(s, 2.0 ** -100)
            assert bool((448 * s >= most - slack).all()) and bool((s >= floor).all()), "a scale that holds the values"
            assert bool(((224 * s < most + slack) | (s == floor)).all()), "the smallest such scale"
            got = values(c1[where], s1[where])
            # one rounding: half a step is 2^-4 of the value, or 2^-10 of the scale below e4m3's normal range
            room = lambda v: torch.maximum(v.abs() * 2.0 ** -4, (2.0 ** -10 * s)[:, None, None])  # noqa: E731
            part = got[:, off:off + rows]
            want = torch.where(x.isinf(), x.sign() * (448 * s)[:, None, None], x)
            assert torch.equal(part.isnan(), want.isnan())
            ok = (part - want).abs() <= room(want) * (1 + 2.0 ** -20) + err.nan_to_num(0, 0, 0)
            assert bool((ok | want.isnan()).all()), float((part - want).abs().max())
            if off:
                old = values(c0[where][:, :off], s0[where])
                same = (s == s0[where].double())[:, None, None]
                ok = torch.where(same, got[:, :off] == old, (got[:, :off] - old).abs() <= room(old))
                assert bool((ok | old.isnan()).all()), "older tokens"
            assert torch.equal(c0[where][:, off + rows:].view(torch.uint8), c1[where][:, off + rows:].view(torch.uint8))
            lo, row = hi, row + rows
    keep = ~touched.to(c0.device)
    assert torch.equal(c0[keep].view(torch.uint8), c1[keep].view(torch.uint8)) and torch.equal(s0[keep], s1[keep])


def attend(q, cache, page_table, lens, starts, *, scale=None, softcap=0.0, slopes=None, causal=True):
    """q [T, H, D]: float64 out, lse, and their bounds; rows of no sequence are NaN."""
    T, H, D = q.shape
    k_codes, v_codes, k_scale, v_scale = cache
    Hkv, page = k_codes.shape[1:3]
    share, scale = H // Hkv, D ** -0.5 if scale is None else scale
    u = torch.finfo(q.dtype).eps / 2
    tiny = {torch.float16: 2.0 ** -25}.get(q.dtype, 2.0 ** -126)
    out, lse = (torch.full(s, math.nan, dtype=torch.float64, device=q.device) for s in ((T, H, D), (T, H)))
    out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    for n, length in enumerate(lens):
        a, b = starts[n], starts[n + 1]
        if a == b:
            continue
        pages = page_table[n][: -(-length // page)]
        wide = lambda codes, s: values(codes[pages], s[pages]).transpose(0, 1).flatten(1, 2)[:, :length].repeat_interleave(share, 0)  # noqa: E731
        k, v = wide(k_codes, k_scale), wide(v_codes, v_scale)
        x = q[a:b].double().transpose(0, 1)
        raw = x @ k.transpose(1, 2) * scale
        z = softcap * torch.tanh(raw / softcap) if softcap else raw
        far = torch.arange(length - (b - a), length, device=q.device)[:, None] - torch.arange(length, device=q.device)
        bias = slopes.double()[:, None, None] * far.abs() if slopes is not None else torch.zeros_like(z)
        z = z - bias
        see = (far >= 0) if causal else torch.ones_like(far, dtype=torch.bool)
        z = torch.where(see, z, -math.inf)
        total = torch.logsumexp(z, -1)
        w = torch.exp(z - total[..., None])
        # a score's error: 2^-19 of the summed product's size, 2^-21 of the cap's and the bias's
        err = 2.0 ** -19 * (x.abs() @ k.abs().transpose(1, 2)) * abs(scale) + 2.0 ** -21 * (softcap + bias)
        err = torch.where(see, err, 0.0).amax(-1, keepdim=True)
        # a weight is rounded to fp16 (2^-11, or 2^-25 of the largest one); V in fp16 relative to the sequence's largest scale
        dw = w * (2.0 ** -11 + 2 * err + (length + 64) * 2.0 ** -24) + 2.0 ** -24
        y = w @ v
        most = v_scale[pages].double().max()
        tol = u * y.abs() + dw @ v.abs() + 2.0 ** -24 * most + tiny
        out[a:b], out_tol[a:b] = y.transpose(0, 1), tol.transpose(0, 1)
        lse[a:b] = total.t()
        # the row's sum: n fp32 terms in any order are off by at most (n - 1) 2^-24 of the sum of their sizes, each
        # term by the exponential's 2 units and its argument's rounding: 32 * 2^-24
        lse_tol[a:b] = (err[..., 0] + (length + 32) * 2.0 ** -24 + 2.0 ** -23 * total.abs()).t()
    return out, lse, out_tol, lse_tol


def check_attend(got, q, cache, page_table, lens, starts, **kw):
    out, lse = torch.cat(got[0], 1).double(), torch.cat(got[1], 0).t().double()
    want, total, tol, lse_tol = attend(torch.cat(q, 1), cache, page_table, lens, starts, **kw)
    rows = ~total[:, 0].isnan()
    assert bool(((out - want).abs() <= tol)[rows].all()), (float((out - want).abs()[rows].max()), float(((out - want).abs() / tol)[rows].max()))
    assert bool(((lse - total).abs() <= lse_tol)[rows].all()), float((lse - total).abs()[rows].max())
    return rows
