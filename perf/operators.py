"""What the attention and key-value cache operators compute, in plain torch, and the cases they are measured on.

The operators work on what the scatter of this library produces: P head groups,
each a ``[B, S, H/P, D]`` tensor.

* ``attention``: scores ``scale * q.k``, optionally capped by ``cap * tanh(x / cap)``,
  plus ``-slope[h] * |position distance|``, under a causal, prefix and document
  mask; the weighted sum of V and the log-sum-exp of every row.  Query i of S_q
  stands at position i + S_k - S_q.
* ``training``: the same forward pass and the gradients of Q, K and V.
* ``append``: new rows of K and V (Q beside them) normalised and rotated at their
  sequence positions; K and V go into a paged cache of 8-bit values (e4m3) with
  one power-of-two scale for each page and head.
* ``attend``: attention of each sequence's newest tokens over that cache.

``own`` chooses between the plain forms and the library's calls.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3_MAX = 448.0
LEAST_EXPONENT = -100  # the scale of a page whose values are all zero is 2^-100
EPS = 1e-6


# ---------------------------------------------------------------- cases
def _attention(name, op, *, groups=1, batch=1, q_len, k_len=None, heads, kv_heads=None, dim, type, softcap=0.0,
               alibi=False, causal=False, prefix=0, docs=0, pad=0, fused=False):
    return dict(name=name, op=op, groups=groups, batch=batch, q_len=q_len, k_len=k_len or q_len, heads=heads,
                kv_heads=kv_heads or heads, dim=dim, type=type, softcap=softcap, alibi=alibi, causal=causal,
                prefix=prefix, docs=docs, pad=pad, fused=fused)


def _cache(name, op, *, groups=1, seqs, length, ragged=False, tokens=1, mixed=False, heads, kv_heads=None, dim, page,
           type, rope="interleaved", norm=True, softcap=0.0, alibi=False, causal=True):
    return dict(name=name, op=op, groups=groups, seqs=seqs, length=length, ragged=ragged, tokens=tokens, mixed=mixed,
                heads=heads, kv_heads=kv_heads or heads, dim=dim, page=page, type=type, rope=rope, norm=norm,
                softcap=softcap, alibi=alibi, causal=causal)


def listed():
    return [
        # the smallest workload of this library (P=2, S=256, H=8, D=64): latency of one short call
        _attention("attention short", "attention", groups=2, q_len=256, heads=8, dim=64, type="fp16", softcap=30.0),
        # packed image prompts of unequal length with padding behind them, at the FLUX-like shape, read from
        # the fused [B, S, H/P, 3*D] payloads
        _attention("attention packed", "attention", groups=4, q_len=4096, heads=24, dim=128, type="bf16", docs=5,
                   pad=100, fused=True),
        # one head group of the video DiT at P = 8: every token sees every token, scores capped
        _attention("attention video", "attention", q_len=32760, heads=5, dim=128, type="bf16", softcap=50.0),
        # training on short causal sequences behind a shared prefix, shared key-value heads
        _attention("training short", "training", groups=2, batch=2, q_len=251, heads=8, kv_heads=4, dim=64, type="fp16",
                   causal=True, prefix=70),
        # the portfolio's odd length with distances as a bias
        _attention("training distance", "training", groups=2, batch=2, q_len=6001, heads=12, dim=64, type="bf16",
                   causal=True, alibi=True),
        # a long video in training: half the video DiT's tokens, one head group of P = 8
        _attention("training video", "training", q_len=16380, heads=5, dim=128, type="bf16"),
        # one new token for each of a few sequences
        _cache("append tokens", "append", seqs=8, length=700, ragged=True, heads=8, kv_heads=8, dim=128, page=16,
               type="bf16"),
        # three latent frames (30 x 52 tokens each) of a streamed video behind earlier ones, all 40 heads in 4 groups
        _cache("append frames", "append", groups=4, seqs=1, length=32760, tokens=4680, heads=40, dim=128, page=64,
               type="bf16"),
        # one new token over a short cache: latency
        _cache("attend short", "attend", seqs=1, length=300, heads=8, kv_heads=8, dim=64, page=16, type="fp16"),
        # many sequences of unequal length, one new token each, eight query heads to a key-value head
        _cache("attend batch", "attend", seqs=64, length=8192, ragged=True, heads=32, kv_heads=4, dim=128, page=64,
               type="bf16", softcap=50.0),
        # one latent frame against the whole streamed video; the tokens of a frame see one another
        _cache("attend frame", "attend", groups=4, seqs=1, length=32760, tokens=1560, heads=40, dim=128, page=64,
               type="bf16", causal=False),
        # one new token for each of many long sequences
        _cache("attend long", "attend", seqs=24, length=65536, ragged=True, heads=16, kv_heads=4, dim=128, page=128,
               type="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "training", "append", "attend"])
    dim, type = rng.choice([64, 128]), rng.choice(["bf16", "fp16"])
    shared = rng.choice([1, 1, 2, 4])
    groups = rng.choice([1, 2])
    kv_heads = groups * rng.randint(1, 4)
    heads = kv_heads * shared
    softcap, alibi = rng.choice([0.0, 0.0, 20.0, 50.0]), rng.random() < 0.3
    if op in ("attention", "training"):
        most = 24000 if op == "attention" else 12000  # the listed ones have five heads
        q_len = _log(rng, 1, max(2, int(most * math.sqrt(5 / heads))))
        mask = rng.choice(["none", "causal", "prefix", "docs", "causal docs", "long"])
        docs = rng.randint(1, 8) if "docs" in mask else 0
        c = _attention("", op, groups=groups, batch=rng.choice([1, 1, 2]) if q_len * heads < 20000 else 1, q_len=q_len,
                       k_len=q_len + _log(rng, 1, 2000) if mask == "long" else None, heads=heads, kv_heads=kv_heads,
                       dim=dim, type=type, softcap=softcap, alibi=alibi, causal=mask in ("causal", "prefix", "causal docs", "long"),
                       prefix=rng.randint(1, q_len) if mask == "prefix" else 0, docs=docs,
                       pad=rng.randint(0, q_len // 4) if docs else 0, fused=shared == 1 and rng.random() < 0.5)
    else:
        seqs = _log(rng, 1, 64)
        tokens = rng.choice([1, 1, _log(rng, 1, 1500 if seqs < 8 else 64)])
        length = tokens + _log(rng, 1, max(2, (60000 if op == "attend" else 200000) // seqs))
        c = _cache("", op, groups=groups, seqs=seqs, length=length, ragged=rng.random() < 0.7, tokens=tokens,
                   mixed=rng.random() < 0.5, heads=heads, kv_heads=kv_heads, dim=dim, page=rng.choice([16, 32, 64, 128]),
                   type=type, rope=rng.choice(["interleaved", "neox"]), norm=rng.random() < 0.7, softcap=softcap,
                   alibi=alibi, causal=rng.random() < 0.7)
    del c["name"]
    return c


# ---------------------------------------------------------------- what a case's layout says (no random numbers)
def _doc_lengths(c, b):
    """Unequal document lengths that fill a row up to its padding."""
    n, room = c["docs"], c["q_len"] - c["pad"]
    weights = [1 + (7 * i + 3 * b) % 5 for i in range(n)]
    ends = [round(room * sum(weights[: i + 1]) / sum(weights)) for i in range(n)]
    return [e - s for s, e in zip([0] + ends, ends)]


def _prefixes(c):
    return [max(0, c["prefix"] - 17 * b) for b in range(c["batch"])]


def _tokens(c):
    """New tokens of each sequence."""
    return [1 + (5 * i + c["tokens"] - 1) % c["tokens"] if c["mixed"] else c["tokens"] for i in range(c["seqs"])]


def _lengths(c):
    """Length of each sequence, its new tokens among them."""
    return [max(t, c["length"] * ((37 * i + c["seqs"] - 1) % c["seqs"] + 1) // c["seqs"] if c["ragged"] else c["length"])
            for i, t in enumerate(_tokens(c))]


def _pairs(c):
    """Visible (query, key) pairs of one head over the batch, and the rows of K that some query sees."""
    if c["op"] in ("attention", "training"):
        sq, sk = c["q_len"], c["k_len"]
        if c["docs"]:
            lens = [n for b in range(c["batch"]) for n in _doc_lengths(c, b)]
            return sum(n * (n + 1) // 2 if c["causal"] else n * n for n in lens)
        if not c["causal"]:
            return c["batch"] * sq * sk
        first = sk - sq
        return sum(sum(max(p, min(sk, first + i + 1), 0) for i in range(sq)) for p in _prefixes(c))
    return sum(t * (n - t) + t * (t + 1) // 2 if c["causal"] else t * n for t, n in zip(_tokens(c), _lengths(c)))


def work(case):
    c = case
    if c["op"] in ("attention", "training"):
        q, kv = c["batch"] * c["q_len"] * c["heads"] * c["dim"] * 2, c["batch"] * c["k_len"] * c["kv_heads"] * c["dim"] * 2
        lse = c["batch"] * c["q_len"] * c["heads"] * 4
        product = 2 * c["dim"] * _pairs(c) * c["heads"]
        if c["op"] == "attention":
            return {"bytes": 2 * q + 2 * kv + lse, "flops": 2 * product}
        return {"bytes": 4 * q + 4 * kv, "flops": 7 * product}
    rows = sum(_tokens(c))
    q, kv = rows * c["heads"] * c["dim"] * 2, rows * c["kv_heads"] * c["dim"]
    if c["op"] == "append":
        return {"bytes": 2 * q + 2 * 3 * kv + rows * c["dim"] * 4, "flops": 10 * rows * c["dim"] * (c["heads"] + c["kv_heads"])}
    cached = sum(_lengths(c)) * c["kv_heads"] * c["dim"]
    return {"bytes": 2 * cached + 2 * q + rows * c["heads"] * 4, "flops": 4 * c["dim"] * _pairs(c) * c["heads"]}


# ---------------------------------------------------------------- inputs
def _rows(gen, *shape, type):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(type)


def _slopes(heads):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)], device="cuda")


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    type, dim, groups = TYPES[c["type"]], c["dim"], c["groups"]
    hq, hk = c["heads"] // groups, c["kv_heads"] // groups
    state = {"case": c, "scale": 1.0 / math.sqrt(dim), "slopes": _slopes(c["heads"]) if c["alibi"] else None}
    if c["op"] in ("attention", "training"):
        batch, sq, sk = c["batch"], c["q_len"], c["k_len"]
        if c["fused"]:
            payload = [_rows(gen, batch, sq, hq, 3 * dim, type=type) for _ in range(groups)]
            state["q"], state["k"], state["v"] = ([x[..., i * dim:(i + 1) * dim] for x in payload] for i in range(3))
        else:
            state["q"] = [_rows(gen, batch, sq, hq, dim, type=type) for _ in range(groups)]
            state["k"] = [_rows(gen, batch, sk, hk, dim, type=type) for _ in range(groups)]
            state["v"] = [_rows(gen, batch, sk, hk, dim, type=type) for _ in range(groups)]
        if c["op"] == "training":
            state["dout"] = [_rows(gen, batch, sq, hq, dim, type=type) for _ in range(groups)]
        state["prefix"] = state["docs"] = None
        if c["prefix"]:
            state["prefix"] = torch.tensor(_prefixes(c), dtype=torch.int32, device="cuda")
        if c["docs"]:
            state["docs"] = torch.tensor(
                [[i for i, n in enumerate(_doc_lengths(c, b)) for _ in range(n)] + [-1] * c["pad"] for b in range(batch)],
                dtype=torch.int32, device="cuda")
        return state
    tokens, lengths, page = _tokens(c), _lengths(c), c["page"]
    most = -(-max(lengths) // page)
    used = [-(-n // page) for n in lengths]
    pages = sum(used) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    # a table row: the sequence's pages, then zeros
    n, at = torch.tensor(used, device="cuda"), torch.arange(most, device="cuda")
    first = torch.cumsum(n, 0) - n
    state["page_table"] = torch.where(at < n[:, None], order[(first[:, None] + at).clamp(max=pages - 1)], 0).to(torch.int32)
    state["lens"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    state["starts"] = torch.tensor([sum(tokens[:i]) for i in range(len(tokens) + 1)], dtype=torch.int32, device="cuda")
    state["max_tokens"], state["max_len"] = max(tokens), max(lengths)
    # what earlier calls left in the cache: values of a page within its scale, pages of different magnitude
    state["cache"] = []
    for _ in range(2):
        size = 2.0 ** -torch.randint(0, 3, (pages, c["kv_heads"]), generator=gen, device="cuda").float()
        codes = torch.randn((pages, c["kv_heads"], page, dim), generator=gen, device="cuda").mul_(64).clamp_(-448, 448)
        state["cache"] += [codes.to(torch.float8_e4m3fn), size / 64]
        del codes
    rows = sum(tokens)
    state["q"] = [_rows(gen, rows, hq, dim, type=type) for _ in range(groups)]
    if c["op"] == "append":
        state["k"] = [_rows(gen, rows, hk, dim, type=type) for _ in range(groups)]
        state["v"] = [_rows(gen, rows, hk, dim, type=type) for _ in range(groups)]
        state["weights"] = [(1 + 0.1 * torch.randn(dim, generator=gen, device="cuda")).to(type) for _ in range(2)] if c["norm"] else [None, None]
        angle = torch.arange(most * page, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(dim // 2, device="cuda", dtype=torch.float64) * 2 / dim)
        state["cos_sin"] = torch.stack([angle.cos(), angle.sin()], -1).float()
    return state


# ---------------------------------------------------------------- plain forms
def _visible(s, c, device):
    """[B, 1, S_q, S_k] truth values, or None where everything is visible."""
    sq, sk = c["q_len"], c["k_len"]
    keys = torch.arange(sk, device=device)
    seen = None
    if c["causal"]:
        seen = keys <= (torch.arange(sq, device=device) + (sk - sq))[:, None]
        seen = (seen | (keys < s["prefix"][:, None, None])) if s["prefix"] is not None else seen[None]
    if s["docs"] is not None:
        same = (s["docs"][:, :, None] == s["docs"][:, None, :]) & (s["docs"] >= 0)[:, :, None]
        seen = same if seen is None else seen & same
    return None if seen is None else seen[:, None]


def _softmax(x):
    """Weights before their division, their sums and the log-sum-exp of the last axis of x, which is overwritten."""
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    return p, total, (top + total.log()).squeeze(-1)


def _heads(groups):
    """P groups [B, S, h, D] as one float32 [B, H, S, D]."""
    return torch.cat(groups, 2).float().transpose(1, 2)


def _plain_attention(s, training):
    c = s["case"]
    type, shared = s["q"][0].dtype, c["heads"] // c["kv_heads"]
    q, k, v = _heads(s["q"]), _heads(s["k"]), _heads(s["v"])
    k, v = k.repeat_interleave(shared, 1), v.repeat_interleave(shared, 1)
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])
    slope = None
    if c["softcap"]:
        x.div_(c["softcap"]).tanh_()
        if training:
            slope = 1 - x * x
        x.mul_(c["softcap"])
    if s["slopes"] is not None:
        far = (torch.arange(c["q_len"], device=x.device) + (c["k_len"] - c["q_len"]))[:, None] - torch.arange(c["k_len"], device=x.device)
        x.sub_(s["slopes"][:, None, None] * far.abs())
    seen = _visible(s, c, x.device)
    if seen is not None:
        x.masked_fill_(~seen, -math.inf)
    p, total, lse = _softmax(x)
    p.div_(torch.where(total == 0, torch.ones_like(total), total))
    split = lambda y: list(y.transpose(1, 2).to(type).chunk(c["groups"], 2))  # noqa: E731
    out = torch.matmul(p, v)
    if not training:
        return {"out": split(out), "lse": list(lse.chunk(c["groups"], 1))}
    dout = _heads(s["dout"])
    dv = torch.matmul(p.transpose(-1, -2), dout)
    dx = torch.matmul(dout, v.transpose(-1, -2))
    dx.sub_((dout * out).sum(-1, keepdim=True)).mul_(p)
    if slope is not None:
        dx.mul_(slope)
    dx.mul_(s["scale"])
    dq, dk = torch.matmul(dx, k), torch.matmul(dx.transpose(-1, -2), q)
    joined = lambda y: y.unflatten(1, (-1, shared)).sum(2)  # noqa: E731
    return {"out": split(out), "dq": split(dq), "dk": split(joined(dk)), "dv": split(joined(dv))}


def _positions(s, rows):
    """Sequence and position of each new row."""
    at = torch.arange(rows, device="cuda")
    seq = torch.searchsorted(s["starts"][1:].contiguous(), at.to(torch.int32), right=True)
    new = s["starts"][1:] - s["starts"][:-1]
    return seq, s["lens"][seq].long() - new[seq] + at - s["starts"][seq]


def _rotated(x, weight, rope, angles):
    """[rows, heads, D] normalised (where there is a weight) and rotated, in float32."""
    x = x.float()
    if weight is not None:
        mean = x.double().square().mean(-1, keepdim=True).float()
        x = x * (1 / torch.sqrt(mean + EPS)) * weight.float()
    cos, sin = angles[:, None, :, 0], angles[:, None, :, 1]
    if rope == "neox":
        a, b = x.chunk(2, -1)
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)


def _exponent(most):
    """The least e with most <= 448 * 2^e, at least LEAST_EXPONENT."""
    part, e = torch.frexp(most)
    e = torch.where(part <= 0.875, e - 9, e - 8)
    return torch.where(most > 0, e, torch.full_like(e, LEAST_EXPONENT)).clamp(min=LEAST_EXPONENT)


def _store(s, x, codes, scales, seq, at):
    """Float32 rows [rows, heads, D] into one half of the cache, in place."""
    page = s["case"]["page"]
    where = s["page_table"][seq, at // page].long()
    pages, row_of = torch.unique(where, return_inverse=True)
    most = torch.zeros((len(pages), x.shape[1]), device=x.device)
    most.scatter_reduce_(0, row_of[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
    first = torch.full((len(pages),), page, device=x.device)  # the first new token of each page
    first.scatter_reduce_(0, row_of, at % page, "amin")
    old = scales[pages]
    new = torch.ldexp(torch.ones_like(most), _exponent(most))
    new = torch.where((first > 0)[:, None], torch.maximum(old, new), new)
    kept = codes[pages].float() * (old / new)[..., None, None]
    before = (torch.arange(page, device=x.device) < first[:, None])[:, None, :, None]
    codes[pages] = torch.where(before, kept, codes[pages].float()).to(codes.dtype)
    scales[pages] = new
    codes[where, :, at % page] = (x / new[row_of][..., None]).to(codes.dtype)


def _plain_append(s):
    c = s["case"]
    q, k, v = (torch.cat(s[n], 1) for n in "qkv")
    seq, at = _positions(s, len(q))
    angles = s["cos_sin"][at]
    k_codes, k_scale, v_codes, v_scale = s["cache"]
    _store(s, _rotated(k, s["weights"][1], c["rope"], angles), k_codes, k_scale, seq, at)
    _store(s, v.float(), v_codes, v_scale, seq, at)
    out = _rotated(q, s["weights"][0], c["rope"], angles).to(q.dtype)
    return {"q": list(out.chunk(c["groups"], 1)), "k": k_codes, "k_scale": k_scale, "v": v_codes, "v_scale": v_scale}


def _plain_attend(s):
    c = s["case"]
    shared, page = c["heads"] // c["kv_heads"], c["page"]
    q = torch.cat(s["q"], 1)
    k_codes, k_scale, v_codes, v_scale = s["cache"]
    seq, at = _positions(s, len(q))
    # queries by sequence, padded: [N, T, H, D]
    new = s["starts"][1:] - s["starts"][:-1]
    slot = torch.arange(len(q), device="cuda") - s["starts"][seq]
    padded = torch.zeros((c["seqs"], s["max_tokens"], c["heads"], c["dim"]), device="cuda")
    padded[seq, slot] = q.float()
    table = s["page_table"].long()
    values = lambda codes, scale: (codes[table].float() * scale[table][..., None, None]).transpose(1, 2).flatten(2, 3)  # noqa: E731
    k, v = values(k_codes, k_scale), values(v_codes, v_scale)  # [N, Hkv, L, D]
    x = torch.matmul(padded.unflatten(2, (-1, shared)).permute(0, 2, 3, 1, 4).flatten(2, 3), k.transpose(-1, -2)).mul_(s["scale"])
    x = x.unflatten(2, (shared, -1))  # [N, Hkv, shared, T, L]
    if c["softcap"]:
        x.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    keys = torch.arange(k.shape[2], device="cuda")
    stands = (s["lens"] - new)[:, None] + torch.arange(s["max_tokens"], device="cuda")  # [N, T]
    far = stands[:, :, None] - keys
    if s["slopes"] is not None:
        x.sub_(s["slopes"].unflatten(0, (-1, shared))[:, :, None, None] * far.abs()[:, None, None])
    seen = keys < s["lens"][:, None, None]
    if c["causal"]:
        seen = seen & (far >= 0)
    x.masked_fill_(~seen[:, None, None], -math.inf)
    p, total, lse = _softmax(x)
    out = torch.matmul(p.flatten(2, 3), v).unflatten(2, (shared, -1)).div_(torch.where(total == 0, torch.ones_like(total), total))
    rows = out.permute(0, 3, 1, 2, 4).flatten(2, 3)[seq, slot].to(q.dtype)
    lse = lse.permute(0, 3, 1, 2).flatten(2, 3)[seq, slot].t()
    return {"out": list(rows.chunk(c["groups"], 1)), "lse": list(lse.chunk(c["groups"], 0))}


# ---------------------------------------------------------------- one pass
def run(state):
    s, c = state, state["case"]
    if own:
        from ulysses_sequence_attention_tf_gb300 import binding
        if c["op"] in ("attention", "training"):
            kw = dict(scale=s["scale"], softcap=c["softcap"], slopes=s["slopes"], causal=c["causal"], prefix=s["prefix"],
                      q_docs=s["docs"], k_docs=s["docs"])
            out, lse = binding.attention(s["q"], s["k"], s["v"], **kw)
            if c["op"] == "attention":
                return {"out": out, "lse": lse}
            dq, dk, dv = binding.attention_backward(s["dout"], s["q"], s["k"], s["v"], out, lse, **kw)
            return {"out": out, "dq": dq, "dk": dk, "dv": dv}
        k_codes, k_scale, v_codes, v_scale = s["cache"]
        cache = binding.PagedCache(k_codes, v_codes, k_scale, v_scale)
        if c["op"] == "append":
            q = binding.kv_append(cache, s["page_table"], s["lens"], s["starts"], s["k"], s["v"], s["q"],
                                  q_weight=s["weights"][0], k_weight=s["weights"][1], eps=EPS, cos_sin=s["cos_sin"],
                                  rope=c["rope"])
            return {"q": q, "k": k_codes, "k_scale": k_scale, "v": v_codes, "v_scale": v_scale}
        out, lse = binding.kv_attend(cache, s["page_table"], s["lens"], s["starts"], s["q"], max_tokens=s["max_tokens"],
                                     max_len=s["max_len"], scale=s["scale"], softcap=c["softcap"], slopes=s["slopes"],
                                     causal=c["causal"])
        return {"out": out, "lse": lse}
    if c["op"] == "append":
        return _plain_append(s)
    if c["op"] == "attend":
        return _plain_attend(s)
    return _plain_attention(s, c["op"] == "training")


# ---------------------------------------------------------------- the definition in 64 bits, head by head
def _exact_head(q, k, v, dout, scale, cap, bias, see):
    """One head, float64: q [n, D], k and v [m, D]; bias(i, j) and see(i, j) take index vectors [n, 1] and [1, m]."""
    out, lse = torch.empty_like(q), torch.empty(len(q), dtype=q.dtype, device=q.device)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    j = torch.arange(len(k), device=q.device)[None]
    step = max(1, (1 << 27) // max(1, len(k)))
    for lo in range(0, len(q), step):
        i = torch.arange(lo, min(lo + step, len(q)), device=q.device)[:, None]
        t = torch.einsum("id,jd->ij", q[lo:lo + step], k) * scale
        if cap:
            t = torch.tanh(t / cap)
        x = (t * cap if cap else t) + bias(i, j)
        x = torch.where(see(i, j), x, torch.tensor(-math.inf, dtype=x.dtype, device=x.device))
        z = torch.logsumexp(x, 1)
        w = torch.where(see(i, j), torch.exp(x - torch.where(z == -math.inf, torch.zeros_like(z), z)[:, None]), torch.zeros_like(x))
        lse[lo:lo + step] = z
        out[lo:lo + step] = w @ v
        if dout is not None:
            g = dout[lo:lo + step]
            dv += w.T @ g
            dw = g @ v.T
            ds = w * (dw - (w * dw).sum(1, keepdim=True)) * scale
            if cap:
                ds = ds * (1 - t.square())
            dq[lo:lo + step] = ds @ k
            dk += ds.T @ q[lo:lo + step]
    return out, lse, dq, dk, dv


def _exact_attention(s, c):
    training, shared = c["op"] == "training", c["heads"] // c["kv_heads"]
    wide = lambda groups: torch.cat([g.double() for g in groups], 2)  # noqa: E731
    q, k, v = wide(s["q"]), wide(s["k"]), wide(s["v"])
    dout = wide(s["dout"]) if training else None
    out, dq, dk, dv = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    lse = torch.zeros((c["batch"], c["heads"], c["q_len"]), dtype=torch.float64, device=q.device)
    ahead = c["k_len"] - c["q_len"]
    for b in range(c["batch"]):
        prefix = int(s["prefix"][b]) if s["prefix"] is not None else 0
        docs = s["docs"][b] if s["docs"] is not None else None

        def see(i, j):
            ok = (j <= i + ahead) | (j < prefix) if c["causal"] else (i >= 0) & (j >= 0)
            return ok if docs is None else ok & (docs[i] == docs[j]) & (docs[i] >= 0)

        for h in range(c["heads"]):
            m = float(s["slopes"][h]) if s["slopes"] is not None else 0.0
            g = h // shared
            o, z, a, e, f = _exact_head(q[b, :, h], k[b, :, g], v[b, :, g], dout[b, :, h] if training else None, s["scale"],
                                        c["softcap"], lambda i, j: -m * (i + ahead - j).abs().double(), see)
            out[b, :, h], lse[b, h], dq[b, :, h] = o, z, a
            dk[b, :, g] += e
            dv[b, :, g] += f
    split = lambda y, axis: list(torch.chunk(y, c["groups"], axis))  # noqa: E731
    if not training:
        return {"out": split(out, 2), "lse": split(lse, 1)}
    return {"out": split(out, 2), "dq": split(dq, 2), "dk": split(dk, 2), "dv": split(dv, 2)}


def _exact_rotated(x, weight, rope, cos, sin):
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * weight.double()
    half = x.shape[-1] // 2
    i = torch.arange(half, device=x.device)
    first, second = (i, i + half) if rope == "neox" else (2 * i, 2 * i + 1)
    y = torch.empty_like(x)
    y[..., first] = x[..., first] * cos - x[..., second] * sin
    y[..., second] = x[..., first] * sin + x[..., second] * cos
    return y


def _exact_append(s, c):
    tokens, lengths, page = _tokens(c), _lengths(c), c["page"]
    at = torch.tensor([n - t + i for n, t in zip(lengths, tokens) for i in range(t)], device="cuda")
    cos, sin = s["cos_sin"].double()[at].unbind(-1)
    cos, sin = cos[:, None], sin[:, None]
    q, k, v = (torch.cat(s[n], 1) for n in "qkv")
    new = [_exact_rotated(k, s["weights"][1], c["rope"], cos, sin), v.double()]
    table = s["page_table"].tolist()
    start, done = 0, []
    state = [x.double() if x.dtype != torch.float8_e4m3fn else x.float().double() for x in s["cache"]]
    for n, (t, length) in enumerate(zip(tokens, lengths)):
        lo = length - t
        while lo < length:
            hi = min(length, (lo // page + 1) * page)
            done.append((table[n][lo // page], lo % page, start, start + hi - lo))
            start, lo = start + hi - lo, hi
    for rows, (codes, scales) in zip(new, (state[:2], state[2:])):
        for where, off, a, b in done:
            most = rows[a:b].abs().amax((0, 2))
            e = torch.ceil(torch.log2(most / E4M3_MAX)).clamp(min=LEAST_EXPONENT)
            scale = torch.exp2(e)
            if off:
                scale = torch.maximum(scale, scales[where])
                codes[where, :, :off] = (codes[where, :, :off] * (scales[where] / scale)[:, None, None]).float().to(torch.float8_e4m3fn).float().double()
            scales[where] = scale
            codes[where, :, off:off + b - a] = (rows[a:b].transpose(0, 1) / scale[:, None, None]).float().to(torch.float8_e4m3fn).float().double()
    out = _exact_rotated(q, s["weights"][0], c["rope"], cos, sin)
    return {"q": list(out.chunk(c["groups"], 1)), "k": state[0], "k_scale": state[1], "v": state[2], "v_scale": state[3]}


def _exact_attend(s, c):
    tokens, lengths, page, shared = _tokens(c), _lengths(c), c["page"], c["heads"] // c["kv_heads"]
    q = torch.cat(s["q"], 1).double()
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    table, start = s["page_table"].tolist(), 0
    for n, (t, length) in enumerate(zip(tokens, lengths)):
        pages = table[n][: -(-length // page)]
        half = lambda codes, scale: (codes[pages].float().double() * scale[pages].double()[..., None, None]).transpose(0, 1).flatten(1, 2)[:, :length]  # noqa: E731
        k, v = half(s["cache"][0], s["cache"][1]), half(s["cache"][2], s["cache"][3])
        see = lambda i, j: j <= i + (length - t) if c["causal"] else (i >= 0) & (j >= 0)  # noqa: E731
        for h in range(c["heads"]):
            m = float(s["slopes"][h]) if s["slopes"] is not None else 0.0
            o, z, *_ = _exact_head(q[start:start + t, h], k[h // shared], v[h // shared], None, s["scale"], c["softcap"],
                                   lambda i, j: -m * (i + (length - t) - j).abs().double(), see)
            out[start:start + t, h], lse[start:start + t, h] = o, z
        start += t
    return {"out": list(out.chunk(c["groups"], 1)), "lse": list(lse.t().chunk(c["groups"], 0))}


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"] == "append":
            return _exact_append(s, case)
        if case["op"] == "attend":
            return _exact_attend(s, case)
        return _exact_attention(s, case)
