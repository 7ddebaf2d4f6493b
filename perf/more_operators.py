"""What rotary positions, linear attention and the page plan of a cache compute, in plain torch, and the cases they are
measured on.

* ``rotary``: heads of Q and K rotated at given positions -- pairs (2i, 2i + 1) or (i, i + R/2) of the first R elements
  of a head, by ``position * frequency[i]``, times a magnitude; the rest of the head is copied.  The inverse rotation
  gives the gradient.
* ``linear``: attention without a softmax over P head groups ``[B, S, H/P, D]``, a decay for each head: with
  ``S_t = e^-decay S_(t-1) + k_t^T v_t`` the output is ``scale * q_t S_t``.  Its state is ``[B, H, D, D]``.
* ``training``: the same and the gradients of Q, K, V and of the state in front.
* ``attend``: each sequence's newest tokens (rows ``[T, H/P, D]``) through the states of a pool, which move on.
* ``plan``: for the requests of a paged cache, from their lengths and how many tokens each one gets: the pages they
  take from a ring of free ones and the pages that ended requests give back, the new lengths, the first row of each
  request, and every row's position and slot in the cache.

``own`` chooses between the plain forms and the library's calls.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- cases
def _rotary(name, *, groups=1, batch=0, tokens, heads, kv_heads=None, dim, rotary=None, type, rope="interleaved",
            scaling="none", factor=1.0, far=0, inverse=False):
    """batch 0: rows [T, heads, D] of as many sequences, each at a position of its own up to `far`."""
    return dict(name=name, op="rotary", groups=groups, batch=batch, tokens=tokens, heads=heads,
                kv_heads=heads if kv_heads is None else kv_heads, dim=dim, rotary=rotary or dim, type=type, rope=rope,
                scaling=scaling, factor=factor, far=far, inverse=inverse)


def _linear(name, op, *, groups=1, batch=1, tokens, mixed=False, heads, dim, type, decay=1.0, state=False, fused=False):
    """attend: `batch` sequences of up to `tokens` new tokens."""
    return dict(name=name, op=op, groups=groups, batch=batch, tokens=tokens, mixed=mixed, heads=heads, dim=dim, type=type,
                decay=decay, state=state, fused=fused)


def _plan(name, *, seqs, tokens, mixed=False, length, page, ended=0, spare=8):
    """Every `ended`-th request has ended (0: none); `spare` pages more than are needed (fewer, where negative)."""
    return dict(name=name, op="plan", batch=seqs, tokens=tokens, mixed=mixed, length=length, page=page, ended=ended, spare=spare)


def listed():
    return [
        # one new token for each of a few long sequences, half of the head rotated, frequencies stretched for a long context
        _rotary("rotary tokens", tokens=24, heads=16, kv_heads=4, dim=128, rotary=64, type="bf16", rope="neox",
                scaling="parts", factor=16.0, far=65536),
        # the gradient with respect to Q and K in front of the rotation, at the portfolio's odd length
        _rotary("rotary gradient", groups=2, batch=2, tokens=6001, heads=12, dim=64, rotary=32, type="fp16", rope="neox",
                inverse=True),
        # the video DiT: all 40 heads in four groups, far into a stream
        _rotary("rotary video", groups=4, batch=1, tokens=32760, heads=40, dim=128, type="bf16", scaling="linear",
                factor=4.0, far=100000),
        # the smallest workload of this library (P=2, S=256, H=8, D=64): latency of one short call
        _linear("linear short", "linear", groups=2, tokens=256, heads=8, dim=64, type="fp16"),
        # the video DiT: 40 heads in four groups, read from the fused [B, S, H/P, 3*D] payloads
        _linear("linear video", "linear", groups=4, tokens=32760, heads=40, dim=128, type="bf16", fused=True),
        # training on short sequences that go on from a state
        _linear("training short", "training", groups=2, batch=2, tokens=251, heads=8, dim=64, type="fp16", state=True),
        # a long video in training, half the video DiT's tokens, one head group of P = 8: few heads, long sequences
        _linear("training video", "training", tokens=16380, heads=5, dim=128, type="bf16", decay=0.25),
        # one new token of one sequence: latency
        _linear("token", "attend", tokens=1, heads=8, dim=64, type="fp16"),
        # one new token for each of many sequences: the states go through once
        _linear("tokens", "attend", batch=64, tokens=1, heads=32, dim=128, type="bf16"),
        # prompts of unequal length
        _linear("prompts", "attend", groups=2, batch=16, tokens=2000, mixed=True, heads=16, dim=128, type="bf16"),
        # one new token for each of many requests: latency
        _plan("plan tokens", seqs=64, tokens=1, length=8192, page=64),
        # many requests at once, some with whole prompts, some ended
        _plan("plan prompts", seqs=512, tokens=256, mixed=True, length=4096, page=16, ended=9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "linear", "training", "attend", "plan"])
    dim, type = rng.choice([64, 128]), rng.choice(["bf16", "fp16"])
    groups = rng.choice([1, 2])
    if op == "plan":
        seqs, tokens = _log(rng, 1, 1024), rng.choice([1, _log(rng, 1, 2000)])
        c = _plan("", seqs=seqs, tokens=max(1, min(tokens, 200000 // seqs)), mixed=rng.random() < 0.6, length=_log(rng, 1, 16384),
                  page=rng.choice([16, 32, 64, 128]), ended=rng.choice([0, 0, 2, 5, 13]), spare=rng.choice([0, 8, 100, -1, -3]))
    elif op == "rotary":
        kv = groups * rng.randint(1, 8)
        heads = kv * rng.choice([1, 1, 2, 4])
        rows = rng.random() < 0.4
        tokens = _log(rng, 1, 4096 if rows else 60000 * 8 // heads)
        rotary = rng.choice([dim, dim, dim // 2, dim // 4, rng.randint(1, dim // 2) * 2])
        c = _rotary("", groups=groups, batch=0 if rows else 1 if tokens > 4000 else rng.choice([1, 2, 3]), tokens=tokens, heads=heads,
                    kv_heads=kv, dim=dim, rotary=rotary, type=type, rope=rng.choice(["interleaved", "neox"]),
                    scaling=rng.choice(["none", "linear", "parts"]), factor=rng.choice([2.0, 4.0, 16.0]),
                    far=_log(rng, 1, 1000000), inverse=rng.random() < 0.3)
    elif op == "attend":
        seqs = _log(rng, 1, 64)
        heads = groups * rng.randint(1, 16)
        tokens = rng.choice([1, 1, rng.randint(2, 16), _log(rng, 1, max(2, 60000 // (seqs * heads)))])
        c = _linear("", op, groups=groups, batch=seqs, tokens=tokens, mixed=rng.random() < 0.6, heads=heads, dim=dim, type=type,
                    decay=rng.choice([1.0, 0.1, 0.01, 0.0]))
    else:
        heads = groups * rng.randint(1, 10)
        tokens = _log(rng, 1, (300000 if op == "linear" else 80000) // heads)
        c = _linear("", op, groups=groups, batch=1 if tokens * heads > 20000 else rng.choice([1, 2, 3]), tokens=tokens, heads=heads,
                    dim=dim, type=type, decay=rng.choice([1.0, 0.1, 0.01, 0.0]), state=rng.random() < 0.5, fused=rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------- what a case's layout says (no random numbers)
def _tokens(c):
    """New tokens of each sequence."""
    if c["op"] == "plan":
        every = [1 + (37 * i) % c["tokens"] if c["mixed"] and i % 3 == 0 else 1 if c["mixed"] else c["tokens"] for i in range(c["batch"])]
        return [-1 if c["ended"] and i % c["ended"] == c["ended"] - 1 else t for i, t in enumerate(every)]
    return [1 + (11 * i + c["tokens"] - 1) % c["tokens"] if c["mixed"] else c["tokens"] for i in range(c["batch"])]


def _lengths(c):
    """plan: cached tokens of each request; some have none yet."""
    return [0 if c["mixed"] and i % 3 == 0 else c["length"] * ((41 * i + 7) % c["batch"] + 1) // c["batch"] for i in range(c["batch"])]


def _pages(c):
    """plan: pages that each request has, and pages that it takes."""
    up = lambda n: -(-n // c["page"])  # noqa: E731
    had = [up(n) for n in _lengths(c)]
    return had, [up(n + t) - h if t > 0 else 0 for n, t, h in zip(_lengths(c), _tokens(c), had)]


def work(case):
    c = case
    if c["op"] == "rotary":
        elements = (c["batch"] or 1) * c["tokens"] * (c["heads"] + c["kv_heads"])
        return {"bytes": 4 * elements * c["dim"], "flops": 3 * elements * c["rotary"]}
    if c["op"] == "plan":
        had, taken = _pages(c)
        rows = sum(max(0, t) for t in _tokens(c))
        given = sum(h for h, t in zip(had, _tokens(c)) if t < 0)
        return {"bytes": 16 * c["batch"] + 8 * rows + 8 * (sum(taken) + given), "flops": 0}
    d, rows = c["dim"], sum(_tokens(c)) if c["op"] == "attend" else c["batch"] * c["tokens"]
    tensor, state = 2 * rows * c["heads"] * d, 4 * c["batch"] * c["heads"] * d * d
    # two products with the state a token, the least that the recurrence allows
    step = 4 * rows * c["heads"] * d * d
    if c["op"] == "attend":
        return {"bytes": 4 * tensor + 2 * state, "flops": step}
    if c["op"] == "linear":
        return {"bytes": 4 * tensor + (2 * state if c["state"] else 0), "flops": step}
    return {"bytes": 8 * tensor + (3 * state if c["state"] else 0), "flops": 7 * step // 2}


# ---------------------------------------------------------------- inputs
def _frequencies(c):
    """Angle of one position for each pair, in 64 bits."""
    i = torch.arange(c["rotary"] // 2, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / c["rotary"])
    if c["scaling"] == "linear":
        return f / c["factor"]
    if c["scaling"] == "parts":  # pairs that turn often in the trained length keep their frequency, slow ones are stretched
        turns = 4096.0 * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        return f * (keep + (1 - keep) / c["factor"])
    return f


def _rows(gen, *shape, type):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(type)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    state = {"case": c}
    if c["op"] == "plan":
        had, taken = _pages(c)
        pages = max(1, sum(had) + max(0, sum(taken) + c["spare"]))
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        most = max(max(h + t for h, t in zip(had, taken)), 1)
        n, at = torch.tensor(had, device="cuda"), torch.arange(most, device="cuda")
        first = torch.cumsum(n, 0) - n
        state["page_table"] = torch.where(at < n[:, None], order[(first[:, None] + at).clamp(max=pages - 1)], 0).to(torch.int32)
        state["lens"], state["new"] = ints(_lengths(c)), ints(_tokens(c))
        head = int(torch.randint(0, pages, (), generator=gen, device="cuda"))
        state["free"] = torch.roll(order, head - sum(had))  # the first free page at the ring's head
        state["span"] = ints([head, pages - sum(had)])
        state["rows"] = sum(max(0, t) for t in _tokens(c))
        return state
    type, dim, groups = TYPES[c["type"]], c["dim"], c["groups"]
    hl = c["heads"] // groups
    if c["op"] == "rotary":
        lead = (c["batch"], c["tokens"]) if c["batch"] else (c["tokens"],)
        state["q"] = [_rows(gen, *lead, hl, dim, type=type) for _ in range(groups)]
        state["k"] = [_rows(gen, *lead, c["kv_heads"] // groups, dim, type=type) for _ in range(groups)]
        state["frequencies"] = _frequencies(c)
        state["magnitude"] = 0.1 * math.log(c["factor"]) + 1.0 if c["scaling"] == "parts" else 1.0
        state["positions"] = None
        if not c["batch"]:
            state["positions"] = torch.randint(0, c["far"] + 1, lead, generator=gen, device="cuda", dtype=torch.int32)
        return state
    lead = (sum(_tokens(c)),) if c["op"] == "attend" else (c["batch"], c["tokens"])
    if c["fused"]:
        payload = [_rows(gen, *lead, hl, 3 * dim, type=type) for _ in range(groups)]
        state["q"], state["k"], state["v"] = ([x[..., i * dim:(i + 1) * dim] for x in payload] for i in range(3))
    else:
        state["q"], state["k"], state["v"] = ([_rows(gen, *lead, hl, dim, type=type) for _ in range(groups)] for _ in range(3))
    heads = torch.arange(c["heads"], device="cuda", dtype=torch.float32)
    state["decay"] = c["decay"] * torch.exp2(-8.0 * (heads + 1) / c["heads"])
    state["scale"] = 1.0 / math.sqrt(dim)
    past = lambda n: 4.0 * torch.randn((n, c["heads"], dim, dim), generator=gen, device="cuda")  # noqa: E731
    if c["op"] == "attend":
        t = _tokens(c)
        state["states"] = past(c["batch"] + 2)
        state["slots"] = torch.randperm(c["batch"] + 2, generator=gen, device="cuda")[:c["batch"]].to(torch.int32)
        state["starts"] = torch.tensor([sum(t[:i]) for i in range(len(t) + 1)], dtype=torch.int32, device="cuda")
        state["max_tokens"] = max(t)
        return state
    state["state"] = past(c["batch"]) if c["state"] else None
    if c["op"] == "training":
        state["dout"] = [_rows(gen, *lead, hl, dim, type=type) for _ in range(groups)]
        state["dstate"] = past(c["batch"]) / 4 if c["state"] else None
    return state


# ---------------------------------------------------------------- plain forms
def _plain_rotary(s):
    c = s["case"]
    if s["positions"] is not None:
        at = s["positions"]
    else:
        at = torch.arange(c["tokens"], device="cuda") + c["far"]
    angle = at.double()[..., None] * s["frequencies"].cuda()
    cos, sin = (angle.cos() * s["magnitude"]).float(), (angle.sin() * s["magnitude"]).float()
    if c["inverse"]:
        sin = -sin
    cos, sin = cos[..., None, :], sin[..., None, :]

    def turned(x):
        y = x[..., :c["rotary"]].float()
        if c["rope"] == "neox":
            a, b = y.chunk(2, -1)
            y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        else:
            a, b = y[..., 0::2], y[..., 1::2]
            y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        return torch.cat([y.to(x.dtype), x[..., c["rotary"]:]], -1)

    return {"q": list(map(turned, s["q"])), "k": list(map(turned, s["k"]))}


def _power(decay, n):
    """e^(-decay n) in 32 bits, [H, ...] for n [...]; 0 where n < 0."""
    x = decay.double().view(-1, *[1] * n.dim()) * n
    return torch.where(n >= 0, torch.exp(-x.clamp(min=0)), torch.zeros_like(x)).float()


def _scan(q, k, v, decay):
    """Outputs (unscaled) and last states of [B, H, S, D] from empty states, chunk by chunk: products inside a chunk,
    and the chunks' states joined by one product with the powers of the decay."""
    size = min(128, q.shape[2])
    pad = -q.shape[2] % size  # in front: zeros there change nothing
    q, k, v = (torch.nn.functional.pad(x, (0, 0, pad, 0)).unflatten(2, (-1, size)) for x in (q, k, v))
    at, chunk = torch.arange(size, device=q.device), torch.arange(q.shape[2] + 1, device=q.device)
    inside = torch.matmul(torch.matmul(q, k.transpose(-1, -2)).mul_(_power(decay, at[:, None] - at)[:, None]), v)
    add = torch.matmul((k * _power(decay, size - 1 - at)[:, None, :, None]).transpose(-1, -2), v)
    carry = _power(decay, (chunk[:, None] - chunk[:-1] - 1) * size)  # [H, chunks + 1, chunks]
    states = torch.matmul(carry, add.flatten(-2)).unflatten(-1, (q.shape[-1], -1))
    inside += torch.matmul(q * _power(decay, at + 1)[:, None, :, None], states[:, :, :-1])
    return inside.flatten(2, 3)[:, :, pad:], states[:, :, -1]


def _heads(groups):
    """P groups [B, S, h, D] as one float32 [B, H, S, D]."""
    return torch.cat(groups, 2).float().transpose(1, 2)


def _plain_linear(s):
    c = s["case"]
    type, decay, scale = s["q"][0].dtype, s["decay"], s["scale"]
    q, k, v = _heads(s["q"]), _heads(s["k"]), _heads(s["v"])
    split = lambda y: list(y.transpose(1, 2).to(type).chunk(c["groups"], 2))  # noqa: E731
    steps = torch.arange(c["tokens"], device="cuda")
    since = _power(decay, steps + 1)[..., None]  # of the state in front, at each token
    whole = _power(decay, torch.tensor(c["tokens"], device="cuda"))[:, None, None] if s["state"] is not None else None
    out, last = _scan(q, k, v, decay)
    if s["state"] is not None:
        out = out + torch.matmul(q * since, s["state"])
        last = last + whole * s["state"]
    found = {"out": split(out * scale), "state": last if c["state"] else None}
    if c["op"] == "training":
        dout = _heads(s["dout"]) * scale
        back = lambda *x: [y.flip(2) for y in x]  # noqa: E731
        dq = _scan(dout, v, k, decay)[0]
        dk = _scan(*back(v, dout, q), decay)[0].flip(2)
        dv, first = _scan(*back(k, q, dout), decay)
        dv = dv.flip(2)
        if s["state"] is not None:
            after = _power(decay, c["tokens"] - 1 - steps)[..., None]
            dq = dq + torch.matmul(dout * since, s["state"].transpose(-1, -2))
            dk = dk + torch.matmul(v * after, s["dstate"].transpose(-1, -2))
            dv = dv + torch.matmul(k * after, s["dstate"])
            first = _power(decay, torch.tensor(1, device="cuda"))[:, None, None] * first + whole * s["dstate"]
        found |= {"dq": split(dq), "dk": split(dk), "dv": split(dv), "dstate": first if c["state"] else None}
    return {n: x for n, x in found.items() if x is not None}


def _plain_attend(s):
    c = s["case"]
    decay, most, slots = s["decay"], s["max_tokens"], s["slots"].long()
    q = torch.cat(s["q"], 1)
    starts = s["starts"].long()
    at = torch.arange(len(q), device="cuda")
    seq = torch.searchsorted(starts[1:].contiguous(), at, right=True)
    step = at - starts[seq]
    place = most - (starts[1:] - starts[:-1])[seq] + step  # sequences end together

    def padded(groups):
        x = torch.zeros((c["batch"], most, c["heads"], c["dim"]), device="cuda")
        x[seq, place] = torch.cat(groups, 1).float()
        return x.transpose(1, 2)

    out, last = _scan(padded(s["q"]), padded(s["k"]), padded(s["v"]), decay)
    past = s["states"][slots]
    count = (starts[1:] - starts[:-1])
    since = torch.arange(1 - most, 1, device="cuda") + count[:, None]  # tokens up to this one, [N, most]
    kept = _power(decay, since).transpose(0, 1)[..., None]
    out = out + torch.matmul(padded(s["q"]) * kept, past)
    s["states"][slots] = last + _power(decay, count).transpose(0, 1)[..., None, None] * past
    rows = (out.transpose(1, 2)[seq, place] * s["scale"]).to(q.dtype)
    return {"out": list(rows.chunk(c["groups"], 1)), "states": s["states"]}


def _plain_plan(s):
    c = s["case"]
    page, rows, table, free = c["page"], s["rows"], s["page_table"].long(), s["free"].long()
    lens, new, most, ring = s["lens"].long(), s["new"].long(), s["page_table"].shape[1], len(s["free"])
    head, count = s["span"].long().unbind(0)
    up = lambda n: (n + page - 1) // page  # noqa: E731
    had = up(lens)
    fits = (new >= 0) & (lens >= 0) & (lens + new <= most * page)
    tokens = torch.where(fits, new, 0)
    need = torch.where(fits, up(lens + tokens) - had, 0)
    granted = fits & (torch.cumsum(need, 0) <= count) & (torch.cumsum(tokens, 0) <= rows)
    tokens, need = torch.where(granted, tokens, 0), torch.where(granted, need, 0)
    given = torch.where(new < 0, had, 0)
    before = lambda n: torch.nn.functional.pad(torch.cumsum(n, 0), (1, 0))  # noqa: E731
    starts, taken, back = before(tokens), before(need), before(given)
    # new pages of each request, in the order of the ring
    col = torch.arange(most, device="cuda") - had[:, None]
    rank = (head + taken[:-1, None] + col) % ring
    table = torch.where((col >= 0) & (col < need[:, None]), free[rank], table)
    # pages of ended requests behind the free ones
    rank = (torch.arange(ring, device="cuda") - head - count) % ring
    of = torch.searchsorted(back[1:].contiguous(), rank, right=True).clamp(max=len(lens) - 1)
    free = torch.where(rank < back[-1], table[of, (rank - back[of]).clamp(0, most - 1)], free)
    # rows
    at = torch.arange(rows, device="cuda")
    seq = torch.searchsorted(starts[1:].contiguous(), at, right=True).clamp(max=len(lens) - 1)
    used = at < starts[-1]
    position = torch.where(used, lens[seq] + at - starts[seq], 0)
    slot = torch.where(used, table[seq, (position // page).clamp(max=most - 1)] * page + position % page, -1)
    s["page_table"].copy_(table)
    s["free"].copy_(free)
    span = torch.stack([(head + taken[-1]) % ring, count - taken[-1] + back[-1]])
    whole = lambda x: x.to(torch.int32)  # noqa: E731
    return {"page_table": s["page_table"], "free": s["free"], "lens": whole(torch.where(new < 0, 0, lens + tokens)),
            "starts": whole(starts), "positions": whole(position), "slots": whole(slot), "span": whole(span)}


# ---------------------------------------------------------------- one pass
def run(state):
    s, c = state, state["case"]
    if own:
        from ulysses_sequence_attention_tf_gb300 import binding
        if c["op"] == "rotary":
            q, k = binding.rope(s["q"], s["k"], positions=s["positions"], first=c["far"], frequencies=s["frequencies"],
                                magnitude=s["magnitude"], rope=c["rope"], inverse=c["inverse"])
            return {"q": q, "k": k}
        if c["op"] == "attend":
            out = binding.linear_attend(s["states"], s["slots"], s["starts"], s["q"], s["k"], s["v"], decay=s["decay"],
                                        scale=s["scale"], max_tokens=s["max_tokens"])
            return {"out": out, "states": s["states"]}
        if c["op"] == "plan":
            p = binding.kv_plan(s["page_table"], s["lens"], s["new"], s["free"], s["span"], page_size=c["page"], rows=s["rows"])
            return {"page_table": s["page_table"], "free": s["free"], "lens": p.lens, "starts": p.starts,
                    "positions": p.positions, "slots": p.slots, "span": p.span}
        kw = dict(decay=s["decay"], scale=s["scale"], state=s["state"])
        out, last = binding.linear_attention(s["q"], s["k"], s["v"], final_state=c["state"], **kw)
        found = {"out": out, "state": last}
        if c["op"] == "training":
            dq, dk, dv, first = binding.linear_attention_backward(s["dout"], s["q"], s["k"], s["v"], dstate=s["dstate"], **kw)
            found |= {"dq": dq, "dk": dk, "dv": dv, "dstate": first}
        return {n: x for n, x in found.items() if x is not None}
    if c["op"] == "rotary":
        return _plain_rotary(s)
    if c["op"] == "attend":
        return _plain_attend(s)
    if c["op"] == "plan":
        return _plain_plan(s)
    return _plain_linear(s)


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_rotary(s, c):
    f = s["frequencies"].cuda()
    at = s["positions"].double() if s["positions"] is not None else torch.arange(c["tokens"], device="cuda").double() + c["far"]
    turn = torch.polar(torch.full_like(at[..., None] * f, s["magnitude"]), at[..., None] * f)[..., None, :]
    if c["inverse"]:
        turn = turn.conj()
    half = torch.arange(c["rotary"] // 2, device="cuda")
    first, second = (half, half + len(half)) if c["rope"] == "neox" else (2 * half, 2 * half + 1)

    def turned(x):
        x = x.double()
        z = torch.complex(x[..., first], x[..., second]) * turn
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    return {"q": [turned(x) for x in s["q"]], "k": [turned(x) for x in s["k"]]}


def _exact_steps(q, k, v, decay, scale, state):
    """[B, S, H, D] in 64 bits, a few tokens at a time: every pair of them, and the state so far."""
    out, step = [], 256
    rate = decay.double()
    for lo in range(0, q.shape[1], step):
        x, y, z = (t[:, lo:lo + step] for t in (q, k, v))
        i = torch.arange(x.shape[1], device=q.device, dtype=torch.float64)
        gone = i[:, None] - i
        weight = torch.exp(-rate[:, None, None] * gone.clamp(min=0)) * (gone >= 0)
        o = torch.einsum("bhij,bjhe->bihe", torch.einsum("bihd,bjhd->bhij", x, y) * weight, z)
        o = o + torch.einsum("bihd,hi,bhde->bihe", x, torch.exp(-rate[:, None] * (i + 1)), state)
        out.append(scale * o)
        left = torch.exp(-rate[:, None] * (len(i) - 1 - i))
        state = torch.exp(-rate * len(i))[:, None, None] * state + torch.einsum("bjhd,hj,bjhe->bhde", y, left, z)
    return torch.cat(out, 1), state


def _exact_linear(s, c):
    wide = lambda groups: torch.cat([g.double() for g in groups], 2)  # noqa: E731
    split = lambda y: list(torch.chunk(y, c["groups"], 2))  # noqa: E731
    empty = torch.zeros((c["batch"], c["heads"], c["dim"], c["dim"]), dtype=torch.float64, device="cuda")
    leaves = [wide(s["q"]), wide(s["k"]), wide(s["v"]), s["state"].double() if c["state"] else empty]
    if c["op"] == "linear":
        out, last = _exact_steps(*leaves[:3], s["decay"], s["scale"], leaves[3])
        return {"out": split(out), "state": last} if c["state"] else {"out": split(out)}
    with torch.enable_grad():
        leaves = [x.requires_grad_() for x in leaves]
        out, last = _exact_steps(*leaves[:3], s["decay"], s["scale"], leaves[3])
        dlast = s["dstate"].double() if c["state"] else empty.detach() * 0
        dq, dk, dv, first = torch.autograd.grad([out, last], leaves, [wide(s["dout"]), dlast])
    found = {"out": split(out.detach()), "state": last.detach(), "dq": split(dq), "dk": split(dk), "dv": split(dv), "dstate": first}
    return found if c["state"] else {n: x for n, x in found.items() if "state" not in n}


def _exact_attend(s, c):
    q, k, v = (torch.cat([g.double() for g in s[n]], 1) for n in "qkv")
    states, out, starts = s["states"].double(), torch.zeros_like(q), s["starts"].tolist()
    for n, slot in enumerate(s["slots"].tolist()):
        a, b = starts[n], starts[n + 1]
        o, last = _exact_steps(q[None, a:b], k[None, a:b], v[None, a:b], s["decay"], s["scale"], states[slot][None])
        out[a:b], states[slot] = o[0], last[0]
    return {"out": list(out.chunk(c["groups"], 1)), "states": states}


def _exact_plan(s, c):
    page, table, free = c["page"], s["page_table"].tolist(), s["free"].tolist()
    lens, new, (head, count) = s["lens"].tolist(), s["new"].tolist(), s["span"].tolist()
    starts, positions, slots, after = [0], [], [], list(lens)
    pages, full = 0, False
    for n, (length, more) in enumerate(zip(lens, new)):
        if more >= 0 and not full:
            need = -(-(length + more) // page) - -(-length // page)
            full = pages + need > count or len(positions) + more > s["rows"]
        if more >= 0 and not full:
            for x in range(need):
                table[n][-(-length // page) + x] = free[(head + pages + x) % len(free)]
            pages += need
            for at in range(length, length + more):
                positions.append(at)
                slots.append(table[n][at // page] * page + at % page)
            after[n] += more
        starts.append(len(positions))
    behind = head + count
    for n, (length, more) in enumerate(zip(lens, new)):
        if more < 0:
            for x in range(-(-length // page)):
                free[behind % len(free)] = table[n][x]
                behind += 1
            after[n] = 0
    fill = s["rows"] - len(positions)
    span = [(head + pages) % len(free), behind - head - pages]
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"page_table": ints(table), "free": ints(free), "lens": ints(after), "starts": ints(starts),
            "positions": ints(positions + [0] * fill), "slots": ints(slots + [-1] * fill), "span": ints(span)}


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"] == "rotary":
            return _exact_rotary(s, case)
        if case["op"] == "attend":
            return _exact_attend(s, case)
        if case["op"] == "plan":
            return _exact_plan(s, case)
        return _exact_linear(s, case)
