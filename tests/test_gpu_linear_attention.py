"""Linear attention with a decay -- forward, gradients, rows of sequences -- against 64 bits (bounds derived in linear_util)."""
import pytest
import torch

from linear_util import check_rows, check_state, power, recurrence, wide

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16
LENGTHS = [1, 2, 7, 16, 17, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257, 400]


@pytest.fixture(scope="module")
def tf():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from ulysses_sequence_attention_tf_gb300 import binding, build
    build.build()
    binding.lib()
    yield binding
    torch.cuda.synchronize()
    assert binding.device_status() == 0


def decays(kind, H):
    h = torch.arange(H, device="cuda", dtype=torch.float32)
    return {"slopes": torch.exp2(-8 * (h + 1) / H), "none": 0 * h, "slow": 1e-4 * (h + 1), "fast": 3.0 + h, "mixed": (h % 2) * 100.0,
            "huge": (h % 2) * 1e30}[kind]


class Case:
    def __init__(self, B, S, H, D, *, P=1, dtype=BF16, decay="slopes", state=False, fused=False, seed=0, size=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: size * torch.randn(s, generator=g, device="cuda")  # noqa: E731
        if fused:
            pay = [r(B, S, H // P, 3 * D).to(dtype) for _ in range(P)]
            self.q, self.k, self.v = ([x[..., i * D:(i + 1) * D] for x in pay] for i in range(3))
        else:
            self.q, self.k, self.v = ([r(B, S, H // P, D).to(dtype) for _ in range(P)] for _ in range(3))
        self.dout = [r(B, S, H // P, D).to(dtype) for _ in range(P)]
        self.decay, self.scale, self.dtype = decays(decay, H), D ** -0.5, dtype
        self.state, self.dstate = (3 * r(B, H, D, D), 3 * r(B, H, D, D)) if state else (None, None)

    def forward(self, tf, **kw):
        out, last = tf.linear_attention(self.q, self.k, self.v, decay=self.decay, state=self.state, final_state=True, **kw)
        want = recurrence(wide(self.q), wide(self.k), wide(self.v), self.decay, kw.get("scale", self.scale),
                          None if self.state is None else self.state.double())
        check_rows("out", out, *want[:2], self.dtype)
        check_state("state", last, *want[2:])
        return out, last

    def backward(self, tf, scale=None, **kw):
        scale = self.scale if scale is None else scale
        got = tf.linear_attention_backward(self.dout, self.q, self.k, self.v, decay=self.decay, scale=scale, state=self.state,
                                           dstate=self.dstate, dstate_out=True, **kw)
        q, k, v, g = wide(self.q), wide(self.k), wide(self.v), wide(self.dout)
        t = lambda x: None if x is None else x.double().transpose(-1, -2)  # noqa: E731
        w = lambda x: None if x is None else x.double()  # noqa: E731
        dq = recurrence(g, v, k, self.decay, scale, t(self.state))
        dk = recurrence(v, g, q, self.decay, scale, t(self.dstate), 1.0, reverse=True)
        dv = recurrence(k, q, g, self.decay, scale, w(self.dstate), 1.0, reverse=True)
        check_rows("dq", got[0], *dq[:2], self.dtype)
        check_rows("dk", got[1], *dk[:2], self.dtype)
        check_rows("dv", got[2], *dv[:2], self.dtype)
        check_state("dstate", got[3], *dv[2:])
        return got


@pytest.mark.parametrize("S", LENGTHS)
@pytest.mark.parametrize("D,dtype", [(64, FP16), (64, BF16), (128, FP16), (128, BF16)])
def test_lengths(tf, S, D, dtype):
    c = Case(2, S, 4, D, P=2, dtype=dtype, state=S % 2 == 1, seed=S)
    c.forward(tf)
    c.backward(tf)


@pytest.mark.parametrize("decay", ["slopes", "none", "slow", "fast", "mixed"])
@pytest.mark.parametrize("S,B,H", [(150, 2, 3), (1200, 1, 2), (3000, 1, 2), (2200, 3, 8)])
@pytest.mark.parametrize("D,dtype", [(64, FP16), (128, BF16)])
def test_decays(tf, decay, S, B, H, D, dtype):
    c = Case(B, S, H, D, dtype=dtype, decay=decay, state=True, fused=True, seed=S)
    c.forward(tf)
    c.backward(tf)


@pytest.mark.parametrize("S", [5, 300, 6000])
def test_a_decay_that_leaves_a_token_alone(tf, S):
    """e^-decay is 0 for every second head: the others' rounding and their own state must not show in it."""
    c = Case(1, S, 2, 64, decay="huge", state=True)
    c.forward(tf)
    c.backward(tf)


@pytest.mark.parametrize("S", [3, 140])
def test_offsets_beyond_32_bits(tf, S):
    """Batch rows 2^31 elements apart, and a state as far into its pool."""
    c = Case(3, S, 2, 128, state=True, decay="slow")
    store, n = torch.empty(2 ** 32 + 2 ** 20, dtype=BF16, device="cuda"), S * 2 * 128

    def far(i, x=None):
        y = store.as_strided((3, S, 2, 128), (2 ** 31, 256, 128, 1), i * n)
        return [y if x is None else y.copy_(x)]

    c.q, c.k, c.v, c.dout = (far(i, x[0]) for i, x in enumerate((c.q, c.k, c.v, c.dout)))
    out, _ = c.forward(tf, out=far(4))
    assert out[0].stride(0) == 2 ** 31
    c.backward(tf, dq=far(4), dk=far(5), dv=far(6))
    del store
    states = torch.empty((70000, 2, 128, 128), dtype=torch.float32, device="cuda")
    slots = [69999, 0, 65537]
    for n, slot in enumerate(slots):
        states[slot] = c.state[n]
    rows = [[x[0].reshape(3 * S, 2, 128)] for x in (c.q, c.k, c.v)]
    starts = torch.arange(0, 3 * S + 1, S, dtype=torch.int32, device="cuda")
    tf.linear_attend(states, torch.tensor(slots, dtype=torch.int32, device="cuda"), starts, *rows, decay=c.decay, max_tokens=S)
    want = recurrence(wide(c.q), wide(c.k), wide(c.v), c.decay, c.scale, c.state.double())
    check_state("state", states[slots], *want[2:])


@pytest.mark.parametrize("B,S,H,P", [(1, 6001, 1, 1), (5, 333, 64, 8), (300, 40, 2, 1), (1, 130, 200, 1)])
def test_shapes(tf, B, S, H, P):
    c = Case(B, S, H, 64, P=P, state=True)
    c.forward(tf)
    if S < 2000:
        c.backward(tf)


@pytest.mark.parametrize("S", [3, 140])
def test_scales(tf, S):
    c = Case(1, S, 2, 64, state=True)
    for scale in (1.0, -0.3, 0.0):
        c.forward(tf, scale=scale)
        c.backward(tf, scale=scale)


@pytest.mark.parametrize("size", [2.0 ** -10, 2.0 ** -4, 60.0])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("S", [5, 300])
def test_sizes_of_fp16(tf, size, D, S):
    """Small inputs lose nothing, and large ones overflow in the result alone.  scale brings the results back to size."""
    c = Case(1, S, 2, D, dtype=FP16, state=True, size=size)
    c.forward(tf, scale=0.02 * size ** -2)
    c.backward(tf, scale=0.02 * size ** -2)


def test_gradients_against_autograd_and_differences(tf):
    c = Case(1, 200, 2, 64, state=True)
    got = c.backward(tf)
    leaves = [x.requires_grad_() for x in (wide(c.q), wide(c.k), wide(c.v), c.state.double())]
    f = lambda q, k, v, s: sum((a * b).sum() for a, b in zip(  # noqa: E731
        recurrence(q, k, v, c.decay, c.scale, s)[::2], (wide(c.dout), c.dstate.double())))
    grads = torch.autograd.grad(f(*leaves), leaves)
    u = torch.finfo(BF16).eps / 2
    for x, want in zip([wide(g) for g in got[:3]] + [got[3].double()], grads):
        assert float((x - want).norm()) <= 2 ** 0.5 * u * float(want.norm())
    with torch.no_grad():
        gen = torch.Generator(device="cuda").manual_seed(3)
        for i, x in enumerate([wide(g) for g in got[:3]] + [got[3].double()]):
            e = torch.randn(x.shape, generator=gen, device="cuda", dtype=torch.float64)
            moved = lambda h: f(*[y + h * e if j == i else y for j, y in enumerate(leaves)])  # noqa: E731
            slope = (moved(0.5) - moved(-0.5))  # f is linear in each of them
            # the error's norm times that of its projection on a random direction: 6 of its deviations
            assert abs(float(slope - (x * e).sum())) <= 6 * 2 ** 0.5 * u * float(x.norm())


def test_streaming_is_the_whole(tf):
    """Chunk after chunk from state to state, in place, is the whole sequence."""
    c = Case(2, 700, 4, 64, P=2, state=True)
    want = recurrence(wide(c.q), wide(c.k), wide(c.v), c.decay, c.scale, c.state.double())
    state, outs, at = c.state.clone(), [], 0
    for n in (1, 128, 1, 3, 200, 300, 67):
        part = [[x[:, at:at + n] for x in t] for t in (c.q, c.k, c.v)]
        out, last = tf.linear_attention(*part, decay=c.decay, state=state, final_state=state)
        assert last is state
        outs.append(out)
        at += n
    assert at == 700
    check_rows("out", [torch.cat(x, 1) for x in zip(*outs)], *want[:2], c.dtype)
    check_state("state", state, *want[2:])


def test_thousands_of_steps_do_not_add_up(tf):
    """lambda near 1, token by token: a state that has gone through 2000 calls."""
    c = Case(1, 2000, 2, 64, decay="slow")
    state = torch.zeros((1, 2, 64, 64), device="cuda")
    for i in range(2000):
        tf.linear_attention([c.q[0][:, i:i + 1]], [c.k[0][:, i:i + 1]], [c.v[0][:, i:i + 1]], decay=c.decay, state=state, final_state=state)
    want = recurrence(wide(c.q), wide(c.k), wide(c.v), c.decay, c.scale)
    check_state("state", state, *want[2:])


# ---------------------------------------------------------------- rows of sequences
class Rows:
    def __init__(self, tokens, H, D, *, P=1, dtype=BF16, front=0, behind=0, extra=2, seed=0, decay="slopes"):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.tokens, self.H, self.D, self.P, self.dtype = tokens, H, D, P, dtype
        self.at = [front]
        for t in tokens:
            self.at.append(self.at[-1] + t)
        self.T = self.at[-1] + behind
        r = lambda: [torch.randn((self.T, H // P, D), generator=g, device="cuda").to(dtype) for _ in range(P)]  # noqa: E731
        self.q, self.k, self.v = r(), r(), r()
        N = len(tokens)
        self.states = 3 * torch.randn((N + extra, H, D, D), generator=g, device="cuda")
        self.slots = torch.randperm(N + extra, generator=g, device="cuda")[:N].to(torch.int32)
        self.starts = torch.tensor(self.at, dtype=torch.int32, device="cuda")
        self.decay = decays(decay, H)

    def run(self, tf, left_out=(), **kw):
        before = self.states.clone()
        out = [torch.full_like(x, 7.0) for x in self.q]
        assert tf.linear_attend(self.states, self.slots, self.starts, self.q, self.k, self.v, out, decay=self.decay, **kw) is out
        touched = torch.zeros(self.T, dtype=torch.bool, device="cuda")
        kept = torch.ones(len(before), dtype=torch.bool, device="cuda")
        for n, t in enumerate(self.tokens):
            if n in left_out or t == 0:
                continue
            a, b, slot = self.at[n], self.at[n + 1], int(self.slots[n])
            touched[a:b], kept[slot] = True, False
            part = lambda ts: wide([x[None, a:b] for x in ts])  # noqa: E731
            want = recurrence(part(self.q), part(self.k), part(self.v), self.decay, self.D ** -0.5, before[slot][None].double())
            check_rows(f"out {n}", [x[None, a:b] for x in out], *want[:2], self.dtype, norm=b - a > 32)
            check_state(f"state {n}", self.states[slot][None], *want[2:])
        assert torch.equal(self.states[kept], before[kept]), "slots that no sequence moves"
        for x in out:
            assert bool((x[~touched] == 7.0).all()), "rows of no sequence"


@pytest.mark.parametrize("tokens", [[1], [1] * 5, [1] * 200, [2, 1, 0, 3], [0, 0], [1, 300, 0, 17, 64, 128, 129], [5] * 30, [1000, 1], [16] * 9,
                                    [33, 0, 1, 1, 90, 256, 31, 2100]])
@pytest.mark.parametrize("D,dtype", [(64, FP16), (128, BF16)])
def test_rows(tf, tokens, D, dtype):
    most = max(max(tokens), 1)
    r = Rows(tokens, 4, D, P=2, dtype=dtype, front=3, behind=most + 2)
    r.run(tf, max_tokens=most)
    r = Rows(tokens, 4, D, P=2, dtype=dtype, front=0, behind=2)
    r.run(tf)


@pytest.mark.parametrize("tokens", [[1, 2, 1], [40, 200, 129]])
def test_other_sequences_and_rows_do_not_matter(tf, tokens):
    """What lies behind a sequence's last row, or belongs to another one, may be anything."""
    r = Rows(tokens, 2, 64, front=5, behind=150)
    for x in r.q + r.k + r.v:
        x[: r.at[0]] = float("nan")
        x[r.at[-1]:] = float("inf")
        x[r.at[1]:r.at[2]] = float("nan")
    bad = int(r.slots[1])
    others = [int(r.slots[n]) for n in (0, 2)]
    before = r.states.clone()
    out = tf.linear_attend(r.states, r.slots, r.starts, r.q, r.k, r.v, decay=r.decay, max_tokens=max(tokens))
    assert bool(r.states[bad].isnan().all())
    for n in (0, 2):
        a, b, slot = r.at[n], r.at[n + 1], int(r.slots[n])
        part = lambda ts: wide([x[None, a:b] for x in ts])  # noqa: E731
        want = recurrence(part(r.q), part(r.k), part(r.v), r.decay, 64 ** -0.5, before[slot][None].double())
        check_rows("out", [x[None, a:b] for x in out], *want[:2], r.dtype, norm=False)
    assert bool(r.states[others].isfinite().all())


@pytest.mark.parametrize("long", [False, True])
def test_sequences_out_of_range_are_left_out(tf, long):
    tokens = [40, 130, 20, 7] if long else [1, 2, 1, 1]
    for what in ("slot", "negative slot", "too long", "starts"):
        r = Rows(tokens, 2, 64, behind=1)
        kw = dict(max_tokens=max(tokens))
        out_ = [1]
        if what == "slot":
            r.slots[1] = len(r.states)
        elif what == "negative slot":
            r.slots[1] = -1
        elif what == "too long":
            kw = dict(max_tokens=max(tokens) - 1)
        else:
            r.starts[4], out_ = r.T + 1, [3]
        before = r.states.clone()
        slots = r.slots.clone()
        out = [torch.full_like(x, 7.0) for x in r.q]
        tf.linear_attend(r.states, r.slots, r.starts, r.q, r.k, r.v, out, decay=r.decay, **kw)
        assert tf.device_status(clear=True) == 8
        for n in out_:
            a, b = r.at[n], r.at[n + 1]
            assert bool((out[0][a:b] == 7.0).all())
            if what in ("too long", "starts"):
                assert torch.equal(r.states[int(slots[n])], before[int(slots[n])])
        for n in range(4):
            if n not in out_:
                assert not torch.equal(r.states[int(slots[n])], before[int(slots[n])])


@pytest.mark.parametrize("most,tokens", [(1, [1, 1, 1, 1]), (300, [300, 1, 60, 200])])
def test_graphs_and_streams(tf, most, tokens):
    """A captured call follows slots, starts and states; two graphs share nothing; another stream works."""
    r = Rows(tokens, 2, 64)
    kw = dict(decay=r.decay, max_tokens=most)
    side = torch.cuda.Stream()
    eager, state = [torch.empty_like(x) for x in r.q], r.states.clone()
    side.wait_stream(torch.cuda.current_stream())
    tf.linear_attend(state, r.slots, r.starts, r.q, r.k, r.v, eager, stream=side, **kw)
    torch.cuda.current_stream().wait_stream(side)
    pool, outs, graphs = [r.states.clone(), r.states.clone()], [], []
    for p in pool:
        outs.append([torch.empty_like(x) for x in r.q])
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            tf.linear_attend(p, r.slots, r.starts, r.q, r.k, r.v, outs[-1], **kw)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for s, g in zip(streams, graphs):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    for p, o in zip(pool, outs):
        assert torch.equal(o[0], eager[0]) and torch.equal(p, state)
    # fewer sequences, others' slots, at the next replay
    r.slots.copy_(r.slots.flip(0))
    want = pool[0].clone()
    tf.linear_attend(want, r.slots, r.starts, r.q, r.k, r.v, eager, **kw)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(pool[0], want) and torch.equal(outs[0][0], eager[0])


def test_training_in_graphs(tf):
    c = Case(1, 1500, 2, 64, state=True)
    out, last = c.forward(tf)
    grads = c.backward(tf)
    new = lambda: [[torch.empty_like(x) for x in t] for t in (c.q, c.q, c.k, c.v)]  # noqa: E731
    got, states = [new(), new()], [[torch.empty_like(c.state) for _ in range(2)] for _ in range(2)]
    graphs = []
    for g, s in zip(got, states):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            tf.linear_attention(c.q, c.k, c.v, g[0], decay=c.decay, state=c.state, final_state=s[0])
            tf.linear_attention_backward(c.dout, c.q, c.k, c.v, *g[1:], decay=c.decay, state=c.state, dstate=c.dstate, dstate_out=s[1])
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for g, s in zip(got, states):  # the same inputs give the same bits
        for a, b in zip(g, (out, *grads[:3])):
            assert torch.equal(a[0], b[0])
        assert torch.equal(s[0], last) and torch.equal(s[1], grads[3])


def test_gradient_of_the_state_in_place_is_refused(tf):
    """The gradients' passes run together: one reads what another would write."""
    c = Case(2, 400, 2, 64, state=True)
    with pytest.raises(tf.TfUlyssesError):
        tf.linear_attention_backward(c.dout, c.q, c.k, c.v, decay=c.decay, state=c.state, dstate=c.dstate, dstate_out=c.dstate)


def test_empty(tf):
    c = Case(2, 0, 2, 64, state=True)
    out, last = tf.linear_attention(c.q, c.k, c.v, decay=c.decay, state=c.state, final_state=True)
    assert out[0].shape == (2, 0, 2, 64) and torch.equal(last, c.state)
    _, last = tf.linear_attention(c.q, c.k, c.v, decay=c.decay, final_state=True)
    assert not bool(last.any())
    dq, dk, dv, first = tf.linear_attention_backward(c.dout, c.q, c.k, c.v, decay=c.decay, state=c.state, dstate=c.dstate)
    assert torch.equal(first, c.dstate) and dk[0].shape == (2, 0, 2, 64)
    c = Case(0, 5, 2, 64)
    out, last = tf.linear_attention(c.q, c.k, c.v, decay=c.decay, final_state=True)
    assert out[0].shape == (0, 5, 2, 64) and last.shape == (0, 2, 64, 64)
    r = Rows([], 2, 64, behind=4)
    r.run(tf, max_tokens=2)
    r = Rows([], 2, 64)
    tf.linear_attend(r.states, r.slots, r.starts, r.q, r.k, r.v, decay=r.decay)


def test_small_results_lie_apart_and_are_ordinary_tensors(tf):
    """They may share an allocation, but no memory; one outlives the others; large ones share nothing."""
    c = Case(2, 40, 4, 64, P=2, state=True)
    out, last = tf.linear_attention(c.q, c.k, c.v, decay=c.decay, state=c.state, final_state=True)
    grads = tf.linear_attention_backward(c.dout, c.q, c.k, c.v, decay=c.decay, state=c.state, dstate=c.dstate)
    for results in ([*out, last], [*grads[0], *grads[1], *grads[2], grads[3]]):
        spans = sorted((x.data_ptr(), x.data_ptr() + x.numel() * x.element_size()) for x in results)
        assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:])) and all(a[0] % 32 == 0 for a in spans)
        assert all(x.is_contiguous() and x.is_leaf and not x.requires_grad and not x.is_inference() for x in results)
    kept, copy = last, last.clone()
    x = out[1].requires_grad_()
    (x.float() * 2).sum().backward()
    assert bool((x.grad == 2).all()) and x._version == 0
    out[0].add_(1)
    assert x._version == 0 and out[0]._version == 1
    del out, x, grads
    torch.full((1 << 20,), float("nan"), device="cuda")
    assert torch.equal(kept, copy)
    with torch.inference_mode():
        out, last = tf.linear_attention(c.q, c.k, c.v, decay=c.decay, state=c.state, final_state=True)
        assert out[0].is_inference() and torch.equal(last, kept)
    c = Case(1, 2100, 4, 128, P=2)
    out, last = tf.linear_attention(c.q, c.k, c.v, decay=c.decay, final_state=True)
    assert len({x.untyped_storage().data_ptr() for x in (*out, last)}) == 3


def test_what_is_not_asked_for(tf):
    c = Case(1, 300, 2, 64)
    out, last = tf.linear_attention(c.q, c.k, c.v, decay=c.decay)
    assert last is None
    # a call that hands out no state may keep fewer parts of the keys: the same bounds, not the same bits
    check_rows("out", out, *recurrence(wide(c.q), wide(c.k), wide(c.v), c.decay, c.scale)[:2], c.dtype)
    dq, dk, dv, first = tf.linear_attention_backward(c.dout, c.q, c.k, c.v, decay=c.decay)
    assert first is None


def test_the_operators_in_a_run(tf):
    """Two steps of generation: the plan's rows are rotated at its positions, go through the paged cache and through
    the states of a linear layer beside it."""
    H, D, page, N = 4, 64, 16, 3
    gen = torch.Generator(device="cuda").manual_seed(1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table, lens, free, span = torch.zeros((N, 8), dtype=torch.int32, device="cuda"), i32([0] * N), i32(list(range(23, -1, -1))), i32([0, 24])
    cache, states, slots = tf.kv_cache(24, H, page, D), torch.zeros((N, H, D, D), device="cuda"), i32([2, 0, 1])
    decay = decays("slopes", H)
    past = [[[] for _ in range(N)] for _ in range(3)]
    for new in ([40, 1, 17], [1, 20, 1]):
        T = sum(new)
        plan = tf.kv_plan(table, lens, i32(new), free, span, page_size=page, rows=T)
        q, k, v = ([torch.randn((T, H, D), generator=gen, device="cuda").to(BF16)] for _ in range(3))
        q, k = tf.rope(q, k, positions=plan.positions, rotary_dim=32)
        where = (table, plan.lens, plan.starts)
        tf.kv_append(cache, *where, k, v, rope=None)
        out, _ = tf.kv_attend(cache, *where, q, max_tokens=max(new))
        fades = tf.linear_attend(states, slots, plan.starts, q, k, v, decay=decay, max_tokens=max(new))
        at = 0
        for n, t in enumerate(new):
            for keep, x in zip(past, (q, k, v)):
                keep[n].append(x[0][at:at + t])
            Q, K, V = (wide([torch.cat(keep[n])[None]]) for keep in past)
            size = Q.shape[2]
            x = Q[:, :, size - t:] @ K.transpose(-1, -2) * D ** -0.5
            seen = torch.arange(size, device="cuda") <= torch.arange(size - t, size, device="cuda")[:, None]
            soft = torch.where(seen, x, -float("inf")).softmax(-1) @ V
            # keys and values in e4m3 (2^-4 each, independent), as the cache's own tests bound them closely
            assert float((wide([out[0][None, at:at + t]]) - soft).norm()) <= 2.0 ** -3 * float(soft.norm())
            want, a, _, _ = recurrence(Q, K, V, decay, D ** -0.5)
            check_rows("fades", [fades[0][None, at:at + t]], want[:, :, size - t:], a[:, :, size - t:], BF16, norm=False)
            at += t
        # every row's slot holds its key
        codes = cache.k.float() * cache.k_scale[..., None, None]
        kept = codes.permute(0, 2, 1, 3).reshape(-1, H, D)[plan.slots.long()].double()
        assert float((kept - k[0].double()).norm()) <= 2.0 ** -4 * float(k[0].double().norm())
        lens, span = plan.lens, plan.span
    assert lens.tolist() == [41, 21, 18] and span.tolist() == [7, 17]


def test_refusals(tf):
    c = Case(1, 4, 2, 64, state=True)
    r = Rows([1, 2], 2, 64)
    kw = dict(decay=c.decay)
    for bad in (dict(decay=None), dict(decay=c.decay[:1]), dict(decay=c.decay.double()), dict(decay=c.decay.cpu()), dict(state=c.state[0]),
                dict(state=c.state.half()), dict(final_state=c.state[:, :1]), dict(out=c.q[:0]), dict(out=[c.q[0].half()])):
        with pytest.raises(ValueError):
            tf.linear_attention(c.q, c.k, c.v, **{**kw, **bad})
    for q, k, v in ((c.q[0], c.k, c.v), (c.q, [c.k[0][:, :3]], c.v), (c.q, c.k, [c.v[0].half()]), ([c.q[0].float()], c.k, c.v),
                    ([c.q[0][0]], [c.k[0][0]], [c.v[0][0]]), ([c.q[0].cpu()], c.k, c.v)):
        with pytest.raises(ValueError):
            tf.linear_attention(q, k, v, **kw)
    for bad in (dict(dstate=c.state[0]), dict(dq=[c.q[0][:, :2]]), dict(dstate_out=c.state.double())):
        with pytest.raises(ValueError):
            tf.linear_attention_backward(c.dout, c.q, c.k, c.v, **kw, **bad)
    args = [r.states, r.slots, r.starts, r.q, r.k, r.v]
    for i, x in ((0, r.states[0]), (0, r.states.half()), (0, r.states[:, :1]), (1, r.slots.long()), (1, r.slots[:1]), (2, r.starts[1:]), (2, None),
                 (3, [r.q[0][None]])):
        with pytest.raises(ValueError):
            tf.linear_attend(*[x if j == i else a for j, a in enumerate(args)], decay=r.decay)
    for bad in (dict(max_tokens=0), dict(max_tokens=r.T + 1)):
        with pytest.raises(tf.TfUlyssesError):
            tf.linear_attend(*args, decay=r.decay, **bad)
    with pytest.raises(tf.TfUlyssesError):
        tf.linear_attention(c.q, c.k, c.v, decay=c.decay, scale=float("nan"))
    assert float(power(c.decay, torch.zeros(1, device="cuda")).max()) == 1.0
