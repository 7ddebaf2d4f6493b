"""The paged key-value cache -- append and attention over it -- against 64 bits (bounds derived in kv_util)."""
import math

import pytest
import torch

import kv_util

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def tf():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from ulysses_sequence_attention_tf_gb300 import binding, build
    build.build()
    binding.lib()
    binding.use_torch_allocator(True)
    yield binding
    torch.cuda.synchronize()
    binding.cache_clear()
    assert binding.device_status() == 0


class Setup:
    """Sequences of given lengths (new tokens among them), pages in random order, a cache with earlier content."""

    def __init__(self, tf, lens, tokens, *, P=1, H=4, Hkv=2, D=64, page=16, dtype=BF16, seed=0, front=0, behind=0, extra=3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens_, self.page, self.D, self.P, self.dtype = list(lens), page, D, P, dtype
        self.starts_ = [front]
        for t in tokens:
            self.starts_.append(self.starts_[-1] + t)
        T = self.T = self.starts_[-1] + behind
        used = [-(-n // page) for n in lens]
        self.most = max(max(used), 1) + 1
        order = torch.randperm(sum(used) + extra, generator=g, device="cuda").tolist()
        self.table_, at = [], 0
        for n in used:
            self.table_.append(order[at:at + n] + [-1] * (self.most - n))
            at += n
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.table, self.lens, self.starts = i32(self.table_), i32(self.lens_), i32(self.starts_)
        self.cache = tf.kv_cache(len(order), Hkv, page, D)
        for codes in self.cache[:2]:  # codes of any value but NaN
            codes.view(torch.uint8).random_(0, 255, generator=g)
            bad = (codes.view(torch.uint8) & 0x7f) == 0x7f
            codes.view(torch.uint8)[bad] = 0x30
        for s in self.cache[2:]:
            s.copy_(torch.exp2(torch.randint(-12, -5, s.shape, generator=g, device="cuda").float()))
        r = lambda h: [torch.randn((T, h // P, D), generator=g, device="cuda").to(dtype) for _ in range(P)]  # noqa: E731
        self.q, self.k, self.v = r(H), r(Hkv), r(Hkv)
        self.weights = [(1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(dtype) for _ in range(2)]
        self.args = (self.cache, self.table, self.lens, self.starts)

    def copy(self):
        return [t.clone() for t in self.cache]

    def append(self, tf, *, rope="interleaved", norm=True, q=True, **kw):
        before = self.copy()
        wq, wk = self.weights if norm else (None, None)
        out = tf.kv_append(*self.args, self.k, self.v, self.q if q else None, rope=rope, q_weight=wq, k_weight=wk, **kw)
        after = self.copy()
        cos_sin = kv_util.table(self.most * self.page, self.D)
        at = torch.zeros(self.T, dtype=torch.long, device="cuda")
        for n, length in enumerate(self.lens_):
            a, b = self.starts_[n], self.starts_[n + 1]
            at[a:b] = torch.arange(length - (b - a), length, device="cuda")
        k, size = kv_util.rotated(torch.cat(self.k, 1), wk, rope, cos_sin, at)
        v = torch.cat(self.v, 1).double()
        where = (self.table_, self.lens_, self.starts_)
        kv_util.check_half((before[0], before[2]), (after[0], after[2]), *where, k, size)
        kv_util.check_half((before[1], before[3]), (after[1], after[3]), *where, v, torch.zeros_like(v))
        if q:
            want, size = kv_util.rotated(torch.cat(self.q if kw.get("q_out") is not self.q else self.kept, 1), wq, rope, cos_sin, at)
            got = torch.cat(out, 1).double()
            a, b = self.starts_[0], self.starts_[-1]
            tol = torch.finfo(self.dtype).eps / 2 * want.abs() + 2.0 ** -20 * size + 2.0 ** -25
            assert bool(((got - want).abs() <= tol)[a:b].all())
        return out

    def attend(self, tf, **kw):
        got = tf.kv_attend(*self.args, self.q, **kw)
        kw = {n: x for n, x in kw.items() if n in ("scale", "softcap", "slopes", "causal")}
        kv_util.check_attend(got, self.q, self.cache, self.table_, self.lens_, self.starts_, **kw)
        return got


LAYOUTS = [([1], [1]), ([300], [1]), ([16], [16]), ([17], [16]), ([130], [130]), ([200, 31, 64, 1], [1, 1, 1, 1]),
           ([100, 0, 33, 257], [7, 0, 33, 100]), ([48, 48], [0, 48])]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("rope", ["interleaved", "neox", None])
def test_append_pages_and_rotations(tf, rope, page, D, dtype):
    for seed, (lens, tokens) in enumerate(LAYOUTS):
        Setup(tf, lens, tokens, page=page, D=D, dtype=dtype, seed=seed).append(tf, rope=rope, norm=seed % 2 == 0)


@pytest.mark.parametrize("P,H,Hkv", [(1, 1, 1), (2, 8, 4), (4, 4, 4), (8, 16, 8), (3, 18, 3)])
def test_append_groups(tf, P, H, Hkv):
    s = Setup(tf, [70, 33], [20, 33], P=P, H=H, Hkv=Hkv, seed=P)
    s.append(tf)
    s.append(tf, q=False)


def test_append_again_changes_nothing(tf):
    s = Setup(tf, [70, 33], [20, 1], seed=5)
    s.append(tf)
    once = s.copy()
    s.append(tf)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(once, s.copy()))


def test_append_token_by_token_grows_a_page_scale(tf):
    s = Setup(tf, [40], [1], page=64, D=64, Hkv=2, seed=6, extra=0)
    for n in range(1, 60):
        s.lens_ = [n]
        s.lens.fill_(n)
        for ts in (s.k, s.v):
            ts[0].copy_(torch.randn_like(ts[0], dtype=torch.float32) * 1.2 ** n)
        s.append(tf, rope=None, norm=False)
    s.attend(tf)


def test_append_values_at_the_ends_of_the_range(tf):
    s = Setup(tf, [48], [48], D=64, seed=7)
    s.v[0][:16] = 0                                   # a page of zeros
    s.v[0][16:32] *= 2.0 ** 120                       # near the type's largest values
    s.v[0][32:48] *= 2.0 ** -120                      # below the smallest scale
    s.v[0][17, 0, 3], s.v[0][18, 1, 5], s.v[0][33, 0, 0] = math.inf, -math.inf, math.nan
    s.k[0][0, 0, :] = 448 / 8                         # exactly the largest code
    s.k[0][:16, 1, :] = 449                           # just above it
    s.append(tf, rope=None, norm=False)


def test_append_strided_rows_and_rows_of_no_sequence(tf):
    s = Setup(tf, [70, 33], [20, 33], P=2, H=4, Hkv=2, front=3, behind=5, seed=8)
    wide = [torch.randn((s.T, 7, s.D), device="cuda").to(BF16) for _ in range(2)]
    s.q, s.k, s.v = [w[:, 0:2] for w in wide], [w[:, 3:4] for w in wide], [w[:, 5:6] for w in wide]
    for ts in (s.q, s.k, s.v):  # what no sequence owns may be anything
        for t in ts:
            t[:3], t[-5:] = math.nan, math.inf
    out = [torch.full((s.T, 2, s.D), 7.0, dtype=BF16, device="cuda") for _ in range(2)]
    s.append(tf, q_out=out)
    for o in out:
        assert bool((o[:3] == 7).all()) and bool((o[-5:] == 7).all())
    got = tf.kv_attend(*s.args, s.q, out)
    kv_util.check_attend(got, s.q, s.cache, s.table_, s.lens_, s.starts_)
    for o in out:
        assert bool((o[:3] == 7).all()) and bool((o[-5:] == 7).all())


def test_append_in_place_with_a_given_table(tf):
    s = Setup(tf, [70], [20], D=128, seed=9)
    s.kept = [t.clone() for t in s.q]
    s.append(tf, q_out=s.q, cos_sin=kv_util.table(s.most * s.page, 128))


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_attend_layouts(tf, causal, page, D, dtype):
    for seed, (lens, tokens) in enumerate(LAYOUTS):
        Setup(tf, lens, tokens, page=page, D=D, dtype=dtype, seed=seed).attend(tf, causal=causal)


@pytest.mark.parametrize("P,H,Hkv", [(1, 1, 1), (1, 8, 1), (2, 8, 4), (4, 4, 4), (8, 16, 8), (3, 18, 3), (1, 40, 2), (1, 96, 1)])
@pytest.mark.parametrize("tokens", [1, 5, 70])
def test_attend_groups_and_shared_heads(tf, P, H, Hkv, tokens):
    Setup(tf, [70, 333], [tokens, 1], P=P, H=H, Hkv=Hkv, seed=P, D=128).attend(tf, max_tokens=tokens)


@pytest.mark.parametrize("tokens", [1, 40])
@pytest.mark.parametrize("cap", [0.0, 3.0, 50.0])
def test_attend_capped_and_biased(tf, cap, tokens):
    s = Setup(tf, [900, 77], [tokens, 40], H=4, Hkv=2, D=64, page=32, seed=11)
    slopes = torch.tensor([0.5, 0.01, 0.0, 2.0], device="cuda")
    s.q = [4 * t for t in s.q]
    s.attend(tf, softcap=cap)
    s.attend(tf, softcap=cap, slopes=slopes, scale=0.3)
    s.attend(tf, softcap=cap, slopes=slopes, causal=False)


@pytest.mark.parametrize("tokens", [1, 3, 100])
def test_attend_long(tf, tokens):
    s = Setup(tf, [9000, 1, 4111], [tokens, 1, 1], H=8, Hkv=1, D=128, page=64, seed=12)
    s.attend(tf)
    s.attend(tf, max_tokens=tokens, max_len=9000)


def test_attend_pages_of_very_different_scales(tf):
    s = Setup(tf, [700], [5], H=4, Hkv=2, D=64, page=16, seed=13, dtype=FP16)
    for x in (s.cache.k_scale, s.cache.v_scale):
        x.copy_(torch.exp2(torch.randint(-30, -8, x.shape, device="cuda").float()))
    s.attend(tf)
    s.cache.v_scale.fill_(2.0 ** -100)  # pages of zeros
    s.cache.v.view(torch.uint8).zero_()
    out, _ = s.attend(tf)
    assert bool((out[0] == 0).all())


def test_attend_does_not_see_what_lies_behind_a_sequence(tf):
    s = Setup(tf, [70, 17], [1, 17], H=4, Hkv=2, page=32, seed=14)
    for n, length in enumerate(s.lens_):
        where, off = s.table_[n][length // 32], length % 32
        for codes in s.cache[:2]:
            codes[where][:, off:] = math.nan
    for x in s.cache[2:]:  # pages that no sequence owns
        x[[i for i in range(len(x)) if i not in sum(s.table_, [])]] = math.nan
    s.attend(tf)
    s.attend(tf, causal=False)


def test_attend_pages_shared_between_sequences(tf):
    s = Setup(tf, [70, 70], [1, 1], H=4, Hkv=2, page=32, seed=15)
    s.table_[1][:2] = s.table_[0][:2]
    s.table.copy_(torch.tensor(s.table_, dtype=torch.int32))
    s.append(tf)
    s.attend(tf)


def test_table_rows_with_a_stride(tf):
    s = Setup(tf, [70, 90], [1, 30], seed=16)
    wide = torch.full((2, s.most + 5), -1, dtype=torch.int32, device="cuda")
    wide[:, :s.most] = s.table
    s.args = (s.cache, wide[:, :s.most], s.lens, s.starts)
    s.append(tf)
    s.attend(tf)


def test_a_cache_beyond_32_bit_offsets(tf):
    s = Setup(tf, [300, 40], [2, 40], H=4, Hkv=2, D=128, page=128, seed=17)
    pages = 2 ** 32 // (2 * 128 * 128) + 40
    big = tf.kv_cache(pages, 2, 128, 128)
    moved = [p + pages - 20 if p >= 0 else p for p in sum(s.table_, [])]
    s.table_ = [moved[:s.most], moved[s.most:]]
    s.table.copy_(torch.tensor(s.table_, dtype=torch.int32))
    for a, b in zip(big, s.cache):
        a[pages - 20:pages - 20 + len(b)] = b
    tail = [t[pages - 20:] for t in big]
    s.args, s.cache = (big, *s.args[1:]), tail
    s.table_ = [[p - (pages - 20) if p >= 0 else p for p in row] for row in s.table_]
    s.append(tf)
    s.attend(tf)


def test_out_of_range_lengths_starts_and_pages_are_left_out(tf):
    def broken(change):
        s = Setup(tf, [70, 33, 20], [20, 3, 1], seed=18)
        change(s)
        before, out = s.copy(), [torch.full_like(t, 7.0) for t in s.q]
        tf.kv_append(*s.args, s.k, s.v, s.q, [t.clone() for t in out])
        assert tf.device_status(clear=True) == 8
        tf.kv_attend(*s.args, s.q, out, max_len=80)
        assert tf.device_status(clear=True) == 8
        return s, before, out

    def seq(n, value):
        return lambda s: s.lens.__setitem__(n, value)

    for n, value in ((0, 2), (0, -1), (0, 10 ** 9), (1, 2 ** 31 - 1)):
        s, before, out = broken(seq(n, value))
        a, b = s.starts_[n], s.starts_[n + 1]
        assert bool((out[0][a:b] == 7).all()) and not bool((out[0][b if n == 0 else 0:b + 3 if n == 0 else a] == 7).any())
    for value in (-5, 10 ** 6):
        s, before, out = broken(lambda s: s.starts.__setitem__(1, value))
        own = [i for i in range(len(s.cache.k)) if i not in sum(s.table_, [])]
        assert torch.equal(s.cache.k[own].view(torch.uint8), before[0][own].view(torch.uint8))
    for value in (-1, 10 ** 6):
        s, before, out = broken(lambda s: s.table.__setitem__((0, 4), value))
        assert not bool((out[0][s.starts_[1]:] == 7).any())
    s = Setup(tf, [70], [1], seed=19)  # longer than the given table
    before = s.copy()
    tf.kv_append(*s.args, s.k, s.v, cos_sin=kv_util.table(69, 64))
    assert tf.device_status(clear=True) == 8
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(before, s.copy()))
    Setup(tf, [70, 9], [3, 1], seed=20).attend(tf, max_tokens=3)
    s = Setup(tf, [70, 9], [3, 1], seed=20)
    out = [torch.full_like(t, 7.0) for t in s.q]
    tf.kv_attend(*s.args, s.q, out, max_tokens=2)
    assert tf.device_status(clear=True) == 8
    assert bool((out[0][:3] == 7).all()) and not bool((out[0][3] == 7).all())


@pytest.mark.parametrize("tokens,D,page", [(1, 64, 64), (1, 128, 16), (100, 128, 64), (100, 64, 16), (300, 128, 128)])
@pytest.mark.parametrize("missing", [(0,), (2, 3), (1, -2)])
def test_keys_of_missing_pages_are_left_out(tf, tokens, D, page, missing):
    """As if the sequence were shorter by them (without mask and bias positions do not matter)."""
    s = Setup(tf, [1000], [tokens], H=4, Hkv=2, D=D, page=page, seed=33)
    used = -(-1000 // page)
    for m in missing:
        s.table[0, m % used] = len(s.cache.k) if m % 2 else -1
    got = tf.kv_attend(*s.args, s.q, causal=False)
    assert tf.device_status(clear=True) == 8
    left = [p for i, p in enumerate(s.table_[0][:used]) if i not in {m % used for m in missing}]
    kv_util.check_attend(got, s.q, s.cache, [left], [1000 - page * len(missing)], s.starts_, causal=False)


def test_captured_and_replayed_as_the_sequences_grow(tf):
    s = Setup(tf, [60, 30, 16], [1, 1, 1], H=4, Hkv=2, page=16, seed=21)
    s.append(tf)
    torch.cuda.synchronize()
    before = s.copy()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = tf.kv_append(*s.args, s.k, s.v, s.q, q_weight=s.weights[0], k_weight=s.weights[1])
        got = tf.kv_attend(*s.args, q, max_tokens=1, max_len=80)
    for t, b in zip(s.cache, before):
        t.copy_(b)
    for step in range(3):
        s.lens_ = [n + 1 for n in s.lens_] if step else s.lens_
        s.lens.copy_(torch.tensor(s.lens_, dtype=torch.int32))
        graph.replay()
        kv_util.check_attend(got, q, s.cache, s.table_, s.lens_, s.starts_)
        # what the graph wrote is what an eager call writes
        graphed, first = s.copy(), [t.clone() for t in q]
        again = tf.kv_append(*s.args, s.k, s.v, s.q, q_weight=s.weights[0], k_weight=s.weights[1])
        assert all(torch.equal(a, b) for a, b in zip(again, first))
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(graphed, s.copy()))
        if step == 0:
            s.table_[2][1] = len(s.cache.k) - 1 if len(s.cache.k) - 1 not in sum(s.table_, []) else [
                i for i in range(len(s.cache.k)) if i not in sum(s.table_, [])][0]
            s.table_[0] = s.table_[0][:4] + [[i for i in range(len(s.cache.k)) if i not in sum(s.table_, [])][0]]
            s.table[2, 1], s.table[0, 4] = s.table_[2][1], s.table_[0][4]


@pytest.mark.parametrize("tokens", [1, 40])
def test_two_calls_at_once(tf, tokens):
    """Calls in flight on two streams, each joining chunks from a workspace of its own."""
    both = [Setup(tf, [9000, 5000 + i], [tokens, tokens], H=8, Hkv=2, D=128, page=64, seed=30 + i) for i in range(2)]
    want = [s.attend(tf) for s in both]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [tf.kv_attend(*s.args, s.q, stream=st) for s, st in zip(both, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(m, n) for a, b in zip(want, got) for x, y in zip(a, b) for m, n in zip(x, y))


REFUSED = {"cache on the CPU": dict(k=lambda t: t.cpu()), "codes of another type": dict(k=lambda t: t.view(torch.uint8)),
           "scales of another shape": dict(v_scale=lambda t: t[:, :1]), "a cache without V": dict(v=lambda t: None),
           "64-bit lengths": dict(lens=lambda t: t.long()), "starts too short": dict(starts=lambda t: t[:-1]),
           "64-bit table": dict(page_table=lambda t: t.long()), "table on the CPU": dict(page_table=lambda t: t.cpu()),
           "table by columns": dict(page_table=lambda t: t.t().contiguous().t()), "one-dimensional table": dict(page_table=lambda t: t[0])}


@pytest.mark.parametrize("how", REFUSED)
def test_refused_caches(tf, how):
    s = Setup(tf, [20, 30], [1, 1])
    names = ("k", "v", "k_scale", "v_scale", "page_table", "lens", "starts")
    x = dict(zip(names, (*s.cache, s.table, s.lens, s.starts)))
    for n, f in REFUSED[how].items():
        x[n] = f(x[n])
    args = ([x[n] for n in names[:4]], x["page_table"], x["lens"], x["starts"])
    before = s.copy()
    with pytest.raises(ValueError):
        tf.kv_attend(*args, s.q)
    with pytest.raises(ValueError):
        tf.kv_append(*args, s.k, s.v, rope=None)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(before, s.cache))


def test_refused_rows(tf):
    s = Setup(tf, [20, 30], [1, 1], H=4, Hkv=2, P=2)
    for k, v, q in ((s.k[:1], s.v, s.q), (s.k, [t.half() for t in s.v], s.q), (s.k, s.v, s.q[:1]), (s.q[0], s.v, s.q),
                    (s.k, s.v, [t[:1] for t in s.q]), ([t[:, :0] for t in s.k], s.v, s.q), (s.k, s.v, [t.float() for t in s.q])):
        with pytest.raises(ValueError):
            tf.kv_append(*s.args, k, v, q)
    for kw in (dict(q_weight=s.weights[0].float()), dict(k_weight=s.weights[1][:8]), dict(rope="other"),
               dict(cos_sin=torch.zeros((50, 64), device="cuda")), dict(q_out=s.k), dict(eps="x")):
        with pytest.raises((ValueError, TypeError)):
            tf.kv_append(*s.args, s.k, s.v, s.q, **kw)
    for kw in (dict(max_tokens=0), dict(max_tokens=3), dict(max_len=0), dict(max_len=10 ** 6), dict(softcap=-1.0), dict(eps=1)):
        with pytest.raises((ValueError, TypeError, tf.TfUlyssesError)):
            tf.kv_attend(*s.args, s.q, **kw)
    for q in ([t[..., :32] for t in s.q], [t.float() for t in s.q], s.q[:1] * 9, [s.q[0], s.q[1][:1]]):
        with pytest.raises((ValueError, tf.TfUlyssesError)):
            tf.kv_attend(*s.args, q)


def test_the_same_inputs_give_the_same_bits_on_any_stream(tf):
    s = Setup(tf, [3000, 500], [1, 9], H=8, Hkv=2, D=128, page=64, seed=22)
    want = s.attend(tf)
    torch.cuda.synchronize()
    for stream in (torch.cuda.Stream(), torch.cuda.Stream()):
        for handle in (stream, stream.cuda_stream):
            got = tf.kv_attend(*s.args, s.q, stream=handle)
            stream.synchronize()
            assert all(torch.equal(a[: s.T], b[: s.T]) for x, y in zip(want, got) for a, b in zip(x, y))


def test_streamed_chunks_agree_with_attention_over_the_whole(tf):
    """Chunks scattered, appended and attended one after another, gathered back: each token sees what it would have
    seen in one causal pass over everything."""
    from attention_util import Reference
    from ulysses_sequence_attention_tf_gb300 import synth
    P, H, D, chunk, chunks, page = 2, 4, 64, 96, 3, 32
    cache = tf.kv_cache(chunk * chunks // page, H, page, D)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    order = i32([list(range(chunk * chunks // page))[::-1]])
    cos_sin = kv_util.table(chunk * chunks, D)
    kept = {n: [] for n in "qkv"}
    for c in range(chunks):
        d = synth.move(synth.qkv_shards(P, 1, chunk // P, H, D, BF16, seed=c), "cuda:0")
        q, k, v, _ = tf.scatter_qkv("stream", d["q"], d["k"], d["v"])
        rows = lambda ts: [t.flatten(0, 1) for t in ts]  # noqa: E731
        at = (order, i32([(c + 1) * chunk]), i32([0, chunk]))
        turned = tf.kv_append(cache, *at, rows(k), rows(v), rows(q), cos_sin=cos_sin)
        out, lse = tf.kv_attend(cache, *at, turned)
        kv_util.check_attend((out, lse), turned, cache, order.tolist(), [(c + 1) * chunk], [0, chunk])
        back, _ = tf.gather_out("stream", [t[None] for t in out])
        assert torch.equal(torch.cat(back, 1)[0], torch.cat(out, 1))
        for n, ts in (("q", turned), ("k", rows(k)), ("v", rows(v))):
            kept[n].append(torch.cat(ts, 1).clone())
        last = torch.cat(out, 1).double()
    q, k, v = (torch.cat(kept[n])[None] for n in "qkv")
    k = kv_util.rotated(k[0], None, "interleaved", cos_sin, torch.arange(chunk * chunks, device="cuda"))[0][None]
    whole = Reference([q], [k], [v], causal=True).out[0].transpose(0, 1)[-chunk:]
    # e4m3 keeps 3 bits of K and V: each rounding is off by at most 2^-4, here about 2^-5.8 on average
    assert float((last - whole).norm() / whole.norm()) < 0.0625
    tf.cache_clear()
