"""Attention over the head groups and its gradient against 64 bits (bounds derived in attention_util)."""
import math

import pytest
import torch

from attention_util import Reference

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


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


def make(P, B, Sq, Sk, Hl, Hkl, D, dtype, seed, fused=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    if fused:
        pay = [r(B, Sq, Hl, 3 * D) for _ in range(P)]
        q, k, v = ([x[..., i * D:(i + 1) * D] for x in pay] for i in range(3))
    else:
        q = [r(B, Sq, Hl, D) for _ in range(P)]
        k = [r(B, Sk, Hkl, D) for _ in range(P)]
        v = [r(B, Sk, Hkl, D) for _ in range(P)]
    return q, k, v, [r(B, Sq, Hl, D) for _ in range(P)]


def both(tf, q, k, v, dout, **kw):
    out, lse = tf.attention(q, k, v, **kw)
    dq, dk, dv = tf.attention_backward(dout, q, k, v, out, lse, **kw)
    ref = Reference(q, k, v, dout, **kw)
    for name, got in (("out", out), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        ref.check(name, got)
    return out, lse, dq, dk, dv


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Sq,Sk", [(1, 1), (1, 300), (300, 1), (127, 129), (128, 128), (256, 384), (257, 255), (700, 513)])
def test_sizes(tf, Sq, Sk, D, dtype):
    both(tf, *make(1, 1, Sq, Sk, 2, 2, D, dtype, Sq + Sk))


@pytest.mark.parametrize("P,B,Hl,Hkl", [(1, 1, 1, 1), (2, 3, 4, 1), (4, 1, 6, 2), (8, 2, 1, 1), (3, 2, 5, 5)])
@pytest.mark.parametrize("causal", [False, True])
def test_groups_and_shared_heads(tf, P, B, Hl, Hkl, causal):
    both(tf, *make(P, B, 200, 200, Hl, Hkl, 64, BF16, P + B), causal=causal)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Sq,Sk", [(1, 1), (130, 130), (300, 300), (100, 400), (400, 100), (513, 770)])
def test_causal_with_and_without_prefix(tf, Sq, Sk, D):
    x = make(2, 2, Sq, Sk, 2, 1, D, FP16, 3)
    both(tf, *x, causal=True)  # Sq > Sk: the first rows see nothing
    for pre in ([0, 1], [Sk // 2, Sk + 50], [Sk, 129]):
        both(tf, *x, causal=True, prefix=torch.tensor(pre, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("cap", [0.5, 5.0, 50.0])
def test_capped_scores(tf, cap, dtype):
    q, k, v, dout = make(1, 2, 200, 333, 2, 2, 128, dtype, 7)
    both(tf, [4 * t for t in q], k, v, dout, softcap=cap)
    both(tf, q, k, v, dout, softcap=cap, scale=0.01)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_distance_bias(tf, cap, causal):
    x = make(2, 1, 300, 450, 2, 2, 64, BF16, 9)
    slopes = torch.tensor([0.5, 0.01, 0.0, 2.0], device="cuda")
    both(tf, *x, slopes=slopes, softcap=cap, causal=causal)


DOCS = {
    "packed": lambda S: [i * 5 // S for i in range(S)],
    "tail": lambda S: [0] * (S // 3) + [1] * (S // 5) + [-1] * (S - S // 3 - S // 5),
    "scattered": lambda S: [(i * 7) % 3 - (i % 11 == 0) * 9 for i in range(S)],
    "all padding": lambda S: [-3] * S,
    "singles": lambda S: list(range(S)),
    "large numbers": lambda S: [2 ** 31 - 1 - i // 100 for i in range(S)],
}


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("S", [1, 257, 640])
@pytest.mark.parametrize("kind", sorted(DOCS))
def test_documents(tf, kind, S, causal):
    x = make(2, 2, S, S, 2, 1, 64, BF16, 11)
    docs = torch.tensor([DOCS[kind](S), DOCS["packed"](S)], dtype=torch.int32, device="cuda")
    both(tf, *x, q_docs=docs, k_docs=docs, causal=causal)


def test_documents_of_unequal_sides_behind_a_prefix(tf):
    q, k, v, dout = make(1, 2, 150, 400, 2, 2, 128, FP16, 13)
    qd = torch.tensor([[i * 3 // 150 for i in range(150)]] * 2, dtype=torch.int32, device="cuda")
    kd = torch.tensor([[i * 4 // 400 for i in range(400)]] * 2, dtype=torch.int32, device="cuda")
    both(tf, q, k, v, dout, q_docs=qd, k_docs=kd, causal=True, prefix=torch.tensor([200, 7], dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("D", [64, 128])
def test_padding_may_hold_anything(tf, D):
    S = 300
    q, k, v, dout = make(1, 2, S, S, 2, 1, D, BF16, 17)
    docs = torch.tensor([[0] * 200 + [-1] * 100, [-1] * 33 + [1] * 100 + [-5] * 40 + [2] * 127], dtype=torch.int32, device="cuda")
    pad = docs < 0
    for ts in (q, k, v, dout):
        ts[0][pad] = math.nan
        ts[0][:, -1] = torch.where(pad[:, -1, None, None], torch.tensor(math.inf, device="cuda", dtype=BF16), ts[0][:, -1])
    kw = dict(q_docs=docs, k_docs=docs)
    out, lse = tf.attention(q, k, v, **kw)
    dq, dk, dv = tf.attention_backward(dout, q, k, v, out, lse, **kw)
    ref = Reference(q, k, v, dout, clean=True, **kw)
    for name, got in (("out", out), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        ref.check(name, got)


@pytest.mark.parametrize("D", [64, 128])
def test_views_into_fused_payloads_and_strided_results(tf, D):
    q, k, v, dout = make(2, 2, 260, 260, 3, 3, D, BF16, 19, fused=True)
    dout = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in dout]  # heads outside tokens
    ref = Reference(q, k, v, dout)
    big = [torch.full((2, 260, 3, 3 * D), 7.0, dtype=BF16, device="cuda") for _ in q]
    out = [t[..., D:2 * D] for t in big]
    out, lse = tf.attention(q, k, v, out)
    ref.check("out", out)
    grads = [torch.full((2, 260, 3, 3 * D), 7.0, dtype=BF16, device="cuda") for _ in q]
    dq, dk, dv = tf.attention_backward(dout, q, k, v, out, lse, *([t[..., i * D:(i + 1) * D] for t in grads] for i in range(3)))
    for name, got in (("dq", dq), ("dk", dk), ("dv", dv)):
        ref.check(name, got)
    for t in big:  # nothing beside the view was written
        assert bool((t[..., :D] == 7).all()) and bool((t[..., 2 * D:] == 7).all())


@pytest.mark.parametrize("D,dtype", [(64, FP16), (128, BF16)])
@pytest.mark.parametrize("P,B,Sq,Sk,Hl,Hkl", [(1, 1, 300, 2200, 1, 1), (1, 1, 2300, 2200, 1, 1), (2, 2, 1100, 3001, 2, 1),
                                              (1, 1, 5000, 1100, 4, 1)])
def test_units_cut_along_the_other_side(tf, P, B, Sq, Sk, Hl, Hkl, D, dtype):
    """Few row tiles over many of the other side: their sums are joined from parts."""
    x = make(P, B, Sq, Sk, Hl, Hkl, D, dtype, Sq)
    both(tf, *x)
    both(tf, *x, softcap=4.0, slopes=torch.linspace(0.0, 0.05, P * Hl, device="cuda"))


def test_large_scores_and_equal_keys(tf):
    q, k, v, dout = make(1, 1, 140, 300, 2, 2, 64, BF16, 23)
    both(tf, [30 * t for t in q], k, v, dout)          # one weight takes nearly all
    both(tf, q, [torch.ones_like(t) for t in k], v, dout)  # all weights equal
    both(tf, q, k, v, dout, scale=0.0)
    both(tf, q, k, v, dout, scale=-0.3)


def test_nothing_to_do(tf):
    empty = lambda *s: [torch.empty(s, dtype=BF16, device="cuda")]  # noqa: E731
    out, lse = tf.attention(empty(1, 0, 2, 64), empty(1, 5, 2, 64), empty(1, 5, 2, 64))
    assert out[0].shape == (1, 0, 2, 64) and lse[0].shape == (1, 2, 0)
    q, _, _, dout = make(1, 2, 5, 5, 2, 2, 64, BF16, 0)
    out, lse = tf.attention(q, empty(2, 0, 2, 64), empty(2, 0, 2, 64))
    assert bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all())
    dq, dk, dv = tf.attention_backward(dout, q, empty(2, 0, 2, 64), empty(2, 0, 2, 64), out, lse)
    assert bool((dq[0] == 0).all()) and dk[0].numel() == 0
    k = [torch.ones((2, 5, 2, 64), dtype=BF16, device="cuda")]
    none = empty(2, 0, 2, 64)
    dq, dk, dv = tf.attention_backward(none, none, k, k, none, [torch.empty((2, 2, 0), device="cuda")],
                                       dk=[torch.ones_like(k[0])], dv=[torch.ones_like(k[0])])
    assert bool((dk[0] == 0).all()) and bool((dv[0] == 0).all())


def test_gradient_against_differences(tf):
    q, k, v, dout = make(1, 1, 70, 90, 2, 1, 64, FP16, 29)
    kw = dict(softcap=5.0, causal=True, slopes=torch.tensor([0.1, 0.02], device="cuda"))
    out, lse = tf.attention(q, k, v, **kw)
    grads = tf.attention_backward(dout, q, k, v, out, lse, **kw)
    loss = lambda *x: float((Reference(*x, **kw).out * dout[0].double().transpose(1, 2)).sum())  # noqa: E731
    gen = torch.Generator(device="cuda").manual_seed(31)
    for n in range(3):  # the derivative along a random direction, central differences of the 64-bit forward pass
        step = torch.randn((q, k, v)[n][0].shape, generator=gen, device="cuda").double()
        moved = lambda e: [[x[0].double() + e * step] if m == n else x for m, x in enumerate((q, k, v))]  # noqa: E731
        h = 1e-4
        want = (loss(*moved(h)) - loss(*moved(-h))) / (2 * h)
        ref = Reference(q, k, v, dout, **kw)
        tol = float((getattr(ref, ("dq_tol", "dk_tol", "dv_tol")[n]) * step.transpose(1, 2).abs()).sum())
        got = float((grads[n][0].double() * step).sum())
        assert abs(got - want) <= tol + 1e-6 * abs(want), (n, got, want, tol)


def test_the_same_inputs_give_the_same_bits(tf):
    x = make(2, 2, 300, 300, 4, 2, 128, BF16, 37)
    kw = dict(causal=True, softcap=30.0)
    a, b = both(tf, *x, **kw), both(tf, *x, **kw)
    for s, t in zip(a, b):
        assert all(torch.equal(m, n) for m, n in zip(s, t))


def test_another_stream(tf):
    x = make(2, 1, 400, 400, 2, 2, 64, BF16, 41)
    want = both(tf, *x)
    torch.cuda.synchronize()
    for stream in (torch.cuda.Stream(), torch.cuda.Stream()):
        out, lse = tf.attention(*x[:3], stream=stream)
        got = (out, lse, *tf.attention_backward(x[3], *x[:3], out, lse, stream=stream.cuda_stream))
        stream.synchronize()
        assert all(torch.equal(m, n) for s, t in zip(want, got) for m, n in zip(s, t))


@pytest.mark.parametrize("Sq,Sk", [(300, 40000), (40000, 300)])
def test_causal_heads_in_blocks(tf, Sq, Sk):
    """Heads whose keys (queries, for dK and dV) are too many to be interleaved all at once: blocks of 3 and 2."""
    both(tf, *make(1, 1, Sq, Sk, 5, 5, 128, BF16, 57), causal=True)


@pytest.mark.parametrize("B,S", [(1, 600), (3, 600), (2, 5000), (70, 300)])
def test_documents_ranked_over_batch_rows(tf, B, S):
    """Row tiles of all batch rows in the order of their work, with ties and with rows of padding only."""
    g = torch.Generator(device="cuda").manual_seed(58)
    docs = torch.randint(0, 3, (B, S), generator=g, device="cuda", dtype=torch.int32).sort(1).values
    docs[0] = -1
    both(tf, *make(2, B, S, S, 1, 1, 64, FP16, 59), q_docs=docs, k_docs=docs, causal=B == 3)


def test_documents_of_any_number(tf):
    docs = torch.full((1, 300), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    docs[:, 10:20], docs[:, 150:], docs[:, 299] = -2 ** 31, 0, -7
    both(tf, *make(1, 1, 300, 300, 2, 1, 64, BF16, 60), q_docs=docs, k_docs=docs)
    docs = torch.zeros((1, 256), dtype=torch.int32, device="cuda")
    docs[:, 3] = -2 ** 31  # the only padding of its tile
    both(tf, *make(1, 1, 256, 256, 2, 1, 64, BF16, 61), q_docs=docs, k_docs=docs)


def test_two_calls_at_once(tf):
    """Calls in flight on two streams, each joining parts from a workspace of its own."""
    x = [make(1, 1, 1100, 3001, 2, 1, 128, BF16, seed) for seed in (51, 52)]
    want = [both(tf, *y) for y in x]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        got = []
        for y, s in zip(x, streams):
            out, lse = tf.attention(*y[:3], stream=s)
            got.append((out, lse, *tf.attention_backward(y[3], *y[:3], out, lse, stream=s)))
        torch.cuda.synchronize()
        assert all(torch.equal(m, n) for a, b in zip(want, got) for s, t in zip(a, b) for m, n in zip(s, t))


def test_many_batch_rows_of_documents(tf):
    """More batch rows than one dimension of a grid may count (65535)."""
    B, S = 65600, 3
    g = torch.Generator(device="cuda").manual_seed(53)
    docs = torch.randint(-1, 2, (B, S), generator=g, device="cuda", dtype=torch.int32)
    both(tf, *make(1, B, S, S, 1, 1, 64, BF16, 54), q_docs=docs, k_docs=docs)


def test_values_of_masked_keys(tf):
    """A key that a row does not see may hold anything in K.  In V too, if it is padding (see above) or lies in a
    tile that the row's 256 rows skip; in a visited tile its weight is 0, and 0 times infinity is NaN."""
    q, k, v, _ = make(1, 1, 512, 512, 1, 1, 64, BF16, 55)
    want, lse = tf.attention(q, k, v, causal=True)
    for bad in (math.nan, math.inf, -math.inf):
        kb, vb = [k[0].clone()], [v[0].clone()]
        kb[0][:, 300:], vb[0][:, 256:] = bad, bad
        out, got = tf.attention(q, kb, vb, causal=True)
        assert torch.equal(out[0][:, :256], want[0][:, :256]) and torch.equal(got[0][..., :300], lse[0][..., :300])


REFUSED = {
    "q no list": lambda a: dict(q=a["q"][0]), "no groups": lambda a: dict(q=[]), "one group more": lambda a: dict(q=a["q"] * 2),
    "no tensor": lambda a: dict(k=[0]), "two types": lambda a: dict(v=[a["v"][0].half()]), "fp32": lambda a: {n: [a[n][0].float()] for n in "qkv"},
    "another batch": lambda a: dict(k=[a["k"][0][:1]], v=[a["v"][0][:1]]), "K and V differ": lambda a: dict(v=[a["v"][0][:, :7]]),
    "another D": lambda a: dict(k=[a["k"][0][..., :32]], v=[a["v"][0][..., :32]]), "three dimensions": lambda a: dict(q=[a["q"][0][0]]),
    "D not innermost": lambda a: dict(q=[a["q"][0].transpose(2, 3).contiguous().transpose(2, 3)]), "q on the CPU": lambda a: dict(q=[a["q"][0].cpu()]),
    "v on the CPU": lambda a: dict(v=[a["v"][0].cpu()]), "broadcast k": lambda a: dict(k=[a["k"][0][:, :1].expand(-1, 8, -1, -1)]),
    "short slopes": lambda a: dict(slopes=torch.zeros(1, device="cuda")), "fp16 slopes": lambda a: dict(slopes=torch.zeros(2, dtype=FP16, device="cuda")),
    "64-bit documents": lambda a: dict.fromkeys(("q_docs", "k_docs"), torch.zeros((2, 8), dtype=torch.int64, device="cuda")),
    "documents of one side": lambda a: dict(q_docs=torch.zeros((2, 8), dtype=torch.int32, device="cuda")),
    "prefix on the CPU": lambda a: dict(causal=True, prefix=torch.zeros(2, dtype=torch.int32)),
    "prefix without causal": lambda a: dict(prefix=torch.zeros(2, dtype=torch.int32, device="cuda")),
    "short out": lambda a: dict(out=[a["q"][0][:, :7]]), "two outs": lambda a: dict(out=a["q"] * 2),
    "fp16 lse": lambda a: dict(lse=[torch.zeros((2, 2, 8), dtype=FP16, device="cuda")]),
    "strided lse": lambda a: dict(lse=[torch.zeros((2, 2, 16), device="cuda")[..., ::2]]),
    "scale no number": lambda a: dict(scale="x"), "scale NaN": lambda a: dict(scale=math.nan), "negative cap": lambda a: dict(softcap=-1.0)}


@pytest.mark.parametrize("how", REFUSED)
def test_refused_tensors(tf, how):
    q, k, v, dout = make(1, 2, 8, 8, 2, 2, 64, BF16, 56)
    args = dict(q=q, k=k, v=v)
    args.update(REFUSED[how](args))
    n = tf.launch_count()
    with pytest.raises((ValueError, TypeError, tf.TfUlyssesError)):
        tf.attention(**args)
    out, lse = args.pop("out", q), args.pop("lse", [torch.zeros((2, 2, 8), device="cuda")])
    with pytest.raises((ValueError, TypeError, tf.TfUlyssesError)):
        tf.attention_backward(dout, args.pop("q"), args.pop("k"), args.pop("v"), out, lse, **args)
    assert tf.launch_count() == n


def test_captured_and_replayed_with_new_inputs(tf):
    x = make(2, 1, 300, 300, 2, 2, 64, BF16, 43)
    docs = torch.tensor([DOCS["packed"](300)], dtype=torch.int32, device="cuda")
    kw = dict(q_docs=docs, k_docs=docs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = tf.attention(*x[:3], **kw)
        grads = tf.attention_backward(x[3], *x[:3], out, lse, **kw)
    for seed in (44, 45):
        for ts, new in zip(x, make(2, 1, 300, 300, 2, 2, 64, BF16, seed)):
            for t, n in zip(ts, new):
                t.copy_(n)
        docs.copy_(torch.tensor([DOCS["tail" if seed == 44 else "scattered"](300)], dtype=torch.int32))
        graph.replay()
        ref = Reference(*x, **kw)
        for name, got in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
            ref.check(name, got)


def test_between_scatter_and_gather(tf):
    """The path of one layer: scatter with norm and rotation, attention, gather; each step as its own test checks it."""
    from ulysses_sequence_attention_tf_gb300 import synth
    P, B, S, H, D = 4, 1, 512, 8, 64
    d = synth.move(synth.qkv_shards(P, B, S // P, H, D, BF16, seed=3, layout="fused"), "cuda:0")
    wq, wk = (w.cuda() for w in synth.norm_weights(D, BF16, seed=3))
    q, k, v, _ = tf.scatter_qkv("layer", d["q"], d["k"], d["v"], norm_rope=True, q_weight=wq, k_weight=wk, layout="fused")
    out, lse = tf.attention(q, k, v, softcap=20.0)
    Reference(q, k, v, softcap=20.0).check("out", out)
    back, _ = tf.gather_out("layer", out)
    whole = torch.cat(out, 2)
    for r in range(P):
        assert torch.equal(back[r], whole[:, r * (S // P):(r + 1) * (S // P)])
    tf.cache_clear()
