"""Rotary positions against complex products in 64 bits.

A result is off by half a step of its type, by the sines' and cosines' error (3e-7 < 2^-21 as the header says) and three
roundings of fp32 (2^-24 each, of terms up to |x0| + |x1|): 2^-20 m (|x0| + |x1|) covers both.
"""
import math

import pytest
import torch

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


def rows(*shape, dtype=BF16, seed=0):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def check(x, y, at, f, *, rope, m=1.0, inverse=False):
    """x, y: [..., tokens, heads, D]; at: [..., tokens]."""
    R, D = 2 * len(f), x.shape[-1]
    assert y.shape == x.shape and y.dtype == x.dtype
    assert torch.equal(y[..., R:].reshape(-1).view(torch.int16), x[..., R:].reshape(-1).view(torch.int16)), "the rest of the head"
    i = torch.arange(R // 2, device="cuda")
    a, b = (i, i + R // 2) if rope == "neox" else (2 * i, 2 * i + 1)
    angle = at.double()[..., None] * f.cuda()
    turn = torch.polar(torch.full_like(angle, m), -angle if inverse else angle)[..., None, :]
    w = x.double()
    z = torch.complex(w[..., a], w[..., b]) * turn
    size = abs(m) * (w[..., a].abs() + w[..., b].abs())
    for got, want in ((y[..., a], z.real), (y[..., b], z.imag)):
        tol = torch.finfo(x.dtype).eps / 2 * want.abs() + 2.0 ** -20 * size + torch.finfo(x.dtype).tiny * torch.finfo(x.dtype).eps
        assert bool(((got.double() - want).abs() <= tol).all()), float(((got.double() - want).abs() / tol).max())
    assert D == x.shape[-1]


@pytest.mark.parametrize("rope", ["interleaved", "neox"])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("D,R", [(64, 64), (128, 128), (128, 64), (64, 16), (128, 96), (64, 24), (64, 20), (128, 2), (64, 6), (8, 8), (8, 4),
                                 (40, 10), (256, 256), (256, 250), (96, 90)])
def test_parts_of_heads(tf, rope, dtype, D, R):
    q, k = [rows(2, 7, 3, D, dtype=dtype, seed=s) for s in (0, 1)], [rows(2, 7, 1, D, dtype=dtype, seed=s) for s in (2, 3)]
    f = tf.rope_frequencies(R)
    q_out, k_out = tf.rope(q, k, first=5, rotary_dim=R, rope=rope)
    at = torch.arange(5, 12, device="cuda").expand(2, 7)
    for x, y in zip(q + k, q_out + k_out):
        check(x, y, at, f, rope=rope)


@pytest.mark.parametrize("shape,heads,kv,P", [((1, 1), 1, 1, 1), ((1, 1), 40, 8, 4), ((3, 5), 6, 2, 2), ((1, 513), 5, 5, 1), ((2, 2047), 3, 1, 1),
                                              ((1, 4096), 24, 24, 4), ((700,), 8, 2, 2), ((1,), 64, 8, 8)])
@pytest.mark.parametrize("rope", ["interleaved", "neox"])
def test_sizes(tf, shape, heads, kv, P, rope):
    q = [rows(*shape, heads // P, 128, seed=g) for g in range(P)]
    k = [rows(*shape, kv // P, 128, seed=9 + g) for g in range(P)]
    at = torch.randint(0, 2 ** 20, shape, device="cuda", dtype=torch.int32)
    f = tf.rope_frequencies(64, scaling="parts", factor=8.0)
    q_out, k_out = tf.rope(q, k, positions=at, frequencies=f, magnitude=1.2, rope=rope)
    for x, y in zip(q + k, q_out + k_out):
        check(x, y, at, f, rope=rope, m=1.2)


@pytest.mark.parametrize("first", [0, -3, 1000000, 2 ** 31 - 8])
def test_far_positions(tf, first):
    """Angles of any position; frequencies beyond a turn and negative ones among them."""
    q = [rows(1, 7, 2, 64)]
    f = torch.cat([tf.rope_frequencies(56), torch.tensor([7.5, -0.3, 0.0, 100.25], dtype=torch.float64)])
    at = torch.arange(first, first + 7, device="cuda", dtype=torch.int64)[None]
    q_out, none = tf.rope(q, first=first, frequencies=f)
    assert none is None
    check(q[0], q_out[0], at, f, rope="interleaved")
    given, _ = tf.rope(q, positions=at.to(torch.int32), frequencies=f)
    assert torch.equal(given[0], q_out[0])


@pytest.mark.parametrize("rope", ["interleaved", "neox"])
@pytest.mark.parametrize("R", [128, 48, 20])
def test_strided_and_in_place(tf, rope, R):
    """Views into fused payloads, broadcast inputs, and rows rotated where they lie."""
    pay = rows(2, 33, 4, 3 * 128)
    q, k = pay[..., :128], pay[..., 128:256]
    f = tf.rope_frequencies(R)
    at = torch.arange(33, device="cuda").expand(2, 33)
    before = pay.clone()
    want_q, want_k = tf.rope([q], [k], rotary_dim=R, rope=rope)
    check(q, want_q[0], at, f, rope=rope)
    check(k, want_k[0], at, f, rope=rope)
    back = tf.rope([q], [k], [q], [k], rotary_dim=R, rope=rope)
    assert back[0][0] is q and torch.equal(q, want_q[0]) and torch.equal(k, want_k[0])
    assert torch.equal(pay[..., 256:], before[..., 256:])
    one = rows(1, 33, 1, 128)
    spread = one.expand(2, 33, 4, 128)
    got, _ = tf.rope([spread], rotary_dim=R, rope=rope)
    check(spread, got[0], at, f, rope=rope)
    # q in place, k elsewhere
    x, y = rows(2, 33, 4, 128, seed=5), rows(2, 33, 2, 128, seed=6)
    want = tf.rope([x], [y], rotary_dim=R, rope=rope)
    q2, k2 = tf.rope([x], [y], [x], None, rotary_dim=R, rope=rope)
    assert torch.equal(x, want[0][0]) and torch.equal(k2[0], want[1][0])


@pytest.mark.parametrize("rope", ["interleaved", "neox"])
def test_offsets_beyond_32_bits(tf, rope):
    """Batch rows 2^31 elements apart, into another tensor and in place."""
    store = torch.empty(2 ** 32 + 2 ** 16, dtype=BF16, device="cuda")
    far = [store.as_strided((3, 5, 2, 64), (2 ** 31, 128, 64, 1), i * 640) for i in range(2)]
    x = rows(3, 5, 2, 64)
    far[0].copy_(x)
    f, at = tf.rope_frequencies(64), torch.arange(5, device="cuda").expand(3, 5)
    for out in (far[1], far[0]):
        tf.rope([far[0]], q_out=[out], rope=rope)
        check(x, out, at, f, rope=rope)


@pytest.mark.parametrize("rope", ["interleaved", "neox"])
def test_inverse_is_the_gradient(tf, rope):
    x, g = rows(1, 50, 2, 64, dtype=FP16), rows(1, 50, 2, 64, dtype=FP16, seed=1)
    f = tf.rope_frequencies(48)
    dx, _ = tf.rope([g], frequencies=f, magnitude=1.25, rope=rope, inverse=True, first=77)
    at = torch.arange(77, 127, device="cuda")[None]
    check(g, dx[0], at, f, rope=rope, m=1.25, inverse=True)
    # against differences: the rotation is linear, so <g, rope(e)> is the derivative along e
    e = rows(1, 50, 2, 64, dtype=FP16, seed=2)
    y, _ = tf.rope([e], frequencies=f, magnitude=1.25, rope=rope, first=77)
    left, right = (g.double() * y[0].double()).sum(), (dx[0].double() * e.double()).sum()
    # half a step of every product's rounded factor, and 2^-20 of both terms
    room = (torch.finfo(FP16).eps / 2 + 2.0 ** -18) * ((g.double() * y[0].double()).abs().sum() + (dx[0].double() * e.double()).abs().sum())
    assert abs(left - right) <= room


@pytest.mark.parametrize("rope", ["interleaved", "neox"])
def test_values_that_are_not_finite(tf, rope):
    """They stay in their pair, and where nothing turns they are copied."""
    x = rows(1, 3, 1, 64)
    x[0, 1, 0, 4], x[0, 2, 0, 63], x[0, 0, 0, 50] = math.inf, math.nan, -math.inf
    y, _ = tf.rope([x], rotary_dim=20, rope=rope, first=9)
    assert torch.equal(y[0][..., 20:].contiguous().view(torch.int16), x[..., 20:].contiguous().view(torch.int16))
    pair = 14 if rope == "neox" else 5
    bad = ~y[0][..., :20].isfinite()
    assert set(map(tuple, bad.nonzero().tolist())) == {(0, 1, 0, 4), (0, 1, 0, pair)}


def test_streams_and_graphs(tf):
    q = [rows(1, 64, 4, 64)]
    at = torch.arange(64, device="cuda", dtype=torch.int32)[None].contiguous()
    want, _ = tf.rope(q, positions=at)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other, _ = tf.rope(q, positions=at, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other[0], want[0])
    out = [torch.empty_like(q[0])]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tf.rope(q, q_out=out, positions=at)
    for first in (0, 1000):
        at.copy_(torch.arange(first, first + 64, device="cuda")[None])
        graph.replay()
        want, _ = tf.rope(q, first=first)
        assert torch.equal(out[0], want[0])


def test_empty(tf):
    q, k = tf.rope([rows(0, 5, 2, 64)], [rows(0, 5, 1, 64)])
    assert q[0].shape == (0, 5, 2, 64) and k[0].shape == (0, 5, 1, 64)
    q, _ = tf.rope([rows(0, 2, 64)])
    assert q[0].shape == (0, 2, 64)


def test_refusals(tf):
    q = [rows(1, 4, 2, 64)]
    pos = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    for kw in (dict(k=[rows(1, 4, 2, 128)]), dict(k=[rows(4, 2, 64)]), dict(k=[rows(1, 5, 2, 64)]), dict(positions=pos[0]),
               dict(positions=pos.long()), dict(positions=pos.cpu()), dict(q_out=[rows(1, 4, 2, 64, dtype=FP16)]), dict(k_out=q),
               dict(frequencies=torch.ones(8)), dict(frequencies=torch.ones(8, dtype=torch.float64, device="cuda")),
               dict(frequencies=torch.ones(8, dtype=torch.float64), rotary_dim=8), dict(rope="half"), dict(first=2 ** 31)):
        with pytest.raises(ValueError):
            tf.rope(q, **kw)
    for kw in (dict(frequencies=torch.ones(33, dtype=torch.float64)), dict(rotary_dim=65), dict(rotary_dim=0), dict(magnitude=math.nan)):
        with pytest.raises(tf.TfUlyssesError):
            tf.rope(q, **kw)
