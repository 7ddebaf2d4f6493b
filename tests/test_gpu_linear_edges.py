"""Linear attention where its numbers reach their ends, against 64 bits (bounds derived in linear_util)."""
import pytest
import torch

from linear_util import check_rows, check_state, recurrence, wide

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16
LARGEST = torch.finfo(torch.float32).max


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


def rows(B, S, H, D, dtype, seed):
    return [torch.randn((B, S, H, D), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)]


def check_all(tf, q, k, v, dout, decay, state, dstate, dtype):
    """Outputs, final state and the gradients of both."""
    scale = q[0].shape[-1] ** -0.5
    Q, K, V, G = (wide(x) for x in (q, k, v, dout))
    flip = lambda x: x.double().transpose(-1, -2)  # noqa: E731
    out, last = tf.linear_attention(q, k, v, decay=decay, state=state, final_state=True)
    want = recurrence(Q, K, V, decay, scale, state.double())
    check_rows("out", out, *want[:2], dtype)
    check_state("state", last, *want[2:])
    dq, dk, dv, first = tf.linear_attention_backward(dout, q, k, v, decay=decay, state=state, dstate=dstate)
    check_rows("dq", dq, *recurrence(G, V, K, decay, scale, flip(state))[:2], dtype)
    check_rows("dk", dk, *recurrence(V, G, Q, decay, scale, flip(dstate), 1.0, reverse=True)[:2], dtype)
    want = recurrence(K, Q, G, decay, scale, dstate.double(), 1.0, reverse=True)
    check_rows("dv", dv, *want[:2], dtype)
    check_state("dstate", first, *want[2:])


@pytest.mark.parametrize("S", [1, 5, 17, 128, 300, 6000])
@pytest.mark.parametrize("D,dtype", [(64, FP16), (128, BF16)])
def test_decays_up_to_the_largest_number(tf, S, D, dtype):
    """Nothing is kept from token to token, whatever the length and however large the decay is; 1e30 and less beside it."""
    decay = torch.tensor([LARGEST, 2.4e38, 1e30, 300.0, 90.0, 0.0], device="cuda")
    q, k, v, dout = (rows(1, S, 6, D, dtype, i) for i in range(4))
    state, dstate = (torch.randn((1, 6, D, D), generator=torch.Generator(device="cuda").manual_seed(i), device="cuda") for i in (5, 6))
    check_all(tf, q, k, v, dout, decay, state, dstate, dtype)


def channels(D, *sizes):
    """[D]: sizes in turn."""
    return torch.tensor(sizes, device="cuda").repeat(D // len(sizes))


@pytest.mark.parametrize("S", [3, 8, 9, 16, 17, 100, 128, 300, 1100])
@pytest.mark.parametrize("D,H", [(64, 2), (128, 2), (64, 400)])
@pytest.mark.parametrize("large,small", [(100.0, 1e-3), (100.0, 1e-5)])
def test_channels_of_unlike_size(tf, S, D, H, large, small):
    """fp16: a key channel far smaller than another keeps its bits in the state, token by token and in chunks.  The state's
    columns are as unlike for dQ."""
    if H > 2 and S > 128:
        return
    size = channels(D, large, small)
    decay = torch.tensor([0.05, 0.4], device="cuda").repeat(H // 2)
    q, k, v, dout = (rows(1, S, H, D, FP16, i) for i in range(4))
    k = [(k[0].float() * size).to(FP16)]
    state, dstate = (torch.randn((1, H, D, D), generator=torch.Generator(device="cuda").manual_seed(i), device="cuda") for i in (5, 6))
    check_all(tf, q, k, v, dout, decay, state * size[:, None], dstate, FP16)


@pytest.mark.parametrize("S", [5, 16, 17, 128, 300, 3000])
@pytest.mark.parametrize("D", [64, 128])
def test_channels_over_the_whole_range_of_fp16(tf, S, D):
    size = channels(D, 8192.0, 1e-6, 1.0, 1e-3)
    decay = torch.tensor([0.0, 0.01, 0.3, 3.0], device="cuda")
    q, k, v = (rows(2, S, 4, D, FP16, i) for i in range(3))
    k = [(k[0].float().clamp(-4, 4) * size).to(FP16)]
    out, last = tf.linear_attention(q, k, v, decay=decay, final_state=True, scale=1e-4)
    want = recurrence(wide(q), wide(k), wide(v), decay, 1e-4)
    check_rows("out", out, *want[:2], FP16)
    check_state("state", last, *want[2:])
    starts, slots = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, S, 2 * S], [1, 0]))
    states = torch.zeros((2, 4, D, D), device="cuda")
    tf.linear_attend(states, slots, starts, *[[x[0].reshape(2 * S, 4, D)] for x in (q, k, v)], decay=decay, max_tokens=S)
    check_state("states", states.flip(0), *want[2:])


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_large_tokens_that_have_faded(tf, reverse, D):
    """fp16: keys 2^29 times as large as a row's own, 10 tokens and more away at a decay of 3, weigh nothing in that row -- also
    not by taking its power of two.  Outputs beyond fp16 are infinite."""
    S, H, scale = 260, 2, 2.0 ** 12
    decay = torch.full((H,), 3.0, device="cuda")
    q, k, v = (rows(1, S, H, D, FP16, i) for i in range(3))
    token = torch.arange(S, device="cuda") % 128
    size = torch.where((token >= 64) == reverse, 2.0 ** 13, 2.0 ** -16)[:, None, None]
    k = [(k[0].float().clamp(-4, 4) * size).to(FP16)]
    if reverse:  # of the gradients: dV_j sums k_j . q_i over later rows i
        got = tf.linear_attention_backward(v, k, q, v, decay=decay, scale=scale)[2]
        want = recurrence(wide(q), wide(k), wide(v), decay, scale, None, 1.0, reverse=True)
    else:
        got, _ = tf.linear_attention(q, k, v, decay=decay, scale=scale)
        want = recurrence(wide(q), wide(k), wide(v), decay, scale)
    check_rows("rows", got, *want[:2], FP16, norm=False)


def test_outputs_over_inputs_are_refused(tf):
    """The passes run together and read ahead; slices of one payload lie apart and are fine."""
    q, k, v, dout = (rows(1, 300, 2, 64, BF16, i) for i in range(4))
    decay = torch.tensor([0.1, 0.2], device="cuda")
    for out in (q, k, v):
        with pytest.raises(tf.TfUlyssesError):
            tf.linear_attention(q, k, v, out, decay=decay)
    for grads in (dict(dq=dout), dict(dq=q), dict(dk=k), dict(dv=v), dict(dk=dout, dv=dout)):
        with pytest.raises(tf.TfUlyssesError):
            tf.linear_attention_backward(dout, q, k, v, decay=decay, **grads)
    with pytest.raises(tf.TfUlyssesError):
        tf.rope(q, k, k, None)
    payload = torch.empty((1, 300, 2, 3 * 64), dtype=BF16, device="cuda")
    into = [[payload[..., i * 64:(i + 1) * 64]] for i in range(3)]
    got = tf.linear_attention_backward(dout, q, k, v, *into, decay=decay)
    for x, y in zip(got, tf.linear_attention_backward(dout, q, k, v, decay=decay)[:3]):
        assert torch.equal(x[0], y[0])


@pytest.mark.parametrize("reverse", [False, True])
def test_large_numbers_far_in_front_of_a_segment(tf, reverse):
    """40 heads of 256 chunks are cut into segments of 37.  The first (reverse: the last) token's key and value of 2^60
    still count behind its segment, at e^-142 and less, where every other number in front is 0."""
    S, H, D, far, scale = 32768, 40, 64, 2.0 ** 40, 2.0 ** 10
    decay = torch.full((H,), 0.03, device="cuda")
    t = torch.arange(S, device="cuda", dtype=torch.float64)
    q, k, v = (torch.zeros((1, S, H, D), dtype=BF16, device="cuda") for _ in range(3))
    first = S - 1 if reverse else 0
    size = rows(1, 1, H, D, BF16, 1)[0][0, 0].float().sign()
    k[0, first, :, 3], v[0, first] = 2.0 ** 60, (size * 2.0 ** 60).to(BF16)
    gone = (t - first).abs()
    q[0, :, :, 3] = torch.where(gone >= 4000, far, 0.0).to(BF16)[:, None]
    if reverse:  # dV_j = scale sum_(i >= j) e^(-decay (i - j)) (k_j . q_i) dout_i
        got = tf.linear_attention_backward([v], [k], [q], [v], decay=decay, scale=scale)[2][0]
    else:
        got = tf.linear_attention([q], [k], [v], decay=decay, scale=scale)[0][0]
    seen = (gone >= 4000) & (gone <= 6500)
    want = scale * far * 2.0 ** 120 * torch.exp(-decay.double()[0] * gone[seen])[:, None, None] * size.double()
    # two roundings to bf16's 8 bits, the result's and the state's or the weight's, half a step of 2^-7 each; the exponents' 2^-24 of
    # 200 and the keys' 2^-16.  A number below 2^-126, bf16's least normal one, need not count in the state: from 246 log 2 / 0.03 =
    # 5684 tokens on 2^120 has faded below it, so 2^-126 far scale = 2^-76 may be missing, where 2^-35 are at stake at the first
    # segment's end
    room = (2 * 2.0 ** -8 + 2.0 ** -14) * want.abs() + 2.0 ** -126 * far * scale
    off = (got[0, seen].double() - want).abs()
    assert bool((off <= room).all()), [(int(i), float(off[i].max()), float(room[i].max())) for i in (off > room).any(-1).any(-1).nonzero()[:3, 0]]


@pytest.mark.parametrize("S", [17, 300])
@pytest.mark.parametrize("D", [64, 128])
def test_small_channels_that_large_queries_bring_up(tf, S, D):
    """fp16: channels of k 2^24 times as small as others, which queries as much larger bring up again, and channels of v 2^22 times
    as small.  The state's tile for q keeps 11 bits of what is above 2^-27 of its largest entry; entries of both are 2^-46 of it,
    and below 2^-27 an entry is off by 2^-38 of the largest (2^-25 of a number in [2^13, 2^14)).  So beside the usual bound an
    output may be off by scale sum_c |q_c| 2^-38 max |S|, S in front of its chunk."""
    decay = torch.tensor([0.01, 0.0], device="cuda")
    q, k, v = (rows(1, S, 2, D, FP16, i) for i in range(3))
    size, of_v = channels(D, 2.0 ** 12, 2.0 ** -12), channels(D, 2.0 ** 10, 2.0 ** 10, 2.0 ** -12, 1.0)
    q, k, v = [(q[0].float() / size).to(FP16)], [(k[0].float() * size).to(FP16)], [(v[0].float() * of_v).to(FP16)]
    out, last = tf.linear_attention(q, k, v, decay=decay, final_state=True, scale=0.05)
    Q, K, V = wide(q), wide(k), wide(v)
    want = recurrence(Q, K, V, decay, 0.05)
    beside = torch.zeros_like(want[1])
    for at in range(128, S, 128):
        front = recurrence(Q[:, :, :at], K[:, :, :at], V[:, :, :at], decay, 0.05)[2]
        beside[:, :, at:] = 0.05 * 2.0 ** -38 * front.abs().amax((-1, -2))[..., None, None] * Q[:, :, at:].abs().sum(-1, keepdim=True)
    check_rows("out", out, want[0], want[1] + beside / (2.0 ** -11 + 2.0 ** -15), FP16)
    check_state("state", last, *want[2:])


@pytest.mark.parametrize("S", [8200, 20000])
def test_one_head_in_many_segments(tf, S):
    """65 and 157 chunks of one head: as many segments as are looked at, of one, two or three chunks."""
    decay = torch.tensor([2e-4], device="cuda")
    q, k, v, dout = (rows(1, S, 1, 64, BF16, i) for i in range(4))
    state, dstate = (torch.randn((1, 1, 64, 64), generator=torch.Generator(device="cuda").manual_seed(i), device="cuda") for i in (5, 6))
    check_all(tf, q, k, v, dout, decay, state, dstate, BF16)


@pytest.mark.parametrize("D,dtype", [(64, FP16), (128, BF16)])
def test_calls_at_once(tf, D, dtype):
    """Calls on streams of their own, beside one another and beside attention, give the bits of the calls alone."""
    q, k, v, dout = (rows(1, 2000, 8, D, dtype, i) for i in range(4))
    decay = torch.exp2(-torch.arange(1.0, 9.0, device="cuda"))
    calls = [lambda: tf.linear_attention(q, k, v, decay=decay)[0], lambda: tf.linear_attention_backward(dout, q, k, v, decay=decay)[1],
             lambda: tf.attention(q, k, v, causal=True)[0], lambda: tf.linear_attention(k, v, q, decay=decay)[0]]
    want = [f()[0].clone() for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = []
    for _ in range(10):
        for f, s in zip(calls, streams):
            with torch.cuda.stream(s):
                got.append(f()[0])
    torch.cuda.synchronize()
    for i, x in enumerate(got):
        assert torch.equal(x, want[i % len(calls)])
