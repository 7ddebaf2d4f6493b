"""Gradients of the attention where rounding, padding and scale show, against 64 bits (bounds derived in attention_util
and beside the tests)."""
import math

import pytest
import torch

from attention_util import Reference
from gradient_util import Gradients

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


def rows(gen, B, S, h, D, dtype, P=1):
    return [torch.randn((B, S, h, D), generator=gen, device="cuda").to(dtype) for _ in range(P)]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("cap", [0.5, 50.0])  # both forms of the cap's tanh
@pytest.mark.parametrize("biased", [False, True])
def test_padding_may_hold_anything_under_a_cap(tf, biased, cap, causal, D, dtype):
    S = 300
    gen = torch.Generator(device="cuda").manual_seed(17)
    q, dout = rows(gen, 2, S, 2, D, dtype), rows(gen, 2, S, 2, D, dtype)
    k, v = rows(gen, 2, S, 1, D, dtype), rows(gen, 2, S, 1, D, dtype)
    docs = torch.tensor([[0] * 200 + [-1] * 100, [-1] * 33 + [1] * 100 + [-5] * 40 + [2] * 127], dtype=torch.int32, device="cuda")
    pad = docs < 0
    kw = dict(q_docs=docs, k_docs=docs, softcap=cap, causal=causal)
    if biased:
        kw["slopes"] = torch.tensor([0.5, 0.01], device="cuda")
    ref = Reference(q, k, v, dout, clean=True, **kw)
    for first, second in ((math.nan, math.inf), (-math.inf, math.nan), (float(torch.finfo(dtype).max),) * 2):
        for ts in (q, k, v, dout):
            ts[0][pad] = first
            ts[0][:, -1] = torch.where(pad[:, -1, None, None], torch.tensor(second, device="cuda", dtype=dtype), ts[0][:, -1])
        out, lse = tf.attention(q, k, v, **kw)
        dq, dk, dv = tf.attention_backward(dout, q, k, v, out, lse, **kw)
        for name, got in (("out", out), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
            ref.check(name, got)


def sharp(tf, q, k, v, dout, *, docs=None, **kw):
    """Gradients against bounds in which the output's rounding has no part but times another rounding."""
    call = dict(kw, **({} if docs is None else dict(q_docs=docs, k_docs=docs)))
    out, lse = tf.attention(q, k, v, **call)
    dq, dk, dv = tf.attention_backward(dout, q, k, v, out, lse, **call)
    ref = Gradients(q, k, v, dout, out, docs=docs, **kw)
    ref.check("dq", dq)
    ref.check("dk", dk)
    Reference(q, k, v, dout, **call).check("dv", dv)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_rows_in_which_few_keys_weigh(tf, cap, D, dtype):
    """Steep distances leave a row one to six of two thousand keys that it sees."""
    gen = torch.Generator(device="cuda").manual_seed(63)
    x = [rows(gen, 1, 2000, 2, D, dtype, P=2) for _ in range(4)]
    for causal in (True, False):
        sharp(tf, *x, slopes=torch.tensor([0.5, 0.63, 1.0, 2.0], device="cuda"), softcap=cap, causal=causal)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_short_documents_behind_long_ones(tf, causal, D, dtype):
    """A document's gradients do not depend on what shares its tiles."""
    gen = torch.Generator(device="cuda").manual_seed(64)
    lens = [1500, 3, 1, 2, 700, 1, 1, 5, 20, 400]
    docs = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens)).to(torch.int32).cuda()[None]
    x = [rows(gen, 1, sum(lens), 2, D, dtype) for _ in range(4)]
    sharp(tf, *x, docs=docs, causal=causal)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("D,Sq,Sk", [(64, 2100, 2100), (128, 2100, 2100), (128, 300, 5000), (64, 20000, 1100)])
def test_keys_and_values_with_a_common_part(tf, Sq, Sk, D, dtype):
    """Their means as large as their spread: what delta lacks adds up over a row (the last two: units in parts)."""
    gen = torch.Generator(device="cuda").manual_seed(65)
    q, dout = rows(gen, 1, Sq, 1, D, dtype), rows(gen, 1, Sq, 1, D, dtype)
    k, v = ([t + 1 for t in rows(gen, 1, Sk, 1, D, dtype)] for _ in range(2))
    sharp(tf, q, k, v, dout)
    sharp(tf, q, k, v, dout, softcap=5.0)
    if Sq == Sk:
        sharp(tf, q, k, v, dout, causal=True)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("D", [64, 128])
def test_one_score_that_dominates(tf, D, dtype):
    gen = torch.Generator(device="cuda").manual_seed(66)
    q, k, v, dout = (rows(gen, 1, 1100, 2, D, dtype) for _ in range(4))
    q[0] += 3 * k[0]  # a query close to the key at its own position
    sharp(tf, q, k, v, dout)
    sharp(tf, q, k, v, dout, causal=True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("factor", [2.0 ** -14, 2.0 ** -10, 1.0, 2.0 ** 8])
@pytest.mark.parametrize("Sq,Sk,kw", [(300, 6000, {}), (2500, 2500, dict(causal=True)), (2500, 2500, dict(softcap=3.0))])
def test_fp16_gradients_of_any_size(tf, Sq, Sk, kw, factor, D):
    """Gradients of the scores are about |dout| / Sk: far below fp16's normal range, or (times large values) above it.
    dout is a multiple of 2^-2 below 4, exact in fp16 times each factor."""
    gen = torch.Generator(device="cuda").manual_seed(67)
    q, k, v = (rows(gen, 1, S, 2, D, FP16) for S in (Sq, Sk, Sk))
    dout = [(4 * t).round().clamp(-15, 15) / 4 * factor for t in rows(gen, 1, Sq, 2, D, FP16)]
    if factor > 1:
        v = [64 * t for t in v]
        k = [t / 16 for t in k]  # dQ stays within fp16
    out, lse = tf.attention(q, k, v, **kw)
    dq, dk, dv = tf.attention_backward(dout, q, k, v, out, lse, **kw)
    # dx is kept times a power of two that puts |dout| |v| at 2^13 or above; below fp16's normal range a
    # rounding is off by 2^-25 at most
    flush = 2.0 ** -38 * max(float(t.double().norm(dim=-1).max()) for t in dout) * max(float(t.double().norm(dim=-1).max()) for t in v)
    ref = Gradients(q, k, v, dout, out, flush=flush, **kw)
    ref.check("dq", dq)
    ref.check("dk", dk)
    assert dv[0].isfinite().all()


def test_fp16_padding_has_no_part_in_the_gradients_size(tf):
    gen = torch.Generator(device="cuda").manual_seed(68)
    q, k, v, dout = (rows(gen, 1, 900, 2, 64, FP16) for _ in range(4))
    dout = [t * 2.0 ** -9 for t in dout]
    docs = torch.tensor([[0] * 700 + [-1] * 200], dtype=torch.int32, device="cuda")
    kw = dict(q_docs=docs, k_docs=docs)
    got = []
    for value in (0.0, 60000.0, math.inf, math.nan):
        for ts in (q, k, v, dout):
            ts[0][:, 700:] = value
        out, lse = tf.attention(q, k, v, **kw)
        got.append(tf.attention_backward(dout, q, k, v, out, lse, **kw))
        assert all(torch.equal(a, b) for x, y in zip(got[0], got[-1]) for a, b in zip(x, y)), value


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap,scale", [(1e-12, 1.0), (1e-30, 0.125), (1e-37, 0.125), (1e27, 1e30), (1e30, 0.125), (1e38, 2.0)])
def test_caps_of_any_size_over_scores_of_zero(tf, cap, scale, D):
    """The cap's polynomial takes factors of scale and cap; rows of zeros weigh all of their keys alike."""
    gen = torch.Generator(device="cuda").manual_seed(69)
    k, v, dout = (rows(gen, 1, 400, 2, D, BF16) for _ in range(3))
    q = [torch.zeros_like(t) for t in dout]
    out, lse = tf.attention(q, k, v, softcap=cap, scale=scale)
    Reference(q, k, v, softcap=0.0, scale=0.0).check("out", out)
    assert bool(((lse[0] - math.log(400)).abs() <= 2.0 ** -16).all())
    if cap >= 1e30:  # scores far below the cap: as without one
        q = rows(gen, 1, 400, 2, D, BF16)
        out, lse = tf.attention(q, k, v, softcap=cap, scale=scale)
        ref = Reference(q, k, v, dout, scale=scale)
        ref.check("out", out)
        for name, got in zip(("dq", "dk", "dv"), tf.attention_backward(dout, q, k, v, out, lse, softcap=cap, scale=scale)):
            ref.check(name, got)
