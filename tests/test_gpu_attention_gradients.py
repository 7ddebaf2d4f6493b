"""Gradients of the attention where rounding, padding and scale show, against 64 bits (bounds derived in attention_util
and beside the tests)."""
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
