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
