"""Outputs that start where an input or another output does are refused before any CUDA call (no GPU needed)."""
import ctypes

import pytest

AT = {n: 0x1000000 * (i + 1) for i, n in enumerate(("q", "k", "v", "dout", "out", "dq", "dk", "dv", "q_out", "k_out"))}


@pytest.fixture(scope="module")
def tf():
    from ulysses_sequence_attention_tf_gb300 import binding, build
    build.build()
    return binding


def arrays(names, over):
    """Two head groups a tensor, 0x100000 apart; over = (tensor, group, tensor, group): the first lies where the second does."""
    at = {n: [AT[n], AT[n] + 0x100000] for n in names}
    if over:
        at[over[0]][over[1]] = at[over[2]][over[3]]
    return {n: (ctypes.c_void_p * 8)(*x) for n, x in at.items()}


def linear(tf, call, over):
    """[2, 4, 4, 64] in two groups; without a workspace of its own and without a GPU a call that is not refused for its
    tensors ends in a CUDA error."""
    a = tf.Linear(2, 2, 4, 8, 64, 1, 0.125, 0x100000)
    st = (tf.Strides * 4)(*[tf.Strides(1024, 256, 64)] * 4)
    L = tf.lib()
    if call == "backward":
        p = arrays(("dout", "q", "k", "v", "dq", "dk", "dv"), over)
        return L.tf_ulysses_linear_attention_backward(ctypes.byref(a), p["dout"], p["q"], p["k"], p["v"], st, None, None, p["dq"], p["dk"],
                                                      p["dv"], None, None, None, 0, None)
    p = arrays(("q", "k", "v", "out"), over)
    if call == "forward":
        return L.tf_ulysses_linear_attention(ctypes.byref(a), p["q"], p["k"], p["v"], st, None, p["out"], None, None, None, 0, None)
    a.B = 1
    pool = tf.LinearPool(0x200000, 4, 1, 0x100000, 0x100000, 4)
    return L.tf_ulysses_linear_attend(ctypes.byref(a), ctypes.byref(pool), p["q"], p["k"], p["v"], st, p["out"], None, None, 0, None)


def rotate(tf, over, k=True):
    f = (ctypes.c_double * 32)(*[1.0] * 32)
    r = tf.Rotary(2, 2, 4, 8, 8, 64, 64, 1, 1, 0, 1.0, ctypes.cast(f, ctypes.POINTER(ctypes.c_double)), None, 0)
    p = arrays(("q", "k", "q_out", "k_out"), over)
    st = (tf.Strides * 2)(*[tf.Strides(1024, 256, 64)] * 2)
    return tf.lib().tf_ulysses_rope(ctypes.byref(r), p["q"], p["k"] if k else None, st, p["q_out"], p["k_out"] if k else None, None, None)


@pytest.mark.parametrize("call,over", [
    ("forward", ("out", 0, "q", 0)), ("forward", ("out", 1, "k", 0)), ("forward", ("out", 0, "v", 1)), ("forward", ("out", 0, "out", 1)),
    ("attend", ("out", 1, "q", 1)), ("attend", ("out", 0, "v", 0)), ("attend", ("out", 1, "out", 0)),
    ("backward", ("dq", 0, "q", 0)), ("backward", ("dq", 1, "dout", 1)), ("backward", ("dk", 0, "v", 1)), ("backward", ("dv", 1, "k", 0)),
    ("backward", ("dq", 0, "dk", 0)), ("backward", ("dk", 1, "dv", 0)), ("backward", ("dv", 0, "dv", 1)),
])
def test_linear_attention(tf, call, over):
    assert linear(tf, call, over) == 1
    message = tf.lib().tf_ulysses_last_error().decode()
    assert "overlaps" in message and over[0] in message and over[2] in message


@pytest.mark.parametrize("over", [("q_out", 0, "k", 0), ("k_out", 1, "q", 1), ("q_out", 0, "k_out", 0), ("q_out", 0, "q_out", 1),
                                  ("k_out", 0, "k_out", 1)])
def test_rotation(tf, over):
    assert rotate(tf, over) == 1
    assert "overlaps" in tf.lib().tf_ulysses_last_error().decode()


def test_groups_in_place_of_one_another(tf):
    """q_out[0] is q[1] and q_out[1] is q[0]."""
    f = (ctypes.c_double * 32)(*[1.0] * 32)
    r = tf.Rotary(2, 2, 4, 8, 8, 64, 64, 1, 1, 0, 1.0, ctypes.cast(f, ctypes.POINTER(ctypes.c_double)), None, 0)
    st = (tf.Strides * 2)(*[tf.Strides(1024, 256, 64)] * 2)
    q, q_out = (ctypes.c_void_p * 8)(AT["q"], AT["k"]), (ctypes.c_void_p * 8)(AT["k"], AT["q"])
    assert tf.lib().tf_ulysses_rope(ctypes.byref(r), q, None, st, q_out, None, st, None) == 1
    assert "overlaps" in tf.lib().tf_ulysses_last_error().decode()
