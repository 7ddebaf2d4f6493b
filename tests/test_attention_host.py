"""Refusals of the attention entry points, before any CUDA call (no GPU needed)."""
import ctypes
import math

import pytest

FAKE = 0x10000


@pytest.fixture(scope="module")
def tf():
    from ulysses_sequence_attention_tf_gb300 import binding, build
    build.build()
    return binding


def describe(tf, **kw):
    a = dict(P=2, B=1, Sq=8, Sk=8, H=4, Hkv=2, D=64, dtype=1, scale=0.125, softcap=0.0, causal=0, slopes=None, prefix=None,
             q_docs=None, k_docs=None)
    a.update(kw)
    return tf.Attention(*[a[n] for n, _ in tf.Attention._fields_])


def forward(tf, a, q=FAKE, k=FAKE, v=FAKE, out=FAKE, strides=None, out_strides=None, lse=None):
    ptrs = [(ctypes.c_void_p * 8)(*([p] * 8)) if p is not None else None for p in (q, k, v, out)]
    st = (tf.Strides * 3)(*(strides or [tf.Strides(8 * 2 * 64, 2 * 64, 64)] * 3))
    return tf.lib().tf_ulysses_attention(ctypes.byref(a), *ptrs[:3], st, ptrs[3],
                                         ctypes.byref(out_strides) if out_strides else None, lse, None, 0, None)


def backward(tf, a, workspace=None, nbytes=0, lse=FAKE, dk=FAKE):
    arr = (ctypes.c_void_p * 8)(*([FAKE] * 8))
    st = (tf.Strides * 5)(*([tf.Strides(8 * 2 * 64, 2 * 64, 64)] * 5))
    return tf.lib().tf_ulysses_attention_backward(
        ctypes.byref(a), arr, arr, arr, arr, arr, (ctypes.c_void_p * 8)(*([lse] * 8)) if lse else None, st, arr,
        (ctypes.c_void_p * 8)(*([dk] * 8)) if dk else None, arr, None, workspace, nbytes, None)


REFUSED = [
    (dict(P=0), 1), (dict(P=9), 1), (dict(B=-1), 1), (dict(Sq=-1), 1), (dict(Sk=-1), 1), (dict(H=0), 1), (dict(Hkv=0), 1),
    (dict(P=4), 2), (dict(H=3), 2), (dict(dtype=2), 4), (dict(dtype=3), 4), (dict(dtype=9), 4), (dict(D=32), 4),
    (dict(D=96), 4), (dict(D=256), 4), (dict(scale=math.nan), 1), (dict(scale=math.inf), 1), (dict(softcap=-1.0), 1),
    (dict(softcap=math.nan), 1), (dict(softcap=math.inf), 1), (dict(causal=2), 1), (dict(prefix=FAKE), 1),
    (dict(q_docs=FAKE), 1), (dict(k_docs=FAKE), 1), (dict(Sq=2 ** 30, Sk=2 ** 30), 4),
]


@pytest.mark.parametrize("kw,status", REFUSED)
def test_descriptions_refused(tf, kw, status):
    a = describe(tf, **kw)
    n = ctypes.c_size_t()
    assert forward(tf, a) == status and tf.lib().tf_ulysses_last_error()
    assert backward(tf, a) == status
    assert tf.lib().tf_ulysses_attention_workspace(ctypes.byref(a), 0, ctypes.byref(n)) == status


def test_pointers_and_strides_refused(tf):
    a = describe(tf)
    for name in ("q", "k", "v", "out"):
        assert forward(tf, a, **{name: None}) == 1
        assert forward(tf, a, **{name: 0}) == 1
        assert forward(tf, a, **{name: FAKE + 8}) == 3
    good = tf.Strides(8 * 2 * 64, 2 * 64, 64)
    assert forward(tf, a, strides=[good, tf.Strides(8 * 2 * 64, 2 * 64 + 4, 64), good]) == 3
    assert forward(tf, a, strides=[good, good, tf.Strides(8 * 2 * 64, -128, 64)]) == 4
    assert forward(tf, a, out_strides=tf.Strides(8 * 2 * 64, 0, 64)) == 1
    assert forward(tf, a, lse=(ctypes.c_void_p * 8)(FAKE, 0)) == 1
    assert tf.lib().tf_ulysses_attention(None, None, None, None, None, None, None, None, None, 0, None) == 1


def test_gradient_needs_its_statistics_and_workspace(tf):
    a = describe(tf)
    n = ctypes.c_size_t()
    assert tf.lib().tf_ulysses_attention_workspace(ctypes.byref(a), 1, ctypes.byref(n)) == 0 and n.value > 0
    assert tf.lib().tf_ulysses_attention_workspace(ctypes.byref(a), 1, None) == 1
    assert backward(tf, a, None, n.value) == 1
    assert backward(tf, a, FAKE, n.value - 1) == 1
    assert backward(tf, a, FAKE + 4, n.value) == 3
    assert backward(tf, a, FAKE, n.value, lse=None) == 1
    assert backward(tf, a, FAKE, n.value, lse=0) == 1
    assert backward(tf, a, FAKE, n.value, dk=0) == 1


def test_tensors_off_the_device_refused(tf):
    """The binding's checks of tensors, which need no GPU to refuse a call."""
    torch = pytest.importorskip("torch")
    calls = tf._torch_calls()
    q = [torch.zeros((1, 8, 2, 64), dtype=torch.bfloat16)]
    before, none = (q, q, q, None, 0.0, None, False, None, None, None, 0, 0), [None] * 5
    with pytest.raises(ValueError, match="on the current device"):
        calls.attention(*before, None, None)
    with pytest.raises(ValueError, match="on the current device"):
        calls.attention_backward(*before, q, q, [torch.zeros((1, 2, 8))], None, None, None)
    for bad in (None, 1, q[0], [], q * 9, [None]):
        with pytest.raises(ValueError):
            calls.attention(bad, *before[1:], None, None)
    with pytest.raises(TypeError):
        calls.attention(*before)
    cache = tf.kv_cache(4, 2, 16, 64, device="cpu")
    where = [torch.zeros(s, dtype=torch.int32) for s in ((1, 2), (1,), (2,))]
    rows = [torch.zeros((3, 2, 64), dtype=torch.bfloat16)]
    with pytest.raises(ValueError, match="page_table"):
        calls.kv_append(*cache, *where, 0, 0, rows, rows, None, None, None, None, 1e-6, 1e4, None, 0)
    with pytest.raises(ValueError, match="page_table"):
        calls.kv_attend(*cache, *where, 0, 0, rows, *none, 0.0, None, True)
    with pytest.raises(ValueError):
        calls.kv_attend(*[None] * 7, 0, 0, rows, *none, 0.0, None, True)
    with pytest.raises(ValueError, match="rope"):
        tf.kv_append(cache, *where, rows, rows, rope="other")


@pytest.mark.parametrize("name", ["attention", "attention_backward", "kv_append", "kv_attend"])
def test_a_call_on_a_stream_takes_the_streams_device(tf, monkeypatch, name):
    """The device that tensors are checked against and the raw stream are those of the stream's context, whose
    device may be another than the caller's; no GPU is needed to see which are handed over."""
    import contextlib

    import torch
    current = [0]

    @contextlib.contextmanager
    def entered(stream):
        before, current[0] = current[0], stream
        try:
            yield
        finally:
            current[0] = before

    class Calls:
        def __getattr__(self, called):
            return lambda *args: (called, args)

    monkeypatch.setattr(tf, "_calls", Calls())
    monkeypatch.setattr(tf, "_on_stream", entered)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 1000 * (device + 1) + current[0], raising=False)
    for stream, device in ((1, 1), (0, 0), (None, 0)):
        called, args = tf._run(name, stream, ("before",), ("after",))
        assert called == name and args == ("before", device, 1001 * device + 1000, "after")
    assert current == [0]


@pytest.mark.parametrize("kw", [dict(softcap=1e-40), dict(softcap=2.0 ** -127, scale=4.0), dict(softcap=3e38), dict(softcap=1e38, scale=1e-3),
                                dict(softcap=1e-45, scale=-1.0), dict(softcap=1e38, scale=1.0)])
def test_caps_out_of_the_kernels_range_refused(tf, kw):
    """Scores are divided by the cap as scale / softcap, in fp32."""
    a = describe(tf, **kw)
    n = ctypes.c_size_t()
    assert forward(tf, a) == 4 and backward(tf, a) == 4
    assert tf.lib().tf_ulysses_attention_workspace(ctypes.byref(a), 0, ctypes.byref(n)) == 4
    c = tf.KvCache(FAKE, FAKE, FAKE, FAKE, 8, 2, 16, 64, 2, 4, FAKE, 4, FAKE, FAKE)
    a = tf.KvAttention(2, 8, 8, 1, 8, 64, kw.get("scale", 0.125), kw["softcap"], 1, None)
    assert tf.lib().tf_ulysses_kv_attend_workspace(ctypes.byref(c), ctypes.byref(a), ctypes.byref(n)) == 4


@pytest.mark.parametrize("kw", [dict(softcap=1e-30), dict(softcap=1e30), dict(softcap=1e38, scale=2.0), dict(softcap=1e-38, scale=0.0),
                                dict(softcap=1e-37, scale=-0.5)])
def test_caps_in_the_kernels_range(tf, kw):
    a, n = describe(tf, **kw), ctypes.c_size_t()
    assert tf.lib().tf_ulysses_attention_workspace(ctypes.byref(a), 1, ctypes.byref(n)) == 0
