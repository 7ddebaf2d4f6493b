"""Refusals of the key-value cache entry points, before any CUDA call (no GPU needed)."""
import ctypes
import math

import pytest

FAKE = 0x10000


@pytest.fixture(scope="module")
def tf():
    from ulysses_sequence_attention_tf_gb300 import binding, build
    build.build()
    return binding


def cache(tf, **kw):
    c = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, num_pages=8, Hkv=4, page_size=16, D=64, N=2, max_pages=4,
             page_table=FAKE, table_stride=4, lens=FAKE, starts=FAKE)
    c.update({n: x for n, x in kw.items() if n in c})
    return tf.KvCache(*[c[n] for n, _ in tf.KvCache._fields_])


def ptrs(p):
    return (ctypes.c_void_p * 8)(*([p] * 8)) if p is not None else None


def append(tf, c, P=2, T=8, H=8, dtype=1, k=FAKE, v=FAKE, q=FAKE, q_out=FAKE, stride=256, o_str=None, nr="given", rope=1, rows=64,
           weight=FAKE, eps=1e-6, cos_sin=FAKE, theta=1e4):
    st = (tf.Strides * 3)(*([tf.Strides(0, stride, 64)] * 3))
    given = tf.NormRope(weight, weight, eps, theta, cos_sin)
    return tf.lib().tf_ulysses_kv_append(ctypes.byref(c), P, T, H, dtype, ptrs(k), ptrs(v), ptrs(q), st, ptrs(q_out),
                                         ctypes.byref(o_str) if o_str else None, ctypes.byref(given) if nr else None, rope, rows, None)


def attend(tf, c, q=FAKE, out=FAKE, lse=None, workspace=None, nbytes=0, stride=256, o_str=None, **kw):
    a = dict(P=2, T=8, H=8, dtype=1, max_tokens=8, max_len=64, scale=0.125, softcap=0.0, causal=1, slopes=None)
    a.update(kw)
    a = tf.KvAttention(*[a[n] for n, _ in tf.KvAttention._fields_])
    n = ctypes.c_size_t()
    asked = tf.lib().tf_ulysses_kv_attend_workspace(ctypes.byref(c), ctypes.byref(a), ctypes.byref(n))
    st = tf.Strides(0, stride, 64)
    status = tf.lib().tf_ulysses_kv_attend(ctypes.byref(c), ctypes.byref(a), ptrs(q), ctypes.byref(st), ptrs(out),
                                           ctypes.byref(o_str) if o_str else None, lse, workspace, nbytes, None)
    return asked, status


CACHES = [
    (dict(num_pages=0), 1), (dict(Hkv=0), 1), (dict(max_pages=0), 1), (dict(N=-1), 1), (dict(Hkv=3), 2), (dict(D=96), 4),
    (dict(D=256), 4), (dict(page_size=8), 4), (dict(page_size=48), 4), (dict(page_size=256), 4), (dict(max_pages=2 ** 27), 4),
    (dict(table_stride=3), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(k_scale=None), 1), (dict(v_scale=None), 1),
    (dict(page_table=None), 1), (dict(lens=None), 1), (dict(starts=None), 1), (dict(k=FAKE + 8), 3), (dict(v=FAKE + 4), 3),
    (dict(v_scale=FAKE + 2), 3), (dict(lens=FAKE + 1), 3),
]


@pytest.mark.parametrize("kw,status", CACHES)
def test_caches_refused(tf, kw, status):
    c = cache(tf, **kw)
    assert append(tf, c) == status and tf.lib().tf_ulysses_last_error()
    assert attend(tf, c) == (status, status)


@pytest.mark.parametrize("kw,status", [
    (dict(P=0), 1), (dict(P=9), 1), (dict(T=-1), 1), (dict(H=7), 2), (dict(H=0), 1), (dict(dtype=2), 4), (dict(dtype=3), 4),
    (dict(k=None), 1), (dict(v=None), 1), (dict(k=0), 1), (dict(v=FAKE + 8), 3), (dict(q=None), 1), (dict(q_out=None), 1),
    (dict(q=FAKE + 4), 3), (dict(stride=-256), 4), (dict(stride=100), 3), (dict(rope=3), 1), (dict(rope=-1), 1), (dict(nr=None), 1),
    (dict(weight=FAKE + 2), 3), (dict(eps=-1.0), 1), (dict(eps=math.nan), 1), (dict(cos_sin=FAKE + 4), 3), (dict(rows=0), 1),
    (dict(cos_sin=None, theta=0.0), 1), (dict(cos_sin=None, theta=math.inf), 1),
])
def test_appends_refused(tf, kw, status):
    assert append(tf, cache(tf), **kw) == status


def test_append_refuses_results_that_overlap(tf):
    assert append(tf, cache(tf), o_str=tf.Strides(0, 0, 64)) == 1


@pytest.mark.parametrize("kw,status", [
    (dict(P=0), 1), (dict(T=-1), 1), (dict(H=6), 2), (dict(H=0), 1), (dict(dtype=2), 4), (dict(max_tokens=0), 1),
    (dict(max_tokens=9), 1), (dict(max_len=0), 1), (dict(max_len=65), 1), (dict(scale=math.nan), 1), (dict(softcap=-1.0), 1),
    (dict(causal=2), 1),
])
def test_attention_refused(tf, kw, status):
    assert attend(tf, cache(tf), **kw) == (status, status)


def test_attention_pointers_refused(tf):
    c = cache(tf)
    for kw, status in ((dict(q=None), 1), (dict(q=0), 1), (dict(q=FAKE + 8), 3), (dict(out=None), 1), (dict(out=0), 1),
                       (dict(stride=100), 3), (dict(o_str=tf.Strides(0, 0, 64)), 1), (dict(lse=(ctypes.c_void_p * 8)(FAKE, 0)), 1)):
        assert attend(tf, c, **kw)[1] == status
