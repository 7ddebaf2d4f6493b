"""Refusals of the rotation, the cache's plan and linear attention before any CUDA call, and the frequencies (no GPU needed)."""
import ctypes
import math

import pytest

FAKE = 0x100000


@pytest.fixture(scope="module")
def tf():
    from ulysses_sequence_attention_tf_gb300 import binding, build
    build.build()
    return binding


def ptrs(p, second=None):
    return (ctypes.c_void_p * 8)(p, *([p if second is None else second] * 7)) if p is not None else None


def strides(tf, n, b, t, h):
    return (tf.Strides * n)(*([tf.Strides(b, t, h)] * n))


# ---------------------------------------------------------------- rotation
def rotate(tf, q=FAKE, k=FAKE, q_out=FAKE + 0x100000, k_out=FAKE + 0x200000, st=(4096, 256, 64), out_st=None, frequency=1.0, second=None,
           null_frequencies=False, **kw):
    r = dict(P=2, B=2, T=16, H=8, Hk=8, D=64, rotary_dim=64, dtype=1, rope=1, inverse=0, magnitude=1.0, positions=None, first=0)
    r.update(kw)
    f = (ctypes.c_double * 128)(*([frequency] * 128))
    c = tf.Rotary(*[r[n] for n in ("P", "B", "T", "H", "Hk", "D", "rotary_dim", "dtype", "rope", "inverse", "magnitude")],
                  ctypes.cast(None if null_frequencies else f, ctypes.POINTER(ctypes.c_double)), r["positions"], r["first"])
    return tf.lib().tf_ulysses_rope(ctypes.byref(c), ptrs(q), ptrs(k), strides(tf, 2, *st), ptrs(q_out, second), ptrs(k_out),
                                    strides(tf, 2, *out_st) if out_st else None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(P=0), 1), (dict(P=9), 1), (dict(B=-1), 1), (dict(T=-1), 1), (dict(H=0), 1), (dict(Hk=0), 1), (dict(H=7), 2), (dict(Hk=3), 2),
    (dict(D=60), 4), (dict(D=264, rotary_dim=64), 4), (dict(D=0), 4), (dict(rotary_dim=0), 1), (dict(rotary_dim=63), 1),
    (dict(rotary_dim=66), 1), (dict(dtype=2), 4), (dict(dtype=3), 4), (dict(rope=0), 1), (dict(rope=3), 1), (dict(inverse=2), 1),
    (dict(magnitude=math.inf), 1), (dict(magnitude=math.nan), 1), (dict(frequency=math.nan), 1), (dict(frequency=math.inf), 1),
    (dict(null_frequencies=True), 1), (dict(q=None), 1), (dict(q_out=None), 1), (dict(k=None), 1), (dict(k_out=None), 1),
    (dict(q=FAKE + 8), 3), (dict(k_out=FAKE + 2), 3), (dict(positions=FAKE + 2), 3), (dict(st=(4096, 252, 64)), 3),
    (dict(st=(4096, -256, 64)), 4), (dict(out_st=(4096, 0, 64)), 1), (dict(out_st=(0, 256, 64)), 1),
    (dict(q_out=FAKE, out_st=(8192, 512, 64)), 1), (dict(q_out=FAKE, out_st=(4096, 256, 64), second=FAKE + 0x100000), 1),
    (dict(B=2 ** 14, T=2 ** 14), 4),
])
def test_rotations_refused(tf, kw, status):
    assert rotate(tf, **kw) == status and tf.lib().tf_ulysses_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(rotary_dim=0), 1), (dict(rotary_dim=3), 1), (dict(rotary_dim=258), 1), (dict(theta=0.0), 1), (dict(theta=math.inf), 1),
    (dict(scaling="linear", factor=0.0), 1), (dict(scaling="linear", factor=math.nan), 1), (dict(scaling="base", rotary_dim=2), 1),
    (dict(scaling="parts", original=0), 1), (dict(scaling="parts", low=4.0, high=4.0), 1), (dict(scaling="parts", high=math.nan), 1),
])
def test_frequencies_refused(tf, kw, status):
    args = dict(rotary_dim=64, factor=2.0)
    args.update(kw)
    with pytest.raises(tf.TfUlyssesError) as e:
        tf.rope_frequencies(**args)
    assert e.value.status == status


@pytest.mark.parametrize("R", [2, 20, 64, 128, 256])
@pytest.mark.parametrize("scaling", [None, "linear", "base", "parts"])
def test_frequencies(tf, R, scaling):
    if scaling == "base" and R == 2:
        return
    got = tf.rope_frequencies(R, 500.0, scaling=scaling, factor=4.0, original=1000, low=1.0, high=8.0).tolist()
    for i, f in enumerate(got):
        base = 500.0 * 4.0 ** (R / (R - 2)) if scaling == "base" else 500.0
        want = base ** (-2 * i / R)
        if scaling == "linear":
            want /= 4
        if scaling == "parts":
            turns = 1000 * want / (2 * math.pi)
            if turns >= 8:
                pass
            elif turns <= 1:
                want /= 4
            else:
                want = want * (turns - 1) / 7 + want / 4 * (8 - turns) / 7
        assert abs(f - want) <= 1e-13 * want
    with pytest.raises(ValueError):
        tf.rope_frequencies(R, scaling="dynamic")


# ---------------------------------------------------------------- plan
def plan(tf, **kw):
    n = iter(range(1, 20))
    a = dict(N=4, max_pages=8, page_size=16, num_pages=32, T=64, table_stride=8)
    for name in ("page_table", "lens", "new_tokens", "free_pages", "free_span", "lens_out", "starts", "positions", "slots", "span_out"):
        a[name] = FAKE + 0x10000 * next(n)
    a.update(kw)
    p = tf.Plan(*[a[name] for name, _ in tf.Plan._fields_])
    return tf.lib().tf_ulysses_kv_plan(ctypes.byref(p), None)


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), 1), (dict(T=-1), 1), (dict(max_pages=0), 1), (dict(num_pages=0), 1), (dict(page_size=24), 4), (dict(page_size=256), 4),
    (dict(N=8193), 4), (dict(T=2 ** 30), 4), (dict(max_pages=2 ** 27, table_stride=2 ** 27), 4), (dict(num_pages=2 ** 27), 4),
    (dict(table_stride=7), 1), (dict(page_table=None), 1), (dict(lens=None), 1), (dict(new_tokens=None), 1), (dict(free_pages=None), 1),
    (dict(free_span=None), 1), (dict(lens_out=None), 1), (dict(starts=None), 1), (dict(positions=None), 1), (dict(slots=None), 1),
    (dict(span_out=None), 1), (dict(lens=FAKE + 2), 3), (dict(starts=FAKE + 1), 3),
    # outputs over inputs or one another
    (dict(lens=FAKE, lens_out=FAKE), 1), (dict(lens=FAKE, lens_out=FAKE + 12), 1), (dict(free_span=FAKE, span_out=FAKE + 4), 1),
    (dict(positions=FAKE, slots=FAKE + 252), 1), (dict(page_table=FAKE, starts=FAKE + 124), 1),
])
def test_plans_refused(tf, kw, status):
    assert plan(tf, **kw) == status and tf.lib().tf_ulysses_last_error()


# ---------------------------------------------------------------- linear attention
def linear(tf, backward=False, q=FAKE, out=FAKE, state=None, last=None, workspace=None, nbytes=0, st=(4096, 256, 64), out_st=None, **kw):
    a = dict(P=2, B=2, S=16, H=8, D=64, dtype=1, scale=0.125, decay=FAKE)
    a.update(kw)
    c = tf.Linear(*[a[n] for n, _ in tf.Linear._fields_])
    n = ctypes.c_size_t()
    asked = tf.lib().tf_ulysses_linear_attention_workspace(ctypes.byref(c), int(backward), ctypes.byref(n))
    o = strides(tf, 3, *out_st) if out_st else None
    if backward:
        got = tf.lib().tf_ulysses_linear_attention_backward(ctypes.byref(c), ptrs(FAKE), ptrs(q), ptrs(FAKE), ptrs(FAKE),
                                                            strides(tf, 4, *st), state, last, ptrs(out), ptrs(FAKE), ptrs(FAKE), o, None,
                                                            workspace, nbytes, None)
    else:
        got = tf.lib().tf_ulysses_linear_attention(ctypes.byref(c), ptrs(q), ptrs(FAKE), ptrs(FAKE), strides(tf, 3, *st), state,
                                                   ptrs(out), o, last, workspace, nbytes, None)
    return asked, got


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("kw,status,asked", [
    (dict(P=0), 1, 1), (dict(P=9), 1, 1), (dict(B=-1), 1, 1), (dict(S=-1), 1, 1), (dict(H=0), 1, 1), (dict(H=7), 2, 2), (dict(D=96), 4, 4),
    (dict(D=256), 4, 4), (dict(dtype=2), 4, 4), (dict(scale=math.nan), 1, 1), (dict(scale=math.inf), 1, 1), (dict(decay=None), 1, 1),
    (dict(decay=FAKE + 2), 3, 3), (dict(S=2 ** 30 + 1), 4, 4), (dict(B=2 ** 20, S=2 ** 20), 4, 4), (dict(B=2 ** 25, S=0, last=FAKE), 4, 4),
    (dict(q=None), 1, 0), (dict(out=None), 1, 0), (dict(q=FAKE + 8), 3, 0), (dict(out=FAKE + 4), 3, 0), (dict(state=FAKE + 4), 3, 0),
    (dict(last=FAKE + 8), 3, 0), (dict(st=(4096, 252, 64)), 3, 0), (dict(st=(4096, 256, -64)), 4, 0), (dict(st=(4096, 0, 64)), 4, 0),
    (dict(out_st=(4096, 256, 0)), 1, 0),
])
def test_linear_attention_refused(tf, kw, status, asked, backward):
    assert linear(tf, backward, **kw) == (asked, status) and tf.lib().tf_ulysses_last_error()


def test_states_that_overlap_are_refused(tf):
    """A final state shifted against the state by less than its size (2 * 8 * 64 * 64 floats)."""
    assert linear(tf, state=FAKE, last=FAKE + 0x10000) == (0, 1)
    assert b"overlaps" in tf.lib().tf_ulysses_last_error()


def attend(tf, q=FAKE, workspace=None, nbytes=0, **kw):
    a = dict(P=2, B=1, S=16, H=8, D=64, dtype=1, scale=0.125, decay=FAKE)
    p = dict(states=FAKE, num_slots=4, N=3, slots=FAKE, starts=FAKE, max_tokens=8)
    a.update({n: x for n, x in kw.items() if n in a})
    p.update({n: x for n, x in kw.items() if n in p})
    a, p = tf.Linear(*[a[n] for n, _ in tf.Linear._fields_]), tf.LinearPool(*[p[n] for n, _ in tf.LinearPool._fields_])
    n = ctypes.c_size_t()
    asked = tf.lib().tf_ulysses_linear_attend_workspace(ctypes.byref(a), ctypes.byref(p), ctypes.byref(n))
    got = tf.lib().tf_ulysses_linear_attend(ctypes.byref(a), ctypes.byref(p), ptrs(q), ptrs(FAKE), ptrs(FAKE), strides(tf, 3, 0, 256, 64),
                                            ptrs(FAKE), None, workspace, nbytes, None)
    return asked, got


@pytest.mark.parametrize("kw,status,asked", [
    (dict(B=2), 1, 1), (dict(N=-1), 1, 1), (dict(num_slots=0), 1, 1), (dict(states=None), 1, 1), (dict(slots=None), 1, 1),
    (dict(starts=None), 1, 1), (dict(states=FAKE + 4), 3, 3), (dict(slots=FAKE + 2), 3, 3), (dict(starts=FAKE + 1), 3, 3),
    (dict(max_tokens=0), 1, 1), (dict(max_tokens=17), 1, 1), (dict(N=2 ** 28), 4, 4), (dict(D=32), 4, 4), (dict(H=3), 2, 2), (dict(q=None), 1, 0),
    (dict(q=FAKE + 4), 3, 0),
])
def test_linear_attend_refused(tf, kw, status, asked):
    assert attend(tf, **kw) == (asked, status) and tf.lib().tf_ulysses_last_error()
