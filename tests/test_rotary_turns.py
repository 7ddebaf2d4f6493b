"""The 64-bit fractions of a turn that stand for frequencies (csrc/rotary_turns.h) against exact rationals, on the CPU."""
import ctypes
import math
import os
import random
import subprocess
from fractions import Fraction

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "ulysses_sequence_attention_tf_gb300", "csrc")

SHIM = r'''
#include "rotary_turns.h"
extern "C" uint64_t turn_fraction(double f) { return tfu::turn_fraction(f); }
'''


@pytest.fixture(scope="module")
def fraction(tmp_path_factory):
    at = tmp_path_factory.mktemp("turns")
    (at / "turns.cpp").write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", f"-I{CSRC}", "-o", at / "turns.so", at / "turns.cpp"], check=True)
    f = ctypes.CDLL(str(at / "turns.so")).turn_fraction
    f.argtypes, f.restype = [ctypes.c_double], ctypes.c_uint64
    return f


def pi(bits):
    """By Machin's formula, floor(pi 2^bits) but for a few units."""
    one = 1 << (bits + 32)

    def arctan(x):
        term, total, n = one // x, one // x, 1
        while term:
            term, n = -term // (x * x), n + 2
            total += term // n
            if abs(term) <= 1:
                break
        return total

    return Fraction(4 * (4 * arctan(5) - arctan(239)), one)


TWO_PI = 2 * pi(400)


def off(got, f):
    """Distance of got 2^-64 from f / 2 pi modulo a turn, in 2^-64."""
    d = (Fraction(got) - Fraction(f) / TWO_PI * 2 ** 64) % 2 ** 64
    return float(min(d, 2 ** 64 - d))


def test_two_pi():
    """Against sine and cosine in 64 bits, and its first binary places."""
    assert math.floor(TWO_PI * 2 ** 61) == 0xc90fdaa22168c234 and abs(math.sin(float(TWO_PI))) < 3e-16


NAMED = [1.0, -1.0, 0.5, 7.5, -0.3, 100.25, -100.25, -1e-6, 1e-20, -1e-20, 1e-300, -5e-324, 0.0, -0.0, math.pi, 2 * math.pi, -2 * math.pi, 1e9, -1e9,
         2.0 ** 52, 2.0 ** 53 + 2, 2.0 ** 59 + 2.0 ** 10, 2.0 ** 60, -2.0 ** 60, math.nextafter(1.0, 0.0)]


@pytest.mark.parametrize("f", NAMED)
def test_named_frequencies(fraction, f):
    # half a unit of the rounding, and 2^60 2^-128 2^64 of 1 / 2 pi's bits that are left out
    assert off(fraction(f), f) <= 0.5 + 2.0 ** -4


def test_random_frequencies(fraction):
    rng = random.Random(1)
    for _ in range(5000):
        f = math.ldexp(rng.uniform(-1, 1), rng.randint(-80, 60))
        assert off(fraction(f), f) <= 0.5 + 2.0 ** -4, f


@pytest.mark.parametrize("theta", [10000.0, 500000.0, 0.01])
def test_far_angles(fraction, theta):
    """Angles of the farthest positions are the exact ones to 2^-33 of a turn, where a product in 64-bit floats is not."""
    for i in range(64):
        f = theta ** (-2 * i / 128)
        for at in (2 ** 31 - 1, -2 ** 31, 12345):
            turn = (at * fraction(f)) % 2 ** 64
            d = (Fraction(turn, 2 ** 64) - Fraction(f) * at / TWO_PI) % 1
            assert min(d, 1 - d) <= Fraction(1, 2 ** 33)


@pytest.mark.parametrize("f", [2.0 ** 60 * 1.0001, -2.0 ** 61, 1e300])
def test_frequencies_beyond_that_are_refused(f):
    from ulysses_sequence_attention_tf_gb300 import binding, build
    build.build()
    one, fake = (ctypes.c_double * 1)(f), (ctypes.c_void_p * 8)(*[0x100000] * 8)
    r = binding.Rotary(1, 1, 4, 2, 2, 64, 2, 1, 1, 0, 1.0, ctypes.cast(one, ctypes.POINTER(ctypes.c_double)), None, 0)
    st = (binding.Strides * 2)(*[binding.Strides(512, 128, 64)] * 2)
    assert binding.lib().tf_ulysses_rope(ctypes.byref(r), fake, None, st, fake, None, None, None) == 4
    assert b"2^60" in binding.lib().tf_ulysses_last_error()


def test_frequencies_out_of_range():
    """A rotary_dim that 32 bits do not hold, and a factor whose base they do not."""
    from ulysses_sequence_attention_tf_gb300 import binding, build
    build.build()
    with pytest.raises(ValueError):
        binding.rope_frequencies(2 ** 32 + 64)
    for factor in (1e300, 1e-300):
        with pytest.raises(binding.TfUlyssesError):
            binding.rope_frequencies(4, 1e10 if factor > 1 else 1e-10, scaling="base", factor=factor)
