"""The polynomials that stand for tanh x / x (csrc/attention_common.cuh): the stored coefficients, evaluated in 64 bits."""
import os
import re

import numpy as np

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ulysses_sequence_attention_tf_gb300", "csrc",
                      "attention_common.cuh")


def test_errors_that_the_comments_state():
    with open(SOURCE) as f:
        text = f.read()

    def value(name):
        return float(np.float32(re.search(rf"\b{name} = (-?[\d.e-]+)f", text).group(1)))

    def worst(name, near, terms):
        x = np.linspace(0.0, value(near), 200001)[1:]
        got = np.polyval([value(f"{name}{i}") for i in reversed(range(terms))], x * x)
        return np.abs(got / (np.tanh(x) / x) - 1).max()

    assert 9.0e-8 < worst("kTanh", "kTanhNear", 5) < 9.2e-8
    assert 1.1e-7 < worst("kTanhNearest", "kTanhNearest", 3) < 1.2e-7
