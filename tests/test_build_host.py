"""When the build compiles again (no GPU needed)."""
import sys


def test_another_torch_or_python_compiles_the_calls_module_again(monkeypatch):
    import torch

    from ulysses_sequence_attention_tf_gb300 import build
    build.build()
    assert not build._calls_stale()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0")
        assert build._calls_stale()
    with monkeypatch.context() as m:
        m.setattr(sys, "version", "another")
        assert build._calls_stale()
    with monkeypatch.context() as m:
        m.setattr(torch, "__file__", "/elsewhere/torch/__init__.py")
        assert build._calls_stale()
    assert not build._calls_stale()
