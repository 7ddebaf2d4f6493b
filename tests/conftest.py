import gc
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built CUDA library")


def pytest_collection_finish(session):
    gc.collect()
    gc.freeze()  # what lives from here on is not looked at again after each test


@pytest.hookimpl(trylast=True)
def pytest_runtest_teardown(item):
    """A captured graph that a test leaves in a reference cycle (an expected exception's frame) is destroyed here: the
    collector may otherwise come to it while a later test captures, which ends that capture."""
    if item.get_closest_marker("gpu"):
        gc.collect()


@pytest.fixture(scope="session")
def olib():
    import oracle
    return oracle.load()
