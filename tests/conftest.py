import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


# Tests that run and have to fail: the value they hold is wrong.
WRONG_VALUES = {
    "tests/test_rope.py::test_frequencies[4-4]":
        "YaRN's ramp is bounded by rot_dim - 1, this value by rot_dim / 2 - 1 (right: tests/test_rope_yarn.py)",
}


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built library")


def pytest_collection_modifyitems(config, items):
    # GPU tests fail loudly (not skip) when the GPU or the library is missing:
    # a silent skip would hide a missing native path on the GPU machine.
    for item in items:
        if item.nodeid in WRONG_VALUES:
            item.add_marker(pytest.mark.xfail(reason=WRONG_VALUES[item.nodeid], strict=True))
