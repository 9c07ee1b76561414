"""perf/operators.py without a GPU: its cases, its work counts and the pieces
of its plain forms that are plain numbers."""
import importlib.util
import os
import random

import numpy as np
import pytest

import attention_quantized_kv_gb300 as kvq

import oracle
from tests import _rope as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ops():
    from attention_quantized_kv_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("operators", os.path.join(ROOT, "perf", "operators.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_listed_cases(ops):
    cases = ops.listed()
    assert len({c["name"] for c in cases}) == len(cases)
    work = [ops.work(c) for c in cases]
    assert all(w["bytes"] > 0 and w["flops"] > 0 for w in work)
    assert max(w["bytes"] for w in work) >= 16 * min(w["bytes"] for w in work)
    for op in ("table", "apply", "append", "shift", "decode"):
        assert sum(c["op"] == op for c in cases) >= 2


def test_drawn_cases(ops):
    rng = random.Random(3)
    most = max(ops.work(c)["bytes"] for c in ops.listed())
    for _ in range(400):
        c = ops.draw(rng)
        assert 0 < ops.work(c)["bytes"] <= most
        assert c["rot"] % 2 == 0 and 2 <= c["rot"] <= 128
        if c["op"] == "append":
            assert sum(ops.counts(c)) == c["tokens"] and min(ops.counts(c)) >= 1
        if c["op"] == "shift":
            assert all(0 <= e <= n for e, n in zip(ops.evicted(c), ops.lengths(c)))


def test_layout_and_signs_are_the_oracles(ops):
    for codec in range(4):
        for side in (0, 1):
            assert (ops.unit_offsets(codec, side) == oracle.unit_offset_table(codec, side)).all()
    assert ops.SIGNS == oracle.turbo_signs().tolist()


@pytest.mark.parametrize("scaling", range(5))
def test_frequencies_are_the_librarys(ops, scaling):
    case = dict(rot=96, base=500000.0, factor=5.5, orig=3000, scaling=ops.SCALINGS[scaling])
    got = np.array(kvq.kvq_rope_freqs(96, 500000.0, scaling, 5.5, 3000))
    assert np.abs(got / np.array(ops.frequencies(case)) - 1).max() <= 2.0 ** -48


def test_plain_angles():
    """The tests' extended-precision angles against integer arithmetic: a
    frequency that is a whole fraction of a turn returns to the same angles."""
    c, s = R.angles64([2 * np.pi / 1024], np.arange(4096))
    assert np.abs(c[:1024] - c[4096 - 1024:]).max() < 1e-12 and np.abs(s[:1024] - s[4096 - 1024:]).max() < 1e-12
