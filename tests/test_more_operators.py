"""perf/more_operators.py without a GPU: its cases, its work counts and how it
spreads rows and lengths over sequences."""
import importlib.util
import os
import random

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ops():
    from attention_quantized_kv_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("more_operators", os.path.join(ROOT, "perf", "more_operators.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _sound(ops, c):
    w = ops.work(c)
    assert w["bytes"] > 0 and w["flops"] > 0
    lens = ops.lengths(c)
    assert len(lens) == c["seqs"] and min(lens) >= 0
    if c["op"] == "prefix":
        sizes = ops.shares(c["seqs"], c["groups"])
        assert sum(sizes) == c["seqs"] and min(sizes) >= 1
        assert len(ops.prefixes(c)) == c["groups"] and max(ops.prefixes(c)) == c["prefix"]
        assert c["n_q"] % c["n_kv"] == 0
        return
    rows = ops.counts(c)
    assert sum(rows) == c["rows"] and min(rows) >= (0 if c["op"] == "read" else 1)
    if c["op"] == "read":
        assert all(n <= have for n, have in zip(rows, lens))
    if c["op"] == "cross":
        assert c["n_q"] % c["n_kv"] == 0 and min(lens) >= 1


def test_listed_cases(ops):
    cases = ops.listed()
    assert len({c["name"] for c in cases}) == len(cases)
    for c in cases:
        _sound(ops, c)
    work = [ops.work(c) for c in cases]
    assert max(w["bytes"] for w in work) >= 16 * min(w["bytes"] for w in work)
    for op in ("prefix", "cross", "append", "read"):
        assert sum(c["op"] == op for c in cases) >= 2


def test_drawn_cases(ops):
    rng = random.Random(3)
    most = {unit: max(ops.work(c)[unit] for c in ops.listed()) for unit in ("bytes", "flops")}
    for _ in range(400):
        c = ops.draw(rng)
        _sound(ops, c)
        assert all(ops.work(c)[unit] <= most[unit] for unit in most)
