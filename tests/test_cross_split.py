"""The bounds of tests/_cross_split.py on the CPU: operands as two fp16 parts meet them, rounded once
they do not."""
import numpy as np
import pytest
import torch

from tests import _cross_split as S
from tests import _encoders as E

F16, Q8, Q4, T4 = 0, 1, 2, 3
SCALE = 1 / np.sqrt(128.0)


def _half(x):
    return x.to(torch.float16).double()


def _parts(x, split):
    """What the operands add up to: two fp16 parts, or one rounding."""
    return _half(x) + (_half(x - _half(x)) if split else 0)


def _cached(codec, n, heads, seed, rows=None):
    """fp64 [heads, n, 128]: what a cache holds of rows [n, heads, 128]."""
    x = np.random.default_rng(seed).standard_normal((n, heads, 128)).astype(np.float32) if rows is None else rows
    y = E.decode(codec, E.encode(codec, x.reshape(-1, 128))).reshape(n, heads, 128)
    return torch.from_numpy(y.astype(np.float64)).transpose(0, 1).contiguous()


@pytest.mark.parametrize("codec", [Q8, Q4, T4])
@pytest.mark.parametrize("T", [1, 2, 33])  # (over hundreds of keys the roundings average out)
@pytest.mark.parametrize("rounded", ["nothing", "keys", "query"])
def test_log_sum_exp(codec, T, rounded):
    if rounded == "query" and codec != T4:
        pytest.skip("fp16 queries are operands as they are")
    k = _cached(codec, T, 2, 3 + T)
    q = _half(torch.from_numpy(np.random.default_rng(T).standard_normal((40, 6, 128))))
    want, tol = S.lse_of(q, [(codec, k)], SCALE)
    x, y = (S.rotated(S.by_head(q, 2)) / 16, S.rotated(k) / 8) if codec == T4 else (S.by_head(q, 2), k)
    x = _parts(x, rounded != "query")
    y = _parts(y, rounded != "keys")
    got = torch.logsumexp(x @ y.transpose(1, 2) * SCALE, -1).reshape(2, 40, 3).transpose(0, 1).reshape(40, 6)
    off = ((got - want).abs() / tol).max()
    assert off <= 1 if rounded == "nothing" else off > 1.5


@pytest.mark.parametrize("codec", [Q8, Q4, T4])
@pytest.mark.parametrize("T", [2, 16, 33])
@pytest.mark.parametrize("split", [True, False])
def test_values(codec, T, split):
    v = _cached(codec, T, 2, 0, S.near_opposites(T, 2, np.random.default_rng(T)))
    want, tol = S.mean_of(v, codec, 2.0 ** -11)
    y = _parts(S.rotated(v) / 8 if codec == T4 else v, split).mean(1)
    got = _half(S.hadamard() @ y.T / 16).T * S.signs() if codec == T4 else _half(y)
    off = ((got - want).abs() / tol).max()
    assert off <= 1 if split else off > 1.5
