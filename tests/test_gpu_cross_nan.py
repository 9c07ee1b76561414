"""Rows that are no numbers: attn_cross and attn_decode_prefix return NaN for every row whose query
or keys hold a NaN, however its keys are split, and leave the other rows alone."""
import numpy as np
import pytest
import torch

import attention_quantized_kv_gb300 as kvq

from tests import _cross as C
from tests import _rope as R
from tests.test_gpu_cross import EPS, _cross_ws, _filled, _prefix_ws, _queries, _values
from tests.test_gpu_rope import _i32

pytestmark = pytest.mark.gpu

SCALE = R.default_scale()
F16, Q8, Q4, T4 = 0, 1, 2, 3
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_quantized_kv_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _nan(out, lse, rows, heads=slice(None)):
    assert out[rows][..., heads, :].isnan().all(), (out[rows][..., heads, :].isnan().float().mean())
    assert lse[rows][..., heads].isnan().all()


@pytest.mark.parametrize("ck,cv", [(F16, F16), (Q8, Q4), (T4, Q8), (Q8, T4)])
@pytest.mark.parametrize("lens,counts", [([20000], [7]), ([700, 90], [300, 41]), ([40, 33], [2, 1]), ([9000], [129])])
@pytest.mark.parametrize("kind", [torch.float16, torch.bfloat16])
def test_queries(ck, cv, lens, counts, kind):
    """One NaN in a query makes its head's row NaN, in items of one piece and of many."""
    n_kv, n_q, total = 2, 6, sum(counts)
    cap = -(-max(lens) // 256) * 256
    L, table = _filled(len(lens), n_kv, n_q, cap, ck, cv, False, lens, 41)
    q = _queries(total, n_q, 3, kind)
    bad = [(0, 4), (total - 1, 0), (total // 2, 3)]
    for r, h in bad:
        q[r, h, 17 * h + 5] = NAN
    out, lse = torch.full_like(q, 7), torch.full((total, n_q), 7.0, device="cuda")
    kvq.attn_cross(L, q, SCALE, out, lse, cap, _cross_ws(L, total, cap), row_start=_i32(np.cumsum([0] + counts)))
    assert L.err.item() == 0
    for r, h in bad:
        _nan(out, lse, slice(r, r + 1), slice(h, h + 1))
    values, at = _values(L, table, lens), 0
    for s, n in enumerate(counts):
        good = torch.ones((n, n_q), dtype=torch.bool, device="cuda")
        for r, h in bad:
            if at <= r < at + n:
                good[r - at, h] = False
        some = q[at:at + n].half().double().nan_to_num()
        ref, tol, rl, rt = C.attend(some, [(ck, cv) + values[s]], SCALE)
        got, eps = out[at:at + n].double(), EPS[kind]
        assert ((got - ref).abs() <= tol * (1 + eps) + eps * ref.abs() + 2.0 ** -25)[good].all()
        assert ((lse[at:at + n].double() - rl).abs() <= rt)[good].all()
        at += n


@pytest.mark.parametrize("first,n", [(0, 20000), (0, 64), (19000, 32), (777, 1), (6400, 6400)])
@pytest.mark.parametrize("rows", [1, 90, 400])
def test_keys(first, n, rows):
    """NaN in one key, in the keys of a whole tile, of a piece, of all: every row of their kv head."""
    L, table = _filled(1, 2, 4, 20224, F16, F16, False, [20000], 42)
    t = torch.arange(first, first + n, device="cuda")
    units = L.k_cache.view(torch.float16).view(2, 20224 // 16, 2048)
    # dim 0 of token row r of a unit of K
    g, rh = (t % 16) & 7, (t % 16) >> 3
    units[1, t // 16, rh * 256 + 4 * g * 8] = NAN
    q = _queries(rows, 4, 4)
    out, lse = torch.full_like(q, 7), torch.full((rows, 4), 7.0, device="cuda")
    kvq.attn_cross(L, q, SCALE, out, lse, 20224, _cross_ws(L, rows, 20224), row_start=_i32([0, rows]))
    _nan(out, lse, slice(0, rows), slice(2, 4))
    assert torch.isfinite(out[:, :2]).all() and torch.isfinite(lse[:, :2]).all()


@pytest.mark.parametrize("cap,lens", [(256, [40, 255, 3, 0]), (4096, [4000, 100, 1, 0])])
@pytest.mark.parametrize("ck,cv", [(F16, F16), (Q8, T4), (T4, Q4)])
def test_queries_behind_a_prefix(cap, lens, ck, cv):
    """Own keys by whole streams and split; a sequence of no own keys; one behind no prefix."""
    L, table = _filled(4, 1, 4, cap, ck, cv, False, lens, 43)
    P, ptable = _filled(1, 1, 4, 5120, ck, cv, False, [5000], 44)
    for bad in range(4):
        q = _queries(4, 4, 5)
        q[bad, 2, 100] = NAN
        out, lse = torch.full_like(q, 7), torch.full((4, 4), 7.0, device="cuda")
        kvq.attn_decode_prefix(L, P, q, SCALE, out, lse, cap, 5120, _prefix_ws(L, P, cap, 5120),
                               group_start=_i32([1, 4]))
        _nan(out, lse, slice(bad, bad + 1), slice(2, 3))
        good = torch.ones((4, 4), dtype=torch.bool, device="cuda")
        good[bad, 2] = False
        assert torch.isfinite(out[good]).all() and torch.isfinite(lse[good]).all()


@pytest.mark.parametrize("cap,length", [(256, 200), (4096, 4000)])
@pytest.mark.parametrize("where", ["own", "prefix"])
@pytest.mark.parametrize("all_keys", [False, True])
def test_keys_behind_a_prefix(cap, length, where, all_keys):
    L, _ = _filled(2, 1, 4, cap, F16, F16, False, [length, 30], 45)
    P, _ = _filled(2, 1, 4, 5120, F16, F16, False, [5000, 300], 46)
    layer, n, c = (L, length, cap) if where == "own" else (P, 5000, 5120)
    t = torch.arange(n if all_keys else 1, device="cuda")
    units = layer.k_cache.view(torch.float16).view(2, c // 16, 2048)
    units[0, t // 16, ((t % 16) >> 3) * 256 + 4 * ((t % 16) & 7) * 8] = NAN
    q = _queries(2, 4, 6)
    out, lse = torch.full_like(q, 7), torch.full((2, 4), 7.0, device="cuda")
    kvq.attn_decode_prefix(L, P, q, SCALE, out, lse, cap, 5120, _prefix_ws(L, P, cap, 5120), group_start=_i32([0, 1, 2]))
    _nan(out, lse, slice(0, 1))
    assert torch.isfinite(out[1]).all() and torch.isfinite(lse[1]).all()


@pytest.mark.parametrize("cv", [F16, Q8])
def test_time(cv):
    """A NaN key of an fp16 cache, whose operands are exact, does not send its rows to the fp32 way:
    that took 44 and 77 ms here, and an ordinary call takes 0.2."""
    L, _ = _filled(1, 2, 8, 20224, F16, cv, False, [20000], 47)
    q = _queries(1000, 8, 8)
    out, lse, ws = torch.empty_like(q), torch.empty((1000, 8), device="cuda"), _cross_ws(L, 1000, 20224)

    def median_ms():
        times = []
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in "ab")
            a.record()
            kvq.attn_cross(L, q, SCALE, out, lse, 20224, ws, row_start=_i32([0, 1000]))
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return sorted(times)[2]

    median_ms()
    usual = median_ms()
    # the last key, dim 0, of both kv heads
    L.k_cache.view(torch.float16).view(2, 20224 // 16, 2048)[:, 19999 // 16, 256 + 4 * 7 * 8] = NAN
    assert median_ms() <= 5 * usual
    _nan(out, lse, slice(0, 1000))
