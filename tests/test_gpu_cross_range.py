"""Finite rows whose products, scores or queries lie beyond fp16's reach: attn_cross and
attn_decode_prefix give what the definition does (tolerances: tests/_cross.py)."""
import numpy as np
import pytest
import torch

import attention_quantized_kv_gb300 as kvq

from tests import _cross as C
from tests import _rope as R
from tests.test_gpu_cross import EPS, _cross_ws, _filled, _prefix_ws, _queries, _values
from tests.test_gpu_rope import _i32, _layer

pytestmark = pytest.mark.gpu

SCALE = R.default_scale()
F16, Q8, Q4, T4 = 0, 1, 2, 3


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_quantized_kv_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _check(out, lse, want, eps, where=""):
    """As tests/_cross.check, outputs beyond their type's range as infinities; the log-sum-exp's last
    place too (2^-23 of it)."""
    ref, tol, rl, rt = want
    top = float(torch.finfo(out.dtype).max)
    g = out.double()
    near = ref.abs() + tol * (1 + eps) + eps * ref.abs() >= top
    assert torch.isfinite(g[~near]).all(), where
    assert not torch.isnan(g).any(), where
    bad = ((g - ref).abs() > tol * (1 + eps) + eps * ref.abs() + 2.0 ** -25) & ~near
    assert not bad.any(), (where, int(bad.sum()))
    diff = (lse.double() - rl).abs()
    assert (diff <= rt + 2.0 ** -23 * rl.abs()).all(), (where, float((diff / rt).max()))


def _rows(n, n_kv, seed, spots, size):
    """fp32 rows of N(0, 1) with values of `size` at the (token, head, dim) of `spots`."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((n, n_kv, 128), generator=g, device="cuda")
    for t, h, d in spots:
        x[t, h, d] = size
    return x


def _two(lens, n_kv, n_q, cap, ck, cv, paged, k_size, v_size, spots):
    """A layer of two sequences, the second with large values in K or V."""
    L, table = _layer(2, n_kv, n_q, cap, ck, cv, paged, 5, fill=0xFF)
    k, v = (torch.cat([_rows(lens[0], n_kv, 50 + i, [], 0), _rows(lens[1], n_kv, 60 + i, spots if size else [], size)])
            for i, size in enumerate((k_size, v_size)))
    kvq.kv_append_rows(L, k, v, row_start=_i32([0, lens[0], sum(lens)]))
    return L, table


# fp16 rows reach the first: 65504 / 127 is 516 in fp16, and 127 * 516 = 65532 rounds to infinity
@pytest.mark.parametrize("ck,cv", [(Q8, Q8), (Q4, Q4), (T4, T4), (F16, Q8), (Q8, F16)])
@pytest.mark.parametrize("size", [65504.0, 3e5, 4e6])
@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("lens,counts,paged", [([300, 700], [40, 33], False), ([100, 9000], [3, 2], True),
                                               ([200, 500], [100, 200], True)])
def test_cached_values(ck, cv, size, side, lens, counts, paged):
    """A few large values in one sequence: its rows, and the other sequence's too."""
    codec = ck if side == "k" else cv
    limit = {F16: 65504.0, Q8: 8.3e6, Q4: 5.2e5, T4: 5e5}[codec]  # codes and scales hold these
    if size > limit:
        size = limit
    n_kv, n_q = 2, 6
    cap = -(-max(lens) // 256) * 256
    spots = [(0, 0, 5), (lens[1] - 1, 1, 127), (lens[1] // 2, 0, 64)]
    L, table = _two(lens, n_kv, n_q, cap, ck, cv, paged, size if side == "k" else 0, size if side == "v" else 0, spots)
    # large keys: queries so small that no row's weight is all on them
    q = _queries(sum(counts), n_q, 7, torch.bfloat16, 2.0 ** -13 if side == "k" else 1.0).half().bfloat16()
    out, lse = torch.full_like(q, 7), torch.full((sum(counts), n_q), 7.0, device="cuda")
    kvq.attn_cross(L, q, SCALE, out, lse, cap, _cross_ws(L, sum(counts), cap), row_start=_i32(np.cumsum([0] + counts)))
    assert L.err.item() == 0
    values, at = _values(L, table, lens), 0
    assert max(float(x.abs().max()) for x in values[1]) >= min(size, 65000.0) * 0.5
    for s, n in enumerate(counts):
        want = C.attend(q[at:at + n].double(), [(ck, cv) + values[s]], SCALE)
        _check(out[at:at + n], lse[at:at + n], want, EPS[q.dtype], s)
        at += n


@pytest.mark.parametrize("pk,pv", [(Q8, Q8), (Q4, T4), (T4, Q8)])
@pytest.mark.parametrize("cap,own", [(256, [40, 255, 0]), (2560, [2500, 3, 0])])
def test_prefix_values(pk, pv, cap, own):
    """The same as a prefix: the tokens give what they give as own keys."""
    L, table = _filled(3, 2, 6, cap, Q8, Q8, False, own, 8)
    P, ptable = _two([30, 3000], 2, 6, 3328, pk, pv, False, 65504.0, 65504.0, [(1000, 0, 9), (2999, 1, 3)])
    q = _queries(3, 6, 8, gain=2.0 ** -12)
    out, lse = torch.full_like(q, 7), torch.full((3, 6), 7.0, device="cuda")
    kvq.attn_decode_prefix(L, P, q, SCALE, out, lse, cap, 3328, _prefix_ws(L, P, cap, 3328), group_start=_i32([0, 1, 3]))
    assert L.err.item() == 0 and P.err.item() == 0
    mine, shared = _values(L, table, own), _values(P, ptable, [30, 3000])
    for s, g in enumerate([0, 1, 1]):
        parts = [(Q8, Q8) + mine[s], (pk, pv) + shared[g]]
        _check(out[s:s + 1], lse[s:s + 1], C.attend(q[s:s + 1].double(), parts, SCALE), EPS[q.dtype], s)


@pytest.mark.parametrize("ck", [F16, Q8, T4])
def test_queries(ck):
    """bf16 queries beyond 65504 (over small keys), and turbo4 ones whose rotation is."""
    L, table = _layer(2, 1, 4, 512, ck, F16, False, 5, fill=0xFF)
    k, v = _rows(500, 1, 70, [], 0) * 2.0 ** -10, _rows(500, 1, 71, [], 0)
    kvq.kv_append_rows(L, k, v, row_start=_i32([0, 200, 500]))
    q = _queries(50, 4, 9, torch.bfloat16)
    q[7] *= 30000.0
    q[8, 1, 3], q[45, 3, 77] = 3e5, -1e6
    signs = torch.from_numpy(C.oracle.turbo_signs().astype(np.float32)).cuda()
    q[30, 2] = (signs * 60000.0).bfloat16()  # the rotation is 8 times that in one place
    out, lse = torch.full_like(q, 7), torch.full((50, 4), 7.0, device="cuda")
    kvq.attn_cross(L, q, SCALE, out, lse, 512, _cross_ws(L, 50, 512), row_start=_i32([0, 20, 50]))
    values, at = _values(L, table, [200, 300]), 0
    for s, n in enumerate([20, 30]):
        _check(out[at:at + n], lse[at:at + n], C.attend(q[at:at + n].double(), [(ck, F16) + values[s]], SCALE),
               EPS[q.dtype], s)
        at += n


@pytest.mark.parametrize("rows,keys", [(1, 700), (90, 300), (300, 5000)])
@pytest.mark.parametrize("size", [300.0, 3000.0, 16000.0])
def test_scores(rows, keys, size):
    """Scores so large that fp32 steps of them exceed a weight's whole range: a key that leads by
    far more than the scores' errors takes all the weight."""
    L, table = _layer(1, 1, 2, 5120, F16, F16, False, 5, fill=0xFF)
    g = torch.Generator(device="cuda").manual_seed(11)
    sign = torch.where(torch.rand((1, 1, 128), generator=g, device="cuda") < 0.5, -1.0, 1.0)
    # scores of size^2 * 128 * (0.5 to 0.9) * scale, and one leader of 1
    share = 0.5 + 0.4 * torch.rand((keys, 1, 1), generator=g, device="cuda")
    lead = keys // 3
    share[lead] = 1.0
    k, v = (size * share * sign).half(), _rows(keys, 1, 72, [], 0).half()
    kvq.kv_append_rows(L, k, v, row_start=_i32([0, keys]))
    away = 1.0 + torch.rand((rows, 2, 1), generator=g, device="cuda")
    q = (size * away * sign).half()
    out, lse = torch.full_like(q, 7), torch.full((rows, 2), 7.0, device="cuda")
    kvq.attn_cross(L, q, SCALE, out, lse, 5120, _cross_ws(L, rows, 5120), row_start=_i32([0, rows]))
    s = torch.einsum("rhd,td->rht", q.double(), k[:, 0].double()) * SCALE
    top = s.amax(-1)
    # 16 * 2^-23 of the score (tests/_cross.py) against a lead of 0.09 of it: 10^4 times as much
    assert (top - s.topk(2, -1).values[..., 1] > 2000).all()
    # the weight's and the output's rounding, 2^-11 each, and ex2.approx's 2^-22
    want = v[lead].double()
    assert ((out.double() - want).abs() <= (2.0 ** -10 + 2.0 ** -20) * want.abs() + 2.0 ** -24).all()
    assert ((lse.double() - top).abs() <= 17 * 2.0 ** -23 * top.abs()).all()
