"""The precision that include/kvq.h states for attn_cross and for a prefix's part: quantized sides and
turbo4 queries as pairs of fp16 numbers, tolerances of tests/_cross_split.py."""
import numpy as np
import pytest
import torch

import attention_quantized_kv_gb300 as kvq

from tests import _cross_split as S
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


def _within(got, want, tol, where):
    off = (got.double() - want).abs() / tol
    assert (off <= 1).all(), (where, float(off.max()))


@pytest.mark.parametrize("ck", [F16, Q8, Q4, T4])
@pytest.mark.parametrize("rows", [1, 40, 300])
@pytest.mark.parametrize("gain", [1.0, 0.1])
def test_log_sum_exp(ck, rows, gain):
    lens = [1, 2, 33, 256, 700]
    L, table = _filled(5, 2, 6, 768, ck, Q8, True, lens, 31)
    q = _queries(5 * rows, 6, 3, gain=gain)
    out, lse = torch.empty_like(q), torch.empty((5 * rows, 6), device="cuda")
    kvq.attn_cross(L, q, SCALE, out, lse, 768, _cross_ws(L, 5 * rows, 768), row_start=_i32(np.arange(6) * rows))
    for s, (k, _) in enumerate(_values(L, table, lens)):
        mine = slice(s * rows, (s + 1) * rows)
        _within(lse[mine], *S.lse_of(q[mine].double(), [(ck, k)], SCALE), lens[s])


def _opposites(n_seqs, n_kv, n_q, cap, cv, paged, lens, seed):
    L, table = _layer(n_seqs, n_kv, n_q, cap, F16, cv, paged, seed, fill=0xFF)
    rng = np.random.default_rng(seed)
    v = torch.from_numpy(np.concatenate([S.near_opposites(n, n_kv, rng) for n in lens])).cuda()
    kvq.kv_append_rows(L, torch.randn_like(v), v, row_start=_i32(np.cumsum([0] + lens)))
    return L, table


@pytest.mark.parametrize("cv", [F16, Q8, Q4, T4])
@pytest.mark.parametrize("rows", [1, 40, 300])
@pytest.mark.parametrize("kind", [torch.float16, torch.bfloat16])
def test_values(cv, rows, kind):
    """Weights that are all one: an output is the values' mean."""
    lens = [2, 16, 33, 64, 130]
    L, table = _opposites(5, 2, 6, 256, cv, True, lens, 32)
    q = torch.zeros((5 * rows, 6, 128), dtype=kind, device="cuda")
    out = torch.full_like(q, 7)
    kvq.attn_cross(L, q, SCALE, out, None, 256, _cross_ws(L, 5 * rows, 256), row_start=_i32(np.arange(6) * rows))
    for s, (_, v) in enumerate(_values(L, table, lens)):
        mean, tol = S.mean_of(v, cv, EPS[kind])
        got = out[s * rows:(s + 1) * rows].view(rows, 2, 3, 128)
        _within(got, mean[None, :, None], tol[None, :, None], lens[s])


@pytest.mark.parametrize("pk", [F16, Q8, Q4, T4])
@pytest.mark.parametrize("pv", [F16, Q8, Q4, T4])
def test_prefixes(pk, pv):
    """A prefix's part, alone and with own fp16 keys."""
    own, shared = [0, 0, 20, 0], [1, 33, 256]
    group_of = [0, 1, 1, 2]
    L, table = _filled(4, 2, 6, 256, F16, F16, False, own, 33)
    P, ptable = _filled(3, 2, 6, 512, pk, Q8, True, shared, 34)
    q = _queries(4, 6, 5)
    out, lse = torch.empty_like(q), torch.empty((4, 6), device="cuda")
    groups = _i32([0, 1, 3, 4])
    kvq.attn_decode_prefix(L, P, q, SCALE, out, lse, 256, 512, _prefix_ws(L, P, 256, 512), group_start=groups)
    mine, theirs = _values(L, table, own), _values(P, ptable, shared)
    for s, g in enumerate(group_of):
        parts = [(pk, theirs[g][0])] + ([(F16, mine[s][0])] if own[s] else [])
        _within(lse[s:s + 1], *S.lse_of(q[s:s + 1].double(), parts, SCALE), s)
    V, vtable = _opposites(3, 2, 6, 256, pv, False, [2, 16, 33], 35)
    q.zero_()
    kvq.attn_decode_prefix(L, V, q, SCALE, out, None, 256, 256, _prefix_ws(L, V, 256, 256), group_start=groups)
    for s, g in enumerate(group_of):
        if not own[s]:
            mean, tol = S.mean_of(_values(V, vtable, [2, 16, 33])[g][1], pv, EPS[q.dtype])
            _within(out[s].view(2, 3, 128), mean[:, None], tol[:, None], s)
