"""Workspaces of attn_cross and attn_decode_prefix: as large as a call of that size can need, and not
written past."""
import numpy as np
import pytest
import torch

import attention_quantized_kv_gb300 as kvq

from tests import _cross as C
from tests import _rope as R
from tests.test_gpu_cross import EPS, _filled, _queries, _values
from tests.test_gpu_rope import _i32

pytestmark = pytest.mark.gpu

SCALE = R.default_scale()
F16, Q8, Q4, T4 = 0, 1, 2, 3
GUARD = 1 << 16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_quantized_kv_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("ck", [F16, T4])
def test_sizes(ck):
    """One row over 256 keys does not need a place for every SM's two tiles; more rows or keys never
    need less."""
    L = kvq.KVLayer(16, 2, 8, 65536, ck, Q8, n_pages=16 * 256)
    size = lambda n, m: kvq.attn_cross_workspace(L, n, m)
    assert size(1, 256) <= 2 << 20
    assert size(16, 1500) <= 21 << 20
    assert size(100000, 65536) <= 41 << 20
    rows, keys = [0, 1, 2, 16, 31, 32, 33, 64, 65, 100, 1000, 100000], [1, 64, 65, 256, 1500, 4096, 65536]
    for m in keys:
        assert all(size(a, m) <= size(b, m) for a, b in zip(rows, rows[1:]))
    for n in rows:
        assert all(size(n, a) <= size(n, b) for a, b in zip(keys, keys[1:]))
    P = kvq.KVLayer(1, 2, 8, 65536, ck, Q8)
    one = kvq.KVLayer(1, 2, 8, 256, F16, F16)
    assert kvq.attn_decode_prefix_workspace(one, P, 256, 256) <= 3 << 20


def _guarded(n):
    ws = torch.full((n + GUARD,), 0x5A, dtype=torch.uint8, device="cuda")
    return ws, ws[:n]


@pytest.mark.parametrize("ck,cv", [(F16, Q8), (Q4, F16), (T4, T4)])
@pytest.mark.parametrize("group", [1, 4, 12])
@pytest.mark.parametrize("lens,counts", [
    ([1], [1]), ([256], [1]), ([300, 0, 17], [1, 1, 1]), ([2000], [10]), ([2000], [33]), ([700, 90], [128, 1]),
    ([700, 90], [129, 32]), ([64] * 40, [1] * 40), ([2048] * 3, [0, 300, 5]), ([65] * 20, [11] * 20)])
def test_nothing_is_written_past(ck, cv, group, lens, counts):
    """Workspaces of exactly the size, calls at and around whole tiles and slices."""
    cap, n_kv, total = 2048, 2, sum(counts)
    L, table = _filled(len(lens), n_kv, n_kv * group, cap, ck, cv, False, lens, 61)
    values = _values(L, table, lens)
    q = _queries(total, n_kv * group, 6)
    for max_len in (max(lens), cap):
        out, lse = torch.full_like(q, 7), torch.full((total, n_kv * group), 7.0, device="cuda")
        ws, mine = _guarded(kvq.attn_cross_workspace(L, total, max_len))
        kvq.attn_cross(L, q, SCALE, out, lse, max_len, mine, row_start=_i32(np.cumsum([0] + counts)))
        assert (ws[len(mine):] == 0x5A).all() and L.err.item() == 0
        at = 0
        for s, n in enumerate(counts):
            if n:
                want = C.attend(q[at:at + n].double(), [(ck, cv) + values[s]], SCALE)
                C.check(out[at:at + n], lse[at:at + n], want, EPS[q.dtype], (max_len, s))
            at += n


@pytest.mark.parametrize("n_seqs,plen,own", [(1, 1, 0), (1, 2000, 40), (3, 300, 255), (40, 2048, 9), (2, 1500, 2000)])
@pytest.mark.parametrize("pk", [F16, T4])
def test_prefixes(n_seqs, plen, own, pk):
    lens = [max(own - 3 * s, 0) for s in range(n_seqs)]
    L, table = _filled(n_seqs, 2, 8, 2048, Q8, Q8, False, lens, 62)
    P, ptable = _filled(1, 2, 8, 2048, pk, Q8, False, [plen], 63)
    own_values, shared = _values(L, table, lens), _values(P, ptable, [plen])
    q = _queries(n_seqs, 8, 7)
    for max_len, max_prefix in ((max(own, 1), plen), (2048, 2048)):
        out, lse = torch.full_like(q, 7), torch.full((n_seqs, 8), 7.0, device="cuda")
        ws, mine = _guarded(kvq.attn_decode_prefix_workspace(L, P, max_len, max_prefix))
        kvq.attn_decode_prefix(L, P, q, SCALE, out, lse, max_len, max_prefix, mine)
        assert (ws[len(mine):] == 0x5A).all() and L.err.item() == 0 and P.err.item() == 0
        for s in range(n_seqs):
            parts = [(Q8, Q8) + own_values[s], (pk, Q8) + shared[0]]
            C.check(out[s:s + 1], lse[s:s + 1], C.attend(q[s:s + 1].double(), parts, SCALE), EPS[q.dtype], s)
