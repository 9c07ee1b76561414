"""Entries of row_start, n_new and group_start that are out of range: the rows of the other sequences
are right, and those behind every sequence stay as they were."""
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


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_quantized_kv_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _holders(start, n):
    """For each of n rows the well-formed sequences that hold it."""
    held = [[] for _ in range(n)]
    for s, (a, b) in enumerate(zip(start, start[1:])):
        if 0 <= a <= b <= n:
            for r in range(a, b):
                held[r].append(s)
    return held


def _bad(start, n):
    """The rows of sequences whose entries are out of range, as far as they are rows."""
    return {r for a, b in zip(start, start[1:]) if not 0 <= a <= b <= n
            for r in range(max(0, min(a, b)), min(n, max(a, b)))}


@pytest.mark.parametrize("bad", [[0, 3, 2, 9], [0, 3, 12, 9], [-1, 3, 6, 9], [0, 3, 6, 10], [5, 3, 6, 8], [0, 2, 4, 3],
                                 [2**31 - 1, 0, 4, 8], [0, -2**31, 4, 8]])
@pytest.mark.parametrize("many", [1, 60])
def test_packed_rows(bad, many):
    """many: entries and rows times this."""
    lens = [400, 600, 40]
    L, table = _filled(3, 2, 4, 768, Q8, Q4, False, lens, 11)
    values, n = _values(L, table, lens), 9 * many
    start = [int(np.clip(x * many, -2**31, 2**31 - 1)) for x in bad]
    q = _queries(n + 3, 4, 8)
    out, lse = torch.full_like(q, 7), torch.full((n + 3, 4), 7.0, device="cuda")
    kvq.attn_cross(L, q[:n], SCALE, out[:n], lse[:n], 768, _cross_ws(L, n, 768), row_start=_i32(start))
    assert L.err.item() == kvq.KVQ_DEVERR_ROWS
    held, loose = _holders(start, n), _bad(start, n)
    for s in range(3):
        mine = [r for r in range(n) if held[r] == [s]]
        if mine:
            want = C.attend(q[mine].double(), [(Q8, Q4) + values[s]], SCALE)
            C.check(out[mine], lse[mine], want, EPS[q.dtype], (bad, s))
    rest = [r for r in range(n + 3) if r >= n or not held[r] and r not in loose]
    assert (out[rest] == 7).all() and (lse[rest] == 7).all()


@pytest.mark.parametrize("bad", [[3, -1, 2], [3, 9, 2], [-2**31, 8, 2**31 - 1]])
def test_padded_rows(bad):
    lens = [400, 600, 40]
    L, table = _filled(3, 2, 4, 768, Q8, Q4, False, lens, 12)
    values = _values(L, table, lens)
    q = _queries(24, 4, 9).view(3, 8, 4, 128)
    out, lse = torch.full_like(q, 7), torch.full((3, 8, 4), 7.0, device="cuda")
    kvq.attn_cross(L, q, SCALE, out, lse, 768, _cross_ws(L, 24, 768), n_new=_i32(bad))
    assert L.err.item() == kvq.KVQ_DEVERR_ROWS
    for s, n in enumerate(bad):
        if 0 <= n <= 8:
            C.check(out[s, :n], lse[s, :n], C.attend(q[s, :n].double(), [(Q8, Q4) + values[s]], SCALE), EPS[q.dtype], s)
            assert (out[s, n:] == 7).all() and (lse[s, n:] == 7).all()


@pytest.mark.parametrize("bad", [[0, 3, 2, 6], [0, 5, 9, 6], [-1, 2, 4, 6], [0, 2, 4, 7], [3, 1, 4, 6],
                                 [0, 2, 2**31 - 1, 4], [-2**31, 2, 4, 5]])
@pytest.mark.parametrize("cap,own", [(256, [40, 255, 0, 3, 17, 100]), (4096, [3000, 3, 0, 90, 1, 700])])
def test_groups(bad, cap, own):
    """Own keys by whole sequences and split.  The workspace holds NaN: no row is taken from it."""
    L, table = _filled(6, 2, 4, cap, Q8, F16, False, own, 13)
    shared = [500, 300, 20]
    P, ptable = _filled(3, 2, 4, 512, Q8, Q4, False, shared, 14)
    q = _queries(6, 4, 10)
    out, lse = torch.full_like(q, 7), torch.full((6, 4), 7.0, device="cuda")
    ws = _prefix_ws(L, P, cap, 512)
    ws.fill_(0xFF)
    kvq.attn_decode_prefix(L, P, q, SCALE, out, lse, cap, 512, ws, group_start=_i32(bad))
    assert P.err.item() == kvq.KVQ_DEVERR_ROWS and L.err.item() == 0
    mine, theirs = _values(L, table, own), _values(P, ptable, shared)
    for s, groups in enumerate(_holders(bad, 6)):
        if len(groups) > 1:
            continue
        parts = [(Q8, F16) + mine[s]] + [(Q8, Q4) + theirs[g] for g in groups]
        C.check(out[s:s + 1], lse[s:s + 1], C.attend(q[s:s + 1].double(), parts, SCALE), EPS[q.dtype], (bad, s))
