"""Own keys behind a prefix: lengths past max_len, unmapped pages and negative lengths, by whole
sequences and split; queries that repeat a row; a prefix for every sequence."""
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


def _run(L, P, q, max_len, groups=None):
    out, lse = torch.full_like(q, 7), torch.full(q.shape[:2], 7.0, device="cuda")
    kvq.attn_decode_prefix(L, P, q, SCALE, out, lse, max_len, P.capacity, _prefix_ws(L, P, max_len, P.capacity),
                           group_start=groups)
    return out, lse


def _check(L, P, own, shared, group_of, q, out, lse):
    for s, g in enumerate(group_of):
        parts = [(L.codec_k, L.codec_v) + own[s]] + ([(P.codec_k, P.codec_v) + shared[g]] if g is not None else [])
        C.check(out[s:s + 1], lse[s:s + 1], C.attend(q[s:s + 1].double(), parts, SCALE), EPS[q.dtype], s)


@pytest.mark.parametrize("ck,cv", [(F16, F16), (Q4, Q4), (T4, Q8)])
@pytest.mark.parametrize("cap", [512, 8192])
def test_lengths(ck, cv, cap):
    """max_len below a length: the bit, and the keys below it; a negative length: none."""
    lens = [cap - 9, 100, 0, 33]
    L, table = _filled(4, 2, 8, cap, ck, cv, False, lens, 81)
    P, ptable = _filled(1, 2, 8, 512, Q8, Q8, False, [300], 82)
    own, shared = _values(L, table, lens), _values(P, ptable, [300])
    q = _queries(4, 8, 3)
    cut = cap - 100
    out, lse = _run(L, P, q, cut)
    assert L.err.item() == kvq.KVQ_DEVERR_MAXLEN and P.err.item() == 0
    own[0] = tuple(x[:, :cut] for x in own[0])
    _check(L, P, own, shared, [0] * 4, q, out, lse)
    L.err.zero_()
    L.seq_lens[3] = -5
    own[3] = tuple(x[:, :0] for x in own[3])
    out, lse = _run(L, P, q, cap)
    assert L.err.item() == 0
    own[0] = _values(L, table, lens[:1])[0]
    _check(L, P, own, shared, [0] * 4, q, out, lse)
    P.seq_lens.fill_(-1)  # and of the prefix
    out, lse = _run(L, P, q, cap)
    assert L.err.item() == 0 and P.err.item() == 0
    _check(L, P, own, [tuple(x[:, :0] for x in shared[0])], [0] * 4, q, out, lse)


@pytest.mark.parametrize("ck,cv", [(F16, Q8), (Q4, T4)])
@pytest.mark.parametrize("cap", [512, 8192])
def test_pages(ck, cv, cap):
    """An unmapped page of one sequence: the bit, the others' rows hold; in the prefix: its own word."""
    lens = [cap - 9, 300, 511]
    L, table = _filled(3, 2, 8, cap, ck, cv, True, lens, 83)
    P, ptable = _filled(2, 2, 8, 768, Q8, Q8, True, [700, 300], 84)
    own, shared = _values(L, table, lens), _values(P, ptable, [700, 300])
    q, groups = _queries(3, 8, 4), _i32([0, 2, 3])
    L.block_table[1, 1] = L.n_pages
    out, lse = _run(L, P, q, cap, groups)
    assert L.err.item() == kvq.KVQ_DEVERR_PAGE and P.err.item() == 0
    for s, g in ((0, 0), (2, 1)):
        want = C.attend(q[s:s + 1].double(), [(ck, cv) + own[s], (Q8, Q8) + shared[g]], SCALE)
        C.check(out[s:s + 1], lse[s:s + 1], want, EPS[q.dtype], s)
    L.err.zero_()
    L.block_table[1, 1] = int(table[1, 1])
    P.block_table[0, 2] = -1
    out, lse = _run(L, P, q, cap, groups)
    assert P.err.item() == kvq.KVQ_DEVERR_PAGE and L.err.item() == 0
    want = C.attend(q[2:].double(), [(ck, cv) + own[2], (Q8, Q8) + shared[1]], SCALE)
    C.check(out[2:], lse[2:], want, EPS[q.dtype], 2)


@pytest.mark.parametrize("kind", [torch.float16, torch.bfloat16])
def test_repeated_queries(kind):
    """Strides of zero: one row for all, one head for all."""
    lens, counts = [700, 33], [90, 3]
    L, table = _filled(2, 2, 8, 768, Q8, Q4, False, lens, 85)
    values, start = _values(L, table, lens), _i32([0, 90, 93])
    for q in (_queries(1, 8, 5, kind).expand(93, 8, 128), _queries(93, 1, 6, kind).expand(93, 8, 128)):
        out, lse = torch.full((93, 8, 128), 7, dtype=kind, device="cuda"), torch.full((93, 8), 7.0, device="cuda")
        kvq.attn_cross(L, q, SCALE, out, lse, 768, _cross_ws(L, 93, 768), row_start=start)
        at = 0
        for s, n in enumerate(counts):
            want = C.attend(q[at:at + n].half().double(), [(Q8, Q4) + values[s]], SCALE)
            C.check(out[at:at + n], lse[at:at + n], want, EPS[kind], s)
            at += n
    assert L.err.item() == 0


def test_a_prefix_for_every_sequence():
    """1024 groups of one sequence, empty ones and prefixes among them."""
    n = 1024
    lens, plens = [(7 * s) % 40 for s in range(n)], [(11 * s) % 60 for s in range(n)]
    L, table = _filled(n, 1, 2, 256, F16, F16, False, lens, 86)
    P, ptable = _filled(n, 1, 2, 256, Q8, Q8, False, plens, 87)
    q = _queries(n, 2, 7)
    out, lse = _run(L, P, q, 256, _i32(np.arange(n + 1)))
    assert L.err.item() == 0 and P.err.item() == 0
    some = [0, 1, 31, 32, 33, 511, 512, 600, 1000, 1022, 1023]
    own, shared = _values(L, table, lens), _values(P, ptable, plens)
    for s in some:
        want = C.attend(q[s:s + 1].double(), [(F16, F16) + own[s], (Q8, Q8) + shared[s]], SCALE)
        C.check(out[s:s + 1], lse[s:s + 1], want, EPS[q.dtype], s)
