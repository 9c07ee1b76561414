"""Query rows against every key of their sequence, and decode steps behind a
shared prefix, against 64 bits (tolerances: tests/_cross.py)."""
import numpy as np
import pytest
import torch

import attention_quantized_kv_gb300 as kvq

from tests import _cross as C
from tests import _rope as R
from tests.test_gpu_rope import _i32, _images, _layer

pytestmark = pytest.mark.gpu

SCALE = R.default_scale()
F16, Q8, Q4, T4 = 0, 1, 2, 3
EPS = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_quantized_kv_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _filled(n_seqs, n_kv, n_q, cap, ck, cv, paged, lens, seed, fill=0xFF):
    """A layer over buffers full of NaN (0xFF bytes), its tokens N(0, 1)."""
    L, table = _layer(n_seqs, n_kv, n_q, cap, ck, cv, paged, seed, fill=fill)
    g = torch.Generator(device="cuda").manual_seed(seed)
    k, v = (torch.randn((n_seqs, max(max(lens), 1), n_kv, 128), generator=g, device="cuda").half() for _ in "kv")
    kvq.kv_append_quantize(L, k, v, _i32(lens))
    return L, table


def _values(L, table, lens):
    """[(k, v)] of every sequence, fp64 [kv heads, length, 128]."""
    images = _images(L, table)
    return [tuple(C.rows_of(im, s, range(n)) for im in images) for s, n in enumerate(lens)]


def _cross_ws(L, n_rows, max_len):
    return torch.zeros(kvq.attn_cross_workspace(L, n_rows, max_len), dtype=torch.uint8, device="cuda")


def _queries(rows, n_q, seed, kind=torch.float16, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (gain * torch.randn((rows, n_q, 128), generator=g, device="cuda")).to(kind)


def _check_rows(L, values, q, out, lse, counts, at=0, where=""):
    for s, n in enumerate(counts):
        if n:
            want = C.attend(q[at:at + n].half().double(), [(L.codec_k, L.codec_v) + values[s]], SCALE)
            C.check(out[at:at + n], None if lse is None else lse[at:at + n], want, EPS[out.dtype], (where, s))
        at += n
    return at


LENS = [300, 0, 1, 15, 16, 17, 127, 128, 129, 1000, 256, 31]
ROWS = [3, 2, 1, 40, 0, 7, 33, 1, 65, 9, 130, 5]


@pytest.mark.parametrize("ck", [F16, Q8, Q4, T4])
@pytest.mark.parametrize("cv", [F16, Q8, Q4, T4])
def test_packed_rows(ck, cv):
    """Every codec pair; ragged rows and lengths, none among both; groups of 1 to 12 heads; the rows
    behind the last sequence stay; what lies behind the lengths is NaN."""
    i = ck + 4 * cv
    n_kv, group = [1, 2, 3][i % 3], [1, 3, 4, 5, 8, 12][i % 6]
    kind = [torch.float16, torch.bfloat16][(ck + cv) % 2]
    n_q, total = n_kv * group, sum(ROWS)
    L, table = _filled(12, n_kv, n_q, 1024, ck, cv, i % 2 == 1, LENS, 10 + i)
    q = _queries(total + 6, n_q, i, kind, 2.0)
    out, lse = torch.full_like(q, 7), torch.full((total + 6, n_q), 7.0, device="cuda")
    start = _i32(np.cumsum([0] + ROWS))
    ws = _cross_ws(L, total + 6, 1024)
    kvq.attn_cross(L, q, SCALE, out, lse, 1024, ws, row_start=start)
    assert L.err.item() == 0
    assert (out[total:] == 7).all() and (lse[total:] == 7).all()
    assert not out[ROWS[0]:ROWS[0] + 2].any()
    _check_rows(L, _values(L, table, LENS), q, out, lse, ROWS)
    again, lse2 = torch.empty_like(out), torch.empty_like(lse)
    kvq.attn_cross(L, q, SCALE, again, lse2, 1024, ws, row_start=start)
    assert torch.equal(again[:total], out[:total]) and torch.equal(lse2[:total], lse[:total])


@pytest.mark.parametrize("kind", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("shift", [0, 3])
def test_padded_strided_rows(kind, shift):
    """Padded rows, q and out views of wider tensors; rows behind a count and around the views stay;
    rows before the first sequence of a packed batch too."""
    n_kv, n_q, lens, counts = 2, 6, [200, 77, 0, 513], [5, 0, 3, 12]
    L, table = _filled(4, n_kv, n_q, 768, Q8, F16, False, lens, 3)
    wide = _queries(4 * 12, n_q + 5, 4, kind).view(4, 12, n_q + 5, 128)
    q = wide[:, :, 2:2 + n_q]
    back = torch.full((4, 12, 2 * n_q, 128), 9, dtype=kind, device="cuda")
    out = back[:, :, n_q:]
    lse = torch.full((4, 12, n_q), 9.0, device="cuda")
    kvq.attn_cross(L, q, SCALE, out, lse, 513, _cross_ws(L, 48, 513), n_new=_i32(counts))
    values = _values(L, table, lens)
    for s, n in enumerate(counts):
        if n:
            want = C.attend(q[s, :n].half().double(), [(Q8, F16) + values[s]], SCALE)
            C.check(out[s, :n], lse[s, :n], want, EPS[kind], s)
        assert (out[s, n:] == 9).all() and (lse[s, n:] == 9).all()
    assert (back[:, :, :n_q] == 9).all()
    # packed, from row `shift` on, without lse
    rows = wide.view(48, n_q + 5, 128)[:, :n_q]
    packed = torch.full((48, n_q, 128), 9, dtype=kind, device="cuda")
    kvq.attn_cross(L, rows, SCALE, packed, None, 768, _cross_ws(L, 48, 768),
                   row_start=_i32(shift + np.cumsum([0] + counts)))
    _check_rows(L, values, rows, packed, None, counts, at=shift)
    assert (packed[:shift] == 9).all() and (packed[shift + sum(counts):] == 9).all()
    assert L.err.item() == 0


@pytest.mark.parametrize("ck,cv,n_kv,group,lens,counts,paged", [
    (Q8, Q8, 2, 4, [20000], [7], False),             # few rows, many keys
    (F16, F16, 1, 8, [9001, 40], [64, 3], True),
    (Q4, Q4, 2, 4, [3000], [500], False),            # many rows
    (F16, Q8, 1, 5, [700, 1500], [300, 411], True),
    (T4, T4, 1, 4, [5000], [129], False),
    (Q8, T4, 8, 1, [257, 1], [1, 1000], False),
])
def test_long(ck, cv, n_kv, group, lens, counts, paged):
    n_q, cap = n_kv * group, -(-max(lens) // 256) * 256
    L, table = _filled(len(lens), n_kv, n_q, cap, ck, cv, paged, lens, 77)
    q = _queries(sum(counts), n_q, 5, gain=1.5)
    out, lse = torch.empty_like(q), torch.empty((sum(counts), n_q), device="cuda")
    kvq.attn_cross(L, q, SCALE, out, lse, cap, _cross_ws(L, sum(counts), cap), row_start=_i32(np.cumsum([0] + counts)))
    assert L.err.item() == 0
    _check_rows(L, _values(L, table, lens), q, out, lse, counts)


@pytest.mark.parametrize("kind", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n_seqs,group", [(1, 1), (5, 4), (40, 12)])
def test_single_tokens(kind, n_seqs, group):
    """One row per sequence, the call's default."""
    n_kv, lens = 2, [(37 * s * s + 5 * s) % 700 for s in range(n_seqs)]
    lens[-1] = 700
    L, table = _filled(n_seqs, n_kv, n_kv * group, 768, Q8, Q4, n_seqs > 1, lens, 8)
    q = _queries(n_seqs, n_kv * group, 6, kind)
    out, lse = torch.full_like(q, 3), torch.full((n_seqs, n_kv * group), 3.0, device="cuda")
    kvq.attn_cross(L, q, SCALE, out, lse, 768, _cross_ws(L, n_seqs, 768))
    assert L.err.item() == 0
    _check_rows(L, _values(L, table, lens), q, out, lse, [1] * n_seqs)


def test_large_scores():
    """Scores far apart (one key takes all the weight) and far from zero."""
    L, table = _filled(2, 1, 4, 512, F16, F16, False, [500, 300], 9)
    q = _queries(40, 4, 7, gain=60.0)
    out, lse = torch.empty_like(q), torch.empty((40, 4), device="cuda")
    kvq.attn_cross(L, q, SCALE, out, lse, 512, _cross_ws(L, 40, 512), row_start=_i32([0, 20, 40]))
    _check_rows(L, _values(L, table, [500, 300]), q, out, lse, [20, 20])


def test_device_conditions():
    """Lengths past max_len, bad row_start entries and unmapped pages set their bits; the other
    sequences' rows hold."""
    lens = [400, 600, 40]
    L, table = _filled(3, 2, 4, 768, Q8, Q8, False, lens, 11)
    values = _values(L, table, lens)
    q = _queries(9, 4, 8)
    out, lse = torch.empty_like(q), torch.empty((9, 4), device="cuda")
    kvq.attn_cross(L, q, SCALE, out, lse, 500, _cross_ws(L, 9, 500), row_start=_i32([0, 3, 6, 9]))
    assert L.err.item() == kvq.KVQ_DEVERR_MAXLEN
    values[1] = tuple(x[:, :500] for x in values[1])
    _check_rows(L, values, q, out, lse, [3, 3, 3])
    for bad in ([0, 3, 2, 9], [0, 3, 12, 9], [-1, 3, 6, 9], [0, 3, 6, 10]):
        L.err.zero_()
        kvq.attn_cross(L, q, SCALE, out, lse, 768, _cross_ws(L, 9, 768), row_start=_i32(bad))
        assert L.err.item() == kvq.KVQ_DEVERR_ROWS, bad
    P, table = _filled(1, 1, 4, 512, F16, Q4, True, [500], 12)
    P.block_table[0, 1] = -1
    kvq.attn_cross(P, q[:2], SCALE, out[:2], lse[:2], 512, _cross_ws(P, 2, 512), row_start=_i32([0, 2]))
    assert P.err.item() == kvq.KVQ_DEVERR_PAGE


def test_empty_batch_and_empty_caches():
    L, _ = _filled(2, 1, 2, 256, F16, F16, False, [0, 0], 13)
    q = _queries(4, 2, 8)
    out, lse = torch.full_like(q, 5), torch.full((4, 2), 5.0, device="cuda")
    ws = _cross_ws(L, 4, 256)
    kvq.attn_cross(L, q[:0], SCALE, out[:0], lse[:0], 256, ws, row_start=_i32([0, 0, 0]))
    assert (out == 5).all()
    kvq.attn_cross(L, q, SCALE, out, lse, 256, ws, row_start=_i32([0, 3, 4]))
    assert not out.any() and torch.isinf(lse).all() and L.err.item() == 0


# ------------------------------------------------------------------ shared prefixes

def _prefix_ws(L, P, max_len, max_prefix):
    return torch.zeros(kvq.attn_decode_prefix_workspace(L, P, max_len, max_prefix), dtype=torch.uint8, device="cuda")


def _check_prefix(L, P, own, shared, group_of, q, out, lse):
    for s, g in enumerate(group_of):
        parts = [(L.codec_k, L.codec_v) + own[s]]
        if g is not None:
            parts.append((P.codec_k, P.codec_v) + shared[g])
        want = C.attend(q[s:s + 1].double(), parts, SCALE)
        C.check(out[s:s + 1], None if lse is None else lse[s:s + 1], want, EPS[torch.float16], (s, g))


@pytest.mark.parametrize("pk,pv", [(F16, F16), (Q8, Q8), (Q4, Q4), (T4, T4), (F16, Q8), (Q8, T4), (T4, Q4)])
@pytest.mark.parametrize("ck,cv", [(F16, F16), (Q8, Q4), (T4, T4)])
def test_groups(pk, pv, ck, cv):
    """Groups of 0, 1 and many, sequences before and behind them, empty prefixes and empty caches."""
    i = pk + 3 * pv + ck
    n_kv, group = [1, 2][i % 2], [1, 4, 5, 8, 12][i % 5]
    n_q = n_kv * group
    lens = [40, 0, 17, 255, 0, 300, 1, 64, 129, 16, 0]
    plens, start = [700, 0, 33, 1, 256], [1, 6, 8, 8, 9, 10]
    L, table = _filled(11, n_kv, n_q, 512, ck, cv, i % 2 == 0, lens, 20 + i)
    P, ptable = _filled(5, n_kv, n_q, 768, pk, pv, i % 3 == 0, plens, 50 + i)
    q = _queries(11, n_q, i, gain=1.5)
    out, lse = torch.full_like(q, 4), torch.full((11, n_q), 4.0, device="cuda")
    ws = _prefix_ws(L, P, 512, 768)
    kvq.attn_decode_prefix(L, P, q, SCALE, out, lse, 512, 768, ws, group_start=_i32(start))
    assert L.err.item() == 0 and P.err.item() == 0
    group_of = [None] * 11
    for g in range(5):
        for s in range(start[g], start[g + 1]):
            group_of[s] = g
    _check_prefix(L, P, _values(L, table, lens), _values(P, ptable, plens), group_of, q, out, lse)


@pytest.mark.parametrize("n_seqs,plen,group,pk,pv", [(1, 5000, 1, F16, F16), (3, 1, 4, Q8, Q8), (70, 3000, 4, Q4, Q4),
                                                     (130, 777, 8, Q8, F16), (33, 4097, 5, T4, T4)])
def test_one_prefix_for_all(n_seqs, plen, group, pk, pv):
    n_kv, lens = 2, [(13 * s + 7) % 200 for s in range(n_seqs)]
    cap = -(-plen // 256) * 256
    L, table = _filled(n_seqs, n_kv, n_kv * group, 256, Q8, Q8, False, lens, 31)
    P, ptable = _filled(1, n_kv, n_kv * group, cap, pk, pv, False, [plen], 32)
    q = _queries(n_seqs, n_kv * group, 9)
    out = torch.empty_like(q)
    kvq.attn_decode_prefix(L, P, q, SCALE, out, None, 256, cap, _prefix_ws(L, P, 256, cap))
    _check_prefix(L, P, _values(L, table, lens), _values(P, ptable, [plen]), [0] * n_seqs, q, out, None)


@pytest.mark.parametrize("ck,cv", [(F16, F16), (Q8, Q4), (F16, T4), (T4, Q8)])
@pytest.mark.parametrize("group", [4, 12])
def test_long_own_keys(ck, cv, group):
    """Few sequences of many own keys, which are split; one of none, one behind no prefix."""
    lens, plens = [2304, 0, 700, 1], [300, 9]
    L, table = _filled(4, 1, group, 2304, ck, cv, ck == Q8, lens, 23)
    P, ptable = _filled(2, 1, group, 512, Q4, F16, False, plens, 24)
    q = _queries(4, group, 15)
    out, lse = torch.empty_like(q), torch.empty((4, group), device="cuda")
    kvq.attn_decode_prefix(L, P, q, SCALE, out, lse, 2304, 512, _prefix_ws(L, P, 2304, 512), group_start=_i32([0, 2, 3]))
    assert L.err.item() == 0 and P.err.item() == 0
    _check_prefix(L, P, _values(L, table, lens), _values(P, ptable, plens), [0, 0, 1, None], q, out, lse)


@pytest.mark.parametrize("n_seqs,n_kv", [(160, 4), (321, 4), (1024, 3)])
def test_many_sequences(n_seqs, n_kv):
    """So many that a block takes two, four or eight of them (the last one less)."""
    lens = [(11 * s) % 70 for s in range(n_seqs)]
    L, table = _filled(n_seqs, n_kv, 2 * n_kv, 256, Q8, T4, False, lens, 25)
    P, ptable = _filled(2, n_kv, 2 * n_kv, 256, Q8, Q8, False, [200, 31], 26)
    q = _queries(n_seqs, 2 * n_kv, 16)
    out, lse = torch.empty_like(q), torch.empty((n_seqs, 2 * n_kv), device="cuda")
    cut = n_seqs // 3
    kvq.attn_decode_prefix(L, P, q, SCALE, out, lse, 256, 256, _prefix_ws(L, P, 256, 256),
                           group_start=_i32([0, cut, n_seqs - 1]))
    assert L.err.item() == 0 and P.err.item() == 0
    own, shared = _values(L, table, lens), _values(P, ptable, [200, 31])
    some = sorted({0, 1, 2, 7, 8, 9, cut - 1, cut, cut + 1, n_seqs // 2, n_seqs - 9, n_seqs - 2, n_seqs - 1})
    for s in some:
        parts = [(Q8, T4) + own[s]] + ([(Q8, Q8) + shared[int(s >= cut)]] if s < n_seqs - 1 else [])
        C.check(out[s:s + 1], lse[s:s + 1], C.attend(q[s:s + 1].double(), parts, SCALE), EPS[torch.float16], s)


def test_views_of_one_pool():
    """Sequences whose block tables share their first pages: the prefix a view over the shared
    pages, the rest a view behind them; the result is attn_decode's over the whole tables."""
    n_seqs, n_kv, n_q, shared = 6, 2, 8, 3
    lens = [shared * 256 + n for n in (0, 5, 300, 256, 77, 511)]
    pages = shared + n_seqs * 2
    table = torch.empty((n_seqs, shared + 2), dtype=torch.int32, device="cuda")
    order = torch.randperm(pages, device="cuda").to(torch.int32)
    table[:, :shared] = order[:shared]
    table[:, shared:] = order[shared:].view(n_seqs, 2)
    whole = kvq.KVLayer(n_seqs, n_kv, n_q, 256 * (shared + 2), Q8, Q8, n_pages=pages, block_table=table)
    k, v = (torch.randn((n_seqs, max(lens), n_kv, 128), device="cuda").half() for _ in "kv")
    k[:, :shared * 256], v[:, :shared * 256] = k[:1, :shared * 256], v[:1, :shared * 256]
    kvq.kv_append_quantize(whole, k, v, _i32(lens))
    view = dict(n_pages=pages, k_cache=whole.k_cache, v_cache=whole.v_cache)
    P = kvq.KVLayer(1, n_kv, n_q, 256 * shared, Q8, Q8, block_table=table[:1, :shared].contiguous(), **view)
    L = kvq.KVLayer(n_seqs, n_kv, n_q, 512, Q8, Q8, block_table=table[:, shared:].contiguous(), **view)
    P.seq_lens.fill_(256 * shared)
    L.seq_lens.copy_(_i32(lens) - 256 * shared)
    q = _queries(n_seqs, n_q, 10)
    out, lse = torch.empty_like(q), torch.empty((n_seqs, n_q), device="cuda")
    kvq.attn_decode_prefix(L, P, q, SCALE, out, lse, 512, 768, _prefix_ws(L, P, 512, 768))
    values = _values(whole, table.cpu().numpy(), lens)
    _check_rows(whole, values, q, out, lse, [1] * n_seqs)


def test_prefix_conditions():
    L, table = _filled(4, 1, 4, 256, F16, F16, False, [10, 20, 30, 40], 14)
    P, ptable = _filled(2, 1, 4, 512, F16, F16, False, [500, 300], 15)
    q = _queries(4, 4, 11)
    out, lse = torch.empty_like(q), torch.empty((4, 4), device="cuda")
    ws = _prefix_ws(L, P, 256, 400)
    kvq.attn_decode_prefix(L, P, q, SCALE, out, lse, 256, 400, ws, group_start=_i32([0, 2, 4]))
    assert P.err.item() == kvq.KVQ_DEVERR_MAXLEN and L.err.item() == 0
    shared = _values(P, ptable, [400, 300])
    _check_prefix(L, P, _values(L, table, [10, 20, 30, 40]), shared, [0, 0, 1, 1], q, out, lse)
    for bad in ([0, 3, 2], [0, 5, 4], [-1, 2, 4], [0, 2, 5]):
        P.err.zero_()
        kvq.attn_decode_prefix(L, P, q, SCALE, out, lse, 256, 512, _prefix_ws(L, P, 256, 512), group_start=_i32(bad))
        assert P.err.item() & kvq.KVQ_DEVERR_ROWS, bad


# ------------------------------------------------------------------ far places

@pytest.mark.parametrize("ck,cv", [(F16, F16), (Q8, F16)])
def test_pages_past_four_gigabytes(ck, cv):
    """Pages whose bytes lie past 2^32: the results of the same pages near the pool's start."""
    n_kv, far = 2, 70000 if ck == Q8 else 36000
    lens, pages = [600, 256], [[far - 1, 3, far - 7], [far - 2, 0, 0]]
    near = [[0, 1, 2], [3, 0, 0]]
    layers = []
    for n_pages, table in ((far, pages), (4, near)):
        L = kvq.KVLayer(2, n_kv, 8, 768, ck, cv, n_pages=n_pages, block_table=torch.tensor(table, dtype=torch.int32, device="cuda"))
        g = torch.Generator(device="cuda").manual_seed(4)
        x = torch.randn((sum(lens), 2 * n_kv, 128), generator=g, device="cuda").half()
        kvq.kv_append_rows(L, x[:, :n_kv], x[:, n_kv:], row_start=_i32([0, 600, 856]))
        assert L.k_cache.numel() > 2 ** 32 or n_pages == 4
        layers.append(L)
    got = []
    for L in layers:
        q = _queries(9, 8, 3)
        out, lse = torch.empty_like(q), torch.empty((9, 8), device="cuda")
        kvq.attn_cross(L, q, SCALE, out, lse, 768, _cross_ws(L, 9, 768), row_start=_i32([0, 4, 9]))
        one, P = torch.empty_like(q[:2]), kvq.KVLayer(1, n_kv, 8, 768, ck, cv, n_pages=L.n_pages, k_cache=L.k_cache,
                                                      v_cache=L.v_cache, block_table=L.block_table[:1].contiguous())
        P.seq_lens.fill_(600)
        kvq.attn_decode_prefix(L, P, q[:2].contiguous(), SCALE, one, None, 768, 768, _prefix_ws(L, P, 768, 768))
        rows = [torch.empty((856, n_kv, 128), dtype=torch.float32, device="cuda") for _ in "kv"]
        kvq.kv_read_rows(L, *rows, row_start=_i32([0, 600, 856]))
        few = [torch.empty((9, n_kv, 128), dtype=torch.float16, device="cuda") for _ in "kv"]
        kvq.kv_read_rows(L, *few, row_start=_i32([0, 4, 9]), first=_i32([590, 250]))
        got.append([out, lse, one, *rows, *few])
        assert L.err.item() == 0 and P.err.item() == 0
    for a, b in zip(*got):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ streams and graphs

def test_graphs_share_a_workspace():
    """Two captured calls over one workspace, replayed in turn with new lengths and queries."""
    lens = [600, 90, 255]
    L, table = _filled(3, 2, 8, 768, Q8, Q8, False, lens, 16)
    P, ptable = _filled(1, 2, 8, 1024, Q4, Q4, False, [1000], 17)
    own, shared = _values(L, table, lens), _values(P, ptable, [1000])
    q, q1 = _queries(20, 8, 12), _queries(3, 8, 13)
    out, out1 = torch.empty_like(q), torch.empty_like(q1)
    lse = torch.empty((20, 8), device="cuda")
    ws = torch.zeros(max(kvq.attn_cross_workspace(L, 20, 768), kvq.attn_decode_prefix_workspace(L, P, 768, 1024)),
                     dtype=torch.uint8, device="cuda")
    start = _i32([0, 9, 9, 20])
    cross = lambda: kvq.attn_cross(L, q, SCALE, out, lse, 768, ws, row_start=start)
    prefix = lambda: kvq.attn_decode_prefix(L, P, q1, SCALE, out1, None, 768, 1024, ws)
    graphs = []
    for f in (cross, prefix):
        f()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f()
        graphs.append(g)
    for step in range(3):
        cut = [max(0, n - 50 * step) for n in lens]
        L.seq_lens.copy_(_i32(cut))
        P.seq_lens.fill_(1000 - 300 * step)
        start.copy_(_i32([0, 9 - step, 9 + step, 20]))
        q.copy_(_queries(20, 8, 20 + step))
        q1.copy_(_queries(3, 8, 30 + step))
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        mine = [tuple(x[:, :n] for x in pair) for n, pair in zip(cut, own)]
        theirs = [tuple(x[:, :1000 - 300 * step] for x in shared[0])]
        _check_rows(L, mine, q, out, lse, [9 - step, 2 * step, 11 - step])
        _check_prefix(L, P, mine, theirs, [0] * 3, q1, out1, None)
    assert L.err.item() == 0 and P.err.item() == 0


def test_two_streams_at_once():
    """Calls on two streams over workspaces of their own, behind work that fills their inputs."""
    lens = [3000, 2000]
    L, table = _filled(2, 2, 8, 3328, F16, Q8, False, lens, 18)
    values = _values(L, table, lens)
    streams = [torch.cuda.Stream() for _ in "ab"]
    qs = [torch.zeros((60, 8, 128), dtype=torch.float16, device="cuda") for _ in "ab"]
    fresh = [_queries(60, 8, 40 + i) for i in (0, 1)]
    outs, wss = [torch.empty_like(q) for q in qs], [_cross_ws(L, 60, 3328) for _ in "ab"]
    start = _i32([0, 25, 60])
    torch.cuda.synchronize()
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                qs[i].copy_(fresh[i])
            kvq.attn_cross(L, qs[i], SCALE, outs[i], None, 3328, wss[i], row_start=start, stream=st)
    torch.cuda.synchronize()
    for i in (0, 1):
        _check_rows(L, values, fresh[i], outs[i], None, [25, 35])


def test_workspace_of_any_contents():
    """Only its size matters: filled with NaN it gives the same bits."""
    L, _ = _filled(2, 2, 8, 2048, Q8, Q4, False, [2000, 1500], 19)
    P, _ = _filled(1, 2, 8, 2048, Q8, Q4, False, [2000], 21)
    q, q1 = _queries(30, 8, 14), _queries(2, 8, 15)
    n = max(kvq.attn_cross_workspace(L, 30, 2048), kvq.attn_decode_prefix_workspace(L, P, 2048, 2048))
    got = []
    for fill in (0, 0xFF):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        out, out1 = torch.empty_like(q), torch.empty_like(q1)
        kvq.attn_cross(L, q, SCALE, out, None, 2048, ws, row_start=_i32([0, 3, 30]))
        kvq.attn_decode_prefix(L, P, q1, SCALE, out1, None, 2048, 2048, ws)
        got.append((out, out1))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
