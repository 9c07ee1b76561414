"""Rows appended without a rotation, and cached rows read back: bit for bit
against the decoders in numpy, each value rounded once to the output's type."""
import numpy as np
import pytest
import torch

import attention_quantized_kv_gb300 as kvq

from tests import _encoders as E
from tests import _rope as R
from tests.test_gpu_rope import _check_caches, _i32, _images, _layer

pytestmark = pytest.mark.gpu

F16, Q8, Q4, T4 = 0, 1, 2, 3
KINDS = {"float16": torch.float16, "bfloat16": torch.bfloat16, "float32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_quantized_kv_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _noise(L, seed):
    """Random bytes in both sides, fp16 scales and values finite."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    for t in (L.k_cache, L.v_cache):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.int32).to(torch.uint8))
    if L.codec_k == F16:
        L.k_cache.copy_(torch.randn(L.k_cache.numel() // 2, generator=g, device="cuda").half().view(torch.uint8))
    if L.codec_v == F16:
        L.v_cache.copy_(torch.randn(L.v_cache.numel() // 2, generator=g, device="cuda").half().view(torch.uint8))


def _same(got, want, dtype):
    """Equal values (NaN equals NaN), the reference rounded to the type."""
    g = got.float().cpu().numpy()
    w = E.as_type(want, dtype).reshape(g.shape)
    nan = np.isnan(w)
    assert (np.isnan(g) == nan).all()
    assert (g[~nan] == w[~nan]).all(), np.argwhere((g != w) & ~nan)[:5]


def _rows(image, seq, tokens):
    return np.stack([[E.decode(image.codec, image.get(seq, h, t)[None])[0] for h in range(image.n_kv)] for t in tokens])


@pytest.mark.parametrize("codec", [F16, Q8, Q4, T4])
@pytest.mark.parametrize("dtype", sorted(KINDS))
@pytest.mark.parametrize("paged", [False, True])
def test_packed(codec, dtype, paged):
    """Any bytes (scales that are infinite or NaN among them): both sides, ragged, rows that begin
    and end inside a unit, rows behind the last sequence as they were."""
    n_kv, cap = 3, 768
    L, table = _layer(5, n_kv, n_kv, cap, codec, codec, paged, 3)
    _noise(L, 5 + codec)
    L.seq_lens.copy_(_i32([768, 300, 5, 0, 257]))
    counts, first = [700, 33, 1, 0, 129], [9, 250, 4, 0, 128]
    total = sum(counts)
    k, v = (torch.full((total + 4, n_kv, 128), 3, dtype=KINDS[dtype], device="cuda") for _ in "kv")
    start = np.cumsum([0] + counts)
    kvq.kv_read_rows(L, k, v, row_start=_i32(start), first=_i32(first))
    assert L.err.item() == 0
    assert (k[total:] == 3).all() and (v[total:] == 3).all()
    for im, t in zip(_images(L, table), (k, v)):
        for s, n in enumerate(counts):
            if n:
                _same(t[start[s]:start[s + 1]], _rows(im, s, range(first[s], first[s] + n)), dtype)


@pytest.mark.parametrize("ck,cv", [(F16, Q8), (Q4, T4), (Q8, Q4), (T4, F16)])
def test_padded_views(ck, cv):
    """Padded rows into views of one fused tensor, sides of two types, one side alone."""
    n_kv = 2
    L, table = _layer(3, n_kv, n_kv, 512, ck, cv, False, 3)
    _noise(L, 9)
    L.seq_lens.copy_(_i32([512, 20, 100]))
    counts = [17, 20, 0]
    images = _images(L, table)
    fused = torch.full((3, 24, 2 * n_kv + 1, 128), 5, dtype=torch.float16, device="cuda")
    kvq.kv_read_rows(L, fused[:, :, :n_kv], fused[:, :, n_kv:2 * n_kv], n_read=_i32(counts))
    alone = torch.full((3, 24, n_kv, 128), 5, dtype=torch.float32, device="cuda")
    kvq.kv_read_rows(L, v=alone, n_read=_i32(counts))
    other = torch.full((3, 24, n_kv, 128), 5, dtype=torch.bfloat16, device="cuda")
    kvq.kv_read_rows(L, k=other, v=alone, n_read=_i32(counts))
    assert L.err.item() == 0
    for s, n in enumerate(counts):
        if n:
            rows = [_rows(im, s, range(n)) for im in images]
            _same(fused[s, :n, :n_kv], rows[0], "float16")
            _same(fused[s, :n, n_kv:2 * n_kv], rows[1], "float16")
            _same(alone[s, :n], rows[1], "float32")
            _same(other[s, :n], rows[0], "bfloat16")
        for t in (fused, alone, other):
            assert (t[s, n:] == 5).all()
    assert (fused[:, :, 2 * n_kv:] == 5).all()


def _equal(a, b):
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


@pytest.mark.parametrize("ck,cv", [(F16, F16), (Q8, Q4), (Q4, T4), (T4, Q8)])
@pytest.mark.parametrize("kinds", [("float16", "float16"), ("float32", "bfloat16"), ("bfloat16", "float32")])
@pytest.mark.parametrize("paged", [False, True])
def test_many_rows(ck, cv, kinds, paged):
    """A large call gives what small ones give, which the other tests compare with the decoders:
    runs of every length and place in a unit, pages that two sequences share, sides of two types."""
    n_kv, cap = 3, 1536
    L, _ = _layer(6, n_kv, n_kv, cap, ck, cv, paged, 3, unmapped=[(2, 1)] if paged else [])
    _noise(L, 31 + ck)
    if paged:  # sequence 1 ends, and sequence 3 begins, in one page
        L.block_table[3, 0] = L.block_table[1, 4]
    L.seq_lens.copy_(_i32([1536, 1100, 900, 40, 1, 700]))
    counts, first = [1500, 1024 + 13, 850, 23, 1, 530], [36, 1037 - 974, 11, 3, 0, 170]
    counts[5] += 20  # behind the sequence
    total = sum(counts)
    start = np.cumsum([0] + counts)
    got = [torch.full((total + 3, n_kv, 128), 3, dtype=KINDS[t], device="cuda") for t in kinds]
    kvq.kv_read_rows(L, *got, row_start=_i32(start), first=_i32(first))
    bits = kvq.KVQ_DEVERR_SEQLEN | (kvq.KVQ_DEVERR_PAGE if paged else 0)
    assert L.err.item() == bits
    want = [torch.full_like(t, 3) for t in got]
    for s, n in enumerate(counts):
        for at in range(0, n, 500):
            m = min(500, n - at)
            rows = [t[start[s] + at:start[s] + at + m] for t in want]
            begin = [0] * 6
            begin[s] = first[s] + at
            kvq.kv_read_rows(L, *rows, row_start=_i32([0] * (s + 1) + [m] * (6 - s)), first=_i32(begin))
    for a, b in zip(got, want):
        assert _equal(a, b)
    pad = torch.full((6, 1600, 2 * n_kv, 128), 3, dtype=KINDS[kinds[0]], device="cuda")  # views, padded
    kvq.kv_read_rows(L, pad[:, :, :n_kv], n_read=_i32(counts), first=_i32(first))
    for s, n in enumerate(counts):
        assert _equal(pad[s, :n, :n_kv], want[0][start[s]:start[s + 1]])
        assert (pad[s, n:] == 3).all() and (pad[s, :, n_kv:] == 3).all()


def test_many_sequences():
    """More sequences than a block keeps the starts of, empty ones among them."""
    n_seqs, n_kv = 300, 4
    L, _ = _layer(n_seqs, n_kv, n_kv, 256, Q8, T4, False, 3)
    _noise(L, 77)
    L.seq_lens.fill_(100)
    counts = [(7 * s) % 26 for s in range(n_seqs)]
    first = [s % 75 for s in range(n_seqs)]
    start = np.cumsum([0] + counts)
    total = int(start[-1])
    assert total >= 8 * n_seqs and total * 2 * n_kv >= 16384
    got = [torch.full((total, n_kv, 128), 3, dtype=torch.float32, device="cuda") for _ in "kv"]
    kvq.kv_read_rows(L, *got, row_start=_i32(start), first=_i32(first))
    assert L.err.item() == 0
    want = [torch.full_like(t, 3) for t in got]
    for lo in range(0, n_seqs, 75):
        rows = [t[start[lo]:start[lo + 75]] for t in want]
        part = np.clip(start, start[lo], start[lo + 75]) - start[lo]
        kvq.kv_read_rows(L, *rows, row_start=_i32(part), first=_i32(first))
    assert all(_equal(a, b) for a, b in zip(got, want))


def test_conditions():
    """Tokens outside a sequence, bad counts and unmapped pages: their bits, their rows untouched."""
    L, table = _layer(2, 2, 2, 512, Q8, Q8, True, 4, unmapped=[(1, 1)])
    _noise(L, 1)
    L.seq_lens.copy_(_i32([100, 512]))
    images = _images(L, table)

    def read(row_start, first, rows=40):
        L.err.zero_()
        k = torch.full((rows, 2, 128), 5, dtype=torch.float32, device="cuda")
        kvq.kv_read_rows(L, k=k, row_start=_i32(row_start), first=_i32(first))
        return k, L.err.item()

    k, err = read([0, 20, 40], [90, 236])
    assert err == kvq.KVQ_DEVERR_SEQLEN
    _same(k[:10], _rows(images[0], 0, range(90, 100)), "float32")
    assert (k[10:20] == 5).all()
    _same(k[20:], _rows(images[0], 1, range(236, 256)), "float32")
    k, err = read([0, 20, 40], [-5, 250])
    assert err == kvq.KVQ_DEVERR_SEQLEN | kvq.KVQ_DEVERR_PAGE
    assert (k[:5] == 5).all() and (k[26:] == 5).all()
    _same(k[5:20], _rows(images[0], 0, range(15)), "float32")
    k, err = read([0, 20, 41], [0, 0])
    assert err == kvq.KVQ_DEVERR_ROWS
    _same(k[:20], _rows(images[0], 0, range(20)), "float32")
    assert (k[20:] == 5).all()
    k, err = read([0, 0, 0], [0, 0])
    assert err == 0 and (k == 5).all()


@pytest.mark.parametrize("ck,cv", [(F16, F16), (Q8, Q4), (Q4, T4), (T4, Q8)])
@pytest.mark.parametrize("counts", [[3, 0, 1, 2], [700, 0, 33, 301]])
@pytest.mark.parametrize("dtype", sorted(KINDS))
def test_append(ck, cv, counts, dtype):
    """Rows of a fused projection appended by rows and by windows, packed and padded: the encoders'
    bytes, and those of kv_append_quantize for fp16; special values among them."""
    n_kv, cap, lens = 4, 1024, [5, 17, 0, 40]
    L, table = _layer(4, n_kv, n_kv, cap, ck, cv, True, 6)
    L.seq_lens.copy_(_i32(lens))
    images = _images(L, table)
    total = sum(counts)
    g = torch.Generator(device="cuda").manual_seed(total)
    kv = torch.randn((total, 2 * n_kv, 128), generator=g, device="cuda").to(KINDS[dtype])
    finite, other = E.special_rows(dtype)
    special = np.concatenate([finite, other])[:total * 2 * n_kv // 2]
    kv.view(-1, 128)[:len(special)] = torch.from_numpy(special).cuda().to(KINDS[dtype])
    k, v = kv[:, :n_kv], kv[:, n_kv:]
    start = np.cumsum([0] + counts)
    kvq.kv_append_rows(L, k, v, row_start=_i32(start))
    assert L.err.item() == 0 and L.seq_lens.tolist() == [a + b for a, b in zip(lens, counts)]
    for im, x in zip(images, (k, v)):
        enc = E.encode(im.codec, x.float().cpu().numpy().reshape(-1, 128)).reshape(total, n_kv, -1)
        for s, n in enumerate(counts):
            for i in range(n):
                for h in range(n_kv):
                    im.put(s, h, lens[s] + i, enc[start[s] + i, h])
    if ck != F16 and cv != F16:  # (a NaN's payload may change)
        _check_caches(L, images)
    # padded, the same rows: the same bytes
    M = kvq.KVLayer(4, n_kv, n_kv, cap, ck, cv, n_pages=L.n_pages, block_table=L.block_table,
                    k_cache=torch.full_like(L.k_cache, 0x5A), v_cache=torch.full_like(L.v_cache, 0x5A))
    M.seq_lens.copy_(_i32(lens))
    pad = torch.zeros((4, max(counts), 2 * n_kv, 128), dtype=KINDS[dtype], device="cuda")
    for s, n in enumerate(counts):
        pad[s, :n] = kv[start[s]:start[s + 1]]
    kvq.kv_append_rows(M, pad[:, :, :n_kv], pad[:, :, n_kv:], n_new=_i32(counts), update_lens=False)
    assert M.seq_lens.tolist() == lens
    assert torch.equal(L.k_cache, M.k_cache) and torch.equal(L.v_cache, M.v_cache)
    if dtype == "float16":
        kvq.kv_append_quantize(M, pad[:, :, :n_kv].contiguous(), pad[:, :, n_kv:].contiguous(), _i32(counts))
        if ck != F16 and cv != F16:
            assert torch.equal(L.k_cache, M.k_cache) and torch.equal(L.v_cache, M.v_cache)
    back = [torch.empty((total, n_kv, 128), dtype=torch.float32, device="cuda") for _ in "kv"]
    kvq.kv_read_rows(L, *back, row_start=_i32(start), first=_i32(lens))
    for im, t in zip(_images(L, table), back):
        for s, n in enumerate(counts):
            if n:
                _same(t[start[s]:start[s + 1]], _rows(im, s, range(lens[s], lens[s] + n)), "float32")


def test_append_conditions():
    """Rows past the capacity and negative lengths: the capacity's bit alone."""
    L, _ = _layer(2, 1, 1, 256, Q8, Q8, False, 7)
    L.seq_lens.copy_(_i32([250, -3]))
    x = torch.randn((20, 1, 128), device="cuda").half()
    kvq.kv_append_rows(L, x, x, row_start=_i32([0, 10, 20]))
    assert L.err.item() == kvq.KVQ_DEVERR_CAPACITY
    assert L.seq_lens.tolist() == [256, -3]


def test_an_encoder_and_its_decoder():
    """A run as a program makes it: an encoder's states written from a fused bf16 projection, a
    target's rows and then single tokens attending them, the states read back; captured in a graph
    and replayed with other states."""
    n_kv, n_q, counts = 2, 8, [300, 129]
    L, table = _layer(2, n_kv, n_q, 512, Q8, Q4, False, 8)
    start, rows = _i32([0, 300, 429]), _i32([0, 40, 61])
    kv = torch.empty((429, 2 * n_kv, 128), dtype=torch.bfloat16, device="cuda")
    q, one = (torch.empty((n, n_q, 128), dtype=torch.bfloat16, device="cuda") for n in (61, 2))
    out, out1 = torch.empty_like(q), torch.empty_like(one)
    back = torch.empty((429, n_kv, 128), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(kvq.attn_cross_workspace(L, n, 512) for n in (61, 2)), dtype=torch.uint8, device="cuda")
    scale = R.default_scale()

    def run():
        L.seq_lens.zero_()
        kvq.kv_append_rows(L, kv[:, :n_kv], kv[:, n_kv:], row_start=start)
        kvq.attn_cross(L, q, scale, out, None, 512, ws, row_start=rows)
        kvq.attn_cross(L, one, scale, out1, None, 512, ws)
        kvq.kv_read_rows(L, v=back, row_start=start)

    from tests import _cross as C
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for seed in (1, 2):
        torch.manual_seed(seed)
        for t in (kv, q, one):
            t.copy_(torch.randn(t.shape, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        assert L.err.item() == 0 and L.seq_lens.tolist() == counts
        images = _images(L, table)
        values = [tuple(C.rows_of(im, s, range(n)) for im in images) for s, n in enumerate(counts)]
        for s, (a, b) in enumerate([(0, 40), (40, 61)]):
            C.check(out[a:b], None, C.attend(q[a:b].half().double(), [(Q8, Q4) + values[s]], scale), 2.0 ** -8, s)
            C.check(out1[s:s + 1], None, C.attend(one[s:s + 1].half().double(), [(Q8, Q4) + values[s]], scale), 2.0 ** -8, s)
        want = torch.cat([v.transpose(0, 1) for _, v in values])
        assert torch.equal(back, want.to(torch.bfloat16))
