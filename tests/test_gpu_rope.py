"""Rotary operators on the GPU against plain references: the angle table in
extended precision, rotated rows and cache bytes bit for bit, the decode step
against the two calls that it replaces, and a run of them together."""
import math

import numpy as np
import pytest
import torch

import attention_quantized_kv_gb300 as kvq

import oracle
from tests import _rope as R
from tests._helpers import ROW, tol

pytestmark = pytest.mark.gpu

SCALE = R.default_scale()
F16, Q8, Q4, T4 = 0, 1, 2, 3


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_quantized_kv_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _bits(x):
    return x.view({1: np.uint8, 2: np.uint16, 4: np.uint32}[x.dtype.itemsize])


def _host(t):
    """A tensor's values as fp32 (bf16 has no numpy type)."""
    return t.detach().float().cpu().numpy()


def _rounded(x32, dtype):
    return torch.from_numpy(np.ascontiguousarray(x32)).to(dtype)


def _same(t, ref):
    """Bit-equal tensors, NaN in the same places."""
    a, b = t.detach().cpu().contiguous(), ref.contiguous()
    nan = torch.isnan(b)
    assert torch.equal(torch.isnan(a), nan)
    iv = {2: torch.int16, 4: torch.int32}[a.element_size()]
    assert torch.equal(torch.where(nan, torch.zeros_like(a), a).view(iv),
                       torch.where(nan, torch.zeros_like(b), b).view(iv))


def _i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def _rope(rot, layout, n_pos, magnitude=1.0, base=500000.0):
    t = R.table32(R.freqs64(rot, base), n_pos)
    return kvq.Rope(table=torch.from_numpy(t).cuda(), layout=layout, magnitude=magnitude), t


# ------------------------------------------------------------------ table

# The fraction of a turn is off by pos * 2^-65 turns (below 2^-42 rad up to
# position 2^20); its conversion to fp32 by half an ulp of at most pi / 4 rad, 0.79 *
# 2^-24; cos and sin by at most an ulp of a value up to 1, 2^-24; the
# reference by 2^-50.  In all below 2^-23.
TABLE_TOL = 2.0 ** -23


@pytest.mark.parametrize("rot,n_pos", [(128, 1), (2, 1), (128, 1023), (34, 777), (6, 4097), (2, 5)])
@pytest.mark.parametrize("scaling", [kvq.KVQ_ROPE_PLAIN, kvq.KVQ_ROPE_YARN])
def test_table(rot, n_pos, scaling):
    freqs = kvq.kvq_rope_freqs(rot, 10000.0, scaling, 4.0, 1024)
    t = torch.full((n_pos + 1, rot // 2, 2), 7.0, device="cuda")
    kvq.kvq_rope_table(freqs, t[:n_pos])
    got = t.cpu().numpy()
    assert (got[n_pos] == 7.0).all()
    c, s = R.angles64(freqs, np.arange(n_pos))
    assert np.abs(got[:n_pos, :, 0] - c).max() <= TABLE_TOL
    assert np.abs(got[:n_pos, :, 1] - s).max() <= TABLE_TOL
    assert (got[0, :, 0] == 1).all() and (got[0, :, 1] == 0).all()


def test_table_far_positions():
    n_pos = 1 << 20
    freqs = kvq.kvq_rope_freqs(64, 10000.0) [:4] + [0.0, 6.283185, 3.0, 1e-9]
    t = torch.empty((n_pos, 8, 2), device="cuda")
    kvq.kvq_rope_table(freqs, t)
    at = np.r_[0:300, n_pos // 2:n_pos // 2 + 300, n_pos - 300:n_pos]
    got = t[torch.from_numpy(at).cuda()].cpu().numpy()
    c, s = R.angles64(freqs, at)
    assert max(np.abs(got[..., 0] - c).max(), np.abs(got[..., 1] - s).max()) <= TABLE_TOL


def test_small_angles_keep_their_relative_precision():
    """sin of a tiny angle is that angle: half an ulp from the conversion, one
    from the sine and one from the angle's 2^-64-turn steps (2^-24 at 1e-9)."""
    f = [1e-9, 3e-7, 1e-4]
    t = torch.empty((9, 3, 2), device="cuda")
    kvq.kvq_rope_table(f, t)
    ref = np.sin(np.arange(1, 9)[:, None] * np.array(f))
    # steps of 2^-64 turns: 2^-65 * 2 pi / 1e-9 = 1.7e-10 relative
    assert (np.abs(t.cpu().numpy()[1:, :, 1] / ref - 1) <= 2.5 * 2.0 ** -23).all()


# ------------------------------------------------------------------ apply

ROTS = [2, 6, 20, 64, 96, 126, 128]


@pytest.mark.parametrize("layout", [R.INTERLEAVED, R.HALF])
@pytest.mark.parametrize("rot", ROTS)
@pytest.mark.parametrize("types", [(torch.float16, torch.float16), (torch.bfloat16, torch.bfloat16),
                                   (torch.float32, torch.float32), (torch.bfloat16, torch.float16),
                                   (torch.float32, torch.float16)])
def test_apply_bits(layout, rot, types):
    """Strided rows of a fused projection, positions in any order, magnitude,
    both directions; outputs have the reference's bits."""
    ti, to = types
    rope, t = _rope(rot, layout, 333, 1.1386294)
    g = torch.Generator().manual_seed(rot + 7 * layout)
    for rows, heads in ((1, 1), (5, 3), (33, 9)):
        wide = torch.randn((rows, heads + 5, 128), generator=g).to(ti)
        pos = torch.randint(0, 333, (rows,), generator=g, dtype=torch.int32)
        out = torch.full((rows + 1, heads, 128), 3.0, dtype=to, device="cuda")
        err = _i32([0])
        for transpose in (False, True):
            kvq.kvq_rope_apply(rope, wide.cuda()[:, 2:2 + heads], out[:rows], pos.cuda(),
                               transpose=transpose, err=err)
            ref = R.rotate(wide[:, 2:2 + heads].float().numpy(), t[pos.numpy()], rot, layout,
                           np.float32(1.1386294), transpose)
            _same(out[:rows], _rounded(ref, to))
        assert (out[rows] == 3.0).all() and err.item() == 0


@pytest.mark.parametrize("layout", [R.INTERLEAVED, R.HALF])
def test_apply_error_against_64_bits(layout):
    """|y - exact| <= (|a| + |b|)(2^-23 + 3 * 2^-24): the table's error, then
    two products and a sum, each rounded once (half an ulp, relative 2^-24)."""
    rope = kvq.Rope(n_pos=2048, layout=layout)
    x = torch.randn((257, 4, 128), device="cuda")
    y = torch.empty_like(x)
    kvq.kvq_rope_apply(rope, x, y, pos0=1700)
    c, s = R.angles64(kvq.kvq_rope_freqs(128), np.arange(1700, 1957))
    ref = R.rotate(x.double().cpu().numpy(), np.stack([c, s], -1), 128, layout)
    a, b = R.planes(128, layout)
    size = np.zeros_like(ref)
    size[..., a] = size[..., b] = (x.abs()[..., a] + x.abs()[..., b]).double().cpu().numpy()
    assert (np.abs(y.double().cpu().numpy() - ref) <= size * 5 * 2.0 ** -24).all()


def test_apply_forms():
    """In place, repeated rows (stride 0), heads outside rows, pos0, int32-far
    strides do not apply: one test per way the same call is made."""
    rope, t = _rope(128, R.HALF, 64)
    x = torch.randn((16, 6, 128), device="cuda").half()
    ref = _rounded(R.rotate(_host(x), t[8:24], 128, R.HALF), torch.float16)
    y = x.clone()
    kvq.kvq_rope_apply(rope, y, y, pos0=8)
    _same(y, ref)
    z = torch.empty((6, 16, 128), dtype=torch.float16, device="cuda").transpose(0, 1)
    kvq.kvq_rope_apply(rope, x, z, pos0=8)
    _same(z, ref)
    one = x[:1].expand(16, 6, 128)
    kvq.kvq_rope_apply(rope, one, y, pos0=8)
    _same(y, _rounded(R.rotate(_host(one), t[8:24], 128, R.HALF), torch.float16))
    qkv = torch.randn((16, 10, 128), device="cuda").half()
    keep = qkv.clone()
    kvq.kvq_rope_apply(rope, qkv[:, :6], qkv[:, :6], pos0=8)
    _same(qkv[:, :6], _rounded(R.rotate(_host(keep[:, :6]), t[8:24], 128, R.HALF), torch.float16))
    assert torch.equal(qkv[:, 6:], keep[:, 6:])
    kvq.kvq_rope_apply(rope, x[:0], y[:0])  # no rows: nothing happens
    with pytest.raises(ValueError):
        kvq.kvq_rope_apply(rope, x, y[:, :5])
    with pytest.raises(ValueError):
        kvq.kvq_rope_apply(rope, x, y, positions=torch.zeros(16, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        kvq.kvq_rope_apply(rope, x, y, positions=_i32(range(15)))
    with pytest.raises(kvq.KVQError):
        kvq.kvq_rope_apply(rope, x[1:], x[:-1])


def test_apply_positions_outside_the_table():
    rope, t = _rope(128, R.INTERLEAVED, 50)
    x = torch.randn((4, 2, 128), device="cuda")
    y, err = torch.empty_like(x), _i32([0])
    kvq.kvq_rope_apply(rope, x, y, _i32([49, -3, 50, 2 ** 31 - 1]), err=err)
    assert err.item() == kvq.KVQ_DEVERR_POS
    _same(y, torch.from_numpy(R.rotate(_host(x), t[[49, 0, 49, 49]], 128, R.INTERLEAVED)))


@pytest.mark.parametrize("layout", [R.INTERLEAVED, R.HALF])
@pytest.mark.parametrize("rot", [6, 64, 128])
def test_apply_special_values(layout, rot):
    """Signed zeros, infinities and NaN pass like the formula's own."""
    rope, t = _rope(rot, layout, 8)
    g = np.random.default_rng(3)
    v = np.array([0.0, -0.0, 1.5, np.inf, -np.inf, np.nan, 6e4, -3e-8], np.float32)
    x = g.choice(v, (8, 3, 128)).astype(np.float16)
    y = torch.empty((8, 3, 128), dtype=torch.float16, device="cuda")
    kvq.kvq_rope_apply(rope, torch.from_numpy(x).cuda(), y, pos0=0)
    with np.errstate(all="ignore"):
        ref = R.rotate(x.astype(np.float32), t, rot, layout)
        _same(y, _rounded(ref, torch.float16))


@pytest.mark.parametrize("layout", [R.INTERLEAVED, R.HALF])
def test_gradient(layout):
    """The transpose against differences: f(x) = <w, R x> is linear, so a
    difference over a step of 1 is the gradient up to the roundings of y
    (|dy| <= 5 * 2^-24 of each operand pair, two evaluations)."""
    rope = kvq.Rope(n_pos=512, rot_dim=96, layout=layout, magnitude=1.2)
    x = torch.randn((3, 2, 128), device="cuda")
    w = torch.randn_like(x)
    g = torch.empty_like(x)
    kvq.kvq_rope_apply(rope, w, g, pos0=300, transpose=True)
    y = torch.empty_like(x)
    for r, h, d in ((0, 0, 0), (1, 1, 47), (2, 0, 48), (0, 1, 95), (1, 0, 96), (2, 1, 127)):
        f = []
        for e in (0.5, -0.5):
            z = x.clone()
            z[r, h, d] += e
            kvq.kvq_rope_apply(rope, z, y, pos0=300)
            f.append((w.double() * y.double()).sum().item())
        # only the two elements of d's plane move; each evaluation is off by at
        # most 1.2 * 8 ulps of |a| + |b| < 12 times |w| < 6
        assert abs(f[0] - f[1] - g[r, h, d].item()) <= 2 * 2 * 1.2 * 12 * 6 * 5 * 2.0 ** -24


# ------------------------------------------------------------------ append

def _layer(n_seqs, n_kv, n_q, cap, ck, cv, paged, seed, fill=0x5A, unmapped=()):
    """A layer over pattern-filled buffers; paged: shuffled pages."""
    table = None
    if paged:
        pps = cap // 256
        n_pages = n_seqs * pps + 2
        table = np.random.default_rng(seed).permutation(n_pages)[:n_seqs * pps].astype(np.int32)
        table = table.reshape(n_seqs, pps)
        for s, p in unmapped:
            table[s, p] = -1
        nb = [n_pages * n_kv * 256 * ROW[c] for c in (ck, cv)]
    else:
        nb = [n_seqs * n_kv * cap * ROW[c] for c in (ck, cv)]
    k, v = (torch.full((n,), fill, dtype=torch.uint8, device="cuda") for n in nb)
    L = kvq.KVLayer(n_seqs, n_kv, n_q, cap, ck, cv, k_cache=k, v_cache=v,
                    n_pages=n_pages if paged else 0,
                    block_table=torch.from_numpy(table).cuda() if paged else None)
    return L, table


def _images(L, table):
    return [R.Cache(c, i, t.cpu().numpy().copy(), L.n_kv_heads, L.capacity, table)
            for i, (c, t) in enumerate(((L.codec_k, L.k_cache), (L.codec_v, L.v_cache)))]


def _check_caches(L, images):
    for im, t in zip(images, (L.k_cache, L.v_cache)):
        got = t.cpu().numpy()
        assert (got == im.data).all(), np.flatnonzero(got != im.data)[:8]


def _append_ref(images, rows, lens, kx, vx, cs, rot, layout, mag):
    """rows: (row, seq, index) of every row to place; kx, vx fp32 [rows, n_kv, 128]."""
    if not rows:
        return
    at = [r for r, _, _ in rows]
    kr = R.rotate(kx[at], cs, rot, layout, mag)
    for im, x in zip(images, (kr, vx[at])):
        n_kv = x.shape[1]
        enc = R.encode_f32(im.codec, x.reshape(-1, 128)).reshape(len(rows), n_kv, -1)
        for j, (_, s, i) in enumerate(rows):
            for h in range(n_kv):
                im.put(s, h, lens[s] + i, enc[j, h])


@pytest.mark.parametrize("ck", [F16, Q8, Q4, T4])
@pytest.mark.parametrize("cv", [F16, Q8, Q4, T4])
@pytest.mark.parametrize("paged", [False, True])
def test_append_packed(ck, cv, paged):
    """Packed rows of sequences with none, one and many tokens, over unit and
    page borders, behind a padded tail: cache bytes, rotated queries, lengths."""
    n_kv, n_q, cap = 3, 6, 768
    counts, lens = [1, 0, 70, 17, 1], [255, 9, 247, 0, 16]
    layout, rot = (R.HALF, 128) if (ck + cv) % 2 else (R.INTERLEAVED, 96)
    ti = [torch.float16, torch.bfloat16, torch.float32][(ck + 2 * cv) % 3]
    rope, t = _rope(rot, layout, cap, 1.25)
    L, table = _layer(5, n_kv, n_q, cap, ck, cv, paged, 4)
    L.seq_lens.copy_(_i32(lens))
    images = _images(L, table)
    total = sum(counts)
    start = np.r_[0, np.cumsum(counts)]
    g = torch.Generator().manual_seed(11 + ck + 4 * cv)
    qkv = torch.randn((total + 4, n_q + 2 * n_kv, 128), generator=g).to(ti)
    dev = qkv.cuda()
    q, k, v = dev.split([n_q, n_kv, n_kv], dim=1)
    q_out = torch.full((total + 4, n_q, 128), 2.0, dtype=torch.float16, device="cuda")
    kvq.kv_append_rope(L, rope, k, v, row_start=_i32(start), q=q, q_out=q_out)
    rows = [(start[s] + i, s, i) for s in range(5) for i in range(counts[s])]
    pos = np.array([lens[s] + i for _, s, i in rows])
    x = qkv.float().numpy()
    _append_ref(images, rows, lens, x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:], t[pos], rot, layout, 1.25)
    _check_caches(L, images)
    _same(q_out[:total], _rounded(R.rotate(x[:total, :n_q], t[pos], rot, layout, 1.25), torch.float16))
    assert (q_out[total:] == 2.0).all()                      # rows behind the last sequence
    assert L.seq_lens.tolist() == [a + b for a, b in zip(lens, counts)]
    assert L.err.item() == 0


@pytest.mark.parametrize("ck,cv,layout,rot", [(F16, Q8, R.HALF, 128), (Q4, F16, R.HALF, 20),
                                              (Q8, T4, R.INTERLEAVED, 6), (T4, Q4, R.HALF, 126)])
@pytest.mark.parametrize("update", [False, True])
def test_append_padded_with_positions(ck, cv, layout, rot, update):
    """Padded rows and explicit positions (in any order, the same one twice)."""
    n_seqs, max_new, n_kv, cap = 4, 37, 2, 512
    counts, lens = [37, 0, 1, 20], [100, 5, 511, 0]
    rope, t = _rope(rot, layout, 999)
    L, table = _layer(n_seqs, n_kv, 4, cap, ck, cv, True, 8)
    L.seq_lens.copy_(_i32(lens))
    images = _images(L, table)
    g = torch.Generator().manual_seed(rot)
    k, v = (torch.randn((n_seqs, max_new, n_kv, 128), generator=g).half() for _ in range(2))
    pos = torch.randint(0, 999, (n_seqs, max_new), generator=g, dtype=torch.int32)
    kvq.kv_append_rope(L, rope, k.cuda(), v.cuda(), n_new=_i32(counts), positions=pos.cuda(),
                       update_lens=update)
    rows = [(s * max_new + i, s, i) for s in range(n_seqs) for i in range(counts[s])]
    p = pos.numpy().reshape(-1)[[r for r, _, _ in rows]]
    _append_ref(images, rows, lens, k.float().numpy().reshape(-1, n_kv, 128),
                v.float().numpy().reshape(-1, n_kv, 128), t[p], rot, layout, 1.0)
    _check_caches(L, images)
    assert L.seq_lens.tolist() == [a + b * update for a, b in zip(lens, counts)]
    assert L.err.item() == 0


WINDOW_COUNTS = [1, 0, 300, 17, 1, 2, 1, 13, 12, 11, 16, 250, 1, 3]
WINDOW_LENS = [255, 9, 247, 0, 16, 510, 31, 3, 4, 5, 240, 77, 0, 254]


@pytest.mark.parametrize("ck", [F16, Q8, Q4, T4])
@pytest.mark.parametrize("cv", [F16, Q8, Q4, T4])
@pytest.mark.parametrize("paged", [False, True])
def test_append_windows(ck, cv, paged):
    """Appends long enough to go by 16-row windows: whole units, incomplete ones
    with few and with many new rows, several sequences in a window, every kind
    of plane and row type, explicit positions, a padded tail."""
    n_kv, n_q, cap, i = 2, 32, 768, ck + 4 * cv + 16 * paged
    layout, rot = [(R.HALF, 128), (R.INTERLEAVED, 96), (R.HALF, 40), (R.HALF, 64), (R.INTERLEAVED, 6),
                   (R.HALF, 32), (R.HALF, 96), (R.HALF, 126), (R.INTERLEAVED, 128)][i % 9]
    ti = [torch.float16, torch.bfloat16, torch.float32][i % 3]
    n_seqs, total = len(WINDOW_COUNTS), sum(WINDOW_COUNTS)
    assert total * (n_q + 2 * n_kv) > 152 * 128               # (the kernel's rule)
    rope, t = _rope(rot, layout, cap, 1.25)
    L, table = _layer(n_seqs, n_kv, n_q, cap, ck, cv, paged, 4)
    L.seq_lens.copy_(_i32(WINDOW_LENS))
    images = _images(L, table)
    start = np.r_[0, np.cumsum(WINDOW_COUNTS)]
    g = torch.Generator().manual_seed(100 + i)
    qkv = torch.randn((total + 21, n_q + 2 * n_kv, 128), generator=g).to(ti)
    q, k, v = qkv.cuda().split([n_q, n_kv, n_kv], dim=1)
    q_out = torch.full((total + 21, n_q, 128), 2.0, dtype=torch.float16, device="cuda")
    pos = None
    if i % 2:
        pos = torch.randint(0, cap, (total + 21,), generator=g, dtype=torch.int32)
    kvq.kv_append_rope(L, rope, k, v, row_start=_i32(start), q=q, q_out=q_out,
                       positions=None if pos is None else pos.cuda())
    rows = [(start[s] + j, s, j) for s in range(n_seqs) for j in range(WINDOW_COUNTS[s])]
    p = np.array([WINDOW_LENS[s] + j for _, s, j in rows]) if pos is None else pos.numpy()[:total]
    x = qkv.float().numpy()
    _append_ref(images, rows, WINDOW_LENS, x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:], t[p], rot, layout, 1.25)
    _check_caches(L, images)
    _same(q_out[:total], _rounded(R.rotate(x[:total, :n_q], t[p], rot, layout, 1.25), torch.float16))
    assert (q_out[total:] == 2.0).all()
    assert L.seq_lens.tolist() == [a + b for a, b in zip(WINDOW_LENS, WINDOW_COUNTS)]
    assert L.err.item() == 0


@pytest.mark.parametrize("ck,cv,rot", [(F16, F16, 128), (Q8, Q4, 40), (T4, Q8, 64)])
def test_append_windows_device_conditions(ck, cv, rot):
    """By windows too: rows past the capacity, on an unmapped page and behind
    bad row starts are skipped, the padded form leaves gaps alone."""
    n_kv, n_q, cap, max_new = 2, 32, 512, 200
    rope, t = _rope(rot, R.HALF, cap)
    lens, counts = [400, 250, 33], [200, 180, 77]
    L, table = _layer(3, n_kv, n_q, cap, ck, cv, True, 3, unmapped=[(1, 1)])
    L.seq_lens.copy_(_i32(lens))
    images = _images(L, table)
    g = torch.Generator().manual_seed(rot)
    k, v = (torch.randn((3, max_new, n_kv, 128), generator=g).half() for _ in "kv")
    q = torch.randn((3, max_new, n_q, 128), generator=g).half()
    q_out = torch.full((3, max_new, n_q, 128), 2.0, dtype=torch.float16, device="cuda")
    assert 3 * max_new * (n_q + 2 * n_kv) > 152 * 128
    kvq.kv_append_rope(L, rope, k.cuda(), v.cuda(), n_new=_i32(counts), q=q.cuda(), q_out=q_out)
    rows = [(s * max_new + i, s, i) for s in range(3) for i in range(counts[s])
            if lens[s] + i < cap and not (s == 1 and lens[s] + i >= 256)]
    pos = np.array([lens[s] + i for _, s, i in rows])
    _append_ref(images, rows, lens, k.float().numpy().reshape(-1, n_kv, 128),
                v.float().numpy().reshape(-1, n_kv, 128), t[pos], rot, R.HALF, 1.0)
    _check_caches(L, images)
    for s in range(3):
        p = np.minimum(cap - 1, lens[s] + np.arange(counts[s]))
        _same(q_out[s, :counts[s]], _rounded(R.rotate(q[s, :counts[s]].float().numpy(), t[p], rot, R.HALF),
                                             torch.float16))
        assert (q_out[s, counts[s]:] == 2.0).all()
    # (positions of the rows past the capacity leave the table too)
    assert L.err.item() == kvq.KVQ_DEVERR_CAPACITY | kvq.KVQ_DEVERR_PAGE | kvq.KVQ_DEVERR_POS
    assert L.seq_lens.tolist() == [512, 430, 110]
    M, _ = _layer(3, n_kv, n_q, cap, ck, cv, True, 3)
    kvq.kv_append_rope(M, rope, k.cuda().view(600, n_kv, 128), v.cuda().view(600, n_kv, 128),
                       row_start=_i32([0, 601, -5, 700]), q=q.cuda().view(600, n_q, 128),
                       q_out=q_out.view(600, n_q, 128))
    assert M.err.item() & kvq.KVQ_DEVERR_ROWS and M.seq_lens.tolist() == [0, 0, 0]


def test_append_long_prompt_many_heads():
    """A prompt of several thousand rows with more query heads than one warp
    takes, q rotated in place."""
    n, n_kv, n_q, cap = 2311, 8, 40, 2560
    rope, t = _rope(128, R.HALF, cap)
    L, table = _layer(1, n_kv, n_q, cap, F16, Q8, False, 1, fill=0)
    images = _images(L, table)
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn((n, n_q, 128), generator=g, device="cuda").half()
    k = torch.randn((n, n_kv, 128), generator=g, device="cuda").half()
    v = torch.randn((n, n_kv, 128), generator=g, device="cuda").half()
    ref = _rounded(R.rotate(_host(q), t[:n], 128, R.HALF), torch.float16)
    kvq.kv_append_rope(L, rope, k, v, row_start=_i32([0, n]), q=q, q_out=q)
    _same(q, ref)
    _append_ref(images, [(i, 0, i) for i in range(n)], [0], _host(k), _host(v), t[:n], 128, R.HALF, 1.0)
    _check_caches(L, images)
    assert L.seq_lens.tolist() == [n]


@pytest.mark.parametrize("codec", [F16, Q8, Q4, T4])
def test_append_without_rotation_is_kv_append_quantize(codec):
    """Position 0 turns nothing (cos 1, sin 0): the bytes of the plain append."""
    rope, _ = _rope(128, R.INTERLEAVED, 4)
    a, _ = _layer(2, 2, 4, 256, codec, codec, False, 0)
    b, _ = _layer(2, 2, 4, 256, codec, codec, False, 0)
    x = torch.randn((2, 21, 2, 128), device="cuda").half()
    y = torch.randn((2, 21, 2, 128), device="cuda").half()
    n = _i32([21, 13])
    zero = torch.zeros((2, 21), dtype=torch.int32, device="cuda")
    kvq.kv_append_rope(a, rope, x, y, n_new=n, positions=zero)
    kvq.kv_append_quantize(b, x, y, n)
    assert torch.equal(a.k_cache, b.k_cache) and torch.equal(a.v_cache, b.v_cache)
    assert a.seq_lens.tolist() == b.seq_lens.tolist() == [21, 13]


def test_append_device_conditions():
    """Capacity, an unmapped page, positions behind the table, bad row starts:
    the bit is set, what can be placed is placed, nothing else is touched."""
    n_kv = 2
    rope, t = _rope(64, R.HALF, 300)
    x = torch.randn((24, n_kv, 128)).half()
    f = x.float().numpy()

    def run(lens, start, **kw):
        L, table = _layer(2, n_kv, 2, 512, F16, Q8, True, 3, **kw)
        L.seq_lens.copy_(_i32(lens))
        images = _images(L, table)
        kvq.kv_append_rope(L, rope, x.cuda(), x.cuda(), row_start=_i32(start))
        return L, images

    # sequence 0 passes the capacity after 4 rows (its positions leave the table)
    L, im = run([508, 3], [0, 12, 24])
    rows = [(i, 0, i) for i in range(4)] + [(12 + i, 1, i) for i in range(12)]
    pos = np.minimum(299, np.array([508 + i for i in range(4)] + [3 + i for i in range(12)]))
    _append_ref(im, rows, [508, 3], f, f, t[pos], 64, R.HALF, 1.0)
    _check_caches(L, im)
    assert L.err.item() == kvq.KVQ_DEVERR_CAPACITY | kvq.KVQ_DEVERR_POS
    assert L.seq_lens.tolist() == [512, 15]
    # sequence 1's second page is not mapped
    L, im = run([0, 250], [0, 12, 24], unmapped=[(1, 1)])
    rows = [(i, 0, i) for i in range(12)] + [(12 + i, 1, i) for i in range(6)]
    pos = np.array([i for _, s, i in rows if s == 0] + [250 + i for _, s, i in rows if s == 1])
    _append_ref(im, rows, [0, 250], f, f, t[pos], 64, R.HALF, 1.0)
    _check_caches(L, im)
    assert L.err.item() == kvq.KVQ_DEVERR_PAGE
    # a row_start behind the rows: sequence 1 keeps its length, sequence 0 is served
    L, im = run([0, 7], [0, 12, 25])
    assert L.err.item() == kvq.KVQ_DEVERR_ROWS and L.seq_lens.tolist() == [12, 7]
    # decreasing
    L, im = run([0, 7], [0, 12, 11])
    assert L.err.item() == kvq.KVQ_DEVERR_ROWS and L.seq_lens.tolist() == [12, 7]
    # negative count in the padded form
    L, _ = _layer(2, n_kv, 2, 512, F16, Q8, True, 3)
    kvq.kv_append_rope(L, rope, x.cuda().view(2, 12, n_kv, 128), x.cuda().view(2, 12, n_kv, 128),
                       n_new=_i32([12, 13]))
    assert L.err.item() == kvq.KVQ_DEVERR_ROWS and L.seq_lens.tolist() == [12, 0]


def test_append_many_sequences():
    """More sequences than threads in a block, most of them idle."""
    n_seqs, n_kv = 700, 1
    rng = np.random.default_rng(9)
    counts = (rng.random(n_seqs) < 0.3).astype(np.int64) * rng.integers(1, 4, n_seqs)
    lens = rng.integers(0, 200, n_seqs).tolist()
    start = np.r_[0, np.cumsum(counts)]
    total = int(start[-1])
    rope, t = _rope(128, R.INTERLEAVED, 256)
    L, table = _layer(n_seqs, n_kv, 1, 256, Q8, Q8, True, 5)
    L.seq_lens.copy_(_i32(lens))
    images = _images(L, table)
    x = torch.randn((total, n_kv, 128)).half()
    kvq.kv_append_rope(L, rope, x.cuda(), x.cuda(), row_start=_i32(start))
    rows = [(start[s] + i, s, i) for s in range(n_seqs) for i in range(counts[s])]
    pos = np.array([lens[s] + i for _, s, i in rows])
    _append_ref(images, rows, lens, x.float().numpy(), x.float().numpy(), t[pos], 128, R.INTERLEAVED, 1.0)
    _check_caches(L, images)
    assert L.seq_lens.tolist() == (np.array(lens) + counts).tolist() and L.err.item() == 0


# ------------------------------------------------------------------ shift

def _fill(L, images, lens, seed):
    """N(0, 1) K rows below the lengths, in the layer and in the images."""
    rng = np.random.default_rng(seed)
    im = images[0]
    for s, n in enumerate(lens):
        x = rng.standard_normal((n, L.n_kv_heads, 128)).astype(np.float16)
        if n:
            enc = oracle.encode_rows(im.codec, x.reshape(-1, 128)).reshape(n, L.n_kv_heads, -1)
            for i in range(n):
                for h in range(L.n_kv_heads):
                    im.put(s, h, i, enc[i, h])
    L.k_cache.copy_(torch.from_numpy(im.data))
    L.seq_lens.copy_(_i32(lens))


@pytest.mark.parametrize("codec", [F16, Q8, Q4, T4])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("layout,rot", [(R.HALF, 128), (R.INTERLEAVED, 128), (R.HALF, 64), (R.HALF, 20),
                                        (R.HALF, 96), (R.INTERLEAVED, 6)])
def test_shift_bits(codec, paged, layout, rot):
    """Deltas of both signs and zero over ragged sequences, odd lengths and an
    empty one: re-encoded bytes; untouched tokens keep theirs."""
    lens = [75, 0, 257, 16]
    rope, t = _rope(rot, layout, 300, 1.5)                   # (the magnitude is not applied)
    L, table = _layer(4, 2, 2, 512, codec, F16, paged, 6)
    images = _images(L, table)
    _fill(L, images, lens, 21)
    rng = np.random.default_rng(7)
    delta = rng.integers(-299, 300, (4, 512)).astype(np.int32)
    delta[rng.random((4, 512)) < 0.3] = 0
    delta[0, :32] = 0
    delta[2, 100:116] = -7                                   # a whole unit, one shift
    kvq.kv_rope_shift(L, rope, torch.from_numpy(delta).cuda())
    im = images[0]
    for s, n in enumerate(lens):
        for i in range(n):
            d = int(delta[s, i])
            if d == 0:
                continue
            raw = np.stack([im.get(s, h, i) for h in range(2)])
            x = oracle.decode_rows(codec, raw).astype(np.float32)  # exact in fp32
            y = R.rotate(x[None], t[[abs(d)]], rot, layout, 1.0, transpose=d < 0)[0]
            enc = R.encode_f32(codec, y)
            for h in range(2):
                im.put(s, h, i, enc[h])
    _check_caches(L, images)
    assert L.err.item() == 0


def test_shift_conditions():
    rope, t = _rope(128, R.HALF, 100)
    L, table = _layer(2, 1, 1, 512, F16, F16, True, 6, unmapped=[(1, 0)])
    images = _images(L, table)
    L.seq_lens.copy_(_i32([2, 3]))
    x = np.random.default_rng(1).standard_normal((2, 128)).astype(np.float32)
    for i in range(2):
        images[0].put(0, 0, i, R.encode_f32(F16, x[i:i + 1])[0])
    L.k_cache.copy_(torch.from_numpy(images[0].data))
    delta = torch.zeros((2, 512), dtype=torch.int32, device="cuda")
    delta[0, 0], delta[0, 1], delta[1, 0] = 2 ** 31 - 1, -2 ** 31, 5
    kvq.kv_rope_shift(L, rope, delta)
    x16 = x.astype(np.float16).astype(np.float32)
    for i, tr in ((0, False), (1, True)):
        y = R.rotate(x16[None, i:i + 1], t[[99]], 128, R.HALF, transpose=tr)[0]
        images[0].put(0, 0, i, R.encode_f32(F16, y)[0])
    _check_caches(L, images)
    assert L.err.item() == kvq.KVQ_DEVERR_POS | kvq.KVQ_DEVERR_PAGE


def test_delta():
    """Against a plain deletion; nothing evicted, everything evicted, the
    first and the last token; entries behind the new length untouched."""
    rng = np.random.default_rng(4)
    lens = [300, 5, 256, 0, 77, 1]
    ev = [sorted(rng.permutation(300)[:120]), [], list(range(256)), [], [0, 76], [0]]
    L, _ = _layer(6, 1, 1, 512, F16, F16, False, 0)
    L.seq_lens.copy_(_i32(lens))
    e = np.zeros((6, 256), np.int32)
    for s, row in enumerate(ev):
        e[s, :len(row)] = row
    delta = torch.full((6, 512), 99, dtype=torch.int32, device="cuda")
    kvq.kv_evict_delta(L, torch.from_numpy(e).cuda(), _i32([len(r) for r in ev]), delta)
    got = delta.cpu().numpy()
    for s, n in enumerate(lens):
        left = np.setdiff1d(np.arange(n), ev[s])
        assert (got[s, :len(left)] == np.arange(len(left)) - left).all()
        assert (got[s, len(left):] == 99).all()


def test_delta_of_long_lists():
    """Lists longer than a block takes at once: scattered, all in a row, at
    both ends, and exactly a block's number of tokens."""
    n, cap = 70000, 70144
    rng = np.random.default_rng(14)
    ev = [np.sort(rng.permutation(n)[:30000]), np.arange(1000, 3500), np.r_[0:700, n - 900:n],
          np.sort(rng.permutation(n)[:256]), np.arange(5, 5 + 257), np.sort(rng.permutation(n)[:69999])]
    L = kvq.KVLayer(len(ev), 1, 1, cap, Q4, Q4)
    L.seq_lens.fill_(n)
    e = np.zeros((len(ev), 70000), np.int32)
    for s, row in enumerate(ev):
        e[s, :len(row)] = row
    delta = torch.full((len(ev), cap), 99, dtype=torch.int32, device="cuda")
    kvq.kv_evict_delta(L, torch.from_numpy(e).cuda(), _i32([len(r) for r in ev]), delta)
    got = delta.cpu().numpy()
    for s in range(len(ev)):
        left = np.setdiff1d(np.arange(n), ev[s])
        assert (got[s, :len(left)] == np.arange(len(left)) - left).all()
        assert (got[s, len(left):] == 99).all()


@pytest.mark.parametrize("layout", [R.INTERLEAVED, R.HALF])
@pytest.mark.parametrize("rot", [40, 128])
def test_append_and_shift_against_64_bits(layout, rot):
    """f16 keys against the fp64 rotation by exact angles.  A key is rounded to
    fp16 once (half a step, 2^-11 of it, 2^-25 below 2^-14) after a rotation
    that is off by (|a| + |b|)(2^-23 + 3 * 2^-24), as in the rows' test."""
    n, cap, at = 700, 1024, 300
    freqs = kvq.kvq_rope_freqs(rot, 10000.0)
    rope = kvq.Rope(n_pos=2048, rot_dim=rot, layout=layout)
    L, _ = _layer(1, 2, 32, cap, F16, F16, False, 0, fill=0)
    L.seq_lens.fill_(at)
    x = torch.randn((n, 2, 128), device="cuda").half()
    q = torch.zeros((n, 32, 128), dtype=torch.float16, device="cuda")
    kvq.kv_append_rope(L, rope, x, x, row_start=_i32([0, n]), q=q, q_out=q)

    def keys():
        c = L.k_cache.cpu().numpy()
        return np.stack([oracle.dequant_stream(F16, 0, c, 2, cap, 0, h, at + n)[at:] for h in (0, 1)], 1)

    def check(x64, pos, transpose=False):
        c, s = R.angles64(freqs, pos)
        ref = R.rotate(x64, np.stack([c, s], -1), rot, layout, transpose=transpose)
        size = np.zeros_like(ref)
        a, b = R.planes(rot, layout)
        size[..., a] = size[..., b] = np.abs(x64[..., a]) + np.abs(x64[..., b])
        got = keys()
        assert (np.abs(got - ref) <= np.abs(ref) * 2.0 ** -11 + size * 6 * 2.0 ** -24 + 2.0 ** -25).all()
        return got

    got = check(x.double().cpu().numpy(), np.arange(at, at + n))
    kvq.kv_rope_shift(L, rope, torch.full((1, cap), -977, dtype=torch.int32, device="cuda"))
    check(got, np.full(n, 977), transpose=True)


# ------------------------------------------------------------------ decode step

def _twin(L, table):
    """The same layer over copies of its buffers."""
    M = kvq.KVLayer(L.n_seqs, L.n_kv_heads, L.n_q_heads, L.capacity, L.codec_k, L.codec_v,
                    k_cache=L.k_cache.clone(), v_cache=L.v_cache.clone(), n_pages=L.n_pages,
                    block_table=L.block_table)
    M.seq_lens.copy_(L.seq_lens)
    return M


def _random_layer(n_seqs, n_kv, n_q, cap, ck, cv, paged, lens, seed):
    L, table = _layer(n_seqs, n_kv, n_q, cap, ck, cv, paged, seed, fill=0)
    g = torch.Generator(device="cuda").manual_seed(seed)
    k, v = (torch.randn((n_seqs, max(lens), n_kv, 128), generator=g, device="cuda").half() for _ in "kv")
    kvq.kv_append_quantize(L, k, v, _i32(lens))
    return L, table


@pytest.mark.parametrize("ck", [F16, Q8, Q4, T4])
@pytest.mark.parametrize("cv", [F16, Q8, Q4, T4])
@pytest.mark.parametrize("paged", [False, True])
def test_decode_step_is_append_then_decode(ck, cv, paged):
    """Bit for bit, three steps in a row: rotation on any dimension, explicit
    positions, groups of 1 to 12 query heads, ragged, empty and full."""
    i = ck + 4 * cv
    n_kv, group = [1, 2, 3][i % 3], [1, 4, 5, 8, 12][i % 5]
    layout, rot = [(R.HALF, 128), (R.INTERLEAVED, 128), (R.HALF, 96), (R.HALF, 20), (R.INTERLEAVED, 6),
                   (R.HALF, 64), (R.HALF, 126)][i % 7]
    n_q, cap, lens = n_kv * group, 1024, [255, 0, 1000, 1024, 16, 777]
    rope, _ = _rope(rot, layout, cap + 1, [1.0, 1.3][i % 2])
    L, table = _random_layer(6, n_kv, n_q, cap, ck, cv, paged, lens, 30 + i)
    M = _twin(L, table)
    ws = torch.zeros(kvq.attn_decode_workspace(L, cap), dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(i)
    for step in range(3):
        q = torch.randn((6, n_q, 128), generator=g, device="cuda").half()
        k, v = (torch.randn((6, n_kv, 128), generator=g, device="cuda").half() for _ in "kv")
        pos = None if step < 2 else torch.randint(0, cap, (6,), generator=g, device="cuda",
                                                  dtype=torch.int32)
        out, lse = torch.full_like(q, 9), torch.full((6, n_q), 9.0, device="cuda")
        kvq.attn_decode_append_rope(L, rope, k, v, q, SCALE, out, lse, cap, ws, positions=pos)
        qr = torch.empty_like(q)
        kvq.kv_append_rope(M, rope, k, v, row_start=_i32(range(7)), q=q, q_out=qr, positions=pos)
        ref, ref_lse = torch.empty_like(out), torch.empty_like(lse)
        kvq.attn_decode(M, qr, SCALE, ref, ref_lse, cap, ws)
        assert torch.equal(L.k_cache, M.k_cache) and torch.equal(L.v_cache, M.v_cache)
        assert L.seq_lens.tolist() == M.seq_lens.tolist()
        assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    assert L.err.item() == M.err.item() == kvq.KVQ_DEVERR_CAPACITY
    assert not ws[:65536].any()


@pytest.mark.parametrize("n_seqs,ck,cv,paged", [(8, F16, Q8, True), (33, Q4, F16, False),
                                                (70, T4, T4, True)])
def test_decode_step_of_many_sequences(n_seqs, ck, cv, paged):
    """From 8 sequences on the step appends in a launch of its own: the bits
    of a step that cannot (a query on an 8-byte boundary), in place too."""
    n_kv, n_q, cap = 2, 6, 512
    lens = [(s * 37) % 511 for s in range(n_seqs)]
    lens[3], lens[5] = 512, 0
    rope, _ = _rope(96, R.HALF, cap, 1.1)
    L, table = _random_layer(n_seqs, n_kv, n_q, cap, ck, cv, paged, lens, 40)
    M, N = _twin(L, table), _twin(L, table)
    ws = torch.zeros(kvq.attn_decode_workspace(L, cap), dtype=torch.uint8, device="cuda")
    buf = torch.randn(n_seqs * n_q * 128 + 4, device="cuda").half()
    q_odd = buf[4:].view(n_seqs, n_q, 128)
    q = q_odd.clone()
    k, v = (torch.randn((n_seqs, n_kv, 128), device="cuda").half() for _ in "kv")
    outs = [torch.empty_like(q) for _ in "ab"]
    lses = [torch.empty((n_seqs, n_q), device="cuda") for _ in "abc"]
    kvq.attn_decode_append_rope(L, rope, k, v, q, SCALE, outs[0], lses[0], cap, ws)
    kvq.attn_decode_append_rope(M, rope, k, v, q_odd, SCALE, outs[1], lses[1], cap, ws)
    kvq.attn_decode_append_rope(N, rope, k, v, q, SCALE, q, lses[2], cap, ws)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], q)
    for X, lse in ((M, lses[1]), (N, lses[2])):
        assert torch.equal(lses[0], lse) and L.seq_lens.tolist() == X.seq_lens.tolist()
        assert torch.equal(L.k_cache, X.k_cache) and torch.equal(L.v_cache, X.v_cache)
        assert X.err.item() == L.err.item() == kvq.KVQ_DEVERR_CAPACITY | kvq.KVQ_DEVERR_POS
    assert not ws[:65536].any()


def test_decode_step_odd_pointers():
    """q on an 8-byte boundary (rows read without the bulk copy)."""
    L, table = _random_layer(3, 2, 8, 512, F16, Q8, False, [300, 17, 0], 3)
    M = _twin(L, table)
    rope, _ = _rope(128, R.HALF, 512)
    ws = torch.zeros(kvq.attn_decode_workspace(L, 512), dtype=torch.uint8, device="cuda")
    buf = torch.randn(3 * 8 * 128 + 4, device="cuda").half()
    q = buf[4:].view(3, 8, 128)
    assert q.data_ptr() % 16 == 8
    k, v = (torch.randn((3, 2, 128), device="cuda").half() for _ in "kv")
    out, ref = torch.empty((3, 8, 128), device="cuda").half(), torch.empty((3, 8, 128), device="cuda").half()
    kvq.attn_decode_append_rope(L, rope, k, v, q, SCALE, out, None, 512, ws)
    kvq.attn_decode_append_rope(M, rope, k, v, q.clone(), SCALE, ref, None, 512, ws)
    assert torch.equal(out, ref) and torch.equal(L.k_cache, M.k_cache)


@pytest.mark.parametrize("n_seqs", [3, 9])
def test_decode_step_every_pointer_odd(n_seqs):
    """q, out, k and v on 8-byte boundaries, few sequences and several."""
    lens = [(300 * s + 17) % 512 for s in range(n_seqs)]
    L, table = _random_layer(n_seqs, 2, 8, 512, F16, Q8, False, lens, 4)
    M = _twin(L, table)
    rope, _ = _rope(128, R.HALF, 512)
    ws = torch.zeros(kvq.attn_decode_workspace(L, 512), dtype=torch.uint8, device="cuda")
    q, k, v, out = (torch.randn(n_seqs * h * 128 + 4, device="cuda").half()[4:].view(n_seqs, h, 128)
                    for h in (8, 2, 2, 8))
    ref = torch.empty((n_seqs, 8, 128), device="cuda").half()
    kvq.attn_decode_append_rope(L, rope, k, v, q, SCALE, out, None, 512, ws)
    kvq.attn_decode_append_rope(M, rope, k.clone(), v.clone(), q.clone(), SCALE, ref, None, 512, ws)
    assert torch.equal(out, ref) and torch.equal(L.k_cache, M.k_cache)
    assert torch.equal(L.v_cache, M.v_cache) and L.seq_lens.tolist() == [n + 1 for n in lens]


def test_decode_step_against_the_oracle():
    """fp64 attention over the cache's own decoded rows, by the rotated query."""
    lens = [1500, 40]
    L, table = _random_layer(2, 2, 8, 2048, Q8, Q8, False, lens, 5)
    rope, t = _rope(128, R.HALF, 2048)
    ws = torch.zeros(kvq.attn_decode_workspace(L, 2048), dtype=torch.uint8, device="cuda")
    q = torch.randn((2, 8, 128), device="cuda").half()
    k, v = (torch.randn((2, 2, 128), device="cuda").half() for _ in "kv")
    out, lse = torch.empty_like(q), torch.empty((2, 8), device="cuda")
    kvq.attn_decode_append_rope(L, rope, k, v, q, SCALE, out, lse, 2048, ws)
    qr = R.rotate(_host(q), t[lens], 128, R.HALF).astype(np.float16)
    kc, vc = L.k_cache.cpu().numpy(), L.v_cache.cpu().numpy()
    ref, ref_lse = oracle.decode_layer(Q8, Q8, kc, vc, 2, 2, 8, 2048, [1501, 41], qr, SCALE)
    vmax = max(oracle.stream_absmax(Q8, 1, vc, 2, 2048, s, h, lens[s] + 1) for s in (0, 1) for h in (0, 1))
    assert np.abs(_host(out) - ref).max() <= tol(vmax)
    assert np.abs(_host(lse) - ref_lse).max() <= 1e-3


def test_decode_step_positions_outside_the_table():
    L, table = _random_layer(2, 1, 2, 512, F16, F16, False, [300, 20], 6)
    M = _twin(L, table)
    rope, _ = _rope(128, R.HALF, 512)
    ws = torch.zeros(kvq.attn_decode_workspace(L, 512), dtype=torch.uint8, device="cuda")
    q, k = torch.randn((2, 2, 128), device="cuda").half(), torch.randn((2, 1, 128), device="cuda").half()
    outs = [torch.empty_like(q) for _ in "ab"]
    kvq.attn_decode_append_rope(L, rope, k, k, q, SCALE, outs[0], None, 512, ws, positions=_i32([-5, 10 ** 9]))
    kvq.attn_decode_append_rope(M, rope, k, k, q, SCALE, outs[1], None, 512, ws, positions=_i32([0, 511]))
    assert torch.equal(*outs) and torch.equal(L.k_cache, M.k_cache)
    assert L.err.item() == kvq.KVQ_DEVERR_POS and M.err.item() == 0


# ------------------------------------------------------------------ far offsets

def test_offsets_past_32_bits():
    """A K side of over 4 GiB (bytes past 2^32) and rows whose strides pass 2^32
    bytes: the last sequence's keys appended, shifted and attended."""
    n_seqs, n_kv, cap = 9, 8, 262144
    L = kvq.KVLayer(n_seqs, n_kv, n_kv, cap, F16, Q4)
    assert L.k_cache.numel() > 2 ** 32
    rope, t = _rope(128, R.HALF, cap)
    at, n, s = cap - 50, 40, n_seqs - 1
    per = cap * 256                                           # one stream's bytes
    L.seq_lens[s] = at
    wide = torch.empty((n, 2 ** 26), dtype=torch.float16, device="cuda")   # 128 MiB between rows
    x = torch.randn((n, n_kv, 128), device="cuda").half()
    wide[:, :n_kv * 128] = x.view(n, -1)
    rows = wide[:, :n_kv * 128].unflatten(1, (n_kv, 128))
    assert rows.stride(0) * 2 * (n - 1) > 2 ** 32
    start = _i32([0] * n_seqs + [n])
    kvq.kv_append_rope(L, rope, rows, rows, row_start=start)
    y = torch.empty_like(x)
    kvq.kvq_rope_apply(rope, rows, y, pos0=at)
    assert L.seq_lens.tolist() == [0] * s + [at + n]

    def stream(h):
        c = L.k_cache[(s * n_kv + h) * per:(s * n_kv + h + 1) * per]
        return c[(at // 16) * 4096:].cpu().numpy()

    base = at // 16 * 16                                      # the first unit's token
    def keys(h):
        return oracle.dequant_stream(F16, 0, np.resize(stream(h), 256 * 256), 1, 256, 0, 0,
                                     at + n - base)[at - base:]

    ref = _rounded(R.rotate(_host(x), t[at:at + n], 128, R.HALF), torch.float16)
    _same(y, ref)
    for h in (0, n_kv - 1):
        assert (keys(h) == ref[:, h].double().numpy()).all()
    delta = torch.zeros((n_seqs, cap), dtype=torch.int32, device="cuda")
    delta[s, at:at + n] = -cap // 2
    kvq.kv_rope_shift(L, rope, delta)
    d = np.full(n, cap // 2)
    ref2 = R.rotate(ref.float().numpy(), t[d], 128, R.HALF, transpose=True).astype(np.float16)
    for h in (0, n_kv - 1):
        assert (keys(h) == ref2[:, h].astype(np.float64)).all()
    assert L.err.item() == 0
    del L, wide, rows
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ together

def _prompt(L, rope, counts, seed, ti=torch.float16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = sum(counts)
    qkv = torch.randn((n, L.n_q_heads + 2 * L.n_kv_heads, 128), generator=g, device="cuda").to(ti)
    q, k, v = qkv.split([L.n_q_heads, L.n_kv_heads, L.n_kv_heads], dim=1)
    q_out = torch.empty((n, L.n_q_heads, 128), dtype=torch.float16, device="cuda")
    kvq.kv_append_rope(L, rope, k, v, row_start=_i32(np.r_[0, np.cumsum(counts)]), q=q, q_out=q_out)
    return q_out


@pytest.mark.parametrize("ck,cv,paged", [(F16, Q8, True), (Q8, Q4, False)])
def test_prompt_decode_evict_decode(ck, cv, paged):
    """A server's run: prompts appended with rotation, prefill attention of the
    rotated queries, decode steps, an eviction that moves the keys back to
    their places, more steps; attention against the oracle at each point."""
    n_kv, n_q, cap = 2, 8, 1024
    rope = kvq.Rope(n_pos=cap, base=500000.0)
    t = rope.table.cpu().numpy()
    L, table = _layer(2, n_kv, n_q, cap, ck, cv, paged, 9, fill=0)
    counts = [601, 333]
    q_rot = _prompt(L, rope, counts, 3)

    def contiguous():
        out = []
        for codec, c in ((L.codec_k, L.k_cache), (L.codec_v, L.v_cache)):
            c = c.cpu().numpy()
            out.append(oracle.from_pool(codec, c, 2, n_kv, cap, table, L.n_pages) if paged else c)
        return out

    kc, vc = contiguous()
    pre = torch.empty((601, n_q, 128), dtype=torch.float16, device="cuda")
    pws = torch.empty(kvq.attn_prefill_workspace(L, 0, 601), dtype=torch.uint8, device="cuda")
    kvq.attn_prefill_chunk(L, 0, 0, q_rot[:601].contiguous(), SCALE, pre, None, pws)
    rows = [0, 17, 600]
    ref, _ = oracle.prefill_chunk(ck, cv, kc, vc, n_kv, n_q, cap, 0, 0, q_rot[:601].cpu().numpy(), SCALE,
                                  rows=rows)
    assert np.abs(_host(pre)[rows] - ref[rows]).max() <= tol(6.0)

    ws = torch.zeros(kvq.attn_decode_workspace(L, cap), dtype=torch.uint8, device="cuda")
    scores = torch.zeros((2, cap), device="cuda")
    g = torch.Generator(device="cuda").manual_seed(8)

    def step(lens):
        q = torch.randn((2, n_q, 128), generator=g, device="cuda").half()
        k, v = (torch.randn((2, n_kv, 128), generator=g, device="cuda").half() for _ in "kv")
        out, lse = torch.empty_like(q), torch.empty((2, n_q), device="cuda")
        kvq.attn_decode_append_rope(L, rope, k, v, q, SCALE, out, lse, cap, ws)
        qr = torch.empty_like(q)
        kvq.kvq_rope_apply(rope, q, qr, positions=_i32(lens))
        kvq.kv_probe_scores(L, qr, SCALE, lse, 0.9, scores)
        kc, vc = contiguous()
        ref, rlse = oracle.decode_layer(ck, cv, kc, vc, 2, n_kv, n_q, cap, [n + 1 for n in lens],
                                        qr.cpu().numpy(), SCALE)
        assert np.abs(_host(out) - ref).max() <= tol(6.0) and np.abs(_host(lse) - rlse).max() <= 1e-3
        return [n + 1 for n in lens]

    lens = step(step(counts))
    before, old = contiguous()[0], list(lens)
    scores, ev, nev = kvq.evict(L, scores, 4, 100, 90, rope=rope)
    assert nev.tolist() == [90, 90]
    lens = [n - 90 for n in lens]
    assert L.seq_lens.tolist() == lens
    # every kept key stands for its old value turned by its move, as re-encoded
    after = contiguous()[0]
    for s in range(2):
        left = np.setdiff1d(np.arange(old[s]), ev[s, :90].cpu().numpy())
        for h in range(n_kv):
            x = oracle.dequant_stream(ck, 0, before, n_kv, cap, s, h, old[s])[left].astype(np.float32)
            d = np.arange(len(left)) - left
            y = R.rotate(x[:, None], t[-d], 128, R.HALF, transpose=True)[:, 0]
            want = np.where((d != 0)[:, None], oracle.decode_rows(ck, R.encode_f32(ck, y)), x)
            got = oracle.dequant_stream(ck, 0, after, n_kv, cap, s, h, lens[s])
            assert (got == want).all()
    step(step(lens))
    assert L.err.item() == 0


def test_shift_agrees_with_appending_at_the_new_positions():
    """f16 keys: an append at p, then a shift by d, against an append at p + d.
    Each of the two roundings to fp16 is off by 2^-11 of an element, the first
    one turned: at most 2^-11 (|a| + |b|) + 2^-11 |y|, and 2^-22 for the rest."""
    rope = kvq.Rope(n_pos=4096)
    x = torch.randn((200, 1, 128), device="cuda").half()
    L, _ = _layer(1, 1, 1, 256, F16, F16, False, 0, fill=0)
    M, _ = _layer(1, 1, 1, 256, F16, F16, False, 0, fill=0)
    p = torch.arange(200, device="cuda", dtype=torch.int32) + 3000
    d = -torch.arange(200, device="cuda", dtype=torch.int32)
    kvq.kv_append_rope(L, rope, x, x, row_start=_i32([0, 200]), positions=p)
    kvq.kv_append_rope(M, rope, x, x, row_start=_i32([0, 200]), positions=p + d)
    delta = torch.zeros((1, 256), dtype=torch.int32, device="cuda")
    delta[0, :200] = d
    kvq.kv_rope_shift(L, rope, delta)
    a, b = (oracle.dequant_stream(F16, 0, c.k_cache.cpu().numpy(), 1, 256, 0, 0, 200) for c in (L, M))
    size = np.hypot(b[:, :64], b[:, 64:])                    # of a plane: |a| + |b| <= sqrt(2) size
    bound = np.tile(size, (1, 2)) * (math.sqrt(2.0) + 1 + 1) * 2.0 ** -11 + 2.0 ** -24
    assert (np.abs(a - b) <= bound).all()


def test_captured_and_on_another_stream():
    """A decode step and an append captured in graphs and replayed, against
    the same calls made eagerly on a side stream."""
    n_kv, n_q, cap, lens = 2, 8, 512, [100, 255, 0]
    rope = kvq.Rope(n_pos=cap)
    base, table = _random_layer(3, n_kv, n_q, cap, F16, Q8, True, lens, 12)
    L, M = _twin(base, table), _twin(base, table)
    q, k, v = (torch.randn((3, h, 128), device="cuda").half() for h in (n_q, n_kv, n_kv))
    wide = torch.randn((5, n_q + 2 * n_kv, 128), device="cuda").bfloat16()
    start = _i32([0, 1, 5, 5])
    ws = {id(x): torch.zeros(kvq.attn_decode_workspace(x, cap), dtype=torch.uint8, device="cuda")
          for x in (L, M)}
    outs = {id(x): (torch.empty_like(q), torch.empty((3, n_q), device="cuda"),
                    torch.empty((5, n_q, 128), dtype=torch.float16, device="cuda")) for x in (L, M)}

    def both(x):
        o, lse, qo = outs[id(x)]
        kvq.attn_decode_append_rope(x, rope, k, v, q, SCALE, o, lse, cap, ws[id(x)])
        a, b, c = wide.split([n_q, n_kv, n_kv], dim=1)
        kvq.kv_append_rope(x, rope, b, c, row_start=start, q=a, q_out=qo)

    warm = _twin(base, table)
    ws[id(warm)], outs[id(warm)] = torch.zeros_like(ws[id(L)]), tuple(torch.empty_like(t) for t in outs[id(L)])
    both(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(L)
    for _ in range(3):
        graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            both(M)
    torch.cuda.synchronize()
    assert L.seq_lens.tolist() == M.seq_lens.tolist() == [106, 270, 3]
    assert torch.equal(L.k_cache, M.k_cache) and torch.equal(L.v_cache, M.v_cache)
    for a, b in zip(outs[id(L)], outs[id(M)]):
        assert torch.equal(a, b)


def test_two_streams_at_once():
    """Appends and decode steps of two layers issued in turn on two streams,
    with nothing between them, against the same calls one after the other."""
    rope = kvq.Rope(n_pos=1024)
    layers = [_random_layer(2, 2, 8, 1024, Q8, F16, i == 1, [400, 33], 50 + i) for i in range(2)]
    pairs = [(L, _twin(L, t)) for L, t in layers]
    g = torch.Generator(device="cuda").manual_seed(5)
    xs = [torch.randn((90, 12, 128), generator=g, device="cuda").half() for _ in range(2)]
    start = _i32([0, 60, 90])

    def calls(L, x, ws, res):
        q, k, v = x.split([8, 2, 2], dim=1)
        kvq.kv_append_rope(L, rope, k, v, row_start=start, q=q, q_out=res[0])
        kvq.attn_decode_append_rope(L, rope, k[:2].contiguous(), v[:2].contiguous(), q[:2].contiguous(),
                                    SCALE, res[1], res[2], 1024, ws)

    def room(L):
        return (torch.zeros(kvq.attn_decode_workspace(L, 1024), dtype=torch.uint8, device="cuda"),
                (torch.empty((90, 8, 128), dtype=torch.float16, device="cuda"),
                 torch.empty((2, 8, 128), dtype=torch.float16, device="cuda"),
                 torch.empty((2, 8), device="cuda")))

    rooms = [[room(L) for L in p] for p in pairs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(6):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                calls(pairs[i][0], xs[i], *rooms[i][0])
    torch.cuda.synchronize()
    for i in (0, 1):
        for _ in range(6):
            calls(pairs[i][1], xs[i], *rooms[i][1])
        a, b = pairs[i]
        assert a.seq_lens.tolist() == b.seq_lens.tolist() == [400 + 6 * 61, 33 + 6 * 31]
        assert torch.equal(a.k_cache, b.k_cache) and torch.equal(a.v_cache, b.v_cache)
        for t, u in zip(rooms[i][0][1], rooms[i][1][1]):
            assert torch.equal(t, u)


def test_evict_and_table_on_another_stream():
    """evict (with and without rope) and a table on a busy stream that is not
    the current one, which goes on to allocate and fill memory of the sizes
    that the call let go of: the results of the same calls made in order."""
    side = torch.cuda.Stream()
    for with_rope in (False, True):
        base, table = _random_layer(2, 2, 4, 1024, Q8, F16, False, [900, 640], 21)
        M = _twin(base, table)
        L = _twin(base, table)
        g = torch.Generator(device="cuda").manual_seed(3)
        scores = torch.rand((2, 1024), generator=g, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        rope = kvq.Rope(n_pos=1024, rot_dim=96, stream=side)
        got = kvq.evict(L, scores, 4, 32, 200, stream=side, rope=rope if with_rope else None)
        sizes = [(t.numel(), t.dtype) for t in (M.k_cache, M.v_cache, M.seq_lens)]
        sizes.append((2 * 1024, torch.int32))
        junk = [torch.full((n,), 77, dtype=t, device="cuda") for n, t in sizes for _ in range(3)]
        torch.cuda.synchronize()
        assert all((t == 77).all() for t in junk)
        same = kvq.Rope(n_pos=1024, rot_dim=96)
        want = kvq.evict(M, scores, 4, 32, 200, rope=same if with_rope else None)
        assert torch.equal(rope.table, same.table)
        for a, b in zip((*got, L.k_cache, L.v_cache, L.seq_lens),
                        (*want, M.k_cache, M.v_cache, M.seq_lens)):
            assert torch.equal(a, b)
        assert L.err.item() == 0


@pytest.mark.parametrize("n_seqs", [3, 9])
def test_two_graphs_share_a_workspace(n_seqs):
    """Decode steps of two layers captured in two graphs over one workspace and
    replayed in turn, between shifts by captured deltas, against eager calls."""
    n_kv, n_q, cap = 2, 8, 512
    rope = kvq.Rope(n_pos=cap)
    lens = [(s * 53) % 490 for s in range(n_seqs)]
    layers = [_random_layer(n_seqs, n_kv, n_q, cap, Q8, F16, i == 1, lens, 70 + i) for i in range(2)]
    pairs = [(L, _twin(L, t)) for L, t in layers]
    ws = torch.zeros(max(kvq.attn_decode_workspace(L, cap) for L, _ in layers), dtype=torch.uint8,
                     device="cuda")
    g = torch.Generator(device="cuda").manual_seed(6)
    q, k, v = (torch.randn((n_seqs, h, 128), generator=g, device="cuda").half() for h in (n_q, n_kv, n_kv))
    delta = torch.randint(-3, 3, (n_seqs, cap), generator=g, device="cuda", dtype=torch.int32)
    outs = [[torch.empty_like(q) for _ in p] for p in pairs]

    def step(L, out):
        kvq.attn_decode_append_rope(L, rope, k, v, q, SCALE, out, None, cap, ws)
        kvq.kv_rope_shift(L, rope, delta)

    warm = _twin(*layers[0])
    step(warm, torch.empty_like(q))
    torch.cuda.synchronize()
    graphs = []
    for i in (0, 1):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            step(pairs[i][0], outs[i][0])
    for _ in range(4):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for i in (0, 1):
        a, b = pairs[i]
        for _ in range(4):
            step(b, outs[i][1])
        assert a.seq_lens.tolist() == b.seq_lens.tolist() == [n + 4 for n in lens]
        assert torch.equal(a.k_cache, b.k_cache) and torch.equal(a.v_cache, b.v_cache)
        assert torch.equal(*outs[i]) and a.err.item() == b.err.item() == 0
