"""Cache bytes of rows that reach the encoders' rare branches: zero blocks, ties
of both signs, quotients next to a rounding boundary, the smallest and largest
scales, infinities and NaN.  Every way into the cache writes the definition's
bytes: appends by rows and by windows, the fused steps, the re-encodings."""
import numpy as np
import pytest
import torch

import attention_quantized_kv_gb300 as kvq

import oracle
from tests import _encoders as E
from tests import _rope as R
from tests.test_gpu_rope import SCALE, _i32, _images, _layer

pytestmark = pytest.mark.gpu

F16, Q8, Q4, T4 = 0, 1, 2, 3
FINITE, OTHER = 0, 1


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_quantized_kv_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _tensor(x, dtype):
    """fp32 values of the type as a tensor of it, NaN with their bits."""
    if dtype == "float32":
        return torch.from_numpy(x.copy()).cuda()
    u = x.view(np.uint32)
    if dtype == "bfloat16":
        return torch.from_numpy((u >> 16).astype(np.uint16).view(np.int16)).view(torch.bfloat16).cuda()
    h = np.where(np.isnan(x), ((u >> 16) & 0x8000) | 0x7c00 | ((u >> 13) & 0x3ff), 0).astype(np.uint16)
    h = np.where(np.isnan(x), h, x.astype(np.float16).view(np.uint16))
    return torch.from_numpy(h.view(np.int16)).view(torch.float16).cuda()


KINDS = [FINITE, OTHER]


def _specials(dtype, kind, n_kv=2):
    """[n, n_kv, 128]: every special row in every head, at another place in each."""
    rows = E.special_rows(dtype)[kind]
    rows = np.concatenate([rows, rows])[:80]
    return np.stack([np.roll(rows, 37 * h, axis=0) for h in range(n_kv)], axis=1)


def _cached(codec, kind, n_kv=2):
    """Canonical rows [n, n_kv, bytes] of one head's special rows and their order turned about, by
    whether all of their values are finite."""
    x = np.concatenate(E.special_rows("float32" if codec else "float16"))
    raw = E.encode(codec, x)
    raw = raw[np.isfinite(E.decode(codec, raw)).all(axis=1) == (kind == FINITE)]
    return np.stack([np.roll(raw, 37 * h, axis=0) for h in range(n_kv)], axis=1)


def _turned(x, rot, layout, magnitude=1.0):
    """Rows at position 0: cos 1, sin 0 (an infinity turns its partner into a NaN)."""
    cs = np.zeros((len(x), rot // 2, 2), np.float32)
    cs[..., 0] = 1
    return R.rotate(x, cs, rot, layout, magnitude)


def _same_rows(codec, got, want):
    """Equal bytes; f16: equal values, NaN for NaN (a NaN's payload is not defined)."""
    if codec == F16:
        a, b = got.view(np.uint16), want.view(np.uint16)
        nan = (b & 0x7fff) > 0x7c00
        assert (((a & 0x7fff) > 0x7c00) == nan).all()
        assert (a[~nan] == b[~nan]).all()
        return
    bad = np.argwhere((got != want).any(axis=-1))
    first = [] if len(bad) == 0 else np.argwhere(got[tuple(bad[0])] != want[tuple(bad[0])])[:4, 0]
    assert len(bad) == 0, (codec, len(bad), bad[:4].tolist(),
                           [(int(i), int(got[tuple(bad[0])][i]), int(want[tuple(bad[0])][i])) for i in first])


def _check_side(L, table, side, want, at):
    """Rows at[j] = (sequence, token) hold want[j] [n_kv, row bytes]; every other byte is the fill's."""
    im = _images(L, table)[side]
    n_kv = L.n_kv_heads
    got = np.stack([np.stack([im.get(s, h, t) for h in range(n_kv)]) for s, t in at])
    _same_rows(im.codec, got, want)
    for s, t in at:
        for h in range(n_kv):
            im.put(s, h, t, 0x5A)
    assert (im.data == 0x5A).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("codec", [F16, Q8, Q4, T4])
@pytest.mark.parametrize("layout,rot", [(R.HALF, 2), (R.HALF, 128), (R.INTERLEAVED, 96)])
@pytest.mark.parametrize("windows", [False, True])
def test_append(kind, codec, dtype, layout, rot, windows):
    """kv_append_rope by rows and by windows of 16 (whole units, incomplete ones with many new rows
    and with few), both sides."""
    n_kv, n_q, cap = 2, 32, 1280
    x = _specials(dtype, kind)
    if windows:
        x = np.concatenate([x] * (600 // len(x) + 1))
    n = len(x)
    assert (n * (2 * n_kv + n_q * windows) > 152 * 128) == windows  # (the kernel's rule)
    counts, lens = [11, n // 2, n - 11 - n // 2 - 5, 5], [0, 3, 250, 14]
    L, table = _layer(4, n_kv, n_q, cap, codec, codec, True, 2)
    L.seq_lens.copy_(_i32(lens))
    t = torch.zeros((4, rot // 2, 2), device="cuda")
    t[..., 0] = 1
    rope = kvq.Rope(table=t, layout=layout)
    dev = _tensor(x, dtype)
    q = torch.zeros((n, n_q, 128), dtype=dev.dtype, device="cuda") if windows else None
    q_out = torch.empty((n, n_q, 128), dtype=torch.float16, device="cuda") if windows else None
    kvq.kv_append_rope(L, rope, dev, dev, row_start=_i32(np.r_[0, np.cumsum(counts)]), q=q, q_out=q_out,
                       positions=torch.zeros(n, dtype=torch.int32, device="cuda"))
    at = [(s, lens[s] + i) for s in range(4) for i in range(counts[s])]
    for side, y in ((0, _turned(x, rot, layout)), (1, x)):
        _check_side(L, table, side, E.encode(codec, y).reshape(n, n_kv, -1), at)
    assert L.err.item() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("windows", [False, True])
def test_append_overflow_after_the_magnitude(kind, dtype, windows):
    """f16 keys that the magnitude takes past 65504 are infinities, 8-bit scales likewise."""
    x = _specials(dtype, kind)
    x = np.concatenate([x] * (600 // len(x) + 1)) if windows else x
    n = len(x)
    for codec in (F16, Q8):
        L, table = _layer(1, 2, 32, 1280, codec, Q8, False, 2)
        t = torch.zeros((1, 64, 2), device="cuda")
        t[..., 0] = 1
        rope = kvq.Rope(table=t, magnitude=30000.0)
        dev = _tensor(x, dtype)
        q = torch.zeros((n, 32, 128), dtype=dev.dtype, device="cuda") if windows else None
        q_out = torch.empty((n, 32, 128), dtype=torch.float16, device="cuda") if windows else None
        kvq.kv_append_rope(L, rope, dev, dev, row_start=_i32([0, n]), q=q, q_out=q_out,
                           positions=torch.zeros(n, dtype=torch.int32, device="cuda"))
        y = _turned(x, 128, R.HALF, np.float32(30000.0))
        _check_side(L, table, 0, E.encode(codec, y).reshape(n, 2, -1), [(0, i) for i in range(n)])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("codec", [Q8, Q4, T4])
def test_append_quantize(kind, codec):
    """kv_append_quantize, few rows (one block) and many."""
    x = _specials("float16", kind)
    for a in (x[:12], x):
        n = len(a)
        L, table = _layer(1, 2, 2, 1280, codec, codec, False, 2)
        dev = _tensor(a, "float16").unsqueeze(0).contiguous()
        kvq.kv_append_quantize(L, dev, dev, _i32([n]))
        want = E.encode(codec, a).reshape(n, 2, -1)
        for side in (0, 1):
            _check_side(L, table, side, want, [(0, i) for i in range(n)])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("codec", [Q8, Q4, T4])
@pytest.mark.parametrize("n_seqs", [5, 24])
@pytest.mark.parametrize("rope", [False, True])
def test_decode_steps(kind, codec, n_seqs, rope):
    """The rows that a decode step appends, in the split kernel and in a launch of its own."""
    x = _specials("float16", kind)
    x = x[:len(x) // n_seqs * n_seqs]
    t = torch.zeros((512, 1, 2), device="cuda")
    t[..., 0] = 1
    r = kvq.Rope(table=t)
    q = torch.zeros((n_seqs, 4, 128), dtype=torch.float16, device="cuda")
    out = torch.empty_like(q)
    L, table = _layer(n_seqs, 2, 4, 512, codec, codec, False, 2)
    ws = torch.zeros(kvq.attn_decode_workspace(L, 512), dtype=torch.uint8, device="cuda")
    steps = x.reshape(-1, n_seqs, 2, 128)
    for a in steps:
        dev = _tensor(a, "float16")
        if rope:
            kvq.attn_decode_append_rope(L, r, dev, dev, q, SCALE, out, None, 512, ws)
        else:
            kvq.attn_decode_append(L, dev, dev, q, SCALE, out, None, 512, ws)
    at = [(s, i) for i in range(len(steps)) for s in range(n_seqs)]
    for side, y in ((0, _turned(x, 2, R.HALF) if rope else x), (1, x)):
        _check_side(L, table, side, E.encode(codec, y).reshape(len(x), 2, -1), at)


def _put_rows(L, table, side, rows, data=0x5A):
    """Canonical rows [n, n_kv, bytes] as tokens 0 .. n - 1 of sequence 0."""
    im = _images(L, table)[side]
    for t in range(len(rows)):
        for h in range(L.n_kv_heads):
            im.put(0, h, t, rows[t, h])
    (L.k_cache, L.v_cache)[side].copy_(torch.from_numpy(im.data))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("codec", [F16, Q8, Q4, T4])
@pytest.mark.parametrize("layout,rot", [(R.HALF, 128), (R.HALF, 20), (R.INTERLEAVED, 96)])
def test_shift(kind, codec, layout, rot):
    """Cached keys whose scales are zeros, infinities and the smallest numbers, f16 keys that are
    infinities and NaN, turned and encoded again."""
    raw = _cached(codec, kind)
    n = len(raw)
    L, table = _layer(1, 2, 2, 512, codec, F16, False, 2)
    _put_rows(L, table, 0, raw)
    L.seq_lens.fill_(n)
    table32 = R.table32(R.freqs64(rot, 10000.0), 64)
    rope = kvq.Rope(table=torch.from_numpy(table32).cuda(), layout=layout)
    delta = np.where(np.arange(512) % 5, np.arange(512) % 61 - 30, 0).astype(np.int32)
    kvq.kv_rope_shift(L, rope, torch.from_numpy(delta).view(1, 512).cuda())
    d = delta[:n]
    y = R.rotate(E.decode(codec, raw.reshape(2 * n, -1)).reshape(n, 2, 128), table32[np.abs(d)], rot, layout,
                 sign=np.where(d < 0, -1, 1))
    want = np.where((d != 0)[:, None, None], E.encode(codec, y).reshape(n, 2, -1), raw)
    _check_side(L, table, 0, want, [(0, i) for i in range(n)])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("src", [F16, Q8, Q4, T4])
@pytest.mark.parametrize("dst", [F16, Q8, Q4, T4])
@pytest.mark.parametrize("side", [0, 1])
def test_requantize(kind, src, dst, side):
    """Re-encoding of the same rows: what the source codec holds, by the append's encoder."""
    raw = _cached(src, kind)
    n = len(raw)
    L, table = _layer(1, 2, 2, 512, src, src, False, 2)
    _put_rows(L, table, side, raw)
    L.seq_lens.fill_(n)
    out = torch.full((2 * 512 * oracle.ROW_BYTES[dst],), 0x5A, dtype=torch.uint8, device="cuda")
    kvq.kv_requantize(L, side, dst, out)
    M, _ = _layer(1, 2, 2, 512, dst, dst, False, 2)
    M.k_cache = M.v_cache = out
    want = E.encode(dst, E.decode(src, raw.reshape(2 * n, -1)))
    if src == F16 and dst == F16:
        want = raw
    _check_side(M, None, side, want.reshape(n, 2, -1), [(0, i) for i in range(n)])
