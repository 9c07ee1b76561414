"""Rotary positions without a GPU: frequencies against their formulas, the
plain references against one another, and every refusal that the host makes."""
import ctypes
import math

import numpy as np
import pytest
import torch

import attention_quantized_kv_gb300 as kvq
from attention_quantized_kv_gb300 import _abi

import oracle
from tests import _rope as R

EINVAL, EUNSUPPORTED, ECAPACITY, EALIGN, EWORKSPACE = 1, 2, 3, 4, 5


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_quantized_kv_gb300 import build
    build.build()


# ------------------------------------------------------------------ frequencies

# pow, log and a handful of operations, each within an ulp or two of double's
# 2^-53: 2^-48 leaves a factor of four over eight of them.
FREQ_TOL = 2.0 ** -48


@pytest.mark.parametrize("rot", [2, 4, 34, 96, 128])
@pytest.mark.parametrize("scaling", range(5))
def test_frequencies(rot, scaling):
    base, s, orig, lo, hi = 50000.0, 6.5, 4096.0, 1.5, 24.0
    got = kvq.kvq_rope_freqs(rot, base, scaling, s, orig, lo, hi)
    n = rot // 2
    assert len(got) == n
    for i in range(n):
        f = base ** (-2.0 * i / rot)
        if scaling == kvq.KVQ_ROPE_LINEAR:
            f = f / s
        elif scaling == kvq.KVQ_ROPE_NTK and n > 1:
            f = (base * s ** (rot / (rot - 2.0))) ** (-2.0 * i / rot)
        elif scaling == kvq.KVQ_ROPE_PARTS:
            keep = (orig * f / (2 * math.pi) - lo) / (hi - lo)
            keep = min(1.0, max(0.0, keep))
            f = f * keep + f / s * (1 - keep)
        elif scaling == kvq.KVQ_ROPE_YARN:
            def at(turns):
                return rot * math.log(orig / (2 * math.pi * turns)) / (2 * math.log(base))
            low, high = max(math.floor(at(hi)), 0), min(math.ceil(at(lo)), n - 1)
            keep = 1 - min(1.0, max(0.0, (i - low) / max(high - low, 0.001)))
            f = f * keep + f / s * (1 - keep)
        assert abs(got[i] - f) <= FREQ_TOL * f, (i, got[i], f)


def test_frequency_limits():
    """The fastest plane keeps its frequency under every blend, the slowest
    gets the whole factor, and a factor of 1 changes nothing."""
    plain = kvq.kvq_rope_freqs(128, 10000.0)
    for scaling in (kvq.KVQ_ROPE_PARTS, kvq.KVQ_ROPE_YARN):
        f = kvq.kvq_rope_freqs(128, 10000.0, scaling, 8.0, 2048)
        assert f[0] == plain[0] and abs(f[-1] * 8.0 / plain[-1] - 1) <= FREQ_TOL
        same = kvq.kvq_rope_freqs(128, 10000.0, scaling, 1.0, 2048)
        assert max(abs(a / b - 1) for a, b in zip(same, plain)) <= FREQ_TOL


@pytest.mark.parametrize("args,status", [
    ((0, 1e4, 0, 1.0, 0, 1, 4), EINVAL), ((3, 1e4, 0, 1.0, 0, 1, 4), EINVAL),
    ((130, 1e4, 0, 1.0, 0, 1, 4), EINVAL), ((128, 1.0, 0, 1.0, 0, 1, 4), EINVAL),
    ((128, math.nan, 0, 1.0, 0, 1, 4), EINVAL), ((128, math.inf, 0, 1.0, 0, 1, 4), EINVAL),
    ((128, 1e4, 5, 1.0, 0, 1, 4), EUNSUPPORTED), ((128, 1e4, -1, 1.0, 0, 1, 4), EUNSUPPORTED),
    ((128, 1e4, 1, 0.5, 0, 1, 4), EINVAL), ((128, 1e4, 1, math.nan, 0, 1, 4), EINVAL),
    ((128, 1e4, 2, math.inf, 0, 1, 4), EINVAL), ((128, 1e300, 2, 1e300, 0, 1, 4), EINVAL),
    ((128, 1e4, 3, 2.0, 0, 1, 4), EINVAL), ((128, 1e4, 3, 2.0, 4096, 4, 4), EINVAL),
    ((128, 1e4, 4, 2.0, 4096, 0, 4), EINVAL), ((128, 1e4, 4, 2.0, 4096, 1, math.inf), EINVAL),
    ((128, 1e4, 4, 2.0, math.nan, 1, 4), EINVAL),
])
def test_frequency_refusals(args, status):
    with pytest.raises(kvq.KVQError) as e:
        kvq.kvq_rope_freqs(*args)
    assert e.value.status == status


# ------------------------------------------------------------------ the references

@pytest.mark.parametrize("layout", [R.INTERLEAVED, R.HALF])
@pytest.mark.parametrize("rot", [2, 34, 128])
def test_reference_rotation_is_a_complex_product(layout, rot):
    rng = np.random.default_rng(5)
    x = rng.standard_normal((7, 3, 128))
    c, s = R.angles64(R.freqs64(rot), np.arange(7) * 1001)
    y = R.rotate(x, np.stack([c, s], -1), rot, layout, 1.25)
    ia, ib = R.planes(rot, layout)
    z = (x[..., ia] + 1j * x[..., ib]) * (1.25 * (c + 1j * s))[:, None]
    assert np.abs(y[..., ia] - z.real).max() < 1e-13 and np.abs(y[..., ib] - z.imag).max() < 1e-13
    assert (y[..., rot:] == x[..., rot:]).all()
    back = R.rotate(y, np.stack([c, s], -1), rot, layout, 1 / 1.25, transpose=True)
    assert np.abs(back - x).max() < 1e-13


def test_reference_encoder_is_the_oracles():
    rng = np.random.default_rng(6)
    x = rng.standard_normal((9, 128)).astype(np.float16)
    for codec in range(4):
        assert (R.encode_f32(codec, x.astype(np.float32)) == oracle.encode_rows(codec, x)).all()


# ------------------------------------------------------------------ refusals of the C ABI

def _rope(**kw):
    v = dict(table=0x10000, n_pos=4096, rot_dim=128, layout=1, magnitude=1.0)
    v.update(kw)
    return _abi.kvq_rope(v["table"], v["n_pos"], v["rot_dim"], v["layout"], v["magnitude"])


def _layer(**kw):
    d = _abi.kvq_layer()
    v = dict(n_seqs=2, n_kv_heads=2, n_q_heads=8, head_dim=128, capacity=512, codec_k=1, codec_v=1,
             pages_per_seq=0, k_cache=0x1000000, v_cache=0x2000000, seq_lens=0x3000000, err=None,
             block_table=None, n_pages=0, reserved=0)
    v.update(kw)
    for k, x in v.items():
        setattr(d, k, x)
    return d


def _rows(**kw):
    v = dict(data=0x4000000, row_stride=1024, head_stride=128, type=0, reserved=0)
    v.update(kw)
    return _abi.kvq_rows(v["data"], v["row_stride"], v["head_stride"], v["type"], v["reserved"])


BAD_ROPES = [({"table": None}, EINVAL), ({"table": 0x10004}, EALIGN), ({"n_pos": 0}, EINVAL),
             ({"rot_dim": 0}, EINVAL), ({"rot_dim": 5}, EINVAL), ({"rot_dim": 130}, EINVAL),
             ({"layout": 2}, EUNSUPPORTED), ({"magnitude": math.nan}, EINVAL),
             ({"magnitude": math.inf}, EINVAL)]


@pytest.mark.parametrize("kw,status", BAD_ROPES)
def test_every_call_refuses_a_bad_rope(kw, status):
    lib, r, L, k = _abi.load(), _rope(**kw), _layer(), _rows()
    y = _rows(data=0x8000000)
    assert lib.kvq_rope_apply(r, k, y, 4, 8, None, 0, 0, None, None) == status
    assert lib.kv_append_rope(L, r, None, k, y, 4, 0x100, None, None, None, 1, None) == status
    assert lib.kv_rope_shift(L, r, 0x100, None) == status
    assert lib.attn_decode_append_rope(L, r, None, 0x100, 0x200, 0x300, 1.0, 0x400, None, 512,
                                       0x1000, 1 << 30, None) == status


def test_missing_rope():
    lib, L, k, y = _abi.load(), _layer(), _rows(), _rows(data=0x8000000)
    assert lib.kvq_rope_apply(None, k, y, 4, 8, None, 0, 0, None, None) == EINVAL
    assert lib.kv_append_rope(L, None, None, k, y, 4, 0x100, None, None, None, 1, None) == EINVAL
    assert lib.kv_rope_shift(L, None, 0x100, None) == EINVAL


def test_table_refusals():
    lib = _abi.load()
    f = (ctypes.c_double * 64)(*([0.5] * 64))
    call = lib.kvq_rope_table
    assert call(None, 128, 16, 0x1000, None) == EINVAL
    assert call(f, 128, 16, None, None) == EINVAL
    assert call(f, 7, 16, 0x1000, None) == EINVAL and call(f, 0, 16, 0x1000, None) == EINVAL
    assert call(f, 130, 16, 0x1000, None) == EINVAL
    assert call(f, 128, 0, 0x1000, None) == EINVAL
    assert call(f, 128, 16, 0x1008, None) == EALIGN
    for bad in (-1e-9, 6.28318531, math.nan, math.inf):
        f[63] = bad
        assert call(f, 128, 16, 0x1000, None) == EINVAL, bad


def test_apply_refusals():
    lib, r = _abi.load(), _rope()
    x, y = _rows(), _rows(data=0x8000000)

    def call(x=x, y=y, n=4, heads=8, pos=None, err=None):
        return lib.kvq_rope_apply(r, x, y, n, heads, pos, 0, 0, err, None)

    assert call(n=0) == 0                                  # nothing to do, nothing launched
    assert call(x=None) == EINVAL and call(y=None) == EINVAL
    assert call(n=-1) == EINVAL and call(n=1 << 31) == EINVAL and call(heads=0) == EINVAL
    assert call(heads=65537) == EINVAL
    assert call(x=_rows(data=None)) == EINVAL and call(x=_rows(reserved=1)) == EINVAL
    assert call(x=_rows(type=3)) == EUNSUPPORTED and call(x=_rows(type=-1)) == EUNSUPPORTED
    assert call(x=_rows(data=0x4000008)) == EALIGN and call(y=_rows(data=0x8000002)) == EALIGN
    assert call(x=_rows(row_stride=1028)) == EALIGN and call(x=_rows(head_stride=129)) == EALIGN
    assert call(x=_rows(row_stride=-1024)) == EINVAL
    assert call(y=_rows(data=0x8000000, type=1)) == EUNSUPPORTED   # fp16 to bf16
    assert call(x=_rows(type=1), y=_rows(data=0x8000000, type=2)) == EUNSUPPORTED
    # an output that shares places between rows or heads
    assert call(y=_rows(data=0x8000000, row_stride=0)) == EINVAL
    assert call(y=_rows(data=0x8000000, head_stride=0)) == EINVAL
    assert call(y=_rows(data=0x8000000, row_stride=896)) == EINVAL
    assert call(y=_rows(data=0x8000000, head_stride=64)) == EINVAL
    # overlapping, but not the same rows
    assert call(y=_rows(data=0x4000000 + 256)) == EINVAL
    assert call(y=_rows(row_stride=2048)) == EINVAL
    assert call(x=_rows(type=2, row_stride=1024), y=_rows(type=0)) == EINVAL
    assert call(pos=0x102) == EALIGN and call(err=0x102) == EALIGN


def test_append_refusals():
    lib, r = _abi.load(), _rope()
    kv = dict(row_stride=256)
    k, v, q = _rows(**kv), _rows(data=0x5000000, **kv), _rows(data=0x6000000)

    def call(L=None, q=None, k=k, v=v, n=4, n_new=0x100, start=None, pos=None, out=None):
        return lib.kv_append_rope(L or _layer(), r, q, k, v, n, n_new, start, pos, out, 1, None)

    assert call(L=_layer(head_dim=64)) == EUNSUPPORTED and call(L=_layer(capacity=500)) == EALIGN
    assert call(k=None) == EINVAL and call(v=None) == EINVAL
    assert call(n=-2) == EINVAL and call(n=1 << 31) == EINVAL
    assert call(n=5) == EINVAL                              # padded: 5 rows of 2 sequences
    assert call(n_new=None) == EINVAL                       # neither form
    assert call(start=0x100) == EINVAL                      # both forms
    assert call(n=0) == 0
    assert call(n_new=None, start=0x102) == EALIGN and call(n_new=0x101) == EALIGN
    assert call(pos=0x106) == EALIGN
    assert call(k=_rows(data=None)) == EINVAL and call(v=_rows(data=0x5000004, **kv)) == EALIGN
    assert call(v=_rows(data=0x5000000, type=1, **kv)) == EUNSUPPORTED   # k and v of two types
    assert call(q=q) == EINVAL and call(out=0x7000000) == EINVAL          # q and q_out go together
    assert call(q=_rows(data=0x6000000, type=2), out=0x7000000) == EUNSUPPORTED
    assert call(q=q, out=0x7000008) == EALIGN
    assert call(q=q, out=0x6000000 + 256) == EINVAL          # q_out over part of q
    assert call(q=q, out=0x4000000) == EINVAL                # over k
    assert call(q=_rows(data=0x6000000, row_stride=2048), out=0x6000000) == EINVAL


def test_shift_and_delta_refusals():
    lib, r, L = _abi.load(), _rope(), _layer()
    assert lib.kv_rope_shift(L, r, None, None) == EINVAL
    assert lib.kv_rope_shift(L, r, 0x102, None) == EALIGN
    assert lib.kv_rope_shift(_layer(codec_k=9), r, 0x100, None) == EUNSUPPORTED
    assert lib.kv_evict_delta(L, None, 0x100, 4, 0x200, None) == EINVAL
    assert lib.kv_evict_delta(L, 0x100, None, 4, 0x200, None) == EINVAL
    assert lib.kv_evict_delta(L, 0x100, 0x100, -1, 0x200, None) == EINVAL
    assert lib.kv_evict_delta(L, 0x100, 0x100, 4, None, None) == EINVAL
    assert lib.kv_evict_delta(L, 0x102, 0x100, 4, 0x200, None) == EALIGN
    many = _layer(n_seqs=65536)
    assert lib.kv_rope_shift(many, r, 0x100, None) == EINVAL
    assert lib.kv_evict_delta(many, 0x100, 0x100, 4, 0x200, None) == EINVAL


def test_decode_refusals():
    lib = _abi.load()

    def call(r=None, L=None, pos=None, k=0x100, v=0x200, q=0x300, out=0x400, lse=None, max_len=512,
             ws=0x1000):
        return lib.attn_decode_append_rope(L or _layer(), r or _rope(), pos, k, v, q, 1.0, out, lse,
                                           max_len, ws, 1 << 30, None)

    assert call(k=None) == EINVAL and call(v=None) == EINVAL and call(q=None) == EINVAL
    assert call(out=None) == EINVAL and call(max_len=0) == EINVAL
    assert call(max_len=513) == ECAPACITY
    assert call(r=_rope(n_pos=511)) == ECAPACITY             # a length the table does not reach
    assert call(pos=0x102) == EALIGN and call(q=0x304) == EALIGN and call(lse=0x402) == EALIGN
    assert call(ws=None) == EWORKSPACE and call(ws=0x1008) == EALIGN


# ------------------------------------------------------------------ refusals of the binding

def test_binding_refuses_host_tensors():
    t = torch.zeros((16, 64, 2))
    x = torch.zeros((4, 8, 128), dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA device"):
        kvq.kvq_rope_table([1.0] * 64, t)
    with pytest.raises(ValueError, match="CUDA device"):
        kvq.Rope(table=t)
    with pytest.raises(ValueError):
        kvq.Rope(table=torch.zeros((16, 65, 2)))
    with pytest.raises(ValueError):
        kvq.Rope(table=torch.zeros((0, 64, 2)))
    with pytest.raises(ValueError, match="layout"):
        kvq.Rope(n_pos=16, layout=7)
    with pytest.raises(ValueError, match="magnitude"):
        kvq.Rope(n_pos=16, magnitude=math.inf)
    with pytest.raises(ValueError, match="CUDA device"):
        kvq.kvq_rope_apply(None, x, x)


def test_row_descriptors():
    """Strides of the views that a model hands over, and what no single stride covers."""
    dev = torch.device("cpu")
    qkv = torch.zeros((5, 12, 128), dtype=torch.bfloat16)
    d, n = kvq._rows(qkv[:, 8:10], 2, dev, "x")
    assert (n, d.row_stride, d.head_stride, d.type) == (5, 12 * 128, 128, 1)
    assert d.data == qkv.data_ptr() + 8 * 128 * 2
    d, n = kvq._rows(qkv.view(1, 5, 12, 128)[:, :, :8], 8, dev, "x")
    assert (n, d.row_stride) == (5, 12 * 128)
    d, n = kvq._rows(torch.zeros((3, 1, 4, 128))[:, :, 1:3], 2, dev, "x")
    assert (n, d.row_stride, d.head_stride) == (3, 512, 128)
    d, n = kvq._rows(torch.zeros((1, 4, 128)).expand(6, 4, 128), 4, dev, "x")
    assert (n, d.row_stride) == (6, 0)
    d, n = kvq._rows(torch.zeros((4, 6, 128)).transpose(0, 1), 4, dev, "x")  # heads outside
    assert (n, d.row_stride, d.head_stride) == (6, 128, 6 * 128)
    for bad in (torch.zeros((5, 12, 256))[..., ::2], torch.zeros((5, 11, 128)), torch.zeros((12, 128)),
                torch.zeros((5, 12, 64)), torch.zeros((5, 12, 128), dtype=torch.float64),
                torch.zeros((3, 9, 12, 128))[:, :4]):
        with pytest.raises(ValueError):
            kvq._rows(bad, 12, dev, "x")


def test_layer_without_an_error_word():
    """err is optional in the C descriptor: a layer may drop or replace its word."""
    L = kvq.KVLayer(1, 1, 1, 256, kvq.KVQ_F16, kvq.KVQ_F16, device="cpu")
    word = L.err
    assert L.desc().err == word.data_ptr()
    L.err = None
    assert not L.desc().err
    L.err = word
    assert L.desc().err == word.data_ptr()


@pytest.mark.parametrize("codec", [kvq.KVQ_F16, kvq.KVQ_Q8_0, kvq.KVQ_Q4_0, kvq.KVQ_TURBO4, 9])
def test_side_bytes_are_the_librarys(codec):
    flat = kvq.KVLayer(3, 2, 4, 512, kvq.KVQ_F16, kvq.KVQ_F16, device="cpu")
    paged = kvq.KVLayer(1, 2, 4, 512, kvq.KVQ_F16, kvq.KVQ_F16, device="cpu", n_pages=7)
    assert kvq._side_bytes(flat, codec) == kvq.kvq_cache_bytes(codec, 3, 2, 512)
    assert kvq._side_bytes(paged, codec) == kvq.kvq_pool_bytes(codec, 7, 2)
