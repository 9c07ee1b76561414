"""The entry points over packed rows without a GPU: what they refuse, before any
device call."""
import ctypes

import pytest

from tests.test_abi import _layer, lib  # noqa: F401

OK, EINVAL, EUNSUPPORTED, ECAPACITY, EALIGN, EWORKSPACE = range(6)
F16, BF16, F32 = range(3)
BIG = 1 << 40


def _rows(data=0x10000000, row=8 * 128, head=128, kind=F16, **kw):
    from attention_quantized_kv_gb300._abi import kvq_rows
    return kvq_rows(data, row, head, kind, kw.get("reserved", 0))


KV = dict(row=2 * 128)  # _layer() has 2 kv heads and 8 query heads


def _cross(lib, layer=None, **kw):  # noqa: F811
    a = dict(q=_rows(), n=4, n_new=None, start=0x400000, scale=0.1, out=_rows(0x20000000), lse=None, max_len=16,
             ws=0x600000, nb=BIG)
    a.update(kw)
    return lib.attn_cross(layer if layer is not None else _layer(n_seqs=2), a["q"], a["n"], a["n_new"], a["start"],
                          a["scale"], a["out"], a["lse"], a["max_len"], a["ws"], a["nb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), EINVAL), (dict(out=None), EINVAL), (dict(max_len=0), EINVAL), (dict(scale=0.0), EINVAL),
    (dict(scale=float("nan")), EINVAL), (dict(scale=-1.0), EINVAL), (dict(scale=float("inf")), EINVAL),
    (dict(max_len=5000), ECAPACITY), (dict(n=-1), EINVAL), (dict(n=1 << 31), EINVAL),
    (dict(start=None), EINVAL),                              # neither form, and not one row each
    (dict(n_new=0x400000), EINVAL),                          # both
    (dict(n_new=0x400000, start=None, n=5), EINVAL),         # padded rows of unequal length
    (dict(start=0x400002), EALIGN), (dict(n_new=0x400001, start=None), EALIGN), (dict(lse=0x700002), EALIGN),
    (dict(q=_rows(kind=F32), out=_rows(0x20000000, kind=F32)), EUNSUPPORTED),
    (dict(out=_rows(0x20000000, kind=BF16)), EUNSUPPORTED), (dict(q=_rows(kind=7)), EUNSUPPORTED),
    (dict(q=_rows(0x10000008)), EALIGN), (dict(q=_rows(row=8 * 128 + 4)), EALIGN), (dict(q=_rows(row=-1024)), EINVAL),
    (dict(q=_rows(reserved=1)), EINVAL), (dict(q=_rows(0)), EINVAL),
    (dict(out=_rows(0x20000000, row=0)), EINVAL), (dict(out=_rows(0x20000000, head=64)), EINVAL),
    (dict(out=_rows()), EINVAL), (dict(out=_rows(0x10000000 + 3 * 2048)), EINVAL),   # q is still read
    (dict(ws=None), EWORKSPACE), (dict(ws=0x600008), EALIGN),
    (dict(n=0), OK),
])
def test_cross_refusals(lib, kw, status):  # noqa: F811
    assert _cross(lib, **kw) == status


def test_layers_are_checked(lib):  # noqa: F811
    n = ctypes.c_size_t(0)
    for kw, status in [(dict(head_dim=64), 2), (dict(codec_k=5), 2), (dict(capacity=1000), 4), (dict(n_seqs=0), 1)]:
        bad, good = _layer(**kw), _layer()
        assert _cross(lib, bad) == status
        assert lib.attn_cross_workspace(bad, 4, 16, n) == status
        assert lib.kv_append_rows(bad, _rows(**KV), _rows(**KV), 4, None, 0x400000, 1, None) == status
        assert lib.kv_read_rows(bad, _rows(**KV), None, 4, None, 0x400000, None, None) == status
        for a, b in ((bad, good), (good, bad)):
            assert lib.attn_decode_prefix_workspace(a, b, 16, 16, n) == status
            assert lib.attn_decode_prefix(a, b, None, 0x10000000, 0.1, 0x20000000, None, 16, 16, 0x600000, BIG,
                                          None) == status
    many = _layer(n_seqs=1025)
    assert _cross(lib, many, n=1025, start=None) == EINVAL
    assert lib.attn_cross_workspace(many, 4, 16, n) == EINVAL
    assert lib.attn_cross_workspace(_layer(), -1, 16, n) == EINVAL
    assert lib.attn_cross_workspace(_layer(), 4, 5000, n) == ECAPACITY
    assert lib.attn_cross_workspace(_layer(), 4, 16, None) == EINVAL


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(start=None), EINVAL), (dict(n_new=0x400000), EINVAL),
    (dict(n=-1), EINVAL), (dict(n_new=0x400000, start=None, n=3), EINVAL), (dict(v=_rows(kind=BF16, **KV)), EUNSUPPORTED),
    (dict(k=_rows(0x10000004, **KV)), EALIGN), (dict(start=0x400002), EALIGN), (dict(n=0), OK),
])
def test_append_refusals(lib, kw, status):  # noqa: F811
    a = dict(k=_rows(**KV), v=_rows(0x20000000, **KV), n=4, n_new=None, start=0x400000)
    a.update(kw)
    assert lib.kv_append_rows(_layer(n_seqs=2), a["k"], a["v"], a["n"], a["n_new"], a["start"], 1, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(k=None, v=None), EINVAL), (dict(start=None), EINVAL), (dict(n_read=0x400000), EINVAL),
    (dict(n=1 << 31), EINVAL), (dict(first=0x400002), EALIGN), (dict(k=_rows(kind=9, **KV)), EUNSUPPORTED),
    (dict(k=_rows(row=0)), EINVAL),                              # rows written to one place
    (dict(v=_rows(**KV)), EINVAL), (dict(v=_rows(0x10000000 + 256, **KV)), EINVAL),
    (dict(k=_rows(row=512), v=_rows(0x10000000 + 256, row=512)), EINVAL),   # heads of both meet
    (dict(k=_rows(row=512), v=_rows(0x10000000 + 512 * 4 + 768, row=512)), EINVAL),  # two rows on, and meeting
    (dict(n=0), OK),
])
def test_read_refusals(lib, kw, status):  # noqa: F811
    a = dict(k=_rows(**KV), v=_rows(0x20000000, **KV), n=4, n_read=None, start=0x400000, first=None)
    a.update(kw)
    assert lib.kv_read_rows(_layer(n_seqs=2), a["k"], a["v"], a["n"], a["n_read"], a["start"], a["first"],
                            None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), EINVAL), (dict(out=None), EINVAL), (dict(scale=0.0), EINVAL), (dict(scale=float("inf")), EINVAL),
    (dict(max_len=0), EINVAL), (dict(max_prefix=0), EINVAL), (dict(max_len=5000), ECAPACITY),
    (dict(max_prefix=5000), ECAPACITY), (dict(prefix=_layer(n_q_heads=4)), EINVAL),
    (dict(prefix=_layer(n_kv_heads=4)), EINVAL), (dict(prefix=_layer(n_seqs=2)), EINVAL),  # no group_start
    (dict(prefix=_layer(n_seqs=1025), groups=0x400000), EINVAL), (dict(groups=0x400002), EALIGN),
    (dict(q=0x10000008), EALIGN), (dict(out=0x20000004), EALIGN), (dict(lse=0x700002), EALIGN),
    (dict(out=0x10000000), EINVAL), (dict(ws=None), EWORKSPACE), (dict(ws=0x600008), EALIGN),
])
def test_prefix_refusals(lib, kw, status):  # noqa: F811
    a = dict(layer=_layer(n_seqs=3), prefix=_layer(), groups=None, q=0x10000000, scale=0.1, out=0x20000000, lse=None,
             max_len=16, max_prefix=16, ws=0x600000, nb=BIG)
    a.update(kw)
    assert lib.attn_decode_prefix(a["layer"], a["prefix"], a["groups"], a["q"], a["scale"], a["out"], a["lse"],
                                  a["max_len"], a["max_prefix"], a["ws"], a["nb"], None) == status
