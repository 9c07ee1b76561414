"""Row counts at and past what the calls over packed rows take, without a GPU."""
import ctypes

import pytest

from tests.test_abi import _layer, lib  # noqa: F401
from tests.test_cross import _cross, _rows

EINVAL = 1


@pytest.mark.parametrize("n", [-1, -2**63, (2**31 - 1) // 8 + 1, 2**31, 2**60, 2**61, 2**62, 2**63 - 1])
def test_row_counts(lib, n):  # noqa: F811
    """8 query heads: 2^60 rows and more times that wrap around 64 bits."""
    size = ctypes.c_size_t(0)
    layer, kv = _layer(n_seqs=2), dict(row=2 * 128)
    assert _cross(lib, layer, n=n) == EINVAL
    assert lib.attn_cross_workspace(layer, n, 16, size) == EINVAL
    assert lib.kv_append_rows(layer, _rows(**kv), _rows(0x20000000, **kv), n, None, 0x400000, 1, None) == EINVAL
    assert lib.kv_read_rows(layer, _rows(**kv), None, n, None, 0x400000, None, None) == EINVAL


BASE = 0x10000000


def _places(r, n, heads):
    size = 4 if r.type == 2 else 2
    return {r.data + (i * r.row_stride + h * r.head_stride) * size + b for i in range(n) for h in range(heads)
            for b in range(0, 128 * size, 16)}


def _meet(a, b, n, heads):
    return bool(_places(a, n, heads) & _places(b, n, heads))


# (k's and v's row and head strides, v's offset from k's in values): views of one tensor
VIEWS = {
    "rows of k and v heads": (4 * 128, 128, 2 * 128),                 # [rows][2][heads][128]
    "heads of k and v": (2 * 2 * 128, 2 * 128, 128),                  # [rows][heads][2][128]
    "heads of k and v, v first": (2 * 2 * 128, 2 * 128, -128),
    "by head": (128, 2 * 4 * 128, 4 * 128),                           # [heads][2][rows][128]
    "by head, beside each other": (2 * 128, 4 * 2 * 128, 128),        # [heads][rows][2][128]
    "three parts": (3 * 2 * 128, 3 * 128, 2 * 128),
    "behind one another": (4 * 128, 128, 4 * 4 * 128),
}


@pytest.mark.parametrize("name", sorted(VIEWS))
@pytest.mark.parametrize("kind", [0, 1, 2])
def test_views_of_one_tensor(lib, name, kind):  # noqa: F811
    """Two kv heads, four rows of two sequences: sides that share no place are taken (here, without a
    GPU, as far as the device)."""
    row, head, at = VIEWS[name]
    size = 4 if kind == 2 else 2
    k, v = _rows(BASE, row, head, kind), _rows(BASE + at * size, row, head, kind)
    assert not _meet(k, v, 4, 2)
    layer = _layer(n_seqs=2)
    assert lib.kv_read_rows(layer, k, v, 4, None, 0x400000, None, None) != EINVAL
    if kind < 2:  # attn_cross: as many heads of queries
        same = _layer(n_seqs=2, n_q_heads=2)
        assert _cross(lib, same, q=k, out=v) != EINVAL


def test_views_that_meet(lib):  # noqa: F811
    """Every small layout of two sets of rows: refused where they share a place (and where the sides'
    strides differ), and no layout of the views above is."""
    layer, taken = _layer(n_seqs=2), 0
    for row in (128, 256, 384, 512, 1024):
        for head in (128, 256, 384, 512, 1024):
            for at in range(-2048, 2049, 64):
                k, v = _rows(BASE, row, head), _rows(BASE + 2 * at, row, head)
                status = lib.kv_read_rows(layer, k, v, 4, None, 0x400000, None, None)
                if _meet(k, v, 4, 2):
                    assert status == EINVAL, (row, head, at)
                taken += status != EINVAL
                other = _rows(BASE + 2 * at, row + 128, head)
                if _meet(k, other, 4, 2):
                    assert lib.kv_read_rows(layer, k, other, 4, None, 0x400000, None, None) == EINVAL
    assert taken > 100
