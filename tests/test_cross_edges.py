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
