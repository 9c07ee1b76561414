"""The numpy encoders of the GPU tests against the oracle's, on rows that reach
the rare branches, and the rule by which the kernels accept their
division-free codes."""
import numpy as np
import pytest

import oracle
from tests import _encoders as E
from tests import _rope as R

F32 = np.float32
MAGIC = F32(12582912.0)  # 1.5 * 2^23


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("codec", range(4))
def test_finite_rows_are_the_oracles(codec, dtype):
    finite, _ = E.special_rows(dtype)
    assert len(finite) > 50
    assert (E.encode(codec, finite) == R.encode_f32(codec, finite)).all()
    if codec != 3:
        ok = np.isfinite(E.decode(codec, E.encode(codec, finite))).all(axis=1)
        assert (E.decode(codec, E.encode(codec, finite))[ok] ==
                oracle.decode_rows(codec, E.encode(codec, finite))[ok]).all()


@pytest.mark.parametrize("codec", [1, 2, 3])
def test_non_finite_rows(codec):
    """A NaN reads back as 0 and moves no other value of its block (turbo4: of its row, which is
    stored as zeros); an infinity makes its block (row) NaN."""
    x = np.random.default_rng(3).standard_normal((1, 128)).astype(F32)
    clean = x.copy()
    x[0, 17] = np.nan
    clean[0, 17] = 0
    got = E.decode(codec, E.encode(codec, x))[0]
    if codec == 3:
        assert (got == 0).all()
    else:
        assert (got == E.decode(codec, E.encode(codec, clean))[0]).all() and got[17] == 0
    x[0, 17] = -np.inf
    got = E.decode(codec, E.encode(codec, x))[0]
    assert np.isnan(got[:32]).all()
    assert np.isnan(got[32:]).all() if codec == 3 else np.isfinite(got[32:]).all()


def _accepted(codec, x, d):
    """The division-free codes and whether the kernels accept a group of eight of them: the
    distances' maxima (minima) over the group, NaN among them."""
    with np.errstate(all="ignore"):
        t = (x * (F32(1) / d).astype(F32)).astype(F32)
        if codec == 1:
            tm = (t + MAGIC).astype(F32)
            fr = (t - (tm - MAGIC).astype(F32)).astype(F32)
            ok = np.abs(fr).max(axis=-1) < F32(0.5) - F32(2.0 ** -14)
            return (tm.view(np.int32) & 255).astype(np.int64), ok
        u = (t + F32(8.5)).astype(F32)
        fm = ((u - F32(0.5)).astype(F32) + MAGIC).astype(F32)
        fr = (u - (fm - MAGIC).astype(F32)).astype(F32)
        ok = (fr.min(axis=-1) > F32(2.0 ** -17)) & (fr.max(axis=-1) < F32(1) - F32(2.0 ** -17))
        return np.minimum((fm.view(np.int32) & 255).astype(np.int64), 15), ok


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("codec", [1, 2])
def test_what_is_accepted_without_a_division_is_exact(codec, dtype):
    """With maxima that keep NaN (numpy's) no group with an infinite 1 / d, an infinity or a NaN is
    accepted with other codes than the definition's."""
    rows = np.concatenate(E.special_rows(dtype))
    by = E.encode(codec, rows).reshape(len(rows), 4, -1)
    x = rows.reshape(-1, 4, 32)
    if codec == 1:
        want = by[:, :, 2:].astype(np.int64)
        d = (np.fmax.reduce(np.abs(x), axis=-1, initial=F32(0))[..., None] / F32(127)).astype(F32)
    else:
        want = np.concatenate([by[:, :, 2:] & 15, by[:, :, 2:] >> 4], axis=-1).astype(np.int64)
        d = (E._signed_max(x) / F32(-8)).astype(F32)
    some = refused = 0
    for g in range(4):
        got, ok = _accepted(codec, x[..., 8 * g:8 * g + 8], d)
        ok &= d[..., 0] != 0
        assert (got[ok] == want[..., 8 * g:8 * g + 8][ok]).all()
        some += ok.sum()
        refused += (~np.isfinite(x[..., 8 * g:8 * g + 8]).all(axis=-1) & ok).sum()
    assert some > 100 and refused == 0
