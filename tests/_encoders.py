"""The row encoders of include/kvq.h in numpy, non-finite values included, and
rows that reach their rare branches."""
import numpy as np

import oracle
from tests._helpers import boundary_rows

F32 = np.float32


def _half(d):
    with np.errstate(over="ignore"):
        return np.ascontiguousarray(d.astype(np.float16)).view(np.uint8).reshape(*d.shape, 2)


def _signed_max(x):
    """The value of largest magnitude along the last axis, the first on ties, NaN left out (0 where
    there is nothing else)."""
    a = np.where(np.isnan(x), F32(-1), np.abs(x))
    j = np.argmax(a, axis=-1)[..., None]
    return np.where(np.take_along_axis(a, j, -1) < 0, F32(0), np.take_along_axis(x, j, -1))


def _levels(x, d):
    with np.errstate(all="ignore"):
        t = np.where(d == 0, F32(0), (x / d).astype(F32))
        u = (t + F32(8.5)).astype(F32)
        q = np.where(np.isnan(u), F32(8), np.minimum(np.trunc(u), F32(15)))
    return q.astype(np.int64) & 15


def fwht(x):
    """Sylvester order, one fp32 addition or subtraction per output and stage."""
    y = x.astype(F32)
    h = 1
    with np.errstate(all="ignore"):
        while h < 128:
            v = y.reshape(-1, 64 // h, 2, h)
            y = np.stack([v[:, :, 0] + v[:, :, 1], v[:, :, 0] - v[:, :, 1]], axis=2).reshape(-1, 128)
            h *= 2
    return y


def encode(codec, x):
    """fp32 [n, 128] -> canonical bytes [n, row bytes]."""
    x = np.ascontiguousarray(x, F32).reshape(-1, 128)
    n = len(x)
    if codec == oracle.F16:
        with np.errstate(over="ignore"):
            return x.astype(np.float16).view(np.uint8).reshape(n, 256)
    if codec == oracle.Q8_0:
        x = x.reshape(n, 4, 32)
        with np.errstate(all="ignore"):
            d = (np.fmax.reduce(np.abs(x), axis=-1, initial=F32(0))[..., None] / F32(127)).astype(F32)
            t = np.where(d == 0, F32(0), (x / d).astype(F32)).astype(np.float64)
            q = np.where(np.isnan(t), 0.0, np.copysign(np.floor(np.abs(t) + 0.5), t))
        b = np.concatenate([_half(d[..., 0]), (q.astype(np.int64) & 255).astype(np.uint8)], axis=-1)
        return b.reshape(n, 136)
    if codec == oracle.Q4_0:
        x = x.reshape(n, 4, 32)
        d = (_signed_max(x) / F32(-8)).astype(F32)
        q = _levels(x, d)
        b = np.concatenate([_half(d[..., 0]), (q[..., :16] | (q[..., 16:] << 4)).astype(np.uint8)], axis=-1)
        return b.reshape(n, 72)
    with np.errstate(all="ignore"):
        y = (fwht(x * oracle.turbo_signs().astype(F32)) * F32(0.125)).astype(F32)
        d = (_signed_max(y) / F32(-8)).astype(F32)
    q = _levels(y, d).reshape(n, 4, 32)
    return np.concatenate([_half(d[:, 0]), (q[..., :16] | (q[..., 16:] << 4)).astype(np.uint8).reshape(n, 64)],
                          axis=-1)


def decode(codec, b):
    """Canonical bytes -> fp32 values, scales that are infinities included."""
    b = np.ascontiguousarray(b).reshape(len(b), -1)
    n = len(b)
    with np.errstate(all="ignore"):
        if codec == oracle.F16:
            return b.view(np.float16).astype(F32)
        if codec == oracle.Q8_0:
            b = b.reshape(n, 4, 34)
            d = np.ascontiguousarray(b[..., :2]).view(np.float16).astype(F32)
            return (d * b[..., 2:].view(np.int8).astype(F32)).reshape(n, 128)
        if codec == oracle.Q4_0:
            b = b.reshape(n, 4, 18)
            d = np.ascontiguousarray(b[..., :2]).view(np.float16).astype(F32)
            q = np.concatenate([b[..., 2:] & 15, b[..., 2:] >> 4], axis=-1).astype(F32) - F32(8)
            return (d * q).reshape(n, 128)
        d = np.ascontiguousarray(b[:, :2]).view(np.float16).astype(F32)
        b = b[:, 2:].reshape(n, 4, 16)
        q = np.concatenate([b & 15, b >> 4], axis=-1).astype(F32).reshape(n, 128) - F32(8)
        return (fwht(d * q) * F32(0.0625)) * oracle.turbo_signs().astype(F32)


LIMITS = {"float16": (2.0 ** -24, 65504.0), "bfloat16": (2.0 ** -133, 3.3e38), "float32": (2.0 ** -149, 3.3e38)}


def as_type(x, dtype):
    """fp32 values rounded to the type, as fp32 (bf16: to nearest even by its bits)."""
    x = np.asarray(x, F32)
    if dtype == "float16":
        with np.errstate(over="ignore"):
            return x.astype(np.float16).astype(F32)
    if dtype == "bfloat16":
        u = x.view(np.uint32).astype(np.uint64)
        r = ((u + 0x7fff + ((u >> 16) & 1)) & 0xffff0000).astype(np.uint32).view(F32)
        return np.where(np.isfinite(x), r, x)
    return x


def special_rows(dtype, seed=5):
    """(finite, other): fp32 rows [n, 128] of values of the type; other: with infinities and NaN,
    or sums that reach them."""
    rng = np.random.default_rng(seed)
    tiny, top = LIMITS[dtype]
    z = rng.standard_normal
    rows = [np.zeros(128), -np.zeros(128), np.where(np.arange(128) % 3, 0.0, -0.0)]
    r = z(128)
    r[32:64] = 0                                    # one zero block, one of negative zeros
    r[96:] = -0.0
    rows.append(r)
    # the largest magnitude with both signs, the first of them positive or negative, in the same
    # and in different 16-byte pieces of a row; every value a tie
    for i, j in ((5, 20), (20, 5), (0, 31), (31, 0), (3, 4), (16, 1), (17, 2)):
        for sign in (1.0, -1.0):
            r = np.clip(z(128), -2.5, 2.5)
            r[i::32] = 3.0 * sign
            r[j::32] = -3.0 * sign
            rows.append(r)
    rows += [np.resize([1.5, -1.5], 128), np.resize([-1.5, 1.5], 128), np.full(128, -0.75), np.full(128, 2.0)]
    r = np.zeros(128)
    r[77] = -4.0                                    # one value in a row (turbo4: 128 ties)
    rows.append(r)
    for codec in (1, 2):
        rows += list(boundary_rows(codec, 6, rng).astype(np.float64))
    # towards and past the smallest scales: 1 / d is infinite below 2^-128
    for e in (1e-30, 4e-37, 3e-38, 1e-38, 2.5e-39, 1e-40, 3e-42, 2e-44):
        rows.append(z(128) * e)
    r = np.zeros(128)                               # 127 : 63.5 and the like by the exact division only
    r[:3], r[40] = (1e-37, -5e-38, 3e-38), 2e-38
    rows.append(r)
    for k in (1, 2, 3, 5, 11, 190, 200, 1000):      # a few steps of the type
        rows.append(np.clip(np.round(z(128) * k / 2), -k, k) * tiny)
        r = np.resize([-1.0, 1.0, 0.0, 0.5], 128) * tiny * k
        rows.append(r)
    for big in (6e4, 8.3e6, 1e7, 1e30):             # fp16 scales that overflow
        rows.append(np.clip(z(128), -1, 1) * min(big, top))
    finite = as_type(np.stack(rows), dtype)
    other = [np.clip(z(128), -1, 1) * min(3.2e38, top)]  # sums that overflow
    for v in (np.nan, -np.nan, np.inf, -np.inf):
        for at in ((0,), (1,), (3, 4), (17,), (31,), (16, 33, 127), tuple(range(0, 128, 4)), (66, 67),
                   tuple(range(32, 64)), tuple(range(128))):
            r = z(128)
            r[list(at)] = v
            other.append(r)
    r = z(128)
    r[9], r[10] = np.inf, -np.inf
    other.append(r)
    r = z(128)
    r[9], r[10], r[60] = np.inf, np.nan, -np.inf
    other.append(r)
    r = z(128) * tiny
    r[5] = np.nan
    other.append(r)
    r = np.zeros(128)
    r[::32] = np.nan
    other.append(r)
    other = as_type(np.stack(other), dtype)
    # NaN of every payload: quiet with all bits set, quiet without any, negative
    bits = other.view(np.uint32).copy()
    at = np.argwhere(np.isnan(other))
    for n, (i, j) in enumerate(at):
        bits[i, j] = (0x7fffe000, 0x7fc00000, 0xffffe000)[n % 3] if dtype == "float16" else \
            (0x7fff0000, 0x7fc00000, 0xffff0000)[n % 3] if dtype == "bfloat16" else \
            (0x7fffffff, 0x7fc00000, 0xffffffff)[n % 3]
    return finite, bits.view(F32)
