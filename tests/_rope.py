"""Plain references of the rotary operators, in numpy: angles in extended
precision, the rotation in fp32 with one rounding per operation (the library's
bits) and in fp64, and rows placed into a cache byte by byte."""
import ctypes
import math

import numpy as np

import oracle

INTERLEAVED, HALF = 0, 1


def freqs64(rot, base=10000.0):
    return [base ** (-2.0 * i / rot) for i in range(rot // 2)]


def angles64(freqs, pos):
    """(cos, sin) [len(pos), len(freqs)] of pos * freq, the product exact: the
    frequency is split into two parts of at most 27 bits, so both products
    with a position below 2^25 are exact in fp64."""
    f = np.asarray(freqs, np.float64)
    c = f * 134217729.0  # 2^27 + 1
    hi = c - (c - f)
    lo = f - hi
    p = np.asarray(pos, np.float64)[:, None]
    a, b = p * hi, p * lo
    return (np.cos(a) * np.cos(b) - np.sin(a) * np.sin(b),
            np.sin(a) * np.cos(b) + np.cos(a) * np.sin(b))


def table32(freqs, n_pos):
    c, s = angles64(freqs, np.arange(n_pos))
    return np.stack([c, s], axis=-1).astype(np.float32)


def planes(rot, layout):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if layout == INTERLEAVED else (i, i + rot // 2)


def rotate(x, cs, rot, layout, magnitude=1.0, transpose=False, sign=None):
    """x [n, heads, 128] by cs [n, rot / 2, 2] in x's precision (fp32: one
    rounding per operation, numpy contracts nothing)."""
    t = x.dtype.type
    c = cs[..., 0].astype(t) * t(magnitude)
    s = cs[..., 1].astype(t) * t(magnitude)
    if transpose:
        s = -s
    if sign is not None:
        s = s * np.asarray(sign, t)[:, None]
    c, s = c[:, None], s[:, None]
    ia, ib = planes(rot, layout)
    y = x.copy()
    with np.errstate(invalid="ignore", over="ignore"):
        y[..., ia] = x[..., ia] * c - x[..., ib] * s
        y[..., ib] = x[..., ia] * s + x[..., ib] * c
    return y


def encode_f32(codec, x):
    """fp32 [n, 128] -> canonical bytes, by the oracle's fp32 block encoders."""
    x = np.ascontiguousarray(x, np.float32).reshape(-1, 128)
    rb = oracle.ROW_BYTES[codec]
    if codec == oracle.F16:
        with np.errstate(over="ignore"):
            return x.astype(np.float16).view(np.uint8).reshape(-1, 256)
    lib = oracle._load()
    fn, step, nb = {oracle.Q8_0: (lib.kvqo_q8_0_encode_block_f32, 32, 34),
                    oracle.Q4_0: (lib.kvqo_q4_0_encode_block_f32, 32, 18),
                    oracle.TURBO4: (lib.kvqo_turbo4_encode_row_f32, 128, 66)}[codec]
    fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    out = np.zeros((x.shape[0], rb), np.uint8)
    for r in range(x.shape[0]):
        for b in range(128 // step):
            rc = fn(x.ctypes.data + (r * 128 + b * step) * 4, out.ctypes.data + r * rb + b * nb)
            assert rc == 0
    return out


class Cache:
    """A side's bytes with rows addressed by (sequence, kv head, token)."""

    def __init__(self, codec, side, data, n_kv, capacity, table=None):
        self.codec, self.data, self.n_kv, self.capacity, self.table = codec, data, n_kv, capacity, table
        self.off = oracle.unit_offset_table(codec, side)
        self.unit_bytes = 16 * oracle.ROW_BYTES[codec]

    def where(self, s, h, t):
        if self.table is None:
            unit = (s * self.n_kv + h) * (self.capacity // 16) + t // 16
        else:
            unit = (int(self.table[s, t // 256]) * self.n_kv + h) * 16 + (t // 16) % 16
        return unit * self.unit_bytes + self.off[t % 16]

    def put(self, s, h, t, row):
        self.data[self.where(s, h, t)] = row

    def get(self, s, h, t):
        return self.data[self.where(s, h, t)]


def half_eps(dtype):
    return {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8, "float32": 2.0 ** -24}[dtype]


def default_scale():
    return 1.0 / math.sqrt(128.0)
