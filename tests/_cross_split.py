"""How far attn_cross, and a prefix's part of attn_decode_prefix, may be off when their operands are
what the header says: a quantized side as two fp16 numbers that add up to it, a turbo4 query as two
parts, fp16 keys and values as they are.  (tests/_cross.py allows for one rounding of each.)

Scores, and with them the log-sum-exp.  Nothing of K is rounded.  A score is summed in fp32, 16
products at a time, each step cut at 2^-23 of the sum of sizes: 8 steps over f16, 16 over pairs, 24
over turbo4's pairs and query parts: e = steps 2^-23 scale max_t sum_i |q_i k_ti|.  turbo4's
rotated query r comes out of seven stages of fp32 sums (7 2^-24 sum |q| / 16 each) and is held to
2^-22 of itself, 2^-25 at least.  The exponent is rounded against the maximum (2^-22 of it), ex2 off
by 2^-22; the sum of T weights takes T / 32 + 20 roundings of 2^-24, its logarithm and the product
with ln 2 2^-22 of the result.

Values, for a query of zeros, whose weights are all 64 and exact in fp16: what is left is the fp32
sums, 2 ceil(T / 16) + 1 steps of 2^-23 of sum |v| / T, a quotient and a factor (2^-22), and the
output's own rounding.  turbo4 values: the same of its rotated values y, each of which reaches every
output by 1/16, and seven stages of 2^-24.
"""
import numpy as np
import torch

F16, Q8, Q4, T4 = 0, 1, 2, 3


def hadamard(device="cpu"):
    i = np.arange(128)
    bits = np.array([[bin(a & b).count("1") for b in i] for a in i])
    return torch.from_numpy(1.0 - 2.0 * (bits % 2)).to(device)


def signs(device="cpu"):
    import oracle
    return torch.from_numpy(oracle.turbo_signs().astype(np.float64)).to(device)


def rotated(x):
    return (x * signs(x.device)) @ hadamard(x.device)


def by_head(q, n_kv):
    """[n, n_q, w] -> [n_kv, n * group, w]."""
    n = q.shape[0]
    return q.reshape(n, n_kv, -1, q.shape[-1]).transpose(0, 1).reshape(n_kv, -1, q.shape[-1])


def scores(q, k, codec, scale):
    """q fp64 [n, n_q, 128], k fp64 [n_kv, T, 128]: scores [n_kv, n * group, T] and how far one may
    be off [n_kv, n * group, 1]."""
    qh = by_head(q, k.shape[0])
    a = qh @ k.transpose(1, 2) * scale
    x, y = (rotated(qh) / 16, rotated(k) / 8) if codec == T4 else (qh, k)
    steps = {F16: 8, T4: 24}.get(codec, 16)
    e = steps * 2.0 ** -23 * scale * (x.abs() @ y.abs().transpose(1, 2)).amax(-1, keepdim=True)
    if codec == T4:
        held = 2.0 ** -22 * x.abs() + 2.0 ** -25 + 7 * 2.0 ** -24 * qh.abs().sum(-1, keepdim=True) / 16
        e = e + scale * (held @ y.abs().transpose(1, 2)).amax(-1, keepdim=True)
    return a, e + 2.0 ** -22 * a.abs().amax(-1, keepdim=True)


def lse_of(q, parts, scale):
    """q over parts [(codec of K, k)]: the log-sum-exp [n, n_q] and its tolerance."""
    got = [scores(q, k, c, scale) for c, k in parts]
    a = torch.cat([x for x, _ in got], -1)
    e = torch.stack([x for _, x in got]).amax(0)[..., 0]
    total = torch.logsumexp(a, -1)
    tol = e + 2.0 ** -22 + (a.shape[-1] / 32 + 20) * 2.0 ** -24 + 2.0 ** -22 * total.abs()
    n = q.shape[0]
    back = lambda x: x.reshape(x.shape[0], n, -1).transpose(0, 1).reshape(n, -1)
    return back(total), back(tol)


def mean_of(v, codec, eps):
    """Values fp64 [n_kv, T, 128]: their mean [n_kv, 128] and how far an output may be from it, eps half
    a step of its type."""
    T = v.shape[1]
    steps = 2 * -(-T // 16) + 1
    mean = v.mean(1)
    if codec == T4:
        y = rotated(v) / 8
        off = (steps * 2.0 ** -23 + 2.0 ** -22) * y.abs().mean(1).sum(-1, keepdim=True) / 16 + \
            7 * 2.0 ** -24 * y.mean(1).abs().sum(-1, keepdim=True) / 16
    else:
        off = (steps * 2.0 ** -23 + 2.0 ** -22) * v.abs().mean(1)
    return mean, off * (1 + eps) + eps * mean.abs() + 2.0 ** -25


def near_opposites(n, heads, rng):
    """fp32 rows [n, heads, 128] in pairs (x, -1.004 x), the last alone for an odd n: their mean is
    small, so that an output shows what is left out of the values."""
    x = rng.standard_normal(((n + 1) // 2, heads, 128))
    return np.stack([x, -1.004 * x], 1).reshape(-1, heads, 128)[:n].astype(np.float32)
