"""Attention over cached rows in 64 bits, and how far fp16 operands may leave it.

With u = 2^-11 / sqrt 3 the root mean square of an fp16 rounding's relative error
(uniform in +-2^-11 where it is largest), a kernel that takes
  K^ = RN16(k)  (f16 keys: exact; turbo4: in the rotated space, the query too)
  P  = RN16(p),  V^ = RN16(v)   (decode: RN16(RN16(p) d) c, two roundings too)
moves a score by ds_t of variance (scale u)^2 sum_i (q_i k_ti)^2, hence an output by sum_t (p_t / L) ((v_tj - o_j) ds_t + v_tj (e_t + e'_t)),
of variance sum_t (p_t / L)^2 ((v_tj - o_j)^2 var(ds_t) + 2 u^2 v_tj^2), and the
log-sum-exp by sum_t (p_t / L) ds_t.  turbo4's rotated query r is rounded once for
all keys: its errors e_i r_i add scale sum_i e_i r_i y_ti to every score, so they do
not average over t but move the log-sum-exp by scale sum_i e_i r_i m_i, m the weighted
mean of the y_t, and an output by scale sum_i e_i r_i c_ij, c the weighted covariance
of y_ti and v_tj.  Eight of these standard deviations hold for
sums of few terms (at most sqrt 3 deviations each) and of many.  Absolute parts:
values below 2^-14 are multiples of 2^-24, 2^-25 off; weights are held as 2^6 p or
more (decode: p), so 2^-25 sum |v| / L covers them.  fp32 sums of T terms: partial
sums of 256, T / 256 + 64 roundings of 2^-24, of L relative to itself (and so of the
log-sum-exp, its logarithm) and of sum p v relative to sum p |v|, both in o.
A score is summed in fp32 too, 16 products at a time, cut at 2^-23 of the largest or of
the sum so far: within e = 16 2^-23 scale max_t sum_i |q_i k_ti|, which moves the
log-sum-exp by e and an output by 2 e sum p |v| / L at most.
turbo4 values: the same in the rotated space y, x_j = sum_i +-y_i / 16.
"""
import numpy as np
import torch

import oracle
from tests import _encoders as E

F16, Q8, Q4, T4 = 0, 1, 2, 3
U = 2.0 ** -11 / 3 ** 0.5


def _hadamard():
    i = np.arange(128)
    bits = np.array([[bin(a & b).count("1") for b in i] for a in i])
    return torch.from_numpy(1.0 - 2.0 * (bits % 2)).cuda()


def rows_of(image, seq, tokens):
    """fp64 [kv heads, n, 128]: the decoded rows of a sequence's tokens (tests._rope.Cache)."""
    got = []
    for h in range(image.n_kv):
        raw = np.stack([image.get(seq, h, t) for t in tokens]) if len(tokens) else \
            np.zeros((0, oracle.ROW_BYTES[image.codec]), np.uint8)
        got.append(E.decode(image.codec, raw) if len(tokens) else np.zeros((0, 128), np.float32))
    return torch.from_numpy(np.stack(got).astype(np.float64)).cuda()


def attend(q, parts, scale):
    """q fp64 [n, n_q, 128] over parts [(codec k, codec v, k, v)], k and v fp64 [kv heads, T, 128]:
    (o, tolerance of o before its own rounding, lse, tolerance of lse)."""
    n, n_q, _ = q.shape
    n_kv = parts[0][2].shape[0]
    T = sum(p[2].shape[1] for p in parts)
    o, tol = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((n, n_q), -float("inf"), dtype=torch.float64, device="cuda")
    ltol = torch.zeros_like(lse)
    if T == 0:
        return o, tol, lse, ltol
    h = _hadamard()
    signs = torch.from_numpy(oracle.turbo_signs().astype(np.float64)).cuda()
    qh = q.reshape(n, n_kv, -1, 128).transpose(0, 1).reshape(n_kv, -1, 128)
    rot = (qh * signs) @ h / 16
    a = torch.cat([qh @ k.transpose(1, 2) for _, _, k, _ in parts], -1) * scale
    top = a.amax(-1, keepdim=True)
    p = torch.exp(a - top)
    L = p.sum(-1, keepdim=True)
    w = p / L
    v = torch.cat([p[3] for p in parts], 1)
    ref = w @ v
    sv, pv, at = 0, 0, 0
    ds = []
    for ck, cv, k, vv in parts:
        t = k.shape[1]
        if ck == F16:
            d = torch.zeros_like(a[..., at:at + t])
        elif ck == T4:
            d = (rot ** 2) @ ((((k * signs) @ h / 8) ** 2).transpose(1, 2))
        else:
            d = (qh ** 2) @ (k ** 2).transpose(1, 2)
        ds.append(d * (scale * U) ** 2)
        at += t
    ds = torch.cat(ds, -1)
    w2 = w ** 2
    # (v - o)^2 ds = v^2 ds - 2 v o ds + o^2 ds
    var = (w2 * ds) @ v ** 2 - 2 * ref * ((w2 * ds) @ v) + ref ** 2 * (w2 * ds).sum(-1, keepdim=True)
    lvar = (w2 * ds).sum(-1, keepdim=True)
    at = 0
    for ck, cv, k, vv in parts:
        if ck == T4 and k.shape[1]:
            y, part = (k * signs) @ h / 8, w[..., at:at + k.shape[1]]
            mean = part @ y
            lvar = lvar + (scale * U) ** 2 * ((rot * mean) ** 2).sum(-1, keepdim=True)
            for i in range(0, rot.shape[1], 64):  # c_ij, 64 rows at a time
                c = torch.einsum("hrt,hti,htj->hrij", part[:, i:i + 64], y, vv) - \
                    mean[:, i:i + 64, :, None] * ref[:, i:i + 64, None, :]
                var[:, i:i + 64] += (scale * U) ** 2 * ((rot[:, i:i + 64, :, None] * c) ** 2).sum(-2)
        at += k.shape[1]
    at = 0
    for ck, cv, k, vv in parts:
        part = w2[..., at:at + k.shape[1]]
        if cv == T4:
            y = (vv * signs) @ h / 8
            var = var + (2 * U ** 2 * part @ y ** 2).sum(-1, keepdim=True) / 256
        else:
            var = var + 2 * U ** 2 * part @ vv ** 2
        at += k.shape[1]
    size = w @ v.abs()
    if any(p[1] == T4 for p in parts):
        size = torch.maximum(size, (w @ v.abs()).amax(-1, keepdim=True))
    e = torch.zeros_like(L)
    for ck, cv, k, vv in parts:
        if k.shape[1]:
            x, y = (rot, (k * signs) @ h / 8) if ck == T4 else (qh, k)
            e = torch.maximum(e, 16 * 2.0 ** -23 * scale * (x.abs() @ y.abs().transpose(1, 2)).amax(-1, keepdim=True))
    bound = 2 * e * size + 8 * var.clamp(min=0).sqrt() + 2.0 ** -24 + 2.0 ** -25 * (v.abs().sum(1, keepdim=True) + 8) / L + \
        2 * (T / 256 + 64) * 2.0 ** -24 * size
    back = lambda x: x.reshape(n_kv, n, -1, x.shape[-1]).transpose(0, 1).reshape(n, n_q, -1)
    err = e + 8 * lvar.sqrt() + 2.0 ** -20 + (T / 256 + 64) * 2.0 ** -24
    total = top + torch.log(L)
    return back(ref), back(bound), back(total)[..., 0], back(err + 2.0 ** -22 * total.abs())[..., 0]


def check(got, got_lse, want, eps, where=""):
    """got [n, n_q, 128] against attend's result; eps: half a step of the output's type."""
    ref, tol, lse, ltol = want
    g = got.double()
    assert torch.isfinite(g).all(), where
    bound = tol * (1 + eps) + eps * ref.abs() + 2.0 ** -25
    bad = (g - ref).abs() > bound
    assert not bad.any(), (where, int(bad.sum()), float(((g - ref).abs() / bound).max()))
    if got_lse is not None:
        empty = torch.isinf(lse)
        assert torch.equal(torch.isinf(got_lse), empty), where
        diff = (got_lse.double() - lse).abs()[~empty]
        assert (diff <= ltol[~empty]).all(), (where, float((diff / ltol[~empty]).max()))
