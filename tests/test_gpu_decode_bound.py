"""The rotary decode step against 64 bits, element by element, within the bound
that its fp16 operands leave.

With p_t = exp(s_t - max s) and L = sum p_t, the step takes
  w_t = RN16(p_t)            |w_t - p_t| <= 2^-11 p_t + 2^-25
  f_t = RN16(w_t d_t)        |f_t - w_t d_t| <= 2^-11 w_t |d_t| + 2^-25
(d_t: the value block's scale; a weight or a product below 2^-14 is a multiple
of 2^-24) into sum_t f_t c_t, c the code (a 4-bit level less its offset of 8).
An f16 value takes w_t alone, a turbo4 row RN16(p_t d_t).  Weights are taken
relative to a running maximum and scaled by factors of at most 1 afterwards,
which leaves the absolute parts below 2^-25.  So before the last rounding (2^-11
of the output, 2^-25 below 2^-14)
  |o_j - exact| <= (2^-11 sum p (|v_j| + |d c_j| (1 + 2^-11))
                    + 2^-25 sum (|v_j| (1 + 2^-11) + |c_j|)) / L
(f16: c = 0; turbo4: 2^-11 sum p |v_j| + 2^-25 sum |c_j|)
and the fp32 parts: a score's 128 products, exact, are added with a relative
error of 2^-23 each at most, so p_t is off by e = 128 * 2^-23 max_t scale
sum_i |q_i k_ti| and 2^-20 for its exponential and the products with scales; the
sums over n tokens, of 4-bit values those of levels and offsets (at most 16 |d|
beside a value), by 2^-23 a step, n / 16 + 64 steps.  For turbo4 values the bound
holds in the rotated space, from which (1/16) sum_i and eight fp32 additions lead
back; for turbo4 keys the query is rotated by eight fp32 additions, held as two
fp16 numbers (2^-22) and multiplied in 256 products.
"""
import numpy as np
import pytest
import torch

import attention_quantized_kv_gb300 as kvq

import oracle
from tests import _encoders as E
from tests import _rope as R
from tests.test_gpu_rope import SCALE, _images, _random_layer

pytestmark = pytest.mark.gpu

F16, Q8, Q4, T4 = 0, 1, 2, 3


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_quantized_kv_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _parts(codec, raw):
    """(v, d, c) of canonical rows [n, bytes], in the space the codec is summed in."""
    n = len(raw)
    if codec == F16:
        v = raw.view(np.float16).astype(np.float64)
        return v, np.zeros_like(v), np.zeros_like(v)
    blocks = raw[:, None] if codec == T4 else raw.reshape(n, 4, -1)
    d = np.ascontiguousarray(blocks[..., :2]).view(np.float16).astype(np.float64)
    d = np.repeat(d.reshape(n, -1), 128 if codec == T4 else 32, axis=1)
    if codec == Q8:
        c = blocks[..., 2:].view(np.int8).astype(np.float64).reshape(n, 128)
    else:
        b = raw[:, 2:].reshape(n, 4, 16) if codec == T4 else blocks[..., 2:]
        c = np.concatenate([b & 15, b >> 4], axis=-1).reshape(n, 128).astype(np.float64) - 8
    return d * c, np.abs(d), np.abs(c)


def _hadamard():
    i = np.arange(128)
    bits = np.array([[bin(a & b).count("1") for b in i] for a in i])
    return 1.0 - 2.0 * (bits % 2)


@pytest.mark.parametrize("ck,cv", [(F16, F16), (F16, Q8), (F16, Q4), (F16, T4), (Q8, Q8), (Q4, Q4), (T4, T4),
                                   (Q4, T4), (T4, Q8)])
@pytest.mark.parametrize("n_seqs,gain", [(2, 1.0), (9, 1.0), (2, 6.0)])
def test_error_of_a_step(ck, cv, n_seqs, gain):
    """Even weights and (gain 6) weights of many magnitudes, most of them subnormal in fp16."""
    n_kv, n_q, cap = 2, 4, 1536
    lens = [1500, 40, 333, 16, 0, 1, 700, 255, 256][:n_seqs]
    L, table = _random_layer(n_seqs, n_kv, n_q, cap, ck, cv, True, lens, 90 + ck + 4 * cv)
    rope = kvq.Rope(n_pos=cap)
    g = torch.Generator(device="cuda").manual_seed(5)
    q = (gain * torch.randn((n_seqs, n_q, 128), generator=g, device="cuda")).half()
    k, v = (torch.randn((n_seqs, n_kv, 128), generator=g, device="cuda").half() for _ in "kv")
    at = L.seq_lens.clone()
    qr = torch.empty_like(q)
    kvq.kvq_rope_apply(rope, q, qr, at)
    out = torch.empty_like(q)
    ws = torch.zeros(kvq.attn_decode_workspace(L, cap), dtype=torch.uint8, device="cuda")
    kvq.attn_decode_append_rope(L, rope, k, v, q, SCALE, out, None, cap, ws)
    got, qr = out.double().cpu().numpy(), qr.double().cpu().numpy()
    images = _images(L, table)
    h = _hadamard()
    signs = oracle.turbo_signs().astype(np.float64)
    worst = 0.0
    for s, n in enumerate(lens):
        for kv in range(n_kv):
            rows = [np.stack([im.get(s, kv, t) for t in range(n + 1)]) for im in images]
            kx = E.decode(ck, rows[0]).astype(np.float64)
            val, d, c = _parts(cv, rows[1])
            size, twice = np.abs(val), (d * c if cv in (Q8, Q4) else np.zeros_like(c))
            for j in range(kv * n_q // n_kv, (kv + 1) * n_q // n_kv):
                a = kx @ qr[s, j] * SCALE
                p = np.exp(a - a.max())[:, None]
                L1 = p.sum()
                ref = (p * val).sum(0) / L1
                fp16 = 2.0 ** -11 * (p * (size + twice * (1 + 2.0 ** -11))).sum(0) + \
                    2.0 ** -25 * ((0 if cv == T4 else size * (1 + 2.0 ** -11)) + c).sum(0)
                e = 128 * 2.0 ** -23 * (np.abs(kx) @ np.abs(qr[s, j])).max() * SCALE + 2.0 ** -20
                if ck == T4:
                    y, rq = np.abs(_parts(T4, rows[0])[0]), np.abs(h @ (signs * qr[s, j])) / 16
                    e = SCALE * ((256 * 2.0 ** -23 + 2.0 ** -22) * (y @ rq).max() +
                                 8 * 2.0 ** -24 * np.abs(qr[s, j]).sum() / 16 * y.sum(1).max()) + 2.0 ** -20
                fp32 = 2 * e * (p * size).sum(0) + \
                    2 * (n / 16 + 64) * 2.0 ** -23 * (p * (size + 16 * d * (cv in (Q4, T4)))).sum(0)
                bound = (fp16 + fp32) / L1
                if cv == T4:
                    bound = np.full(128, (bound + 8 * 2.0 ** -24 * np.abs(ref)).sum() / 16)
                    ref = (ref @ h) / 16 * signs
                bound = bound * (1 + 2.0 ** -11) + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25
                err = np.abs(got[s, j] - ref)
                assert (err <= bound).all(), (s, j, (err / bound).max())
                worst = max(worst, (err / bound).max())
    assert worst > 1e-3                                       # (a bound that says something)
