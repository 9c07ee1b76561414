"""Device conditions of the rotary decode step: the error bits are those of the
two calls that it stands for, whatever the number of sequences."""
import numpy as np
import pytest
import torch

import attention_quantized_kv_gb300 as kvq

from tests import _rope as R
from tests.test_gpu_rope import SCALE, _i32, _random_layer, _rope, _twin

pytestmark = pytest.mark.gpu

F16, Q8 = 0, 1


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_quantized_kv_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("n_seqs", [1, 3, 7, 8, 9])
@pytest.mark.parametrize("positions", [None, "inside", "outside"])
@pytest.mark.parametrize("odd", [-1, -300, 512])
def test_error_bits_of_a_step(n_seqs, positions, odd):
    """A sequence of negative length (no token, no keys) or one at its capacity, by its own length
    and by the caller's positions."""
    n_kv, n_q, cap = 2, 8, 512
    lens = [(s * 61) % 500 for s in range(n_seqs)]
    L, table = _random_layer(n_seqs, n_kv, n_q, cap, F16, Q8, False, lens, 13)
    L.seq_lens[n_seqs - 1] = odd
    M = _twin(L, table)
    rope, _ = _rope(128, R.HALF, cap)
    pos = None
    if positions:
        pos = _i32(np.arange(n_seqs) + 5)
        if positions == "outside":
            pos[n_seqs - 1] = 512
    g = torch.Generator(device="cuda").manual_seed(n_seqs)
    q, k, v = (torch.randn((n_seqs, h, 128), generator=g, device="cuda").half() for h in (n_q, n_kv, n_kv))
    ws = torch.zeros(kvq.attn_decode_workspace(L, cap), dtype=torch.uint8, device="cuda")
    out, ref, qr = (torch.full_like(q, 9) for _ in range(3))
    lse, ref_lse = (torch.full((n_seqs, n_q), 9.0, device="cuda") for _ in range(2))
    kvq.attn_decode_append_rope(L, rope, k, v, q, SCALE, out, lse, cap, ws, positions=pos)
    kvq.kv_append_rope(M, rope, k, v, row_start=_i32(range(n_seqs + 1)), q=q, q_out=qr, positions=pos)
    kvq.attn_decode(M, qr, SCALE, ref, ref_lse, cap, ws)
    want = kvq.KVQ_DEVERR_CAPACITY
    if positions == "outside" or positions is None:
        want |= kvq.KVQ_DEVERR_POS
    assert L.err.item() == M.err.item() == want
    assert L.seq_lens.tolist() == M.seq_lens.tolist() == [n + 1 for n in lens[:-1]] + [odd]
    assert torch.equal(L.k_cache, M.k_cache) and torch.equal(L.v_cache, M.v_cache)
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
