"""Rows beside each other in one tensor: attn_cross's q and out, kv_read_rows's k and v."""
import numpy as np
import pytest
import torch

import attention_quantized_kv_gb300 as kvq

from tests import _cross as C
from tests import _rope as R
from tests.test_gpu_cross import EPS, _cross_ws, _filled, _queries, _values
from tests.test_gpu_rope import _i32

pytestmark = pytest.mark.gpu

SCALE = R.default_scale()
F16, Q8, Q4, T4 = 0, 1, 2, 3


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_quantized_kv_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


# name: (fused shape of n rows and h heads, the two parts' views [n, h, 128])
LAYOUTS = {
    "heads of both in a row": (lambda n, h: (n, 2 * h, 128), lambda t, h: (t[:, :h], t[:, h:])),
    "both in a head": (lambda n, h: (n, h, 2, 128), lambda t, h: (t[:, :, 0], t[:, :, 1])),
    "rows of both in a head": (lambda n, h: (h, 2, n, 128), lambda t, h: (t[:, 0].transpose(0, 1), t[:, 1].transpose(0, 1))),
    "both in a head's row": (lambda n, h: (h, n, 2, 128), lambda t, h: (t[:, :, 1].transpose(0, 1), t[:, :, 0].transpose(0, 1))),
}


@pytest.mark.parametrize("name", sorted(LAYOUTS))
@pytest.mark.parametrize("counts", [[3, 0, 2], [150, 40, 1]])
@pytest.mark.parametrize("kind", [torch.float16, torch.bfloat16])
def test_queries_and_results(name, counts, kind):
    lens, n_q = [700, 33, 5], 6
    shape, parts = LAYOUTS[name]
    L, table = _filled(3, 2, n_q, 768, Q8, Q8, False, lens, 71)
    n = sum(counts)
    fused = torch.full(shape(n, n_q), 9, dtype=kind, device="cuda")
    q, out = parts(fused, n_q)
    q.copy_(_queries(n, n_q, 8, kind))
    before = q.clone()
    kvq.attn_cross(L, q, SCALE, out, None, 768, _cross_ws(L, n, 768), row_start=_i32(np.cumsum([0] + counts)))
    assert L.err.item() == 0 and torch.equal(q, before)
    values, at = _values(L, table, lens), 0
    for s, m in enumerate(counts):
        if m:
            want = C.attend(before[at:at + m].half().double(), [(Q8, Q8) + values[s]], SCALE)
            C.check(out[at:at + m], None, want, EPS[kind], s)
        at += m


@pytest.mark.parametrize("name", sorted(LAYOUTS))
@pytest.mark.parametrize("counts", [[3, 0, 2], [1500, 700, 1]])
@pytest.mark.parametrize("kind", [torch.float16, torch.float32])
def test_sides(name, counts, kind):
    """Row by row and by units: what separate tensors get."""
    shape, parts = LAYOUTS[name]
    L, _ = _filled(3, 4, 4, 1536, Q8, T4, True, [1500, 700, 1] if max(counts) > 3 else [5, 0, 2], 72)
    n, start = sum(counts), _i32(np.cumsum([0] + counts))
    k, v = parts(torch.full(shape(n + 2, 4), 9, dtype=kind, device="cuda"), 4)
    kvq.kv_read_rows(L, k, v, row_start=start)
    want = [torch.full((n + 2, 4, 128), 9, dtype=kind, device="cuda") for _ in "kv"]
    kvq.kv_read_rows(L, *want, row_start=start)
    assert L.err.item() == 0
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
