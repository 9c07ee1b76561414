"""What evict hands over to another stream than the current one: every tensor
that the work there reads or writes, the rope's table among them."""
import types

import pytest
import torch

import attention_quantized_kv_gb300 as kvq

from tests.test_gpu_rope import F16, Q8, _random_layer, _twin


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_quantized_kv_gb300 import build
    build.build()


class _Tensors(list):
    def has(self, t):
        return any(x is t for x in self)


@pytest.mark.parametrize("with_rope", [False, True])
@pytest.mark.parametrize("paged", [False, True])
def test_everything_is_handed_over(monkeypatch, with_rope, paged):
    """On the CPU: the kernels' arguments against what was handed over before the first call."""
    L = kvq.KVLayer(2, 1, 2, 512, kvq.KVQ_F16, kvq.KVQ_Q8_0, device="cpu", n_pages=4 if paged else 0)
    L.err = L.err if paged else None                          # (the word is optional)
    rope = types.SimpleNamespace(table=torch.zeros((512, 64, 2)), n_pos=512, _check_on=lambda d: None)
    scores = torch.zeros((2, 512))
    handed, used = _Tensors(), _Tensors()
    monkeypatch.setattr(kvq, "_hand_over", lambda stream, *t: handed.extend(t))

    def call(layer, *args, **kw):
        used.extend(x for x in (layer.k_cache, layer.v_cache, layer.seq_lens, layer.err, layer.block_table, *args)
                    if isinstance(x, torch.Tensor))
        used.extend(x.table for x in args if x is rope)

    for name in ("kv_evict_select", "kv_compact", "kv_evict_delta", "kv_rope_shift"):
        monkeypatch.setattr(kvq, name, call)
    kvq.evict(L, scores, 4, 4, 8, stream=object(), rope=rope if with_rope else None)
    assert used.has(L.k_cache) and used.has(scores) and used.has(rope.table) == with_rope
    assert all(handed.has(t) for t in used)


@pytest.mark.gpu
@pytest.mark.parametrize("paged", [False, True])
def test_a_rope_and_a_layer_that_go_away(paged):
    """A rope built on the current stream and a layer, both dropped while the other stream is still
    busy, their sizes allocated and filled again: the results of the same calls made in order."""
    side = torch.cuda.Stream()
    base, table = _random_layer(2, 2, 4, 1024, Q8, F16, paged, [900, 640], 23)
    L, M = _twin(base, table), _twin(base, table)
    for X in (L, M):
        X.block_table = None if base.block_table is None else base.block_table.clone()
    scores = torch.rand((2, 1024), device="cuda")
    kvq.Rope(n_pos=1024, rot_dim=96)                          # (its memory goes back to the pool)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = kvq.evict(L, scores, 4, 32, 200, stream=side, rope=kvq.Rope(n_pos=1024, rot_dim=96))
    k, v, lens = L.k_cache, L.v_cache, L.seq_lens
    del L
    junk = [torch.full((n,), 77, dtype=t, device="cuda")
            for n, t in ((1024 * 96, torch.float32), (8, torch.int32), (1, torch.int32)) for _ in range(4)]
    torch.cuda.synchronize()
    assert all((t == 77).all() for t in junk)
    want = kvq.evict(M, scores, 4, 32, 200, rope=kvq.Rope(n_pos=1024, rot_dim=96))
    assert M.err.item() == 0
    for a, b in zip((*got, k, v, lens), (*want, M.k_cache, M.v_cache, M.seq_lens)):
        assert torch.equal(a, b)
