"""Calls at the binding's edges: batches without a row, layers without a buffer, the current
stream."""
import pytest
import torch

import attention_quantized_kv_gb300 as kvq
from attention_quantized_kv_gb300 import _abi

from tests import test_rope as T

EINVAL = 1


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_quantized_kv_gb300 import build
    build.build()


@pytest.mark.parametrize("packed", [False, True])
def test_an_append_of_no_rows_takes_queries(packed):
    """The tensors of an empty batch have no address: q without a row goes with a q_out of NULL."""
    lib, L, r = _abi.load(), T._layer(), T._rope()
    none = T._rows(data=None, row_stride=0)
    n_new, start = (None, 0x100) if packed else (0x100, None)
    for q in (None, none):
        assert lib.kv_append_rope(L, r, q, none, none, 0, n_new, start, None, None, 1, None) == 0
    # with rows the two go together, as before
    some = T._rows(row_stride=256)
    assert lib.kv_append_rope(L, r, T._rows(), some, some, 4, n_new, start, None, None, 1, None) == EINVAL


@pytest.mark.parametrize("buffer", ["k_cache", "v_cache", "seq_lens"])
def test_a_layer_without_a_buffer_is_refused(buffer):
    L = kvq.KVLayer(1, 1, 1, 256, kvq.KVQ_F16, kvq.KVQ_F16, device="cpu")
    setattr(L, buffer, None)
    with pytest.raises(kvq.KVQError) as e:
        kvq.attn_decode_workspace(L, 256)
    assert e.value.status == EINVAL


def test_public_ways_where_torch_has_no_private_ones():
    assert kvq._private("_no_such_name", torch.cuda.current_device) is torch.cuda.current_device


@pytest.mark.gpu
def test_the_current_stream_and_device():
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(stream):
            assert kvq._stream_ptr(None) == kvq._stream_ptr(stream) == stream.cuda_stream
    assert kvq._current_device() == torch.cuda.current_device()


@pytest.mark.gpu
@pytest.mark.parametrize("packed", [False, True])
def test_empty_batches(packed):
    L = kvq.KVLayer(2, 2, 4, 256, kvq.KVQ_Q8_0, kvq.KVQ_F16)
    L.k_cache.fill_(7)
    L.seq_lens.fill_(9)
    rope = kvq.Rope(n_pos=256)
    lead = (0,) if packed else (2, 0)
    k = torch.empty((*lead, 2, 128), dtype=torch.bfloat16, device="cuda")
    q = torch.empty((*lead, 4, 128), dtype=torch.bfloat16, device="cuda")
    out = torch.empty((*lead, 4, 128), dtype=torch.float16, device="cuda")
    which = {"row_start": torch.zeros(3, dtype=torch.int32, device="cuda")} if packed else \
        {"n_new": torch.zeros(2, dtype=torch.int32, device="cuda")}
    kvq.kv_append_rope(L, rope, k, k, q=q, q_out=out, **which)
    kvq.kv_append_rope(L, rope, k, k, **which)
    kvq.kvq_rope_apply(rope, q.view(0, 4, 128), out.view(0, 4, 128))
    assert (L.k_cache == 7).all() and L.seq_lens.tolist() == [9, 9] and L.err.item() == 0
