"""attention_quantized_kv_gb300: attention over a block-quantized KV cache on GB300.

A thin Python layer over libkvq's C ABI (include/kvq.h).  PyTorch provides
device memory and streams; every step of the path (quantize-on-append,
split-K decode attention with its log-sum-exp merge, chunked-prefill
attention, the degrade ladder's re-encode, probe-scored eviction, rotary
positions) runs in the library's sm_103a kernels.  The functions below only
marshal arguments: they take torch tensors, pass their device pointers and
raise ``KVQError`` on a non-zero status.
"""
from __future__ import annotations

import ctypes
import functools
import math
from array import array

import torch

from . import _abi
from ._abi import (KVQ_F16, KVQ_Q8_0, KVQ_Q4_0, KVQ_TURBO4, KVQ_DEVERR_CAPACITY,
                   KVQ_DEVERR_EVICT,
                   KVQ_DEVERR_MAXLEN, KVQ_DEVERR_PAGE, KVQ_DEVERR_SEQLEN, KVQ_DEVERR_TIMEOUT,
                   KVQ_DEVERR_POS, KVQ_DEVERR_ROWS, KVQ_ROPE_HALF, KVQ_ROPE_INTERLEAVED,
                   KVQ_ROPE_LINEAR, KVQ_ROPE_NTK, KVQ_ROPE_PARTS, KVQ_ROPE_PLAIN, KVQ_ROPE_YARN,
                   kvq_layer)

__all__ = ["KVQ_F16", "KVQ_Q8_0", "KVQ_Q4_0", "KVQ_TURBO4", "CODEC_NAMES", "KVQError", "KVLayer",
           "kv_append_quantize", "attn_decode_workspace", "attn_decode", "attn_decode_append",
           "attn_prefill_workspace", "attn_prefill_chunk", "kvq_row_bytes", "kvq_cache_bytes",
           "kvq_pool_bytes", "KVQ_DEVERR_PAGE", "kv_requantize", "degrade", "aggregate_bpv",
           "ladder_next", "default_scale", "KVQ_DEVERR_EVICT", "kv_probe_scores",
           "kv_evict_select", "kv_compact", "evict", "KVQ_DEVERR_POS", "KVQ_DEVERR_ROWS",
           "KVQ_ROPE_HALF", "KVQ_ROPE_INTERLEAVED", "KVQ_ROPE_PLAIN", "KVQ_ROPE_LINEAR",
           "KVQ_ROPE_NTK", "KVQ_ROPE_PARTS", "KVQ_ROPE_YARN", "Rope", "kvq_rope_freqs",
           "kvq_rope_table", "kvq_rope_apply", "kv_append_rope", "kv_evict_delta",
           "kv_rope_shift", "attn_decode_append_rope"]

CODEC_NAMES = {KVQ_F16: "f16", KVQ_Q8_0: "q8_0", KVQ_Q4_0: "q4_0", KVQ_TURBO4: "turbo4"}
HEAD_DIM = 128


class KVQError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = _abi.load().kvq_status_str(status).decode()
        super().__init__(f"{where}: {msg} (status {status})")
        self.status = status


def _check(status: int, where: str) -> None:
    if status != 0:
        raise KVQError(status, where)


def _private(name: str, public):
    """torch._C's function, or the public way to the same where a version has none."""
    return getattr(torch._C, name, None) or public


_current_device = _private("_cuda_getDevice", torch.cuda.current_device)
_raw_stream = _private("_cuda_getCurrentRawStream",
                       lambda device: torch.cuda.current_stream(device).cuda_stream)


def _stream_ptr(stream) -> int:
    """The stream's handle; without one the current stream's, read without building a
    torch.cuda.Stream object (0.2 instead of 3.0 us a call)."""
    if stream is not None:
        return int(stream.cuda_stream)
    return _raw_stream(_current_device())


def _hand_over(stream, *tensors) -> None:
    """Tensors of the current stream's (or None) are used on another one next: that stream waits for
    what fills them, and their memory is given to nothing else before its work on them is done."""
    if stream is None:
        return
    current = torch.cuda.current_stream(tensors[0].device)
    if stream == current:
        return
    stream.wait_stream(current)
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def default_scale(head_dim: int = HEAD_DIM) -> float:
    return 1.0 / math.sqrt(head_dim)


def kvq_row_bytes(codec: int, head_dim: int = HEAD_DIM) -> int:
    return int(_abi.load().kvq_row_bytes(codec, head_dim))


def kvq_cache_bytes(codec: int, n_seqs: int, n_kv_heads: int, capacity: int,
                    head_dim: int = HEAD_DIM) -> int:
    return int(_abi.load().kvq_cache_bytes(codec, n_seqs, n_kv_heads, capacity, head_dim))


def kvq_pool_bytes(codec: int, n_pages: int, n_kv_heads: int,
                   head_dim: int = HEAD_DIM) -> int:
    return int(_abi.load().kvq_pool_bytes(codec, n_pages, n_kv_heads, head_dim))


class KVLayer:
    """One layer's cache: torch-owned device buffers plus the C descriptor.

    ``k_cache``/``v_cache`` are uint8 tensors in the layout of include/kvq.h,
    ``seq_lens`` int32 [n_seqs] and ``err`` one int32 error word.  Paged
    layers (``n_pages`` > 0) hold page pools instead, and ``block_table``
    (int32 [n_seqs][capacity / 256], device) maps each sequence's pages to
    pool pages (-1: not mapped; default: every page mapped, in order).
    """

    def __init__(self, n_seqs: int, n_kv_heads: int, n_q_heads: int, capacity: int,
                 codec_k: int, codec_v: int, device="cuda", head_dim: int = HEAD_DIM,
                 k_cache=None, v_cache=None, n_pages: int = 0, block_table=None):
        self.n_seqs, self.n_kv_heads, self.n_q_heads = n_seqs, n_kv_heads, n_q_heads
        self.capacity, self.codec_k, self.codec_v, self.head_dim = (capacity, codec_k, codec_v,
                                                                    head_dim)
        self.n_pages = int(n_pages)
        self.block_table = None
        if self.n_pages > 0:
            pps = capacity // 256
            if block_table is None:
                block_table = torch.arange(n_seqs * pps, dtype=torch.int32,
                                           device=device).reshape(n_seqs, pps)
            assert block_table.dtype == torch.int32 and block_table.shape == (n_seqs, pps)
            self.block_table = block_table.contiguous()
            kb = kvq_pool_bytes(codec_k, self.n_pages, n_kv_heads, head_dim)
            vb = kvq_pool_bytes(codec_v, self.n_pages, n_kv_heads, head_dim)
        else:
            kb = kvq_cache_bytes(codec_k, n_seqs, n_kv_heads, capacity, head_dim)
            vb = kvq_cache_bytes(codec_v, n_seqs, n_kv_heads, capacity, head_dim)
        if kb < 0 or vb < 0:
            raise ValueError("invalid cache geometry (capacity must be a multiple of 256, "
                             "head_dim 128, codecs f16/q8_0/q4_0/turbo4)")
        self.k_cache = k_cache if k_cache is not None else torch.empty(kb, dtype=torch.uint8,
                                                                        device=device)
        self.v_cache = v_cache if v_cache is not None else torch.empty(vb, dtype=torch.uint8,
                                                                        device=device)
        assert self.k_cache.numel() == kb and self.v_cache.numel() == vb
        self.seq_lens = torch.zeros(n_seqs, dtype=torch.int32, device=device)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        self._desc = None
        self._desc_key = None

    def desc(self) -> kvq_layer:
        """The C descriptor (rebuilt only when a buffer was replaced)."""
        key = (_ptr(self.k_cache), _ptr(self.v_cache), _ptr(self.seq_lens), _ptr(self.err),
               self.codec_k, self.codec_v, _ptr(self.block_table), self.n_pages)
        if self._desc is None or self._desc_key != key:
            d = kvq_layer()
            d.n_seqs, d.n_kv_heads, d.n_q_heads = self.n_seqs, self.n_kv_heads, self.n_q_heads
            d.head_dim, d.capacity = self.head_dim, self.capacity
            d.codec_k, d.codec_v, d.reserved = self.codec_k, self.codec_v, 0
            d.k_cache, d.v_cache, d.seq_lens, d.err = key[:4]
            if self.n_pages > 0:
                d.pages_per_seq, d.block_table, d.n_pages = (self.capacity // 256,
                                                             _ptr(self.block_table), self.n_pages)
            else:
                d.pages_per_seq, d.block_table, d.n_pages = 0, None, 0
            self._desc, self._desc_key = d, key
        return self._desc


def kv_append_quantize(layer: KVLayer, k_new, v_new, n_new, update_lens: bool = True,
                       stream=None) -> None:
    """k_new, v_new: fp16 [n_seqs, max_new, n_kv, 128]; n_new: int32 [n_seqs] (device)."""
    assert k_new.dtype == torch.float16 and v_new.dtype == torch.float16
    assert k_new.is_contiguous() and v_new.is_contiguous() and n_new.dtype == torch.int32
    max_new = int(k_new.shape[1])
    d = layer.desc()
    _check(_abi.load().kv_append_quantize(ctypes.byref(d), _ptr(k_new), _ptr(v_new),
                                          _ptr(n_new), max_new, int(bool(update_lens)),
                                          _stream_ptr(stream)), "kv_append_quantize")


def attn_decode_workspace(layer: KVLayer, max_len: int) -> int:
    """Bytes of decode workspace; allocate it zero-filled (torch.zeros)."""
    n = ctypes.c_size_t(0)
    d = layer.desc()
    _check(_abi.load().attn_decode_workspace(ctypes.byref(d), int(max_len), ctypes.byref(n)),
           "attn_decode_workspace")
    return int(n.value)


def attn_decode(layer: KVLayer, q, scale: float, out, lse, max_len: int, workspace,
                stream=None) -> None:
    """q, out: fp16 [n_seqs, n_q, 128]; lse: fp32 [n_seqs, n_q] or None."""
    assert q.dtype == torch.float16 and out.dtype == torch.float16 and q.is_contiguous()
    d = layer.desc()
    _check(_abi.load().attn_decode(ctypes.byref(d), _ptr(q), float(scale), _ptr(out), _ptr(lse),
                                   int(max_len), _ptr(workspace), int(workspace.numel() *
                                                                      workspace.element_size()),
                                   _stream_ptr(stream)), "attn_decode")


def attn_decode_append(layer: KVLayer, k_new, v_new, q, scale: float, out, lse, max_len: int,
                       workspace, stream=None) -> None:
    """One decode step in one launch: append k_new / v_new (fp16 [n_seqs, n_kv, 128], one
    token per sequence), attend seq_lens + 1 keys, advance seq_lens.  q, out: fp16
    [n_seqs, n_q, 128]; lse: fp32 [n_seqs, n_q] or None; workspace as attn_decode."""
    assert k_new.dtype == torch.float16 and v_new.dtype == torch.float16
    assert k_new.is_contiguous() and v_new.is_contiguous()
    assert q.dtype == torch.float16 and out.dtype == torch.float16 and q.is_contiguous()
    d = layer.desc()
    _check(_abi.load().attn_decode_append(ctypes.byref(d), _ptr(k_new), _ptr(v_new), _ptr(q),
                                          float(scale), _ptr(out), _ptr(lse), int(max_len),
                                          _ptr(workspace),
                                          int(workspace.numel() * workspace.element_size()),
                                          _stream_ptr(stream)), "attn_decode_append")


def attn_prefill_workspace(layer: KVLayer, q_start: int, n_q_tok: int) -> int:
    n = ctypes.c_size_t(0)
    d = layer.desc()
    _check(_abi.load().attn_prefill_workspace(ctypes.byref(d), int(q_start), int(n_q_tok),
                                              ctypes.byref(n)), "attn_prefill_workspace")
    return int(n.value)


def attn_prefill_chunk(layer: KVLayer, seq: int, q_start: int, q, scale: float, out, lse,
                       workspace, stream=None) -> None:
    """q, out: fp16 [n_q_tok, n_q, 128]; lse: fp32 [n_q_tok, n_q] or None."""
    assert q.dtype == torch.float16 and out.dtype == torch.float16 and q.is_contiguous()
    d = layer.desc()
    _check(_abi.load().attn_prefill_chunk(ctypes.byref(d), int(seq), int(q_start),
                                          int(q.shape[0]), _ptr(q), float(scale), _ptr(out),
                                          _ptr(lse), _ptr(workspace),
                                          int(workspace.numel() * workspace.element_size()),
                                          _stream_ptr(stream)), "attn_prefill_chunk")


# --------------------------------------------------------------------------- degrade ladder

@functools.lru_cache(maxsize=None)
def _row_bytes(codec: int) -> int:
    return kvq_row_bytes(codec)


def _side_bytes(layer: KVLayer, codec: int) -> int:
    """kvq_pool_bytes / kvq_cache_bytes of a side of this layer in a codec (-1: no such codec)."""
    tokens = layer.n_pages * 256 if layer.n_pages > 0 else layer.n_seqs * layer.capacity
    row = _row_bytes(codec)
    return row * layer.n_kv_heads * tokens if row > 0 else -1


def kv_requantize(layer: KVLayer, side: int, dst_codec: int, dst_cache, stream=None) -> None:
    """Re-encode side ``side`` (0 = K, 1 = V) of ``layer`` with ``dst_codec`` into
    ``dst_cache`` (uint8 device tensor of kvq_cache_bytes(dst_codec, ...) bytes)."""
    assert dst_cache.dtype == torch.uint8 and dst_cache.is_contiguous()
    nb = _side_bytes(layer, dst_codec)
    if dst_cache.numel() != nb:
        raise ValueError(f"dst_cache must hold {nb} bytes")
    d = layer.desc()
    _check(_abi.load().kv_requantize(ctypes.byref(d), int(side), int(dst_codec), _ptr(dst_cache),
                                     _stream_ptr(stream)), "kv_requantize")


def degrade(layer: KVLayer, side: int, dst_codec: int, stream=None) -> None:
    """Move one side of ``layer`` to ``dst_codec``: a new, zeroed cache buffer
    (torch allocation; rows past the lengths stay zero), the re-encode, then
    the layer points at the new buffer."""
    nb = _side_bytes(layer, dst_codec)
    src = layer.k_cache if side == 0 else layer.v_cache
    dst = torch.zeros(nb, dtype=torch.uint8, device=src.device)
    kv_requantize(layer, side, dst_codec, dst, stream)
    if side == 0:
        layer.k_cache, layer.codec_k = dst, dst_codec
    else:
        layer.v_cache, layer.codec_v = dst, dst_codec


def aggregate_bpv(codecs) -> float:
    arr = (ctypes.c_int32 * len(codecs))(*[int(c) for c in codecs])
    v = float(_abi.load().kvq_aggregate_bpv(arr, len(codecs)))
    if v < 0:
        raise ValueError("invalid codecs")
    return v


def ladder_next(codecs, floor_bpv: float, order=None):
    """(tensor, codec) of the next banded degrade step, or None."""
    arr = (ctypes.c_int32 * len(codecs))(*[int(c) for c in codecs])
    if order is None:
        ordp, n_order = None, 0
    else:
        ordp = (ctypes.c_int32 * len(order))(*[int(t) for t in order])
        n_order = len(order)
    t, k = ctypes.c_int32(-1), ctypes.c_int32(-1)
    _check(_abi.load().kvq_ladder_next(arr, len(codecs), ordp, n_order, float(floor_bpv),
                                       ctypes.byref(t), ctypes.byref(k)), "kvq_ladder_next")
    return None if t.value < 0 else (t.value, k.value)


# --------------------------------------------------------------------------- probe eviction

def kv_probe_scores(layer: KVLayer, q, scale: float, lse, decay: float, scores,
                    stream=None) -> None:
    """Fold one probe into ``scores`` (fp32 [n_seqs, capacity], device, in place):
    score = decay * score + the softmax mass the decode query ``q`` (fp16
    [n_seqs, n_q, 128]) puts on each token, summed over the query heads; ``lse``
    is attn_decode's fp32 [n_seqs, n_q] output for the same q and scale."""
    assert q.dtype == torch.float16 and q.is_contiguous()
    assert lse.dtype == torch.float32 and lse.is_contiguous()
    assert scores.dtype == torch.float32 and scores.is_contiguous()
    assert scores.numel() == layer.n_seqs * layer.capacity
    assert lse.numel() == layer.n_seqs * layer.n_q_heads
    d = layer.desc()
    _check(_abi.load().kv_probe_scores(ctypes.byref(d), _ptr(q), float(scale), _ptr(lse),
                                       float(decay), _ptr(scores), _stream_ptr(stream)),
           "kv_probe_scores")


def kv_evict_select(layer: KVLayer, scores, n_sink: int, n_recent: int, n_evict: int, evict,
                    n_evicted, stream=None) -> None:
    """Per sequence, the n_evict lowest (score, position) middle positions in
    increasing order into ``evict`` (int32 [n_seqs, n_evict]) and their count
    into ``n_evicted`` (int32 [n_seqs])."""
    assert scores.dtype == torch.float32 and scores.numel() == layer.n_seqs * layer.capacity
    assert evict.dtype == torch.int32 and evict.numel() >= layer.n_seqs * max(int(n_evict), 0)
    assert n_evicted.dtype == torch.int32 and n_evicted.numel() == layer.n_seqs
    d = layer.desc()
    _check(_abi.load().kv_evict_select(ctypes.byref(d), _ptr(scores), int(n_sink), int(n_recent),
                                       int(n_evict), _ptr(evict), _ptr(n_evicted),
                                       _stream_ptr(stream)), "kv_evict_select")


def kv_compact(layer: KVLayer, evict, n_evicted, k_dst, v_dst, scores=None, scores_dst=None,
               lens_dst=None, stream=None) -> None:
    """Remove the listed positions (``evict`` int32 [n_seqs, max_evict]) from both
    sides into ``k_dst``/``v_dst`` (uint8, the sizes of the layer's caches);
    optionally the scores and the new lengths too."""
    assert evict.dtype == torch.int32 and evict.dim() == 2 and evict.is_contiguous()
    assert n_evicted.dtype == torch.int32 and n_evicted.numel() == layer.n_seqs
    assert k_dst.dtype == torch.uint8 and v_dst.dtype == torch.uint8
    if k_dst.numel() != _side_bytes(layer, layer.codec_k) or \
            v_dst.numel() != _side_bytes(layer, layer.codec_v):
        raise ValueError("k_dst / v_dst must have the sizes of the layer's caches")
    d = layer.desc()
    _check(_abi.load().kv_compact(ctypes.byref(d), _ptr(evict), _ptr(n_evicted),
                                  int(evict.shape[1]), _ptr(k_dst), _ptr(v_dst), _ptr(scores),
                                  _ptr(scores_dst), _ptr(lens_dst), _stream_ptr(stream)),
           "kv_compact")


def evict(layer: KVLayer, scores, n_sink: int, n_recent: int, n_evict: int, stream=None,
          rope: "Rope | None" = None):
    """Select and remove up to n_evict tokens per sequence: new zeroed cache
    buffers (torch allocations), the layer repointed at them and at the new
    lengths.  With ``rope`` the kept keys are rotated to their new positions
    too (a token's position is its place in the cache again).  On another
    stream than the current one the work starts behind the current stream's.
    Returns (compacted scores, evict list, n_evicted)."""
    dev = layer.k_cache.device
    if rope is not None:
        rope._check_on(dev)
        if rope.n_pos < layer.capacity:
            raise ValueError("evict: the rope's table must cover the layer's capacity")
    ev = torch.zeros((layer.n_seqs, max(int(n_evict), 1)), dtype=torch.int32, device=dev)
    nev = torch.zeros(layer.n_seqs, dtype=torch.int32, device=dev)
    k_dst = torch.zeros_like(layer.k_cache)
    v_dst = torch.zeros_like(layer.v_cache)
    s_dst = torch.zeros_like(scores)
    lens = torch.empty_like(layer.seq_lens)
    delta = torch.empty((layer.n_seqs, layer.capacity if rope is not None else 0),
                        dtype=torch.int32, device=dev)
    _hand_over(stream, ev, nev, k_dst, v_dst, s_dst, lens, delta, scores, layer.k_cache,
               layer.v_cache, layer.seq_lens, layer.block_table, layer.err,
               None if rope is None else rope.table)
    kv_evict_select(layer, scores, n_sink, n_recent, n_evict, ev, nev, stream)
    kv_compact(layer, ev, nev, k_dst, v_dst, scores, s_dst, lens, stream)
    if rope is not None:
        kv_evict_delta(layer, ev, nev, delta, stream)
    layer.k_cache, layer.v_cache, layer.seq_lens = k_dst, v_dst, lens
    if rope is not None:
        kv_rope_shift(layer, rope, delta, stream)
    return s_dst, ev, nev


# --------------------------------------------------------------------------- rotary positions

_ROW_TYPES = {torch.float16: _abi.KVQ_T_F16, torch.bfloat16: _abi.KVQ_T_BF16,
              torch.float32: _abi.KVQ_T_F32}


def _need(t, dtype, shape, device, what: str):
    """A contiguous tensor of this type and shape on this device; its pointer."""
    if t.dtype != dtype or t.device != device or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what}: needs a contiguous {dtype} tensor of shape {tuple(shape)} on "
                         f"{device}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _cuda_device(t, what: str):
    """The device of a tensor, which has to be the current CUDA device."""
    d = t.device
    if d.type != "cuda" or d.index != _current_device():
        raise ValueError(f"{what}: tensors must be on the current CUDA device, got {d}")
    return d


def _layer_on(layer: KVLayer, device, what: str) -> None:
    if layer.k_cache.device != device:
        raise ValueError(f"{what}: the layer is on {layer.k_cache.device}, expected {device}")


def _rows(t, n_heads: int, device, what: str):
    """(descriptor, rows) of rows [..., n_heads, 128]: one stride for all leading dimensions."""
    kind = _ROW_TYPES.get(t.dtype)
    shape, st = t.shape, t.stride()
    if kind is None:
        raise ValueError(f"{what}: rows are float16, bfloat16 or float32, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{what}: on {t.device}, expected {device}")
    dims = len(shape)
    if dims not in (3, 4) or shape[-1] != HEAD_DIM or shape[-2] != n_heads:
        raise ValueError(f"{what}: needs [rows, {n_heads}, {HEAD_DIM}] or [seqs, rows, {n_heads}, "
                         f"{HEAD_DIM}], got {tuple(shape)}")
    if st[-1] != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    n, row = shape[-3], st[-3]
    if dims == 4:
        if shape[0] > 1 and n > 1 and st[0] != n * row:
            raise ValueError(f"{what}: sequences must be evenly spaced rows (stride {st[0]}, "
                             f"expected {n * row})")
        if n == 1:
            row = st[0]
        n *= shape[0]
    return _abi.kvq_rows(t.data_ptr(), row if n > 1 else 0, st[-2] if n_heads > 1 else 0, kind), n


def kvq_rope_freqs(rot_dim: int = HEAD_DIM, base: float = 10000.0, scaling: int = KVQ_ROPE_PLAIN,
                   factor: float = 1.0, orig_len: float = 0.0, low: float = 1.0,
                   high: float | None = None) -> list:
    """Radians per position of each of the rot_dim / 2 planes.  ``low`` and ``high`` are the
    turns over ``orig_len`` positions between which KVQ_ROPE_PARTS and KVQ_ROPE_YARN blend the
    scaled frequency into the plain one.  ``high`` defaults to 32 for KVQ_ROPE_YARN, as Peng et
    al. 2023 have it, and to 4 for KVQ_ROPE_PARTS (a narrower blend than their 1 to 32)."""
    if high is None:
        high = 32.0 if scaling == KVQ_ROPE_YARN else 4.0
    out = array("d", bytes(8 * max(1, int(rot_dim) // 2)))
    _check(_abi.load().kvq_rope_freqs(int(rot_dim), float(base), int(scaling), float(factor),
                                      float(orig_len), float(low), float(high),
                                      out.buffer_info()[0]), "kvq_rope_freqs")
    return out.tolist()


def kvq_rope_table(freqs, table, stream=None) -> None:
    """(cos, sin)(p * freqs[i]) for every position p into ``table`` (fp32
    [n_pos, len(freqs), 2], device)."""
    dev = _cuda_device(table, "kvq_rope_table")
    n = len(freqs)
    ptr = _need(table, torch.float32, (table.shape[0], n, 2), dev, "kvq_rope_table: table")
    f = array("d", freqs)
    _check(_abi.load().kvq_rope_table(f.buffer_info()[0], 2 * n, table.shape[0], ptr,
                                      _stream_ptr(stream)), "kvq_rope_table")


class Rope:
    """Rotary positions: the angle table of ``n_pos`` positions (built on the device, or the
    caller's fp32 [n_pos, rot_dim / 2, 2] ``table``) and the C descriptor over it.

    ``layout``: KVQ_ROPE_HALF pairs (i, i + rot_dim / 2), KVQ_ROPE_INTERLEAVED (2i, 2i + 1).
    ``magnitude`` multiplies cos and sin; None means 1, and 0.1 ln(factor) + 1 for
    KVQ_ROPE_YARN (Peng et al. 2023).  The other arguments are kvq_rope_freqs'."""

    def __init__(self, n_pos: int = 0, rot_dim: int = HEAD_DIM, base: float = 10000.0,
                 layout: int = KVQ_ROPE_HALF, scaling: int = KVQ_ROPE_PLAIN, factor: float = 1.0,
                 orig_len: float = 0.0, low: float = 1.0, high: float | None = None,
                 magnitude: float | None = None, table=None, device="cuda", stream=None):
        if magnitude is None:
            magnitude = 0.1 * math.log(factor) + 1.0 if scaling == KVQ_ROPE_YARN else 1.0
        if layout not in (KVQ_ROPE_HALF, KVQ_ROPE_INTERLEAVED):
            raise ValueError("layout must be KVQ_ROPE_HALF or KVQ_ROPE_INTERLEAVED")
        if not math.isfinite(magnitude):
            raise ValueError("magnitude must be finite")
        if table is None:
            freqs = kvq_rope_freqs(rot_dim, base, scaling, factor, orig_len, low, high)
            if n_pos <= 0:
                raise ValueError("n_pos must be positive")
            table = torch.empty((n_pos, len(freqs), 2), dtype=torch.float32, device=device)
            if table.is_cuda:
                _hand_over(stream, table)
            kvq_rope_table(freqs, table, stream)
        elif table.dim() != 3 or table.shape[0] < 1 or not 1 <= table.shape[1] <= HEAD_DIM // 2:
            raise ValueError(f"table must be [n_pos, rot_dim / 2, 2], got {tuple(table.shape)}")
        dev = _cuda_device(table, "Rope")
        ptr = _need(table, torch.float32, (table.shape[0], table.shape[1], 2), dev, "Rope: table")
        self.table, self.layout, self.magnitude = table, int(layout), float(magnitude)
        self.n_pos, self.rot_dim = int(table.shape[0]), 2 * int(table.shape[1])
        self._desc = _abi.kvq_rope(ptr, self.n_pos, self.rot_dim, self.layout, self.magnitude)

    def desc(self) -> _abi.kvq_rope:
        return self._desc

    def _check_on(self, device) -> None:
        if self.table.device != device:
            raise ValueError(f"the rope's table is on {self.table.device}, expected {device}")


def kvq_rope_apply(rope: Rope, x, y, positions=None, pos0: int = 0, transpose: bool = False,
                   err=None, stream=None) -> None:
    """Rotate the rows ``x`` (float16, bfloat16 or float32 [rows, heads, 128], strided) into ``y``
    (x's type or float16; may be x).  ``positions``: int32 [rows], or row r is at pos0 + r.
    ``transpose``: the gradient with respect to x, given that with respect to y.  ``err``: int32
    word for KVQ_DEVERR_POS.  Like every call here it writes through pointers: autograd neither
    records it nor sees that y (or x, in place) changed."""
    dev = _cuda_device(x, "kvq_rope_apply")
    rope._check_on(dev)
    if x.dim() != 3 or y.shape != x.shape:
        raise ValueError(f"kvq_rope_apply: x {tuple(x.shape)} and y {tuple(y.shape)} must be "
                         "[rows, heads, 128]")
    heads = x.shape[1]
    xd, n = _rows(x, heads, dev, "kvq_rope_apply: x")
    yd, _ = _rows(y, heads, dev, "kvq_rope_apply: y")
    pos = None if positions is None else _need(positions, torch.int32, (n,), dev,
                                               "kvq_rope_apply: positions")
    word = None if err is None else _need(err, torch.int32, (1,), dev, "kvq_rope_apply: err")
    _check(_abi.load().kvq_rope_apply(rope.desc(), xd, yd, n, heads, pos, int(pos0),
                                      int(bool(transpose)), word, _stream_ptr(stream)),
           "kvq_rope_apply")


def kv_append_rope(layer: KVLayer, rope: Rope, k, v, n_new=None, row_start=None, q=None,
                   q_out=None, positions=None, update_lens: bool = True, stream=None) -> None:
    """Rotate the new keys and append them with the values; rotate the queries beside them.

    Packed rows: k, v [rows, n_kv, 128] and ``row_start`` int32 [n_seqs + 1] (sequence s has rows
    row_start[s] .. row_start[s + 1] - 1; the rows behind the last are padding).  Padded rows: k,
    v [n_seqs, max_new, n_kv, 128] and ``n_new`` int32 [n_seqs].  float16, bfloat16 or float32,
    strided (views of a fused projection).  ``q``: rows of n_q heads, same leading shape and
    type, rotated into ``q_out`` (float16, contiguous).  ``positions``: int32, one per row;
    without it a row's position is its place in the cache."""
    dev = _cuda_device(k, "kv_append_rope")
    rope._check_on(dev)
    _layer_on(layer, dev, "kv_append_rope")
    if (n_new is None) == (row_start is None):
        raise ValueError("kv_append_rope: give n_new (padded rows) or row_start (packed rows)")
    lead = k.shape[:-2]
    if n_new is not None:
        if len(lead) != 2 or lead[0] != layer.n_seqs:
            raise ValueError("kv_append_rope: padded rows are [n_seqs, max_new, n_kv, 128]")
        n_ptr, s_ptr = _need(n_new, torch.int32, (layer.n_seqs,), dev, "kv_append_rope: n_new"), None
    else:
        if len(lead) != 1:
            raise ValueError("kv_append_rope: packed rows are [rows, n_kv, 128]")
        n_ptr, s_ptr = None, _need(row_start, torch.int32, (layer.n_seqs + 1,), dev,
                                   "kv_append_rope: row_start")
    if v.shape != k.shape or v.dtype != k.dtype:
        raise ValueError("kv_append_rope: k and v must have one shape and type")
    kd, n = _rows(k, layer.n_kv_heads, dev, "kv_append_rope: k")
    vd, _ = _rows(v, layer.n_kv_heads, dev, "kv_append_rope: v")
    qd = out = None
    if q is not None:
        if q_out is None or q.shape[:-2] != lead or q.dtype != k.dtype:
            raise ValueError("kv_append_rope: q needs q_out, and k's leading shape and type")
        qd, _ = _rows(q, layer.n_q_heads, dev, "kv_append_rope: q")
        out = _need(q_out, torch.float16, q.shape, dev, "kv_append_rope: q_out")
    elif q_out is not None:
        raise ValueError("kv_append_rope: q_out without q")
    pos = None if positions is None else _need(positions, torch.int32, lead, dev,
                                               "kv_append_rope: positions")
    _check(_abi.load().kv_append_rope(layer.desc(), rope.desc(), qd, kd, vd, n, n_ptr, s_ptr, pos,
                                      out, int(bool(update_lens)), _stream_ptr(stream)),
           "kv_append_rope")


def kv_evict_delta(layer: KVLayer, evict, n_evicted, delta, stream=None) -> None:
    """How far kv_compact moves each kept token (new minus old position, <= 0) into ``delta``
    (int32 [n_seqs, capacity]); ``layer`` as it was before the eviction."""
    dev = _cuda_device(delta, "kv_evict_delta")
    _layer_on(layer, dev, "kv_evict_delta")
    if evict.dim() != 2:
        raise ValueError("kv_evict_delta: evict must be [n_seqs, max_evict]")
    ev = _need(evict, torch.int32, (layer.n_seqs, evict.shape[1]), dev, "kv_evict_delta: evict")
    nev = _need(n_evicted, torch.int32, (layer.n_seqs,), dev, "kv_evict_delta: n_evicted")
    out = _need(delta, torch.int32, (layer.n_seqs, layer.capacity), dev, "kv_evict_delta: delta")
    _check(_abi.load().kv_evict_delta(layer.desc(), ev, nev, int(evict.shape[1]), out,
                                      _stream_ptr(stream)), "kv_evict_delta")


def kv_rope_shift(layer: KVLayer, rope: Rope, delta, stream=None) -> None:
    """Rotate the cached keys of token t of sequence s by ``delta[s, t]`` positions, in place
    (int32 [n_seqs, capacity]; 0 leaves the token's bytes as they are)."""
    dev = _cuda_device(delta, "kv_rope_shift")
    _layer_on(layer, dev, "kv_rope_shift")
    rope._check_on(dev)
    d = _need(delta, torch.int32, (layer.n_seqs, layer.capacity), dev, "kv_rope_shift: delta")
    _check(_abi.load().kv_rope_shift(layer.desc(), rope.desc(), d, _stream_ptr(stream)),
           "kv_rope_shift")


def attn_decode_append_rope(layer: KVLayer, rope: Rope, k_new, v_new, q, scale: float, out, lse,
                            max_len: int, workspace, positions=None, stream=None) -> None:
    """attn_decode_append with the rotation in it: the new keys are rotated before they are
    encoded and q before it attends, by ``positions`` (int32 [n_seqs]) or by the lengths before
    the step."""
    dev = _cuda_device(q, "attn_decode_append_rope")
    _layer_on(layer, dev, "attn_decode_append_rope")
    rope._check_on(dev)
    kv_shape = (layer.n_seqs, layer.n_kv_heads, HEAD_DIM)
    q_shape = (layer.n_seqs, layer.n_q_heads, HEAD_DIM)
    what = "attn_decode_append_rope: "
    k_ptr = _need(k_new, torch.float16, kv_shape, dev, what + "k_new")
    v_ptr = _need(v_new, torch.float16, kv_shape, dev, what + "v_new")
    q_ptr = _need(q, torch.float16, q_shape, dev, what + "q")
    o_ptr = _need(out, torch.float16, q_shape, dev, what + "out")
    l_ptr = None if lse is None else _need(lse, torch.float32, q_shape[:2], dev, what + "lse")
    pos = None if positions is None else _need(positions, torch.int32, (layer.n_seqs,), dev,
                                               what + "positions")
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(what + f"workspace must be contiguous on {dev}")
    _check(_abi.load().attn_decode_append_rope(
        layer.desc(), rope.desc(), pos, k_ptr, v_ptr, q_ptr, float(scale), o_ptr, l_ptr,
        int(max_len), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _stream_ptr(stream)), "attn_decode_append_rope")
