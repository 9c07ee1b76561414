"""kv_append_rows into fp16 sides: every cached value is its input's, rounded once, at its own place,
and the bytes are kv_append_quantize's; NaN may change its payload and nothing else."""
import numpy as np
import pytest
import torch

import attention_quantized_kv_gb300 as kvq

from tests import _encoders as E
from tests.test_gpu_rope import _i32, _images, _layer

pytestmark = pytest.mark.gpu

F16, Q8, Q4, T4 = 0, 1, 2, 3
KINDS = {"float16": torch.float16, "bfloat16": torch.bfloat16, "float32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_quantized_kv_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _placed(image, lens, counts, values):
    """Rows of values [total, n_kv, 128] (fp16) in their places of an image; which of its bytes
    hold a NaN."""
    nan = np.zeros(image.data.shape, bool)
    at = 0
    for s, n in enumerate(counts):
        for i in range(n):
            for h in range(image.n_kv):
                row = values[at + i, h]
                image.put(s, h, lens[s] + i, row.view(np.uint8))
                nan[image.where(s, h, lens[s] + i)] = np.repeat(np.isnan(row), 2)
        at += n
    return nan


def _differ(got, image, nan):
    """Bytes that are not the image's; at NaN: 16-bit words that are none."""
    off = (got != image.data) & ~nan
    halves = got.view(np.float16)
    return int(off.sum()) + int((nan.reshape(-1, 2)[:, 0] & ~np.isnan(halves)).sum())


@pytest.mark.parametrize("ck,cv", [(F16, F16), (F16, Q8), (T4, F16)])
@pytest.mark.parametrize("counts", [[3, 0, 1, 2], [700, 0, 33, 301], [16, 16, 5, 2000]])
@pytest.mark.parametrize("dtype", sorted(KINDS))
@pytest.mark.parametrize("paged", [False, True])
def test_values(ck, cv, counts, dtype, paged):
    """By rows and by windows, packed and padded, whole and incomplete units."""
    n_kv, cap, lens = 4, 2304, [5, 17, 0, 40]
    L, table = _layer(4, n_kv, n_kv, cap, ck, cv, paged, 6)
    L.seq_lens.copy_(_i32(lens))
    images = _images(L, table)
    total = sum(counts)
    g = torch.Generator(device="cuda").manual_seed(total)
    kv = torch.randn((total, 2 * n_kv + 1, 128), generator=g, device="cuda").to(KINDS[dtype])
    rows = np.concatenate(E.special_rows(dtype))
    rows = rows[:total * (2 * n_kv + 1) // 2]
    flat = kv.view(-1, 128)
    flat[-len(rows):] = torch.from_numpy(rows).cuda().to(KINDS[dtype])  # NaN, infinities, past 65504
    sides = kv[:, 1:1 + n_kv], kv[:, 1 + n_kv:]
    start = np.cumsum([0] + counts)
    kvq.kv_append_rows(L, *sides, row_start=_i32(start))
    assert L.err.item() == 0
    with np.errstate(over="ignore"):
        halves = [x.float().cpu().numpy().astype(np.float16) for x in sides]
    masks = []
    for side, (image, x) in enumerate(zip(images, halves)):
        got = (L.k_cache, L.v_cache)[side].cpu().numpy()
        masks.append(None)
        if image.codec == F16:
            masks[side] = _placed(image, lens, counts, x)
            assert _differ(got, image, masks[side]) == 0
            # (the comparison sees heads, rows and dims that change places)
            for wrong in (x[:, ::-1], np.roll(x, 1, 0), np.roll(x, 1, 2)):
                other = _images(L, table)[side]
                nan = _placed(other, lens, counts, np.ascontiguousarray(wrong))
                assert _differ(got, other, nan) > 0
    # read back: the input rounded to fp16
    back = [torch.empty((total, n_kv, 128), dtype=torch.float32, device="cuda") for _ in "kv"]
    kvq.kv_read_rows(L, *back, row_start=_i32(start), first=_i32(lens))
    for codec, b, x in zip((ck, cv), back, halves):
        if codec == F16:
            b = b.cpu().numpy()
            assert np.array_equal(b, x.astype(np.float32), equal_nan=True)
    # padded rows, and kv_append_quantize's: the same bytes
    pad = torch.zeros((4, max(counts), 2 * n_kv, 128), dtype=KINDS[dtype], device="cuda")
    for s, n in enumerate(counts):
        pad[s, :n] = kv[start[s]:start[s + 1], 1:]
    calls = [lambda M: kvq.kv_append_rows(M, pad[:, :, :n_kv], pad[:, :, n_kv:], n_new=_i32(counts))]
    if dtype == "float16":
        calls.append(lambda M: kvq.kv_append_quantize(M, pad[:, :, :n_kv].contiguous(), pad[:, :, n_kv:].contiguous(),
                                                      _i32(counts)))
    for call in calls:
        M, _ = _layer(4, n_kv, n_kv, cap, ck, cv, paged, 6)
        M.seq_lens.copy_(_i32(lens))
        call(M)
        assert M.seq_lens.tolist() == L.seq_lens.tolist()
        for side, mask in enumerate(masks):
            a, b = ((x.k_cache, x.v_cache)[side].cpu().numpy() for x in (L, M))
            if mask is None:
                assert np.array_equal(a, b)
            else:
                assert np.array_equal(a[~mask], b[~mask])
                assert np.isnan(b[mask].view(np.float16)).all()
