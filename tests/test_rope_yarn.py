"""YaRN frequencies against values worked out by hand, among them contexts in
which even the slowest plane makes a whole turn: the ramp over the planes then
ends past the last one (at most at index rot_dim - 1)."""
import math

import pytest

import attention_quantized_kv_gb300 as kvq

TOL = 2.0 ** -48  # a handful of operations in double, as in the other tests of frequencies


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_quantized_kv_gb300 import build
    build.build()


# Base 16, so that f_i = 16^(-2i / rot); orig_len = 2 pi 2^e, so that at(2^k) = (rot / 8) (e - k).
@pytest.mark.parametrize("rot,e,low,high,want", [
    # 8 dims, f = 1, 1/2, 1/4, 1/8: at(8) = 1.5 -> l = 1, at(1) = 4.5 -> h = 5, past the last plane;
    # keep = 1, 1, 3/4, 1/2 and 1/4 of the rest
    (8, 4.5, 1.0, 8.0, [1.0, 0.5, 0.25 * 13 / 16, 0.125 * 5 / 8]),
    # l = 2, at(1) = 20.5 bounded by h = 7: keep = 1, 1, 1, 4/5
    (8, 20.5, 1.0, 2.0 ** 18, [1.0, 0.5, 0.25, 0.125 * 17 / 20]),
    # the last plane makes less than a turn: l = 0, h = 3; keep = 1, 2/3, 1/3, 0
    (8, 2.5, 1.0, 4.0, [1.0, 0.5 * 3 / 4, 0.25 / 2, 0.125 / 4]),
    # 4 dims, f = 1, 1/4: l = 0, at(1) = 2.25 -> h = 3 = rot - 1: keep = 1, 2/3
    (4, 4.5, 1.0, 8.0, [1.0, 0.25 * 3 / 4]),
    # 2 dims, f = 1: l = 0, h = 1
    (2, 4.5, 1.0, 8.0, [1.0]),
])
def test_hand_worked(rot, e, low, high, want):
    got = kvq.kvq_rope_freqs(rot, 16.0, kvq.KVQ_ROPE_YARN, 4.0, 2 * math.pi * 2.0 ** e, low, high)
    assert len(got) == len(want)
    for i, (a, b) in enumerate(zip(got, want)):
        assert abs(a - b) <= TOL * b, (i, a, b)


def test_long_original_context():
    """128 dims, base 10^4, 65536 positions, 1 to 32 turns: at(32) = 40.2 and at(1) = 64.3, so plane
    i keeps 1 - (i - 40) / 25 from plane 40 on; the last one 2 / 25."""
    plain = kvq.kvq_rope_freqs(128, 10000.0)
    got = kvq.kvq_rope_freqs(128, 10000.0, kvq.KVQ_ROPE_YARN, 4.0, 65536)
    for i in range(64):
        keep = min(1.0, (65 - i) / 25)
        assert abs(got[i] / plain[i] - (keep + (1 - keep) / 4)) <= TOL, i


def test_a_context_whose_last_planes_make_no_turn():
    """32768 positions: at(32) = 35.4, at(1) = 59.5, the ramp ends at plane 60 as before."""
    plain = kvq.kvq_rope_freqs(128, 10000.0)
    got = kvq.kvq_rope_freqs(128, 10000.0, kvq.KVQ_ROPE_YARN, 4.0, 32768)
    for i in range(64):
        keep = min(1.0, max(0.0, (60 - i) / 25))
        assert abs(got[i] / plain[i] - (keep + (1 - keep) / 4)) <= TOL, i
