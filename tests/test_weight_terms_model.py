"""The cut of a softmax weight into three e5m2 terms (split_weight of
decode_diff_tc.cuh), in numpy, bit for bit: every fp16 value in [0, 2^15] is
t1 + t2 2^-4 + t3 2^-8 exactly, and every step stays within fp16."""
import numpy as np


def near(bits):
    return ((bits.astype(np.uint32) + 0x80) & 0xFF00).astype(np.uint16)


def split(bits):
    terms = []
    for m in range(2):
        lead = near(bits)
        terms.append(lead)
        rest = bits.view(np.float16) - lead.view(np.float16)
        exact = bits.view(np.float16).astype(np.float64) - lead.view(np.float16).astype(np.float64)
        assert np.all(rest == exact)
        scaled = rest * np.float16(16)
        assert np.all(scaled == 16 * exact)
        bits = scaled.view(np.uint16)
    assert not (bits & 0xFF).any()  # the last is an e5m2 value as it stands
    return [*terms, bits & np.uint16(0xFF00)]


def test_every_weight_is_the_sum_of_its_terms():
    bits = np.arange(0x7800 + 1, dtype=np.uint16)
    t = [x.view(np.float16).astype(np.float64) for x in split(bits)]
    assert np.array_equal(t[0] + t[1] / 16 + t[2] / 256, bits.view(np.float16).astype(np.float64))
    assert max(np.abs(x).max() for x in t) <= 2.0 ** 15


def test_packed_pairs_do_not_touch_each_other():
    """The kernel adds to both halves of a word at once: no carry leaves the lower one, signs included."""
    lo = np.concatenate([np.arange(0x7800 + 1), np.arange(0x8000, 0xF800 + 1)]).astype(np.uint32)
    for hi in (0x0000, 0x7800, 0xF800, 0x3C7F):
        word = (np.uint32(hi) << np.uint32(16)) | lo
        lead = (word + np.uint32(0x00800080)) & np.uint32(0xFF00FF00)
        assert np.array_equal((lead & 0xFFFF).astype(np.uint16), near(lo.astype(np.uint16)))
        assert np.all(lead >> 16 == near(np.array([hi], np.uint16))[0])
