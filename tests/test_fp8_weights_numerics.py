"""The numeric facts that the chunk attention's weights rest on for FP8 caches (csrc/chunk_attn.cu,
split_weights), checked on every value.

A weight 2^(s - m + 8), below 2^12, is rounded to f16 and written as an e4m3 and an e5m2 value whose
products with V go into one sum: from 256 up its first three bits as e5m2 and the rest as e4m3, below
the e4m3 value first. The steps run in f16."""

import numpy as np

from oracle import codecs


def weights():
    bits = np.arange(0, 0x7C00, dtype=np.uint16)
    v = bits.view(np.float16)
    return v[v < 4096.0]


def e5m2(x):
    """f16 to the nearest e5m2 value (ties to even): e5m2 is f16's first byte."""
    bits = x.view(np.uint16).astype(np.uint32)
    low, odd = bits & 0xFF, (bits >> 8) & 1
    up = (low > 0x80) | ((low == 0x80) & (odd == 1))
    return (((bits >> 8) + up) << 8).astype(np.uint16).view(np.float16)


def split(v):
    """The kernel's steps: (e4m3 part, e5m2 part, first), float64."""
    rounded = ((v.view(np.uint16).astype(np.uint32) + 0x80) & 0xFF00).astype(np.uint16).view(np.float16)
    first = np.where(v >= 256.0, rounded, np.float16(0.0))
    rest = v - first  # f16
    assert (rest.astype(np.float64) == v.astype(np.float64) - first).all()
    a = codecs.e4m3_round(rest.astype(np.float64))
    b = e5m2((v.astype(np.float64) - a).astype(np.float16))
    return a, b.astype(np.float64), first.astype(np.float64)


def test_sum_of_the_parts_over_every_weight():
    v = weights()
    a, b, first = split(v)
    x = v.astype(np.float64)
    err = np.abs(x - (a + b))
    power = 2.0 ** np.floor(np.log2(np.maximum(x, 2.0 ** -24)))
    full = x >= 2.0 ** -6
    assert (err[full] <= 2.0 ** -8 * power[full]).all()
    assert (err[~full] <= 2.0 ** -14).all()
    assert (err[~full] <= np.maximum(x[~full] / 8, 2.0 ** -17)).all()
    # nothing saturates, and a large weight's e5m2 part is the one that was taken out first
    assert np.abs(a).max() <= 256.0 and np.abs(b).max() <= 4096.0
    assert (b[x >= 256.0] == first[x >= 256.0]).all()


def test_small_weights_keep_their_sum():
    # thousands of weights far below the largest (2^8): an e4m3 pair has no step below 2^-9
    rng = np.random.default_rng(3)
    w = np.exp2(rng.normal(-10.0, 1.44, 100000)).astype(np.float16)
    a, b, _ = split(w)
    total = w.astype(np.float64).sum()
    assert abs((a + b).sum() - total) <= 0.005 * total
    pair = np.exp2(-4.0) * w.astype(np.float64)  # (2^4 is what a pair had for the largest)
    hi = codecs.e4m3_round(pair)
    lo = codecs.e4m3_round(pair - hi)
    assert (hi + lo).sum() < 0.2 * pair.sum()
