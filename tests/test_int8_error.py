"""Quantisation error of the int8 cache (a scale per block of 16 tokens and head)
beside e4m3 with one calibrated scale a head, on CPU through the oracle's write.

Rounding to a step of D leaves an error of D / sqrt(12) (rms) in values that are
spread over many steps.  Int8: D = a / 127 with a the largest of n = 16 * head_size
magnitudes, E[a^2] from the distribution function erf(a / sqrt 2)^n.  e4m3: D =
2^(k - 3) for magnitudes in [2^k, 2^(k + 1)) of the scaled values; the scale that
puts the largest at 448 is a power of two here, so k is that of the value itself.
Blocks x heads = 800 maxima, whose squares spread by 15 %, set E[a^2] to 0.5 %:
3 % is six of that."""
import math

import numpy as np
import pytest
import torch

from oracle import int8 as O8

NB, HEADS = 200, 4


def int8_error(x):
    nb, _, h, d = x.shape
    codes, scales = np.zeros(x.shape, np.int8), np.zeros((nb, h), np.float32)
    O8.write(x.reshape(-1, h, d), x.reshape(-1, h, d), np.arange(nb)[None], np.array([16 * nb]),
             np.array([0, 16 * nb]), codes, codes.copy(), scales, scales.copy())
    return O8.widen(codes, scales) - x


def e4m3_error(x):
    scale = 2.0 ** np.ceil(np.log2(np.abs(x).max((0, 1, 3), keepdims=True) / 448))
    y = torch.from_numpy((x / scale).astype(np.float32)).to(torch.float8_e4m3fn)
    return y.float().numpy() * scale - x


def rms(x):
    return float(np.sqrt(np.mean(np.square(x, dtype=np.float64))))


@pytest.mark.parametrize("d", [64, 128])
def test_channels_of_like_size(d):
    x = np.random.default_rng(d).standard_normal((NB, 16, HEADS, d)).astype(np.float32)
    a = np.linspace(0, 8, 80001)
    below = np.array([math.erf(t / math.sqrt(2)) for t in a]) ** (16 * d)
    top2 = float(np.sum(2 * a * (1 - below)) * (a[1] - a[0]))     # E[a^2]
    int8 = math.sqrt(top2 / 12) / 127
    share = [(math.erf(2.0 ** (k + 1) / math.sqrt(2)) - math.erf(2.0 ** k / math.sqrt(2)), k)
             for k in range(-8, 4)]
    e4m3 = math.sqrt(sum(p * 4.0 ** (k - 3) for p, k in share) / 12)
    assert abs(rms(int8_error(x)) / int8 - 1) < 0.03
    assert abs(rms(e4m3_error(x)) / e4m3 - 1) < 0.03
    assert 0.27 < int8 / e4m3 < 0.34          # "about a third"


def test_channels_of_different_size_take_the_largest_ones_step():
    """Every element is off by half a step of its block's largest channel at most,
    so where a few channels are far larger the others lose what e4m3 keeps."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((NB, 16, HEADS, 128)).astype(np.float32)
    x[..., 5] *= 64
    small = np.delete(np.arange(128), 5)
    step = np.abs(x).max((1, 3), keepdims=True) / 127
    off = int8_error(x)
    assert (np.abs(off) <= step * (0.5 + 2.0 ** -16)).all()
    # (the large channel alone sets the step: at least 64 * 1.0 / 127 in most blocks,
    # error rms over 0.1; e4m3's is below 2^-4 of each value)
    assert rms(off[..., small]) > 0.1 > 2.0 ** -4 > rms(e4m3_error(x)[..., small])
