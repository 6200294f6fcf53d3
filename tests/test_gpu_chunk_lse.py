"""The log-sum-exp of chunk attention as an fp32 output, for every mask, both head dims and both kinds of pages,
and its refusals of a scale beyond fp32.

Tolerance: a score is a sum of d <= 128 exact products, each addition off by 2^-24 of the partial sum; partial
sums are below sum |q k| scale, at most 20 here; the exponentials are off by 2.5e-7, a sum of n of them by
(n / 64 + 64) 2^-24, the logarithm by 2^-22, and references up to 2^5 are added to it: 2e-5 in all for an LSE of
order 1 and more."""

from __future__ import annotations

import numpy as np
import pytest

import exact_attention_116_b200 as fa
from chunk_cases import Batch, call, np64

pytestmark = pytest.mark.gpu

MASKS = {"causal": (True, (-1, -1), 0), "full": (False, (-1, -1), 0), "window": (True, (100, -1), 0),
         "sinks": (True, (100, -1), 5), "both": (False, (90, 30), 0), "far": (True, (20, -1), 200),
         "own": (True, (0, -1), 0)}
SHAPES = [([130, 1, 300, 0, 7], [700, 520, 300, 10, 128], 4, 2), ([1, 4, 1], [3000, 260, 90], 8, 2),
          ([16, 3], [5000, 40], 16, 1), ([1], [20000], 4, 4)]


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mask", list(MASKS))
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_the_log_sum_exp_under_every_mask(shape, mask, d, f8):
    causal, window, sinks = MASKS[mask]
    new, keys, Hq, Hkv = SHAPES[shape]
    b = Batch(new, keys, Hq, Hkv, d, 32, f8, seed=shape + d)
    _, lse = call(b.gpu(), None, causal, window, sinks)
    fa.check()
    ref = b.reference(d ** -0.5, causal, window, sinks)[1]
    dead = ~np.isfinite(ref)
    assert np.array_equal(dead, np64(lse) == -np.inf)
    err = np.abs(np.where(dead, 0, np64(lse)) - np.where(dead, 0, ref)).max()
    assert err <= 2e-5 * max(1.0, np.abs(ref[~dead]).max()), err


@pytest.mark.parametrize("scale", [1e39, -1e39, float("inf"), float("nan")])
def test_a_scale_beyond_fp32_is_refused_as_elsewhere(scale):
    t = Batch([2], [9], 2, 1, 64, 16, False).gpu()
    with pytest.raises(fa.FaError):
        call(t, scale)
