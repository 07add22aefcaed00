"""How near the balance loss's probabilities are to 64-bit arithmetic where they are small."""
import numpy as np
import pytest
import torch

import mxref
from gpu_util import dev, host
from test_gpu_9_balance import run

pytestmark = pytest.mark.gpu

LOG2E = 1.0 / np.log(2.0)
U = 2.0 ** -24


def bound(d):
    """The relative error of exp(-d) / sum, d >= 0 below the row's maximum, as 2^t: t = d log2 e is rounded
    once (half an ulp of t, which the row's shared shift moves by 2^-8 at most, times ln 2) and its constant is off by 0.225 * 2^-24; 2^t to an ulp (2 units), as
    in the largest term (2 more); the sum, its reciprocal, and three products: 6."""
    ulp = np.exp2(np.floor(np.log2(d * LOG2E + 2.0 ** -7)) - 23)
    return 0.5 * ulp * np.log(2.0) + (0.225 * d + 10) * U


@pytest.mark.parametrize("top", [10.3, -3.7, 0.0, 60000.7, 65535.99])
def test_small_probabilities(top):
    """One token: prob_mean is its probabilities.  2047 logits 40 to 85 below the largest (2^-58 to 2^-123),
    so that the sum is the largest term's 1."""
    E = 2048
    rng = np.random.default_rng(5)
    x = (top - rng.uniform(40, 85, (1, E))).astype(np.float32)
    x[0, 77] = top
    _, prob, _, _ = run(dev(x), np.zeros((1, 1), np.int32), None)
    want = mxref.balance(x.astype(np.float64), np.zeros((1, 1), np.int32))[1]
    d = x[0, 77].astype(np.float64) - x[0].astype(np.float64)
    err = np.abs(host(prob).astype(np.float64) / want - 1)
    print("units", (err / U).max(), (err / bound(d)).max())
    assert np.all(err <= bound(d))


@pytest.mark.parametrize("top", [65536.0, 1e5, -70000.0, 2.0 ** 24, 1e30, np.finfo(np.float32).max,
                                 np.finfo(np.float32).min / 2])
def test_large_logits(top):
    """Maxima whose product with log2 e rounds by more than an exponent holds, or overflows: the neighbours
    of the maximum in fp32, and far ones, against 64 bits."""
    E = 64
    x = np.full((3, E), np.float32(top), np.float32)
    for j in range(1, E):
        x[1, j] = np.nextafter(x[1, j - 1], np.float32(-np.inf))
    x[2, 1:] = np.linspace(-1, 0.99, E - 1).astype(np.float32) * np.float32(abs(top))
    idx = np.zeros((3, 1), np.int32)
    x64 = x.astype(np.float64)
    _, prob, _, grad = run(dev(x), idx, None)
    _, want, _, gradf, p, f = mxref.balance(x64, idx)
    d = np.minimum(x64.max(1, keepdims=True) - x64, 150)
    # the difference itself is rounded here too: d more units
    e = (bound(d) + d * U) * p + 2.0 ** -126
    assert np.all(np.abs(host(prob) - want) <= (e + p * e.sum(1, keepdims=True)).sum(0) / 3 + 8 * U * want)
    g = gradf(1.0)
    assert np.all(np.isfinite(host(grad)))
    dev_f = np.abs(f - 1.0 / E)
    tol = E / 3 * (p * (dev_f + (p * dev_f).sum(1, keepdims=True)) * (2 * bound(d) + 2 * d * U + 30 * U) + 2.0 ** -120)
    assert np.all(np.abs(host(grad) - g) <= tol)
