"""MXFP4, the grouped product and the balance loss in 64 bits, from their definitions (numpy)."""
from __future__ import annotations

import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# the magnitudes where the nearest level changes; at an equal distance the even code wins
BORDERS = (LEVELS[1:] + LEVELS[:-1]) / 2


def nearest(a):
    """The code (0..7) of the level nearest to each magnitude."""
    a = np.asarray(a, np.float64)
    up = np.searchsorted(BORDERS, a, side="right")     # a border itself goes up ...
    down = np.searchsorted(BORDERS, a, side="left")    # ... or stays down
    return np.where(up % 2 == 0, up, down)


def scale_byte(amax):
    """amax float64 (finite, of fp32 values) -> byte."""
    m, e = np.frexp(np.asarray(amax, np.float64))
    return np.where(amax > 0, np.maximum(e - 1 - 2 + 127, 0), 0).astype(np.int64)


def encode(x):
    """x [rows, n] -> (codes [rows, n/2] uint8, scales [rows, n/32] uint8)."""
    x = np.asarray(x, np.float64)
    v = x.reshape(x.shape[0], -1, 32)
    bad = ~np.isfinite(v).all(-1)
    v = np.where(bad[..., None], 0.0, v)
    byte = scale_byte(np.abs(v).max(-1))
    q = v * np.exp2(127.0 - byte)[..., None]
    c = nearest(np.abs(q)) + 8 * np.signbit(q)
    c = np.where(bad[..., None], 0, c).reshape(x.shape).astype(np.uint8)
    return c[:, 0::2] | (c[:, 1::2] << 4), np.where(bad, 255, byte).astype(np.uint8)


def levels(codes):
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = LEVELS[c & 7]
    return np.where(c & 8, -v, v)


def decode(codes, scales):
    s = np.exp2(scales.astype(np.float64) - 127.0)
    s = np.where(scales == 255, np.nan, s)
    v = levels(codes)
    return (v.reshape(*scales.shape, 32) * s[..., None]).reshape(v.shape)


def grouped(a, w, offsets):
    """a [rows, k], w [E, N, k] float64 -> y and sum |a||w|, [rows, N]; rows past offsets[E] are 0."""
    y = np.zeros((a.shape[0], w.shape[1]))
    s = np.zeros_like(y)
    for e in range(w.shape[0]):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        if r.stop > r.start:
            y[r] = a[r] @ w[e].T
            s[r] = np.abs(a[r]) @ np.abs(w[e]).T
    return y, s


def silu(g):
    return g / (1.0 + np.exp(-np.clip(g, -700, 700)))


def check_codes(codes, scales, h, d):
    """codes, scales are a right MXFP4 form of some values within d of h [rows, n]."""
    rows, n = h.shape
    lo_a = np.maximum(np.abs(h) - d, 0).reshape(rows, -1, 32).max(-1)
    hi_a = (np.abs(h) + d).reshape(rows, -1, 32).max(-1)
    b = scales.astype(np.int64)
    assert np.all(b >= scale_byte(lo_a)) and np.all(b <= scale_byte(hi_a)), "scale bytes"
    got = levels(codes)
    inv = np.repeat(np.exp2(127.0 - b), 32, axis=1)

    def rounded(v):
        q = v * inv
        return np.copysign(LEVELS[nearest(np.abs(q))], q)

    assert np.all(got >= rounded(h - d)) and np.all(got <= rounded(h + d)), "codes"


def balance(logits, idx, valid=None):
    """counts [E + 1], prob_mean [E], loss and the function grad(g) -> [T, E]."""
    x = np.asarray(logits, np.float64)
    T, E = x.shape
    K = idx.shape[1]
    on = np.ones(T, bool) if valid is None else np.asarray(valid) != 0
    n = int(on.sum())
    p = np.zeros((T, E))
    top = np.where(on, np.where(on[:, None], x, 0).max(1), -np.inf)
    rows = np.flatnonzero(top > -np.inf)
    ex = np.exp(x[rows] - top[rows, None])
    p[rows] = ex / ex.sum(1, keepdims=True)
    counts = np.zeros(E + 1, np.int64)
    ids = idx[on].reshape(-1)
    np.add.at(counts, ids[(ids >= 0) & (ids < E)], 1)
    counts[E] = n
    f = counts[:E] / max(n * K, 1)
    prob = p.sum(0) / max(n, 1)

    def grad(g):
        return g * E / max(n, 1) * p * (f - (p @ f)[:, None])

    return counts, prob, E * float(f @ prob), grad, p, f
