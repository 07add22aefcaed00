"""The 16-bit experts' training operators in 64 bits, from their definitions (torch, on the inputs' device),
and what the rounding of fp32 sums allows."""
from __future__ import annotations

import numpy as np
import torch

from gpu_util import dev, gpu_maps

DT = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
GUARD = 0xAB


def guarded(rows, cols, dtype, gap=0, first=0, extra=3):
    """A [rows, cols] matrix inside a larger buffer, every byte GUARD: `gap` values between rows, the first
    `first` values in.  Returns (buffer, matrix)."""
    ld = cols + gap
    whole = torch.empty(first + (rows + extra) * ld, dtype=dtype, device="cuda")
    whole.view(torch.uint8).fill_(GUARD)
    return whole, whole[first:first + rows * ld].view(rows, ld)[:, :cols]


def untouched(whole, part, live=None):
    """Every byte of the buffer outside the first `live` rows of the part is GUARD still."""
    keep = whole.clone()
    live = part.shape[0] if live is None else live
    inner = keep[part.storage_offset():].as_strided((live, part.shape[1]), (part.stride(0), 1))
    inner.view(torch.int16 if part.element_size() == 2 else torch.int32).fill_(
        -0x5455 if part.element_size() == 2 else -0x54545455)
    return bool((keep.view(torch.uint8) == GUARD).all())


def matrix(x, gap=0, first=0):
    """x's values in rows `gap` apart."""
    whole, part = guarded(*x.shape, x.dtype, gap, first)
    whole.view(torch.uint8).fill_(0xFF)      # NaN in every type: what is read outside the rows shows
    part.copy_(x)
    return part


class Routes:
    """Routes of T tokens to K of E experts, some tokens padded (ids -1), and the library's maps of them."""

    def __init__(self, T, K, E, seed, skew=0.0, pad=0.0):
        rng = np.random.default_rng(seed)
        logits = rng.standard_normal((T, E)) - skew * np.log(1.0 + rng.permutation(E))
        idx = np.argsort(-logits, axis=1, kind="stable")[:, :K].astype(np.int32)
        idx[rng.random(T) < pad] = -1
        self.T, self.K, self.E, self.R = T, K, E, T * K
        res, out = gpu_maps(idx, E, 0)
        self.idx = dev(idx)
        self.offsets, self.src, self.slot = out["offsets"], out["src"], out["slot"].view(T, K)
        self.at = [int(v) for v in res["offsets"]]
        self.live = self.at[-1]
        self.token = self.src[:self.live].long() // K

    def experts(self):
        for e in range(self.E):
            if self.at[e + 1] > self.at[e]:
                yield e, slice(self.at[e], self.at[e + 1])


def half_step(t, y):
    """How far rounding to t moves y, the smallest subnormal's half with it."""
    f = torch.finfo(t)
    return y.abs() * (f.eps / 2) + f.tiny * f.eps / 2


def within(got, want, tol):
    """got is want but for tol and the rounding to got's type."""
    want, got64 = want.double(), got.double()
    bad = ~((got64 - want).abs() <= tol + half_step(got.dtype, want.abs() + tol))
    if bool(bad.any()):
        at = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{int(bad.sum())} of {bad.numel()} off, first at {at}: {got64[at].item()!r} for "
                             f"{want[at].item()!r} +- {torch.as_tensor(tol).expand_as(want)[at].item():.3g}")


def sum_bound(n, s):
    """fp32 sums of n exact products in any order, each addition off by 2^-23 (truncation allowed for) of a
    partial sum that s, the sum of magnitudes, bounds."""
    return n * 2.0 ** -23 * s


def grouped(r, a, w):
    """a [live, k], w [E, N, k] -> sums and sums of magnitudes [live, N]."""
    y = torch.zeros(r.live, w.shape[1], dtype=torch.float64, device="cuda")
    s = torch.zeros_like(y)
    for e, rows in r.experts():
        wt = w[e].double().t().contiguous()
        y[rows] = a[rows].double() @ wt
        s[rows] = a[rows].double().abs() @ wt.abs()
    return y, s


def weight_grad(r, grad, a):
    """[E, N, k] and magnitudes."""
    y = torch.zeros(r.E, grad.shape[1], a.shape[1], dtype=torch.float64, device="cuda")
    s = torch.zeros_like(y)
    for e, rows in r.experts():
        gt, x = grad[rows].double().t().contiguous(), a[rows].double()
        y[e], s[e] = gt @ x, gt.abs() @ x.abs()
    return y, s


def sigmoid_error(g):
    """The kernels' sigmoid, relative: the exponent's argument and constant, exponential, sum, reciprocal."""
    return (1.25 * g.abs() + 8) * 2.0 ** -24


def swiglu(g, u, dg, du):
    """silu(g) u, and how far it is off where gate and up are off by dg and du (|silu'| < 1.1)."""
    silu = g * torch.sigmoid(g)
    h = silu * u
    return h, (1.1 * dg * (u.abs() + du) + silu.abs() * du + h.abs() * sigmoid_error(g)
               + 2.0 ** -119 * u.abs())


def swiglu_grad(d, g, u, tol):
    """The gradients of gate and up from d, that of silu(g) u, and how far they are off where d is by tol.
    For gate: s (1 + g (1 - s)) with s off by s delta has s delta (1 + |g|), from 1 - s again as much and
    a rounding of it, and four roundings of products."""
    s = torch.sigmoid(g)
    delta = sigmoid_error(g)
    a, b = u * s * (1 + g * (1 - s)), g * s
    scale = s * (1 + g.abs())
    ea = u.abs() * (scale * (2 * delta + 8 * 2.0 ** -24) + 2.0 ** -119 * (1 + g.abs()))
    eb = b.abs() * (delta + 4 * 2.0 ** -24) + 2.0 ** -119 * g.abs()
    return d * a, tol * (a.abs() + ea) + d.abs() * ea, d * b, tol * (b.abs() + eb) + d.abs() * eb
