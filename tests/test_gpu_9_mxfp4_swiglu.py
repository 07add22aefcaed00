"""The SwiGLU epilogue far from zero: gates whose exponential leaves fp32's range, with exact sums."""
import numpy as np
import pytest
import torch

import mxref
from test_gpu_9_mxfp4 import product
from gpu_util import host
from quantized_expert_grouped_amd import abi

pytestmark = pytest.mark.gpu

GATES = [-87, -88, -89, -90, -95, -103, -104, -120, -127, -80, -60, -40, -17, -1, 0, 1, 17, 40, 60, 80, 87, 88,
         89, 90, 103, 104, 120, 127, -2, 2, -3, 3]


def whole_number(v):
    """128 values in MXFP4 whose sum is the integer v, |v| < 128: multiples of 8 in the first block (scale 16),
    the rest in the second (scale 1)."""
    x = np.zeros(128)
    a, s = abs(v), np.sign(v)
    hi = a // 8 * 8
    for lv in (96, 64, 48, 32, 24, 16, 8):
        for j in range(2):
            if hi >= lv and (hi - lv) in (0, 8, 16, 24, 32, 48, 64, 96):
                i = int(np.flatnonzero(x[:32] == 0)[0])
                x[i] = s * lv
                hi -= lv
    assert hi == 0
    for j, b in enumerate((4, 2, 1)):
        if a % 8 & b:
            x[32 + j] = s * b
    assert x.sum() == v
    return x


@pytest.mark.parametrize("R", [5, 1300])
@pytest.mark.parametrize("shift", [0, 60, 100])
def test_gates_whose_exponential_leaves_the_range(R, shift):
    """Gates are small integers, the same in the 32 columns of a scale, ups powers of two: sums are exact, so h is
    silu(g) u to the epilogue's own error, (1.25 |g| + 8) 2^-24.  From g = -88 on silu(g), below 2^-119, may
    count as zero: h lies between its value and -0."""
    N = 32 * len(GATES)
    codes = np.zeros((2, N, 64), np.uint8)
    scales = np.full((2, N, 4), 127, np.uint8)
    for b, g in enumerate(GATES):
        x = whole_number(g).reshape(4, 32)
        sc = np.array([131, 127, 127, 127])
        lv = (np.abs(x) / np.exp2(sc - 127.0)[:, None]).ravel()
        code = np.array([int(np.flatnonzero(mxref.LEVELS == v)[0]) for v in lv]) + 8 * (x.ravel() < 0)
        code = code.astype(np.uint8)
        codes[0, 32 * b:32 * b + 32] = code[0::2] | code[1::2] << 4
        scales[0, 32 * b:32 * b + 32] = sc
    codes[1, :, 0] = 2                                        # up: 1.0 times a scale of its own
    scales[1, :, 0] = 127 + shift + (np.arange(N) % 3)
    a = np.ones((R, 128))
    ac, as_ = mxref.encode(a)
    wc, ws = codes.reshape(1, 2 * N, 64), scales.reshape(1, 2 * N, 4)
    y, _ = mxref.grouped(mxref.decode(ac, as_), mxref.decode(wc, ws), [0, R])
    g, u = y[:, :N], y[:, N:]
    assert np.array_equal(g[0, ::32], GATES) and np.array_equal(u[0], np.exp2(shift + np.arange(N) % 3))
    offsets = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    out, os_ = product(wc, ws, offsets, ac, as_, R, None, 1, abi.MX_SWIGLU_MXFP4)
    got_c, got_s = host(out), host(os_)
    h = mxref.silu(g) * u
    d = np.abs(h) * (1.25 * np.abs(g) + 8) * 2.0 ** -24
    exact = np.flatnonzero(np.array(GATES) > -88)
    cols = (32 * exact[:, None] + np.arange(32)).ravel()
    half = (16 * exact[:, None] + np.arange(16)).ravel()
    mxref.check_codes(got_c[:, half], got_s[:, exact], h[:, cols], d[:, cols])
    v = mxref.decode(got_c, got_s)
    low = np.repeat(np.array(GATES) <= -88, 32)
    assert np.all(v[:, low] <= 0) and np.all(v[:, low] >= 1.5 * h[:, low] - 2.0 ** -127)
