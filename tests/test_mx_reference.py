"""The 64-bit reference of the MXFP4 tests against closed forms, and the host's refusals of the MXFP4,
combine and balance entry points (CPU only: no call here reaches a kernel)."""
import numpy as np
import pytest
import torch

import mxref
from quantized_expert_grouped_amd import abi


def test_levels_and_ties():
    assert mxref.nearest([0, .25, .26, .75, .74, 1.25, 1.75, 2.5, 2.51, 3.5, 5.0, 5.1, 9]).tolist() == \
        [0, 0, 1, 2, 1, 2, 4, 4, 5, 6, 6, 7, 7]
    assert mxref.scale_byte(np.array([0.0, 1.0, 4.0, 7.9, 8.0, 2.0 ** -126, 2.0 ** -140])).tolist() == \
        [0, 125, 127, 127, 128, 0, 0]


def test_encode_decode_round_trip():
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 256, (5, 64), dtype=np.uint8)
    codes[:, ::16] |= 6                        # an element of magnitude 4 or 6: the scale is the block's
    scales = rng.integers(1, 253, (5, 4), dtype=np.uint8)
    c, s = mxref.encode(mxref.decode(codes, scales))
    assert np.array_equal(c, codes) and np.array_equal(s, scales)
    x = np.zeros((1, 64))
    x[0, 3], x[0, 40] = np.inf, -0.0
    c, s = mxref.encode(x)
    assert s.tolist() == [[255, 0]] and c[0, 20] == 8 and c.sum() == 8


def test_balance_reference_against_differences():
    rng = np.random.default_rng(1)
    T, E, K, g = 9, 7, 2, 0.7
    x = rng.standard_normal((T, E))
    idx = np.argsort(-x, 1)[:, :K].astype(np.int32)
    valid = (np.arange(T) % 4 != 1).astype(np.uint8)
    counts, _, loss, grad, _, f = mxref.balance(x, idx, valid)
    gr = grad(g)
    for t, j in ((0, 0), (1, 2), (4, 6), (8, 3)):
        d = np.zeros_like(x)
        d[t, j] = 1e-5
        diff = g * (mxref.balance(x + d, idx, valid)[2] - mxref.balance(x - d, idx, valid)[2]) / 2e-5
        assert abs(diff - gr[t, j]) < 1e-9
    u = mxref.balance(np.zeros((E, E)), np.arange(E, dtype=np.int32)[:, None])
    assert abs(u[2] - 1) < 1e-12 and counts[E] == valid.sum()


def test_quantize_host_checks():
    q, d = abi.lib().moe_mxfp4_quantize, abi.lib().moe_mxfp4_dequantize
    p = 1 << 20
    for fn, a in ((q, lambda **k: (k.get("x", p), k.get("dt", 0), k.get("ld", 64), k.get("rows", 2),
                                   k.get("n", 64), k.get("c", p), k.get("s", p), None)),
                  (d, lambda **k: (k.get("c", p), k.get("s", p), k.get("rows", 2), k.get("n", 64),
                                   k.get("x", p), k.get("dt", 0), k.get("ld", 64), None))):
        for bad in (dict(x=None), dict(c=None), dict(s=None), dict(rows=0), dict(n=0), dict(n=-32),
                    dict(x=p + 4), dict(c=p + 8), dict(ld=63), dict(ld=65), dict(ld=0), dict(ld=-64)):
            assert fn(*a(**bad)) == -1, bad
        for bad in (dict(n=40), dict(dt=3), dict(dt=-1), dict(rows=(1 << 30) + 1)):
            assert fn(*a(**bad)) == -2, bad
    assert d(p, p, 2, 64, p, 2, 64, None) == -2           # fp16 values
    assert q(p, 1, 68, 2, 64, p, p, None) == -1           # 136 bytes between bf16 rows


def test_mm_host_checks():
    p = 1 << 20
    names = ["w", "ws", "n", "k", "off", "E", "a", "as_", "n_act", "src", "K", "rows", "epi", "out",
             "outs", "stream"]
    ok = [p, p, 64, 256, p, 4, p, p, 8, None, 1, 8, 0, p, None, None]

    def call(**kw):
        a = list(ok)
        for k, v in kw.items():
            a[names.index(k)] = v
        return abi.lib().moe_mxfp4_mm_grouped(*a)

    for bad in (dict(w=None), dict(ws=None), dict(off=None), dict(a=None), dict(as_=None),
                dict(out=None), dict(n=0), dict(k=0), dict(E=0), dict(rows=0), dict(n_act=0),
                dict(src=p, K=0), dict(epi=3), dict(epi=-1), dict(epi=2), dict(rows=9), dict(w=p + 8),
                dict(a=p + 4), dict(ws=p + 2), dict(as_=p + 1), dict(out=p + 8)):
        assert call(**bad) == -1, bad
    for bad in (dict(n=48), dict(k=192), dict(E=2049), dict(n=32 << 16),
                dict(rows=1 << 28, n_act=1 << 28), dict(src=p, K=65), dict(n=1 << 20, k=1 << 13),
                dict(n=1 << 19, k=1 << 13, epi=2, outs=p), dict(n_act=1 << 25, k=256),
                dict(rows=1 << 27, n_act=1 << 27, k=128, n=1 << 14)):
        assert call(**bad) == -2, bad


def test_combine_and_balance_host_checks():
    L, p = abi.lib(), 1 << 20
    assert L.moe_combine_bf16(None, p, p, 2, 2, 64, p, None) == -1
    assert L.moe_combine_bf16(p, p, p, 0, 2, 64, p, None) == -1
    assert L.moe_combine_bf16(p + 2, p, p, 2, 2, 64, p, None) == -1
    assert L.moe_combine_bf16(p, p, p, 2, 2, 60, p, None) == -2
    assert L.moe_combine_bf16(p, p, p, 2, 65, 64, p, None) == -2
    assert L.moe_combine_bf16(p, p, p, (1 << 23) + 1, 1, 64, p, None) == -2
    size = abi.balance_workspace_size(100, 64)
    assert size > 0 and abi.balance_workspace_size(0, 64) == 0
    assert abi.balance_workspace_size(100, 2049) == 0

    def fwd(lg=p, dt=0, ld=64, T=100, E=64, idx=p, K=4, c=p, pm=p, lo=p, ws=p, nb=size):
        return L.moe_balance_loss(lg, dt, ld, T, E, idx, K, None, c, pm, lo, ws, nb, None)

    def bwd(lg=p, dt=0, ld=64, T=100, E=64, c=p, K=4, g=p, ldg=64):
        return L.moe_balance_loss_backward(lg, dt, ld, T, E, c, K, None, None, g, ldg, None)

    for bad in (dict(lg=None), dict(idx=None), dict(c=None), dict(pm=None), dict(lo=None),
                dict(ws=None), dict(T=0), dict(E=0), dict(K=0), dict(K=65), dict(ld=63),
                dict(lg=p + 2), dict(ws=p + 1)):
        assert fwd(**bad) == -1, bad
    assert fwd(dt=3) == -2 and fwd(E=2049, ld=4096) == -2 and fwd(E=128, ld=128, K=65) == -2
    assert fwd(nb=size - 1) == -3
    for bad in (dict(lg=None), dict(c=None), dict(g=None), dict(T=0), dict(K=65), dict(ld=63),
                dict(ldg=63), dict(g=p + 1)):
        assert bwd(**bad) == -1, bad
    assert bwd(dt=5) == -2 and bwd(E=2049, ld=4096, ldg=4096) == -2


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64)
    c, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    for call in (lambda: abi.mxfp4_quantize(x, c, s), lambda: abi.mxfp4_dequantize(c, s, x),
                 lambda: abi.mxfp4_mm_grouped(torch.zeros(2, 32, 64, dtype=torch.uint8), c, c, c, s, x),
                 lambda: abi.combine_bf16(x.bfloat16(), c, x[:, :1], x),
                 lambda: abi.balance_loss(x, torch.zeros(4, 2, dtype=torch.int32), c, c, c, c),
                 lambda: abi.balance_loss_backward(x, c, 2, x)):
        with pytest.raises(ValueError):
            call()
