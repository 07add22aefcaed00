"""The router's balance loss, counts and gradient on the GPU against the 64-bit reference."""
import numpy as np
import pytest
import torch

import mxref
from gpu_util import dev, empty, host, note
from quantized_expert_grouped_amd import abi

pytestmark = pytest.mark.gpu

DT = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
TINY = {"float32": 2.0 ** -149, "bfloat16": 2.0 ** -133, "float16": 2.0 ** -24}


def case(T, E, K, valid, seed, spread=1.0):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((T, E)) * spread).astype(np.float32)
    idx = np.argsort(-(x + np.linspace(0, 2, E)), 1)[:, :K].astype(np.int32)
    v = None
    if valid == "some":
        v = (rng.random(T) < 0.7).astype(np.uint8) * rng.integers(1, 256, T).astype(np.uint8)
        v[0] = 0
    elif valid == "none":
        v = np.zeros(T, np.uint8)
    return x, idx, v


def run(xt, idx, v, g=None, grad=None):
    T, E = xt.shape
    K = idx.shape[1]
    counts = torch.full((E + 4,), -5, dtype=torch.int32, device="cuda")
    prob, loss = torch.full((E + 3,), -5.0, device="cuda"), torch.full((4,), -5.0, device="cuda")
    ws = empty(abi.balance_workspace_size(T, E), torch.uint8)
    ws.fill_(0xEE)
    vt = None if v is None else dev(v)
    if grad is None:
        grad = torch.empty_like(xt)
    note(f"balance T={T} E={E} K={K} {xt.dtype}")
    abi.balance_loss(xt, dev(idx), counts[:E + 1], prob[:E], loss[:1], ws, valid=vt)
    gt = None if g is None else torch.full((1,), g, device="cuda")
    abi.balance_loss_backward(xt, counts[:E + 1], K, grad, valid=vt, grad_loss=gt)
    torch.cuda.synchronize()
    assert bool((counts[E + 1:] == -5).all()) and bool((prob[E:] == -5).all()) and bool((loss[1:] == -5).all())
    return counts[:E + 1], prob[:E], loss[:1], grad


def check(xt, idx, v, dtype, g, got):
    T, E = xt.shape
    K = idx.shape[1]
    x = xt.double().cpu().numpy()
    counts, prob, loss, grad, p, f = mxref.balance(x, idx, v)
    n = max(int(counts[E]), 1)
    assert np.array_equal(host(got[0]), counts)
    # a probability: 2^t within 2 ulp, t = d log2 e of a rounded difference d by a rounded constant
    # (each a relative 2^-24 of t at most, the constant's a quarter of that: 2.25 |d| 2^-24 of the
    # power), the sum of E terms over a lane's E / 64 and 6 steps across lanes, the quotient, the
    # product
    on = np.ones(T, bool) if v is None else v != 0
    fin = np.isfinite(x) & on[:, None]
    d = np.where(fin, np.where(fin, x, -1e300).max(1, keepdims=True) - np.where(fin, x, 0.0), 0.0)
    eps = (2.25 * np.minimum(d, 150) + E / 64 + 16) * 2.0 ** -24
    eps = eps + (p * eps).sum(1, keepdims=True)      # the sum's own terms carry theirs
    tiny = 2.0 ** -126                               # smaller exponentials may be flushed
    dp = p * eps + tiny
    # a column's sum: at most T / groups / 16 + 16 + 256 / 8 + 8 additions of positive terms, and 1
    # / n
    adds = T / min(T, 256) / 16 + 60
    dprob = dp.sum(0) / n + prob * adds * 2.0 ** -24
    assert np.all(np.abs(host(got[1]) - prob) <= dprob)
    dl = E * float(f @ dprob) + loss * (E / 256 + 24) * 2.0 ** -24
    assert abs(float(host(got[2])[0]) - loss) <= dl + 2.0 ** -126
    # gradient: p (f_j - 1/E - sum p (f - 1/E)); f - 1/E to 8 roundings
    dev_f = f - 1.0 / E
    dot_abs = (p * np.abs(dev_f)).sum(1, keepdims=True)
    err = p * (np.abs(dev_f) + dot_abs) * (eps + (p * eps).sum(1, keepdims=True) + (E / 64 + 24) * 2.0 ** -24)
    err = err + tiny * (np.abs(dev_f) + dot_abs)
    want = grad(g)
    tol = abs(g) * E / n * err
    tol = tol + HALF[dtype] * (np.abs(want) + tol) + TINY[dtype]
    gr = got[3].double().cpu().numpy()
    assert np.all(np.abs(gr - want) <= tol)
    assert np.all(gr[~on] == 0)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,E,K,valid", [
    (1, 1, 1, "all"), (1, 512, 10, "all"), (2, 2, 1, "all"), (5, 3, 2, "some"), (16, 64, 8, "all"),
    (17, 65, 64, "some"), (100, 200, 6, "some"), (257, 512, 10, "all"), (300, 2048, 4, "some"),
    (5000, 128, 4, "some"), (1030, 1000, 2, "all"), (4100, 8, 2, "some"), (33, 60, 3, "none")])
def test_balance(T, E, K, valid, dtype):
    x, idx, v = case(T, E, K, valid, T + E)
    g = 37.5 if T > 1 else -2.0
    xt = dev(x).to(DT[dtype])
    check(xt, idx, v, dtype, g, run(xt, idx, v, g))


@pytest.mark.parametrize("dtype,E,pad", [("float32", 96, 5), ("bfloat16", 96, 1), ("float32", 130, 2),
                                         ("float16", 256, 8), ("bfloat16", 64, 4)])
def test_balance_rows_apart_and_in_place(dtype, E, pad):
    """Rows of logits and of the gradient with gaps, an unaligned first row, and the gradient written over
    the logits: what lies between the rows keeps its values."""
    T, K = 77, 3
    x, idx, v = case(T, E, K, "some", E)
    whole = torch.full((T + 1, E + pad), 9.0, device="cuda", dtype=DT[dtype])
    xt = whole.view(-1)[1:1 + T * (E + pad)].view(T, E + pad)[:, :E]
    xt.copy_(dev(x))
    gw = torch.full((T, E + 3), 9.0, device="cuda", dtype=DT[dtype])
    got = run(xt, idx, v, 2.0, gw[:, :E])
    check(xt, idx, v, dtype, 2.0, got)
    assert bool((gw[:, E:] == 9.0).all())
    first = gw[:, :E].clone()
    run(xt, idx, v, 2.0, xt)
    assert torch.equal(xt, first)
    assert int((whole == 9.0).sum()) >= whole.numel() - T * E


def test_balance_masked_logits_and_stray_values():
    """-inf logits, rows of nothing else, the type's lowest value, NaN and inf in rows that are not valid,
    ids outside [0, E), the same id twice, wide logits."""
    T, E, K = 60, 130, 4
    x, idx, _ = case(T, E, K, "all", 8, spread=30.0)
    v = np.ones(T, np.uint8)
    x[3] = -np.inf
    x[4, 1:] = -np.inf
    x[5, ::2] = -np.inf
    x[6] = np.finfo(np.float32).min
    x[7, 5:] = np.finfo(np.float32).min
    x[8], v[8] = np.nan, 0
    x[9, 3], v[9] = np.inf, 0
    idx[10] = [-1, E, 2 ** 31 - 1, 7]
    idx[11] = 5
    xt = dev(x)
    check(xt, idx, v, "float32", 3.0, run(xt, idx, v, 3.0))


def test_gradient_against_differences_of_the_loss():
    """Central differences of the reference's loss (counts fixed) at the GPU's own logits."""
    T, E, K, step = 12, 20, 2, 1e-4
    x, idx, v = case(T, E, K, "some", 11)
    got = run(dev(x), idx, v, None)
    gr = host(got[3]).astype(np.float64)
    for t in range(T):
        for j in range(0, E, 3):
            d = np.zeros((T, E))
            d[t, j] = step
            diff = (mxref.balance(x + d, idx, v)[2] - mxref.balance(x - d, idx, v)[2]) / (2 * step)
            # a third derivative of p is at most p, times f E / n: 8 * step^2 bounds it, besides
            # fp32
            assert abs(diff - gr[t, j]) <= 8 * step ** 2 + 1e-6


def test_balance_repeats_bit_for_bit():
    x, idx, v = case(3000, 512, 10, "some", 2)
    xt = dev(x)
    a = run(xt, idx, v, 1.0)
    for _ in range(3):
        for p, q in zip(a, run(xt, idx, v, 1.0)):
            assert torch.equal(p, q)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("E", [3, 64, 130, 512])
def test_balance_of_a_valid_row_without_a_softmax_is_nan(E, dtype):
    """A NaN among the logits, nothing but NaN, NaN among -inf, +inf: the loss, every mean and that row's
    gradient are NaN, the counts and the other rows' gradients as without it."""
    T, K = 20, 2
    x, idx, v = case(T, E, K, "all", 3 * E)
    clean = run(dev(x).to(DT[dtype]), idx, v, 2.0)
    for kind in range(4):
        y = x.copy()
        if kind == 0:
            y[7, E // 2] = np.nan
        elif kind == 1:
            y[7] = np.nan
        elif kind == 2:
            y[7] = -np.inf
            y[7, E - 1] = np.nan
        else:
            y[7, 0] = np.inf
        counts, prob, loss, grad = run(dev(y).to(DT[dtype]), idx, v, 2.0)
        assert torch.equal(counts, clean[0])
        assert bool(prob.isnan().all()) and bool(loss.isnan().all())
        assert bool(grad[7].isnan().all())
        rest = torch.arange(T, device="cuda") != 7
        assert torch.equal(grad[rest], clean[3][rest])


@pytest.mark.parametrize("gap", [False, True])
def test_balance_of_more_rows_than_the_wavefronts_see_at_once(gap):
    """More than 64 rows to each of the largest grid's wavefronts, all valid and with runs of invalid rows
    that are longer than what one wavefront looks ahead."""
    T, E, K = 2 * 64 * 4096 + 777, 4, 2
    x, idx, _ = case(T, E, K, "all", 21)
    v = None
    if gap:
        v = np.zeros(T, np.uint8)
        v[5::7001] = 1
        v[-700:] = 255
        v[70000:70100] = 3
    xt = dev(x)
    check(xt, idx, v, "float32", 1e3, run(xt, idx, v, 1e3))
