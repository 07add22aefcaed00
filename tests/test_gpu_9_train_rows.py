"""Rows to the experts and back with their gradients, and the routing weights' gradient, on the GPU against
the definitions in 64 bits."""
import numpy as np
import pytest
import torch

from gpu_util import dev, note
from quantized_expert_grouped_amd import abi
from trainref import DT, Routes, guarded, matrix, untouched, within

pytestmark = pytest.mark.gpu

# T, K, E, H, gap and first value of the rows, padded share
SHAPES = [(1, 1, 1, 1, 0, 0, 0.0), (1, 10, 16, 2048, 0, 0, 0.0), (3, 2, 4, 7, 1, 1, 0.0), (17, 10, 64, 2048, 0, 0, 0.0),
          (61, 3, 8, 1001, 0, 0, 0.3), (40, 1, 5, 512, 8, 8, 0.5), (33, 64, 70, 65, 3, 5, 0.2), (5, 9, 12, 8200, 0, 0, 0.0),
          (700, 4, 32, 264, 24, 0, 0.1), (9, 17, 40, 20000, 0, 4, 0.0), (12, 2, 3, 513, 7, 3, 1.0)]


def rand(rng, dtype, *shape):
    return dev(rng.standard_normal(shape).astype(np.float32)).to(DT[dtype])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,K,E,H,gap,first,pad", SHAPES)
def test_dispatch_bytes(dtype, T, K, E, H, gap, first, pad):
    r = Routes(T, K, E, T + H, pad=pad)
    x = matrix(rand(np.random.default_rng(H), dtype, T, H), gap, first)
    whole, out = guarded(r.R, H, DT[dtype], gap, first)
    note(f"dispatch {dtype} {T}x{H} K={K}")
    abi.dispatch_rows(x, r.src, out, K=K)
    assert torch.equal(out[:r.live], x[r.token])
    assert untouched(whole, out, r.live)


def test_dispatch_keeps_every_bit_and_skips_strays():
    bits = torch.arange(1 << 16, dtype=torch.int32, device="cuda").to(torch.int16).view(64, 1024)
    src = torch.arange(63, -1, -1, dtype=torch.int32, device="cuda") * 2
    src[5], src[6], src[7] = -1, 128, 2 ** 31 - 1
    for dtype in (torch.bfloat16, torch.float16):
        whole, out = guarded(64, 1024, dtype)
        abi.dispatch_rows(bits.view(dtype), src, out, K=2)
        got = out.view(torch.int16)
        keep = torch.ones(64, dtype=torch.bool, device="cuda")
        keep[5:8] = False
        assert torch.equal(got[keep], bits.flip(0)[keep])
        assert bool((out[5:8].contiguous().view(torch.uint8) == 0xAB).all())


@pytest.mark.parametrize("dtype,odtype", [("float32", "float32"), ("bfloat16", "bfloat16"), ("bfloat16", "float32"),
                                          ("float16", "float16"), ("float16", "float32")])
@pytest.mark.parametrize("T,K,E,H,gap,first,pad", SHAPES)
def test_combine_and_gradients(dtype, odtype, T, K, E, H, gap, first, pad):
    r = Routes(T, K, E, T + H, pad=pad)
    rng = np.random.default_rng(T * H)
    rows = matrix(rand(rng, dtype, r.R, H), gap, first)
    rows[r.live:] = float("nan")                     # rows that no route names
    w = dev(rng.standard_normal((T, K)).astype(np.float32))
    res, g = (matrix(rand(rng, odtype, T, H), gap, first) for _ in range(2))
    there = (r.slot >= 0).unsqueeze(-1)
    each = torch.where(there, rows.double()[r.slot.long().clamp(min=0)], 0.0)
    note(f"combine {dtype} -> {odtype} {T}x{H} K={K}")
    for weights, residual in ((w, res), (w, None), (None, None), (None, res)):
        c = (weights.double() if weights is not None else torch.ones_like(w).double()).unsqueeze(-1) * each
        whole, out = guarded(T, H, DT[odtype], gap, first)
        abi.combine_rows(rows, r.slot, weights, out, residual=residual)
        want, mags = c.sum(1), c.abs().sum(1)
        if residual is not None:
            want, mags = want + residual.double(), mags + residual.double().abs()
        within(out, want, (K + 1) * 2.0 ** -24 * mags)      # an fma each
        assert untouched(whole, out)
        if residual is not None:                            # onto the residual itself
            over = matrix(residual, gap, first)
            abi.combine_rows(rows, r.slot, weights, over, residual=over)
            assert torch.equal(over, out)
    note("combine backward")
    for weights in (w, None):
        whole, grad_rows = guarded(r.R, H, DT[dtype], gap, first)
        grad_w = torch.full((T, K), 7.0, device="cuda")
        abi.combine_rows_backward(g, r.slot, weights, grad_rows, rows=rows, grad_w=grad_w)
        wr = (weights if weights is not None else torch.ones_like(w)).double().view(-1)[r.src[:r.live].long()]
        within(grad_rows[:r.live], wr.unsqueeze(1) * g.double()[r.token],
               2.0 ** -24 * (wr.unsqueeze(1) * g.double()[r.token]).abs())
        assert untouched(whole, grad_rows, r.live)
        dots = g.double().unsqueeze(1) * each
        within(grad_w, dots.sum(-1), H * 2.0 ** -24 * dots.abs().sum(-1))
        assert bool((grad_w[r.slot < 0] == 0).all())
        only = torch.empty_like(grad_w)                     # each alone, and in place
        abi.combine_rows_backward(g, r.slot, weights, rows=rows, grad_w=only)
        assert torch.equal(only, grad_w)
        alone = guarded(r.R, H, DT[dtype], gap, first)[1]
        abi.combine_rows_backward(g, r.slot, weights, alone)
        assert torch.equal(alone[:r.live], grad_rows[:r.live])
        over = matrix(rows, gap, first)
        abi.combine_rows_backward(g, r.slot, weights, over, rows=over, grad_w=only.zero_())
        assert torch.equal(only, grad_w) and torch.equal(over[:r.live], grad_rows[:r.live])


def test_combine_of_infinities_and_nans():
    """They stay in the columns and tokens they are in; slots out of range are not looked at."""
    rows = torch.ones(6, 40, device="cuda", dtype=torch.bfloat16)
    rows[0, 3], rows[1, 4], rows[5] = float("inf"), float("nan"), float("nan")
    slot = torch.tensor([[0, 1], [2, 3], [4, 6], [-1, -(2 ** 31)], [2 ** 31 - 1, 2]], dtype=torch.int32, device="cuda")
    w = torch.full((5, 2), 0.5, device="cuda")
    out = torch.empty(5, 40, device="cuda")
    abi.combine_rows(rows, slot, w, out)
    want = torch.tensor([1.0, 1.0, 0.5, 0.0, 0.5], device="cuda").unsqueeze(1).repeat(1, 40)
    want[0, 3], want[0, 4] = float("inf"), float("nan")
    assert torch.equal(out.nan_to_num(7.0), want.nan_to_num(7.0))
    grad_w = torch.empty(5, 2, device="cuda")
    abi.combine_rows_backward(torch.ones(5, 40, device="cuda"), slot, w, rows=rows, grad_w=grad_w)
    assert grad_w[1:].tolist() == [[40.0, 40.0], [40.0, 0.0], [0.0, 0.0], [0.0, 40.0]]
    assert grad_w[0, 0].isinf() and grad_w[0, 1].isnan()


def test_gradients_against_differences():
    """The combine is linear in the rows and in the weights: steps of a power of two change it by the gradient
    but for fp32's rounding."""
    r = Routes(50, 3, 9, 4, pad=0.1)
    rng = np.random.default_rng(4)
    rows, w, g = rand(rng, "float32", r.R, 37), rand(rng, "float32", 50, 3), rand(rng, "float32", 50, 37)

    def loss(rows, w):
        out = torch.empty(50, 37, device="cuda")
        abi.combine_rows(rows, r.slot, w, out)
        return float((out.double() * g.double()).sum())

    grad_rows, grad_w = torch.zeros_like(rows), torch.empty_like(w)
    abi.combine_rows_backward(g, r.slot, w, grad_rows, rows=rows, grad_w=grad_w)
    scale = float((g.double().abs().sum()) * (1 + w.abs().max()) * (1 + rows.abs().max())) * 2.0 ** -22
    for _ in range(6):
        v, u = rand(rng, "float32", r.R, 37), rand(rng, "float32", 50, 3)
        d = loss(rows + v, w) - loss(rows - v, w)
        assert abs(d - 2 * float((grad_rows.double() * v.double())[:r.live].sum())) <= 8 * scale
        d = loss(rows, w + u) - loss(rows, w - u)
        assert abs(d - 2 * float((grad_w.double() * u.double()).sum())) <= 8 * scale


# ---- the routing weights' gradient --------------------------------------------------------------
ROUTES = [(1, 1, 1, 0), (1, 512, 10, 0), (5, 7, 7, 3), (61, 512, 10, 0), (300, 2048, 64, 0), (1000, 33, 2, 1), (4097, 128, 8, 8)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,E,K,gap", ROUTES)
def test_route_gradient(dtype, T, E, K, gap):
    rng = np.random.default_rng(T + E)
    idx = np.argsort(rng.standard_normal((T, E)), axis=1)[:, :K].astype(np.int32)
    idx[rng.random((T, K)) < 0.1] = -1
    idx[rng.random((T, K)) < 0.05] = E
    if K > 1 and T > 4:
        idx[3, 1] = idx[3, 0] = 2                              # an expert twice
    idx, gw = dev(idx), rand(rng, "float32", T, K)
    gw[(idx < 0) | (idx >= E)] = float("nan")                  # not looked at
    w = torch.softmax(rand(rng, "float32", T, K), 1)
    on = (idx >= 0) & (idx < E)
    g = torch.where(on, gw.double(), 0.0)
    mean, mags = (w.double() * g).sum(1, keepdim=True), (w.double() * g.abs()).sum(1, keepdim=True)
    each = torch.where(on, w.double() * (g - mean), 0.0)
    tol = torch.where(on, w.double() * ((K + 2) * 2.0 ** -24 * mags + 2 * 2.0 ** -24 * (g - mean).abs()), 0.0)
    want = torch.zeros(T, E + 1, dtype=torch.float64, device="cuda")
    err = torch.zeros_like(want)
    at = torch.where(on, idx.long(), E)
    want.scatter_add_(1, at, each)
    err.scatter_add_(1, at, tol + 2.0 ** -24 * each.abs())
    want, err = want[:, :E], err[:, :E]
    whole, grad = guarded(T, E, DT[dtype], gap, gap)
    note(f"route_topk_backward {dtype} {T}x{E} K={K}")
    abi.route_topk_backward(idx, w, gw, grad)
    within(grad, want, err)
    assert untouched(whole, grad)
    before = matrix(rand(rng, dtype, T, E), gap, gap)
    onto = matrix(before, gap, gap)
    abi.route_topk_backward(idx, w, gw, onto, accumulate=True)
    both = want + before.double()
    within(onto, both, err + 2.0 ** -24 * both.abs())


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("T,E,K,gap", ROUTES[2:5])
def test_route_gradient_weight_of_a_route_without_an_expert(T, E, K, gap, value):
    """Neither the weight nor its gradient of such a route is looked at: the same bits as with zeros."""
    rng = np.random.default_rng(T + E + 1)
    idx = np.argsort(rng.standard_normal((T, E)), axis=1)[:, :K].astype(np.int32)
    idx[rng.random((T, K)) < 0.2] = -1
    idx[rng.random((T, K)) < 0.1] = E
    idx[0, 0] = -1
    idx, gw, w = dev(idx), rand(rng, "float32", T, K), torch.softmax(rand(rng, "float32", T, K), 1)
    off = (idx < 0) | (idx >= E)
    got = []
    for v in (0.0, value):
        grad = torch.empty(T, E, device="cuda")
        note(f"route_topk_backward {T}x{E} K={K}, weights without an expert {v}")
        abi.route_topk_backward(idx, w.masked_fill(off, v), gw.masked_fill(off, v), grad)
        got.append(grad)
    assert bool(off.any()) and bool(torch.isfinite(got[0]).all())
    assert torch.equal(got[0], got[1])


def test_route_gradient_against_the_routers_differences():
    """Central differences of the library's own router: the loss is sum w c."""
    T, E, K = 40, 64, 6
    rng = np.random.default_rng(9)
    logits, c = rand(rng, "float32", T, E), rand(rng, "float32", T, K)

    def weights(x):
        idx, w = torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda")
        abi.route_topk(x, K, idx, w)
        return idx, w

    idx, w = weights(logits)
    grad = torch.empty(T, E, device="cuda")
    abi.route_topk_backward(idx, w, c, grad)
    h = 2.0 ** -8
    for k in range(K):                                          # step the k-th chosen logit of every token
        step = torch.zeros(T, E, device="cuda").scatter_(1, idx[:, k:k + 1].long(), h)
        (ia, wa), (ib, wb) = weights(logits + step), weights(logits - step)

        def by_id(i, v):                                        # the step may swap two picks
            return torch.zeros(T, E, dtype=torch.float64, device="cuda").scatter_(1, i.long(), v.double())

        same = (torch.sort(ia).values == torch.sort(ib).values).all(1)
        cost = by_id(idx, c)
        d = ((by_id(ia, wa) - by_id(ib, wb)) * cost).sum(1) / (2 * h)
        got = grad.gather(1, idx[:, k:k + 1].long())[:, 0].double()
        # the third derivative of a softmax is below 1 in magnitude: h^2 / 6 each; weights are off by 2^-22
        tol = c.double().abs().sum(1) * (h * h / 6 + 2.0 ** -22 / h) + 1e-6
        assert int(same.sum()) > T // 2 and bool(((d - got).abs() <= tol)[same].all())
