"""The grouped 16-bit product and its gradients on the GPU against the definitions in 64 bits, within the
rounding of fp32 sums and one rounding of the result."""
import numpy as np
import pytest
import torch

from gpu_util import dev, note
from quantized_expert_grouped_amd import abi
from trainref import (DT, Routes, grouped, guarded, matrix, sum_bound, swiglu, swiglu_grad, untouched, weight_grad,
                      within)

pytestmark = pytest.mark.gpu

HALVES = ["bfloat16", "float16"]
# T, K, E, N, k, gather, skew, padded share, gap between rows
SHAPES = [
    (1, 1, 1, 8, 8, False, 0.0, 0.0, 0), (1, 2, 8, 64, 256, True, 0.0, 0.0, 0), (3, 1, 2, 96, 72, True, 0.0, 0.0, 8),
    (5, 3, 40, 160, 2048, True, 0.0, 0.0, 0), (1, 10, 512, 64, 1032, True, 0.0, 0.0, 0),
    (33, 1, 1, 224, 640, True, 0.0, 0.2, 16), (130, 4, 16, 256, 512, True, 0.7, 0.0, 0),
    (300, 1, 3, 288, 904, False, 1.5, 0.1, 8), (257, 6, 64, 64, 1000, True, 0.2, 0.0, 0),
    (64, 8, 2048, 32, 136, True, 0.0, 0.0, 0), (700, 2, 3, 520, 264, True, 3.0, 0.05, 0),
    (1000, 1, 1, 384, 1160, False, 0.0, 0.0, 24), (2500, 2, 9, 136, 648, False, 0.4, 0.3, 0),
    (900, 1, 1, 1032, 64, False, 0.0, 0.0, 0), (2100, 1, 1, 520, 2056, True, 0.0, 0.0, 8),
    (513, 4, 5, 768, 328, True, 0.5, 0.0, 0), (40, 2, 3, 64, 64, True, 0.0, 1.0, 0),
    # more experts than lanes in the tiles of each size; workgroups that walk through several tiles; parts of
    # an expert's rows; tiles of more rows than one
    (2000, 4, 300, 72, 200, True, 0.3, 0.0, 0), (3000, 4, 130, 264, 136, True, 0.2, 0.1, 8),
    (1600, 4, 64, 1024, 1032, True, 0.5, 0.1, 0), (1600, 4, 64, 1032, 1024, False, 0.5, 0.1, 0),
    (6000, 2, 3, 328, 200, True, 0.6, 0.0, 0), (5000, 1, 1, 2056, 264, False, 0.0, 0.0, 0),
]


class Case:
    def __init__(self, dtype, T, K, E, N, k, gather, skew, pad, gap):
        self.r = r = Routes(T, K, E, T + N + k, skew, pad)
        self.rng = np.random.default_rng(T * 7 + N)
        self.dtype, self.gap, self.N, self.k = DT[dtype], gap, N, k
        self.a = matrix(self.rand(T if gather else r.R, k), gap)
        if not gather:
            self.a[r.live:] = float("nan")                      # rows behind the last expert's
        self.src = r.src if gather else None
        self.rows = self.a[r.token] if gather else self.a[:r.live]   # what each live row reads
        self.kw = dict(src=self.src, K=K)
        note(f"{dtype} T={T} K={K} E={E} N={N} k={k} gather={gather} live={r.live}")

    def rand(self, *shape):
        return dev(self.rng.standard_normal(shape).astype(np.float32)).to(self.dtype)

    def weights(self, E, N, k):
        return (self.rand(E, N, k).float() / k ** 0.5).to(self.dtype)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("T,K,E,N,k,gather,skew,pad,gap", SHAPES)
def test_product(dtype, T, K, E, N, k, gather, skew, pad, gap):
    c = Case(dtype, T, K, E, N, k, gather, skew, pad, gap)
    r, w = c.r, c.weights(E, N, k)
    bias = c.rand(E, N)
    y, s = grouped(r, c.rows, w)
    tol = sum_bound(k, s)
    per_row = bias.double()[torch.repeat_interleave(torch.arange(E, device="cuda"), r.offsets.diff().long())]
    for odtype in (c.dtype, torch.float32):
        whole, out = guarded(r.R, N, odtype, gap)
        abi.mm_grouped(w, r.offsets, c.a, out, **c.kw)
        within(out[:r.live], y, tol)
        assert untouched(whole, out, r.live)
        res = matrix(c.rand(r.R, N).to(odtype), gap)
        full = y + per_row + res[:r.live].double()
        whole, both = guarded(r.R, N, odtype, gap)
        abi.mm_grouped(w, r.offsets, c.a, both, bias=bias, residual=res, **c.kw)
        within(both[:r.live], full, tol + 2 * 2.0 ** -24 * (s + per_row.abs() + res[:r.live].double().abs()))
        assert untouched(whole, both, r.live)
        over = matrix(res, gap)                                  # onto the residual itself
        abi.mm_grouped(w, r.offsets, c.a, over, bias=bias, residual=over, **c.kw)
        assert torch.equal(over[:r.live], both[:r.live])


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("T,K,E,N,k,gather,skew,pad,gap", SHAPES)
def test_swiglu_product(dtype, T, K, E, N, k, gather, skew, pad, gap):
    c = Case(dtype, T, K, E, N, k, gather, skew, pad, gap)
    r, w = c.r, c.weights(E, 2 * N, k)
    for bias in (None, c.rand(E, 2 * N)):
        y, s = grouped(r, c.rows, w)
        tol = sum_bound(k, s)
        if bias is not None:
            per_row = bias.double()[torch.repeat_interleave(torch.arange(E, device="cuda"), r.offsets.diff().long())]
            y, tol = y + per_row, tol + 2.0 ** -24 * (s + per_row.abs())
        h, dh = swiglu(y[:, :N], y[:, N:], tol[:, :N], tol[:, N:])
        whole, out = guarded(r.R, N, c.dtype, gap)
        zw, z = guarded(r.R, 2 * N, c.dtype, gap)
        abi.mm_grouped(w, r.offsets, c.a, out, bias=bias, swiglu=True, z=z, **c.kw)
        within(z[:r.live], y, tol)
        within(out[:r.live], h, dh)
        assert untouched(whole, out, r.live) and untouched(zw, z, r.live)
        alone = guarded(r.R, N, c.dtype, gap)[1]
        abi.mm_grouped(w, r.offsets, c.a, alone, bias=bias, swiglu=True, **c.kw)
        assert torch.equal(alone[:r.live], out[:r.live])


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("T,K,E,N,k,gather,skew,pad,gap", SHAPES)
def test_input_gradient(dtype, T, K, E, N, k, gather, skew, pad, gap):
    c = Case(dtype, T, K, E, N, k, gather, skew, pad, gap)
    r, w = c.r, c.weights(E, N, k)
    g = matrix(c.rand(r.R, N), gap)
    g[r.live:] = float("nan")
    y, s = grouped(r, g[:r.live], w.transpose(1, 2))
    tol = sum_bound(N, s)
    for odtype in (c.dtype, torch.float32):
        whole, out = guarded(r.R, k, odtype, gap)
        abi.mm_grouped_dgrad(w, r.offsets, g, out)
        within(out[:r.live], y, tol)
        assert untouched(whole, out, r.live)
    z = matrix((c.rand(r.R, 2 * k).float() * 4).to(c.dtype), gap)
    zl = z[:r.live].double()
    dg, eg, du, eu = swiglu_grad(y, zl[:, :k], zl[:, k:], tol)
    whole, out = guarded(r.R, 2 * k, c.dtype, gap)
    abi.mm_grouped_dgrad(w, r.offsets, g, out, z=z)
    within(out[:r.live, :k], dg, eg)
    within(out[:r.live, k:], du, eu)
    assert untouched(whole, out, r.live)
    abi.mm_grouped_dgrad(w, r.offsets, g, z, z=z)                # over z itself
    assert torch.equal(z[:r.live], out[:r.live])


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("T,K,E,N,k,gather,skew,pad,gap", SHAPES)
def test_weight_gradient(dtype, T, K, E, N, k, gather, skew, pad, gap):
    c = Case(dtype, T, K, E, N, k, gather, skew, pad, gap)
    r = c.r
    g = matrix(c.rand(r.R, N), gap)
    g[r.live:] = float("nan")
    y, s = weight_grad(r, g[:r.live], c.rows)
    counts = r.offsets.diff().double()
    tol = sum_bound(counts.view(-1, 1, 1), s)
    b, sb = weight_grad(r, g[:r.live], torch.ones(r.live, 1, device="cuda"))
    size = abi.mm_grouped_wgrad_workspace_size(r.R, N, k, E)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") if size else None
    for odtype in (c.dtype, torch.float32):
        whole, out = guarded(E * N, k, odtype)
        bw, gb = guarded(E, N, odtype)
        abi.mm_grouped_wgrad(g, r.offsets, c.a, out.view(E, N, k), ws, grad_bias=gb, **c.kw)
        within(out.view(E, N, k), y, tol)
        within(gb, b[..., 0], sum_bound(counts.view(-1, 1), sb[..., 0]))
        assert untouched(whole, out) and untouched(bw, gb)
        alone = guarded(E * N, k, odtype)[1]
        abi.mm_grouped_wgrad(g, r.offsets, c.a, alone.view(E, N, k), ws, **c.kw)
        assert torch.equal(alone, out)


def test_gradients_against_differences():
    """The product is linear in its rows and weights: whole steps change it by the gradients but for the
    rounding of fp32 sums.  Small whole numbers, so every sum is exact."""
    r = Routes(70, 2, 5, 3, 0.5)
    rng = np.random.default_rng(3)
    N, k = 40, 56

    def ints(*shape):
        return dev(rng.integers(-3, 4, shape).astype(np.float32)).bfloat16()

    w, a, g, v, u = ints(5, N, k), ints(70, k), ints(r.R, N), ints(5, N, k), ints(70, k)

    def loss(a, w):
        out = torch.empty(r.R, N, device="cuda")
        abi.mm_grouped(w, r.offsets, a, out, src=r.src, K=2)
        return float((out.double() * g.double()).sum())

    rows, token, grad_w = (torch.empty(s, device="cuda") for s in ((r.R, k), (70, k), (5, N, k)))
    abi.mm_grouped_dgrad(w, r.offsets, g, rows)
    abi.combine_rows(rows, r.slot, None, token)
    ws = torch.empty(abi.mm_grouped_wgrad_workspace_size(r.R, N, k, 5), dtype=torch.uint8, device="cuda")
    abi.mm_grouped_wgrad(g, r.offsets, a, grad_w, ws, src=r.src, K=2)
    assert loss(a + u, w) - loss(a - u, w) == 2 * float((token.double() * u.double()).sum())
    assert loss(a, w + v) - loss(a, w - v) == 2 * float((grad_w.double() * v.double()).sum())


def test_swiglu_gradient_against_differences():
    """Of 64-bit arithmetic: the identity as weights, so that the product's rows are z's SwiGLU."""
    n = 64
    rng = np.random.default_rng(5)
    offsets = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
    w = torch.eye(n, device="cuda").bfloat16().unsqueeze(0)
    z = dev((6 * rng.standard_normal((300, 2 * n))).astype(np.float32)).bfloat16()
    g = dev(rng.standard_normal((300, n)).astype(np.float32)).bfloat16()
    out = torch.empty_like(z)
    abi.mm_grouped_dgrad(w, offsets, g, out, z=z)

    def f(z):
        return z[:, :n] * torch.sigmoid(z[:, :n]) * z[:, n:]

    h = 2.0 ** -10
    for half in (0, 1):
        step = torch.zeros(1, 2 * n, dtype=torch.float64, device="cuda")
        step[:, half * n:(half + 1) * n] = h
        d = (f(z.double() + step) - f(z.double() - step)) / (2 * h) * g.double()
        # |silu'''| < 1: h^2 / 6 of the up's, and fp32's part, far below bf16's half step
        tol = (h * h / 6 + 2.0 ** -18) * (1 + z.double()[:, n:].abs()) * (1 + z.double()[:, :n].abs()) * g.double().abs()
        within(out[:, half * n:(half + 1) * n], d, tol)


@pytest.mark.parametrize("dtype", HALVES)
def test_gates_from_one_end_to_the_other(dtype):
    """silu and its gradient where the exponential runs out of range: no NaN, and the limits' values."""
    n = 512
    g = torch.linspace(-120, 120, n, device="cuda").to(DT[dtype])
    one = torch.ones(1, 8, device="cuda", dtype=DT[dtype])
    offsets = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    w = torch.zeros(1, 2 * n, 8, device="cuda", dtype=DT[dtype])
    w[0, :n, 0], w[0, n:, 1] = g, 1.0
    out, z = torch.empty(1, n, device="cuda", dtype=DT[dtype]), torch.empty(1, 2 * n, device="cuda", dtype=DT[dtype])
    abi.mm_grouped(w, offsets, one, out, swiglu=True, z=z)
    assert torch.equal(z[0, :n], g)
    y = g.double().unsqueeze(0)
    zero = torch.zeros_like(y)
    within(out, *swiglu(y, torch.ones_like(y), zero, zero))
    eye = torch.eye(n, device="cuda").to(DT[dtype]).unsqueeze(0)
    back = torch.empty_like(z)
    abi.mm_grouped_dgrad(eye, offsets, torch.ones(1, n, device="cuda", dtype=DT[dtype]), back, z=z)
    dg, eg, du, eu = swiglu_grad(torch.ones_like(y), y, torch.ones_like(y), zero)
    within(back[:, :n], dg, eg)
    within(back[:, n:], du, eu)


@pytest.mark.parametrize("T,N,k", [(70, 64, 200), (3, 64, 200), (1500, 512, 264)])
def test_infinities_and_nans_stay_in_their_rows_and_columns(T, N, k):
    r = Routes(T, 2, 4, 8)
    rng = np.random.default_rng(8)
    a = dev(rng.standard_normal((T, k)).astype(np.float32)).bfloat16()
    w = dev(rng.standard_normal((4, N, k)).astype(np.float32)).bfloat16()
    a[1, 7], w[2, 5, 3] = float("nan"), float("inf")
    out = torch.zeros(r.R, N, device="cuda")
    abi.mm_grouped(w, r.offsets, a, out, src=r.src, K=2)
    expert = torch.repeat_interleave(torch.arange(4, device="cuda"), r.offsets.diff().long())
    bad = (r.token == 1).unsqueeze(1) | ((expert == 2).unsqueeze(1) & (torch.arange(N, device="cuda") == 5))
    assert torch.equal(~out.isfinite(), bad)
    g = dev(rng.standard_normal((r.R, N)).astype(np.float32)).bfloat16()
    g[0, 3] = float("inf")                                      # a row of the first expert that has some
    da = torch.zeros(r.R, k, device="cuda")
    abi.mm_grouped_dgrad(w, r.offsets, g, da)
    bad = torch.zeros_like(da, dtype=torch.bool)
    bad[0], bad[:, 3] = True, expert == 2
    bad[0] = True
    assert torch.equal(~da.isfinite(), bad)
    ws = torch.empty(abi.mm_grouped_wgrad_workspace_size(r.R, N, k, 4), dtype=torch.uint8, device="cuda")
    dw, db = torch.zeros(4, N, k, device="cuda"), torch.zeros(4, N, device="cuda")
    abi.mm_grouped_wgrad(g, r.offsets, a, dw, ws, src=r.src, K=2, grad_bias=db)
    bad = torch.zeros_like(dw, dtype=torch.bool)
    bad[expert[r.token == 1], :, 7] = True
    bad[expert[0], 3, :] = True
    assert torch.equal(~dw.isfinite(), bad)
    assert torch.equal(torch.nonzero(~db.isfinite()), torch.stack([expert[0], torch.tensor(3, device="cuda")]).unsqueeze(0))


def test_strays_read_the_nearest_row():
    """A src outside the activations stays in bounds."""
    offsets = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    a = torch.eye(8, device="cuda").bfloat16()[:3].contiguous()
    w = torch.eye(8, device="cuda").bfloat16().unsqueeze(0)
    src = torch.tensor([-5, 7, 2, 2 ** 30 - 1], dtype=torch.int32, device="cuda")
    out = torch.empty(4, 8, device="cuda")
    abi.mm_grouped(w, offsets, a, out, src=src, K=2)
    assert out.argmax(1).tolist() == [0, 2, 1, 2]
    dw = torch.empty(1, 8, 8, device="cuda")
    ws = torch.empty(abi.mm_grouped_wgrad_workspace_size(4, 8, 8, 1), dtype=torch.uint8, device="cuda")
    abi.mm_grouped_wgrad(torch.ones(4, 8, device="cuda").bfloat16(), offsets, a, dw, ws, src=src, K=2)
    assert dw[0, 0].tolist() == [1.0, 1.0, 2.0, 0, 0, 0, 0, 0]


def test_rows_past_31_bits():
    """Outputs and gradients whose bytes lie more than 4 GiB in: the last expert's rows."""
    rows, n = 300000, 8192                                       # 4.9 GB of bf16
    offsets = torch.tensor([0, 17, 17, rows - 300, rows], dtype=torch.int32, device="cuda")
    a = torch.zeros(rows, 8, device="cuda", dtype=torch.bfloat16)
    a[:, 0] = 1.0
    a[rows - 300:, 0] = torch.arange(300, device="cuda").remainder(7).bfloat16()
    w = torch.ones(4, n, 8, device="cuda", dtype=torch.bfloat16)
    out = torch.empty(rows, n, device="cuda", dtype=torch.bfloat16)
    abi.mm_grouped(w, offsets, a, out)
    assert torch.equal(out[::1001], a[::1001, :1].expand(-1, n))
    assert torch.equal(out[rows - 300:], a[rows - 300:, :1].expand(-1, n))
    back = torch.empty(rows, 8, device="cuda")
    abi.mm_grouped_dgrad(w, offsets, out, back)
    assert torch.equal(back, (n * a[:, :1].float()).expand(-1, 8))
    dw, db = torch.empty(4, n, 8, device="cuda"), torch.empty(4, n, device="cuda")
    ws = torch.empty(abi.mm_grouped_wgrad_workspace_size(rows, n, 8, 4), dtype=torch.uint8, device="cuda")
    abi.mm_grouped_wgrad(out, offsets, a, dw, ws, grad_bias=db)
    last = a[rows - 300:, 0].double()
    want = [17.0, 0.0, float(rows - 317), float((last * last).sum())]
    assert [dw[e, 5].tolist() for e in range(4)] == [[v] + [0.0] * 7 for v in want]
    assert db[:, n - 1].tolist() == [17.0, 0.0, float(rows - 317), float(last.sum())]


# int32's ends among the routes, with rows enough for the few-rows kernel and for the tiles of each size;
# the last: weight gradients in 256 x 256 tiles with the rows in parts
STRAYS = [2 ** 31 - 1, 2 ** 30, 2 ** 30 - 1, -1, -2 ** 31, 7, 0, 2 ** 31 - 2, 1]


@pytest.mark.parametrize("K", [1, 3, 32, 64])
@pytest.mark.parametrize("rows,N,k", [(9, 64, 264), (400, 2056, 264), (4500, 2056, 264), (9000, 2056, 264), (3000, 2048, 2048)])
def test_strays_of_every_size_read_the_nearest_row(rows, N, k, K):
    n_act = 5
    rng = np.random.default_rng(rows + K)
    offsets = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    a = dev(rng.integers(-3, 4, (n_act, k)).astype(np.float32)).bfloat16()
    w = dev(rng.integers(-3, 4, (1, 2 * N, k)).astype(np.float32)).bfloat16()
    route = np.resize(np.array(STRAYS, np.int64), rows)
    route[::5] = rng.integers(0, n_act * K, len(route[::5]))
    row = dev(np.clip(route, 0, None) // K).clamp(max=n_act - 1)
    src = dev(route.astype(np.int32))
    note(f"strays rows={rows} N={N} k={k} K={K}")
    out, z = torch.empty(rows, N, device="cuda"), torch.empty(rows, 2 * N, device="cuda", dtype=torch.bfloat16)
    abi.mm_grouped(w[:, :N].contiguous(), offsets, a, out, src=src, K=K)
    want = a.double()[row] @ w[0].double().t().contiguous()       # whole numbers: sums are exact
    assert torch.equal(out.double(), want[:, :N])
    abi.mm_grouped(w, offsets, a, torch.empty(rows, N, device="cuda", dtype=torch.bfloat16), src=src, K=K, swiglu=True, z=z)
    assert torch.equal(z, want.bfloat16())
    g = dev(rng.integers(-3, 4, (rows, N)).astype(np.float32)).bfloat16()
    size = abi.mm_grouped_wgrad_workspace_size(rows, N, k, 1)
    ws, dw = torch.empty(size, dtype=torch.uint8, device="cuda"), torch.empty(1, N, k, device="cuda")
    abi.mm_grouped_wgrad(g, offsets, a, dw, ws, src=src, K=K)
    assert torch.equal(dw[0].double(), g.double().t().contiguous() @ a.double()[row])


@pytest.mark.parametrize("rows", [1, 300])
def test_gradients_of_large_gates_and_ups(rows):
    """Finite gates, ups and gradients whose product without the sigmoid leaves fp32's range: the gradient is
    finite wherever the definition's is, and 0 far on the negative side."""
    gates = [-3e38, -1e36, -1e20, -200.0, -89.0, -86.0, -80.0, -40.0, -3.0, 0.0, 3.0, 90.0, 1e4, -1e37, 5.0, -87.0]
    ups = [1.0, -1e36, 3e38, 1e-3]
    n = len(gates) * len(ups)
    z = torch.empty(rows, 2 * n, device="cuda", dtype=torch.bfloat16)
    z[:, :n] = torch.tensor(gates, device="cuda").repeat_interleave(len(ups)).bfloat16()
    z[:, n:] = torch.tensor(ups, device="cuda").repeat(len(gates)).bfloat16()
    w = torch.eye(n, device="cuda").bfloat16().unsqueeze(0)
    offsets = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    for d in (1e4, 1e38, -1e-4):
        grad = torch.full((rows, n), d, device="cuda").bfloat16()
        out = torch.empty_like(z)
        note(f"large gates rows={rows} d={d}")
        abi.mm_grouped_dgrad(w, offsets, grad, out, z=z)
        g, u = z[:, :n].double(), z[:, n:].double()
        dg, eg, du, eu = swiglu_grad(grad.double(), g, u, torch.zeros_like(g))
        top = float(torch.finfo(torch.bfloat16).max)
        for got, want, err in ((out[:, :n], dg, eg), (out[:, n:], du, eu)):
            fits = want.abs() + err < top / 2
            within(got[fits], want[fits], err[fits])
            assert bool((got[g < -100] == 0).all()) and not bool(got.isnan().any())
        assert 2 * int(fits.sum()) > fits.numel()


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("rows", [400, 17000, 33000])
def test_gates_from_one_end_to_the_other_in_the_tiles(rows, dtype):
    """As for one row, through the tiles' own epilogues: 128 x 128, forward in 256 x 256, both in 256 x 256."""
    n = 512
    g = torch.linspace(-120, 120, n, device="cuda").to(DT[dtype])
    one = torch.ones(rows, 8, device="cuda", dtype=DT[dtype])
    offsets = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    w = torch.zeros(1, 2 * n, 8, device="cuda", dtype=DT[dtype])
    w[0, :n, 0], w[0, n:, 1] = g, 1.0
    out, z = (torch.empty(rows, c, device="cuda", dtype=DT[dtype]) for c in (n, 2 * n))
    note(f"gates in tiles rows={rows} {dtype}")
    abi.mm_grouped(w, offsets, one, out, swiglu=True, z=z)
    assert bool((z[:, :n] == g).all()) and bool((z[:, n:] == 1).all())
    y = g.double().unsqueeze(0)
    zero = torch.zeros_like(y)
    within(out[:1], *swiglu(y, torch.ones_like(y), zero, zero))
    assert torch.equal(out, out[:1].expand_as(out))
    eye = torch.eye(n, device="cuda").to(DT[dtype]).unsqueeze(0)
    back = torch.empty_like(z)
    abi.mm_grouped_dgrad(eye, offsets, torch.ones(rows, n, device="cuda", dtype=DT[dtype]), back, z=z)
    dg, eg, du, eu = swiglu_grad(torch.ones_like(y), y, torch.ones_like(y), zero)
    within(back[:1, :n], dg, eg)
    within(back[:1, n:], du, eu)
    assert torch.equal(back, back[:1].expand_as(back))


# as SHAPES: 64 to 128 tiles of 256 x 256, so their rows come in parts
PARTS = [(1500, 2, 2, 2048, 1032, True, 0.0, 0.1, 8), (3000, 1, 1, 2056, 2048, True, 0.0, 0.0, 0),
         (4000, 2, 2, 1536, 1544, True, 2.0, 0.0, 0), (2100, 3, 3, 1032, 1800, False, 0.0, 0.2, 16),
         (3000, 1, 2, 1544, 1536, False, 4.0, 0.0, 0)]


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("T,K,E,N,k,gather,skew,pad,gap", PARTS)
def test_weight_gradient_in_parts_of_large_tiles(dtype, T, K, E, N, k, gather, skew, pad, gap):
    assert abi.mm_grouped_wgrad_workspace_size(T * K, N, k, E) > 0
    test_weight_gradient(dtype, T, K, E, N, k, gather, skew, pad, gap)
