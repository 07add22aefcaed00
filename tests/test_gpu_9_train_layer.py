"""MoeTrainLayer: a run of the training operators as a program uses them, against 64-bit references stage by
stage and autograd as a whole; captured and replayed, on two streams, with padded tokens."""
import numpy as np
import pytest
import torch

from gpu_util import dev, note
from quantized_expert_grouped_amd import abi
from quantized_expert_grouped_amd.layer import MoeTrainLayer
from trainref import (DT, grouped, half_step, sum_bound, swiglu, swiglu_grad, weight_grad, within)

pytestmark = pytest.mark.gpu

# T, H, F, E, K, padded share: few rows an expert, tiles of 128, tiles of 256, odd sizes, one expert
SIZES = [(5, 256, 128, 64, 3, 0.0), (150, 264, 136, 8, 2, 0.2), (3000, 512, 768, 16, 4, 0.1), (700, 1032, 520, 3, 2, 0.0),
         (90, 64, 40, 1, 1, 0.0)]


class Case:
    def __init__(self, T, H, F, E, K, pad, dtype="bfloat16", seed=0, bias=True, max_tokens=None):
        self.rng = np.random.default_rng(seed + T)
        self.T, self.H, self.F, self.E, self.K, self.dtype = T, H, F, E, K, DT[dtype]
        self.gu, self.dn = self.rand(E, 2 * F, H, by=H ** -0.5), self.rand(E, H, F, by=F ** -0.5)
        self.gb, self.db = (self.rand(E, 2 * F), self.rand(E, H)) if bias else (None, None)
        self.x, self.g = self.rand(T, H), self.rand(T, H)
        bias = -0.7 * np.log(1.0 + self.rng.permutation(E))
        self.logits = dev((self.rng.standard_normal((T, E)) + bias).astype(np.float32))
        self.padded = dev(self.rng.random(T) < pad)
        self.layer = MoeTrainLayer(self.gu, self.dn, max_tokens or T, K, self.gb, self.db)

    def rand(self, *shape, by=1.0):
        return dev((by * self.rng.standard_normal(shape)).astype(np.float32)).to(self.dtype)

    def route(self):
        idx, w = self.layer.route(self.logits)
        return idx.masked_fill_(self.padded.unsqueeze(1), -1), w

    def step(self):
        """Routing, forward, backward, the router's gradient on top of the balance loss's."""
        idx, w = self.route()
        out = self.layer.forward(self.x, idx, w)
        valid = (~self.padded).to(torch.uint8)
        counts, prob, loss, onto = self.layer.balance(self.logits, idx, valid=valid)
        grads = self.layer.backward(self.g)
        grads["logits"] = self.layer.route_backward(idx, w, grads["w"], onto)
        return {"out": out, "counts": counts, "loss": loss, **grads}


def bits(r):
    torch.cuda.synchronize()
    return {k: v.contiguous().view(torch.uint8).cpu() for k, v in r.items()}


def same(a, b):
    return a.keys() == b.keys() and all(torch.equal(a[k], b[k]) for k in a)


class Rows:
    """What trainref's references need of the layer's maps."""

    def __init__(self, c):
        self.E, self.at = c.E, c.layer.offsets.tolist()
        self.live = self.at[-1]
        self.src = c.layer.src[:self.live].long()
        self.token = self.src // c.K
        self.slot = c.layer.slot[:c.T * c.K].view(c.T, c.K).long()

    def experts(self):
        for e in range(self.E):
            if self.at[e + 1] > self.at[e]:
                yield e, slice(self.at[e], self.at[e + 1])

    def per_row(self, b):
        counts = torch.tensor(self.at, device="cuda").diff()
        return b.double()[torch.repeat_interleave(torch.arange(self.E, device="cuda"), counts)]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("size", SIZES)
def test_each_stage(size, bias, dtype):
    """Every stage against the definition applied to what the stage before it left."""
    c = Case(*size, dtype=dtype, bias=bias, max_tokens=size[0] + 3)
    note(f"MoeTrainLayer {size} {dtype} bias={bias}")
    idx, w = c.route()
    out = c.layer.forward(c.x, idx, w).clone()
    r, la = Rows(c), c.layer
    y, s = grouped(r, c.x[r.token], c.gu)
    tol = sum_bound(c.H, s)
    if bias:
        y, tol = y + r.per_row(c.gb), tol + 2.0 ** -24 * (s + r.per_row(c.gb).abs())
    z = la.z[:r.live].clone()
    within(z, y, tol)
    h = la.h[:r.live].clone()
    within(h, *swiglu(y[:, :c.F], y[:, c.F:], tol[:, :c.F], tol[:, c.F:]))
    y, s = grouped(r, h, c.dn)
    tol = sum_bound(c.F, s)
    if bias:
        y, tol = y + r.per_row(c.db), tol + 2.0 ** -24 * (s + r.per_row(c.db).abs())
    rows = la.rows[:r.live].clone()
    within(rows, y, tol)
    there = (r.slot >= 0).unsqueeze(-1)
    each = torch.where(there, rows.double()[r.slot.clamp(min=0)], 0.0) if r.live else torch.zeros(
        c.T, c.K, c.H, dtype=torch.float64, device="cuda")
    part = w.double().unsqueeze(-1) * each
    within(out, part.sum(1), (c.K + 1) * 2.0 ** -24 * part.abs().sum(1))

    g = la.backward(c.g)
    dots = c.g.double().unsqueeze(1) * each
    within(g["w"], dots.sum(-1), c.H * 2.0 ** -24 * dots.abs().sum(-1))
    want = w.double().view(-1)[r.src].unsqueeze(1) * c.g.double()[r.token]
    d_rows = want.to(c.dtype)                          # one rounding: checked through what is made of it
    err = 2.0 ** -24 * want.abs() + half_step(c.dtype, want) * 2
    y, s = weight_grad(r, d_rows, h)
    _, e = weight_grad(r, err, h.abs())
    n = torch.tensor(r.at, device="cuda").diff().double()
    within(g["down"], y, sum_bound(n.view(-1, 1, 1), s) + e)
    if bias:
        y, s = weight_grad(r, d_rows, torch.ones(r.live, 1, device="cuda"))
        _, e = weight_grad(r, err, torch.ones(r.live, 1, device="cuda"))
        within(g["down_bias"], y[..., 0], sum_bound(n.view(-1, 1), s[..., 0]) + e[..., 0])
    y, s = grouped(r, d_rows, c.dn.transpose(1, 2))
    _, e = grouped(r, err, c.dn.transpose(1, 2).abs())
    dz = la.z[:r.live].clone()
    zd = z.double()
    dg, eg, du, eu = swiglu_grad(y, zd[:, :c.F], zd[:, c.F:], sum_bound(c.H, s) + e)
    within(dz[:, :c.F], dg, eg)
    within(dz[:, c.F:], du, eu)
    y, s = weight_grad(r, dz, c.x[r.token])
    within(g["gate_up"], y, sum_bound(n.view(-1, 1, 1), s))
    if bias:
        y, s = weight_grad(r, dz, torch.ones(r.live, 1, device="cuda"))
        within(g["gate_up_bias"], y[..., 0], sum_bound(n.view(-1, 1), s[..., 0]))
    y, s = grouped(r, dz, c.gu.transpose(1, 2))
    d_in = la.rows[:r.live]
    within(d_in, y, sum_bound(2 * c.F, s))
    each = torch.where(there, d_in.double()[r.slot.clamp(min=0)], 0.0) if r.live else each
    within(g["x"], each.sum(1), c.K * 2.0 ** -24 * each.abs().sum(1))


def test_against_autograd_as_a_whole():
    """The whole chain's gradients are autograd's of the same layer in 64 bits, within what the roundings
    between its stages add up to: 6 of 2^-9 each (a half step of bfloat16, relative to the 2-norm, is below
    2^-9), in h, rows, the rows' gradient, z's, and the result, and z itself."""
    c = Case(600, 256, 128, 8, 2, 0.1)
    idx, w = c.route()
    out = c.layer.forward(c.x, idx, w)
    g = c.layer.backward(c.g, grad_dtype=torch.float32)
    leaves = {k: v.double().requires_grad_() for k, v in
              dict(x=c.x, w=w, gate_up=c.gu, down=c.dn, gate_up_bias=c.gb, down_bias=c.db).items()}
    total = torch.zeros(c.T, c.H, dtype=torch.float64, device="cuda")
    for e in range(c.E):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        z = leaves["x"][t] @ leaves["gate_up"][e].t() + leaves["gate_up_bias"][e]
        h = z[:, :c.F] * torch.sigmoid(z[:, :c.F]) * z[:, c.F:]
        y = (h @ leaves["down"][e].t() + leaves["down_bias"][e]) * leaves["w"][t, k].unsqueeze(1)
        total = total.index_add(0, t, y)
    total.backward(c.g.double())
    tol = 6 * 2.0 ** -9
    total = total.detach()
    assert float((out.double() - total).norm() / total.norm()) <= tol
    assert g["gate_up"].dtype == torch.float32 and g["x"].dtype == c.dtype
    for k, v in leaves.items():
        assert float((g[k].double() - v.grad).norm() / v.grad.norm()) <= tol, k


def test_residual_and_float32_out():
    c = Case(*SIZES[1])
    idx, w = c.route()
    plain = c.layer.forward(c.x, idx, w, out=torch.empty(c.T, c.H, device="cuda"))
    res = torch.randn(c.T, c.H, device="cuda")
    both = c.layer.forward(c.x, idx, w, out=torch.empty_like(res), residual=res)
    within(both, plain.double() + res.double(), 4 * 2.0 ** -24 * (plain.abs() + res.abs()).double() + 1e-6)
    over = res.clone()
    assert torch.equal(c.layer.forward(c.x, idx, w, out=over, residual=over), both)
    a = c.layer.backward(c.g.float())
    c.layer.forward(c.x, idx, w)
    assert same(bits(a), bits(c.layer.backward(c.g.float())))


def test_weights_are_held_not_copied():
    c = Case(*SIZES[1])
    idx, w = c.route()
    a = c.layer.forward(c.x, idx, w)
    c.dn.mul_(2.0)
    c.db.mul_(2.0)
    assert torch.equal(c.layer.forward(c.x, idx, w), a * 2)     # a power of two: the same roundings


def test_replays_from_a_graph():
    """Two steps captured once each, replayed with eager work and synchronizations between, then on other
    inputs: every result equal to the eager step's bytes."""
    cases = [Case(*SIZES[2]), Case(*SIZES[1], dtype="float16", seed=9)]
    eager = [bits(c.step()) for c in cases]
    graphs = []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        note(f"capture T={c.T}")
        with torch.cuda.graph(g):
            results = c.step()
        graphs.append((g, results))
    for _ in range(3):
        for c, (g, results), want in zip(cases, graphs, eager):
            for t in (*results.values(), c.layer.rows, c.layer.h, c.layer.z, c.layer.src):
                t.zero_()
            c.layer.wgrad_ws.fill_(0xFF)
            g.replay()
            assert same(bits(results), want)
            assert same(bits(c.step()), want)
    for c, (g, results), old in zip(cases, graphs, eager):
        c.x.mul_(-1.5)
        c.logits.neg_()
        c.padded.logical_not_()
        g.replay()
        got = bits(results)
        assert same(bits(c.step()), got) and not same(got, old)


def test_two_layers_on_two_streams():
    cases = [Case(*SIZES[2], seed=1), Case(*SIZES[3], seed=2)]
    want = [bits(c.step()) for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for c, st in zip(cases, streams):
            with torch.cuda.stream(st):
                got.append(c.step())
    for r, wt in zip(got, want):
        assert same(bits(r), wt)


def test_every_token_padded():
    c = Case(40, 128, 64, 4, 2, 0.0)
    c.padded.fill_(True)
    r = c.step()
    for k in ("out", "x", "w", "gate_up", "down", "gate_up_bias", "down_bias", "logits"):
        assert bool((r[k] == 0).all()), k


def test_an_sgd_step_runs_and_fewer_tokens_than_the_buffers():
    c = Case(33, 128, 64, 4, 2, 0.0, max_tokens=64)
    before = c.gu.clone()
    r = c.step()
    c.gu.sub_(0.01 * r["gate_up"])
    assert not torch.equal(before, c.gu) and all(bool(v.isfinite().all()) for v in c.step().values())


def test_backward_follows_a_forward_once():
    c = Case(*SIZES[0])
    with pytest.raises(ValueError, match="follows a forward"):
        c.layer.backward(c.g)
    idx, w = c.route()
    c.layer.forward(c.x, idx, w)
    with pytest.raises(ValueError):
        c.layer.backward(c.g[:2])
    with pytest.raises(ValueError):
        c.layer.backward(c.g, grad_dtype=torch.float64)
    c.layer.backward(c.g)                                        # the refused calls left the forward's state
    with pytest.raises(ValueError, match="follows a forward"):
        c.layer.backward(c.g)


def test_refusals_leave_nothing_enqueued(monkeypatch):
    c = Case(*SIZES[1])
    idx, w = c.route()
    done = []
    monkeypatch.setattr(abi, "build_maps", lambda *a, **k: done.append("maps"))
    x = c.x
    wide = torch.zeros(c.T, 2 * c.H, dtype=c.dtype, device="cuda")
    for bad in (x.float(), x[:, :8], x[0].expand(c.T, c.H), x.cpu(), x.t().contiguous().t(), wide[:, 4:4 + c.H],
                torch.zeros(c.T, c.H + 4, dtype=c.dtype, device="cuda")[:, :c.H]):
        with pytest.raises(ValueError):
            c.layer.forward(bad, idx, w)
    for bad in (x.double(), x[:1], wide[:, 1:1 + c.H], torch.empty(c.T, c.H, dtype=torch.float16, device="cuda")):
        with pytest.raises(ValueError):
            c.layer.forward(x, idx, w, out=bad)
    for kw in (dict(residual=x.float()), dict(residual=x[:1]), dict(out=torch.empty(c.T, c.H, device="cuda"), residual=x)):
        with pytest.raises(ValueError):
            c.layer.forward(x, idx, w, **kw)
    with pytest.raises(ValueError):
        c.layer.forward(x, idx.long(), w)
    with pytest.raises(ValueError):
        c.layer.forward(x, idx, w[:, :1])
    assert not done and c.layer.kept is None


def test_every_iteration_on_two_streams():
    """As test_two_layers_on_two_streams, with each iteration's results compared."""
    cases = [Case(*SIZES[2], seed=3), Case(*SIZES[3], seed=4)]
    want = [bits(c.step()) for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for c, st in zip(cases, streams):
            with torch.cuda.stream(st):
                got.append(c.step())
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        assert same(bits(r), want[i % 2]), i
