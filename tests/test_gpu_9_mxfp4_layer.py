"""MoeMxfp4Layer at sizes whose products take the wide kernel: against the 64-bit reference stage by stage,
captured and replayed, and two layers at once."""
import numpy as np
import pytest
import torch

import mxref
from gpu_util import dev, host, note
from quantized_expert_grouped_amd.layer import MoeMxfp4Layer
from test_gpu_9_mxfp4 import exact_f64, sum_bound

pytestmark = pytest.mark.gpu

# T, H, F, E, K: gate/up and down in the 128 x 128 tile (down's K a last stage of 128 values); gate/up in 256 x
# 64; both in 128 x 192; gate/up in 256 x 256
SIZES = [(1500, 512, 384, 16, 4), (700, 512, 512, 140, 4), (2048, 1024, 1024, 64, 4), (4100, 512, 1024, 16, 4)]


class Case:
    def __init__(self, T, H, F, E, K, seed, max_tokens=None, **options):
        rng = np.random.default_rng(seed)
        self.T, self.H, self.F, self.E, self.K = T, H, F, E, K

        def weights(N, k):
            return (rng.integers(0, 256, (E, N, k // 2), dtype=np.uint8),
                    rng.integers(119, 123, (E, N, k // 32), dtype=np.uint8))

        self.gu, self.dn = weights(2 * F, H), weights(H, F)
        self.x = dev(rng.standard_normal((T, H)).astype(np.float32))
        bias = -0.5 * np.log(1.0 + rng.permutation(E))         # some experts take more rows than others
        self.logits = dev((rng.standard_normal((T, E)) + bias).astype(np.float32))
        self.layer = MoeMxfp4Layer([dev(v) for v in self.gu], [dev(v) for v in self.dn],
                                   max_tokens=max_tokens or T, K=K, **options)

    def run(self):
        self.idx, self.w = self.layer.route(self.logits)
        balance = self.layer.balance(self.logits, self.idx)
        return [self.layer.forward(self.x, self.idx, self.w), self.idx, self.w, *balance]

    def bytes(self, results):
        torch.cuda.synchronize()
        la, R = self.layer, self.T * self.K
        inner = [la.src[:R], la.slot[:R], la.offsets, la.x_codes[:self.T], la.h_codes[:R], la.h_scales[:R], la.rows[:R]]
        return [t.cpu().contiguous().view(torch.uint8).numpy().copy() for t in [*results, *inner]]


def same(a, b):
    return all(np.array_equal(p, q) for p, q in zip(a, b, strict=True))


@pytest.mark.parametrize("T,H,F,E,K,options", [(*s, {}) for s in SIZES] + [
    (*SIZES[0], dict(rows_dtype=torch.float32)), (1, 512, 384, 16, 4, dict(rows_dtype=torch.float32))])
def test_layer_against_the_reference(T, H, F, E, K, options):
    """Each stage against the reference applied to the stage before it as the GPU left it."""
    c = Case(T, H, F, E, K, T, max_tokens=T + 13, **options)
    note(f"MoeMxfp4Layer T={T} H={H} F={F} E={E} K={K} {options}")
    out, idx, w, counts = c.run()[:4]
    la, R = c.layer, T * K
    off, src, slot = host(la.offsets), host(la.src)[:R], host(la.slot)[:R]
    assert np.array_equal(host(counts)[:E], np.diff(off)) and int(host(counts)[E]) == T
    ec, es = mxref.encode(host(c.x))
    assert np.array_equal(host(la.x_codes)[:T], ec) and np.array_equal(host(la.x_scales)[:T], es)
    y, s = mxref.grouped(mxref.decode(ec, es)[src // K], mxref.decode(*c.gu), off)
    tol = sum_bound(H, s)
    g, u = y[:, :F], y[:, F:]
    h = mxref.silu(g) * u
    # |silu'| < 1.1; the epilogue's own error is (1.25 |g| + 8) 2^-24 of h
    dh = 1.1 * tol[:, :F] * (np.abs(u) + tol[:, F:]) + np.abs(mxref.silu(g)) * tol[:, F:] + \
        np.abs(h) * (1.25 * np.abs(g) + 8) * 2.0 ** -24 + 2.0 ** -119 * np.abs(u)
    hc, hs = host(la.h_codes)[:R], host(la.h_scales)[:R]
    mxref.check_codes(hc, hs, h, dh)
    y2, s2 = mxref.grouped(mxref.decode(hc, hs), mxref.decode(*c.dn), off)
    assert la.rows.dtype == options.get("rows_dtype", torch.bfloat16)
    half = 2.0 ** -8 if la.rows.dtype == torch.bfloat16 else 0.0
    rows = exact_f64(la.rows[:R])
    assert np.all(np.abs(rows - y2) <= sum_bound(F, s2) * (1 + half) + half * np.abs(y2))
    own = host(w).astype(np.float64)[..., None] * rows[slot.reshape(T, K)]
    assert np.all(np.abs(exact_f64(out) - own.sum(1)) <= K * 2.0 ** -24 * np.abs(own).sum(1))


def test_layer_replays_from_a_graph():
    """Captured once each, replayed with eager work between the replays, then on changed inputs: every result
    and every buffer equal to the eager call's bytes."""
    cases = [Case(*SIZES[0], 1), Case(*SIZES[3], 2)]
    eager, graphs = [], []
    for c in cases:
        eager.append(c.bytes(c.run()))
    for c in cases:
        g = torch.cuda.CUDAGraph()
        note(f"capture T={c.T}")
        with torch.cuda.graph(g):
            results = c.run()
        graphs.append((g, results))
    for _ in range(3):
        for c, (g, results), want in zip(cases, graphs, eager):
            for t in (*results, c.layer.rows, c.layer.h_codes, c.layer.src):
                t.zero_()
            g.replay()
            assert same(c.bytes(results), want)
    for c, (g, results), old in zip(cases, graphs, eager):
        c.x.mul_(1.75)
        c.logits.neg_()
        g.replay()
        got = c.bytes(results)
        assert same(c.bytes(c.run()), got) and not same(got, old)


def test_two_layers_on_two_streams():
    cases = [Case(*SIZES[1], 3), Case(*SIZES[0], 4)]
    want = [c.bytes(c.run()) for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        got = []
        for c, st in zip(cases, streams):
            with torch.cuda.stream(st):
                got.append(c.run())
    for c, r, wt in zip(cases, got, want):
        assert same(c.bytes(r), wt)


def test_routes_out_of_range_add_nothing():
    """Ids outside [0, E) through the whole layer: the output is that of the routes that are left."""
    c = Case(*SIZES[0], 5)
    idx, w = c.layer.route(c.logits)
    flat = idx.view(-1)
    flat[::7] = -1
    flat[3::11] = c.E
    out = host(c.layer.forward(c.x, idx, w)).astype(np.float64)
    ids, slot = host(idx), host(c.layer.slot).reshape(c.T, c.K)
    on = (ids >= 0) & (ids < c.E)
    assert np.array_equal(slot >= 0, on) and 0 < on.sum() < on.size
    rows = exact_f64(c.layer.rows)
    own = np.where(on[..., None], host(w).astype(np.float64)[..., None] * rows[np.maximum(slot, 0)], 0.0)
    assert np.all(np.abs(out - own.sum(1)) <= c.K * 2.0 ** -24 * np.abs(own).sum(1))
    assert int(host(c.layer.offsets)[c.E]) == on.sum()


@pytest.mark.parametrize("T,H,F,E,K", [(37, 256, 128, 8, 3), SIZES[0], (5, 128, 128, 1, 1), (600, 128, 256, 1, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_tokens_of_each_type_in_rows_with_gaps(T, H, F, E, K, dtype):
    """x as every second row of a wider matrix, and into an out of the caller's: the bytes of the contiguous
    call.  One expert for all tokens among the sizes."""
    c = Case(T, H, F, E, K, 6)
    whole = torch.full((2 * T, H + 16), 7.0, device="cuda", dtype=dtype)
    x = whole[::2, 8:8 + H]
    x.copy_(c.x)
    idx, w = c.layer.route(c.logits)
    want = c.layer.forward(x.contiguous(), idx, w).clone()
    out = torch.full((T + 1, H), 5.0, device="cuda")
    assert c.layer.forward(x, idx, w, out=out[:T]).data_ptr() == out.data_ptr()
    assert torch.equal(out[:T], want) and bool((out[T] == 5.0).all())
    ec, es = mxref.encode(exact_f64(x))
    assert np.array_equal(host(c.layer.x_codes)[:T], ec) and np.array_equal(host(c.layer.x_scales)[:T], es)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_balance_of_padded_logits_in_rows_with_gaps(dtype):
    c = Case(*SIZES[0], 7)
    whole = torch.full((c.T, c.E + 5), 7.0, device="cuda", dtype=dtype)
    logits = whole[:, 3:3 + c.E]
    logits.copy_(c.logits)
    idx, _ = c.layer.route(c.logits)
    valid = (torch.arange(c.T, device="cuda") % 5 != 2).to(torch.uint8)
    g = torch.full((1,), 64.0, device="cuda")
    want = c.layer.balance(logits.contiguous(), idx, valid=valid, grad_loss=g)
    for a, b in zip(c.layer.balance(logits, idx, valid=valid, grad_loss=g), want, strict=True):
        assert torch.equal(a, b)
    counts, prob, loss, grad = want
    n = int(valid.sum())
    ref = mxref.balance(exact_f64(logits), host(idx), host(valid))
    assert np.array_equal(host(counts), ref[0]) and int(counts[c.E]) == n
    assert abs(float(loss) - ref[2]) <= 1e-5 * ref[2]
    assert grad.dtype == dtype and bool((grad[valid == 0] == 0).all())
    one = c.layer.balance(logits, idx, valid=valid)[3]                # without grad_loss: 1
    # 64 is a power of two: the same roundings but where a value is subnormal
    tiny = torch.finfo(dtype).tiny
    assert bool(((grad.double() - 64 * one.double()).abs() <= 64 * tiny).all())
