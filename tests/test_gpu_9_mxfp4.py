"""MXFP4 on the GPU against the 64-bit reference: quantisation byte for byte, the grouped product within
the rounding of its fp32 sums, the bf16 combine, and the whole expert path made of them."""
import numpy as np
import pytest
import torch

import mxref
from gpu_util import dev, empty, gpu_maps, host, note
from quantized_expert_grouped_amd import abi
from quantized_expert_grouped_amd.layer import MoeMxfp4Layer

pytestmark = pytest.mark.gpu

DT = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
GUARD = 0xAB


def guarded(shape, dtype):
    """A buffer with 64 rows more than it needs, every byte GUARD: (whole, the part to use)."""
    t = torch.empty((shape[0] + 64, *shape[1:]), dtype=dtype, device="cuda")
    t.view(torch.uint8).fill_(GUARD)
    return t, t[:shape[0]]


def untouched(whole, rows):
    assert bool((whole[rows:].contiguous().view(torch.uint8) == GUARD).all())


def quantize(x):
    rows, n = x.shape
    cw, c = guarded((rows, n // 2), torch.uint8)
    sw, s = guarded((rows, n // 32), torch.uint8)
    note(f"mxfp4_quantize {rows}x{n} {x.dtype} ld={x.stride(0)}")
    abi.mxfp4_quantize(x, c, s)
    torch.cuda.synchronize()
    untouched(cw, rows)
    untouched(sw, rows)
    return c, s


def exact_f64(t):
    return t.double().cpu().numpy()


# ---- quantisation ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,n,pad", [(1, 32, 0), (1, 2048, 0), (3, 96, 0), (257, 128, 8),
                                        (65, 4128, 0), (7, 2080, 96), (1000, 512, 0)])
def test_quantize_bytes(dtype, rows, n, pad):
    rng = np.random.default_rng(rows + n)
    x = rng.standard_normal((rows, n + pad)) * np.exp2(rng.integers(-12, 6, (rows, 1)))
    x[rows // 2] = 0.0
    x[0, :32] *= 1e-4
    xt = dev(x.astype(np.float32)).to(DT[dtype])[:, :n]
    c, s = quantize(xt)
    ec, es = mxref.encode(exact_f64(xt))
    assert np.array_equal(host(s), es)
    assert np.array_equal(host(c), ec)


def test_quantize_borders_and_extremes():
    """Every border between codes and the fp32 numbers next to it, at several scales (subnormal and
    near the range's top among them), both signs; amax next to a power of two; zeros of both signs;
    subnormal blocks; blocks with an infinity or a NaN."""
    blocks = []
    pts = np.concatenate([mxref.BORDERS, mxref.LEVELS[1:], [7.0, 7.75]]).astype(np.float32)
    near = np.concatenate([np.nextafter(pts, np.float32(0)), pts, np.nextafter(pts, np.float32(9))])
    for e in (0, -20, 40, 123, -100, -125, -126, -127):
        for sign in (1, -1):
            for i in range(0, len(near), 31):
                v = np.zeros(32, np.float32)
                part = near[i:i + 31]
                v[:len(part)] = sign * part
                v[31] = 4.0
                blocks.append(np.ldexp(v, e).astype(np.float32))
    for top in (1.0, 2.0 ** 127, 2.0 ** -126, 2.0 ** -149, 2.0 ** -130):
        for a in (np.nextafter(np.float32(top), np.float32(0)), np.float32(top),
                  np.nextafter(np.float32(top), np.float32(np.inf))):
            v = np.full(32, a, np.float32) * np.linspace(-1, 1, 32).astype(np.float32)
            v[5] = a
            blocks.append(v)
    z = np.zeros(32, np.float32)
    z[::2] = -0.0
    blocks.append(z)
    for bad in (np.inf, -np.inf, np.nan):
        v = np.linspace(-3, 3, 32).astype(np.float32)
        v[17] = bad
        blocks.append(v)
    blocks.append(np.full(32, np.finfo(np.float32).max, np.float32))
    x = np.stack(blocks).reshape(len(blocks), 32)
    c, s = quantize(dev(x))
    ec, es = mxref.encode(x)
    assert np.array_equal(host(s), es)
    assert np.array_equal(host(c), ec)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_dequantize_every_code_and_scale(dtype):
    codes = np.tile(np.arange(256, dtype=np.uint8).reshape(16, 16), (16, 1))     # 256 rows of 32
    codes = np.repeat(codes, 16, axis=0)
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, axis=1).reshape(-1, 1)
    whole = torch.full((len(codes), 40), 7.0, device="cuda", dtype=DT[dtype])
    y = whole[:, :32]
    note(f"mxfp4_dequantize every code {dtype}")
    abi.mxfp4_dequantize(dev(codes), dev(scales), y)
    with np.errstate(over="ignore"):
        want = mxref.decode(codes, scales).astype(np.float32)   # 6 * 2^127 is beyond fp32: inf
    assert np.array_equal(host(y.float()), want, equal_nan=True)
    assert bool((whole[:, 32:] == 7.0).all())


# ---- the grouped product --------------------------------------------------------------------
def weights(rng, E, N, k):
    codes = rng.integers(0, 256, (E, N, k // 2), dtype=np.uint8)
    scales = rng.integers(117, 124, (E, N, k // 32), dtype=np.uint8)
    return codes, scales


def routes(rng, T, K, E, skew):
    w = np.exp(-skew * np.arange(E))
    p = np.log(w / w.sum())[rng.permutation(E)]
    return np.argsort(-(p + rng.gumbel(size=(T, E))), 1)[:, :K].astype(np.int32)


def product(wc, ws, offsets, ac, as_, rows, src, K, epi):
    n_out = wc.shape[1]
    swig = epi == abi.MX_SWIGLU_MXFP4
    shape = (rows, n_out // 4) if swig else (rows, n_out)
    dt = torch.uint8 if swig else torch.float32 if epi == abi.MX_F32 else torch.bfloat16
    ow, out = guarded(shape, dt)
    sw, os_ = guarded((rows, n_out // 64), torch.uint8) if swig else (None, None)
    note(f"mxfp4_mm rows={rows} N={n_out} k={2 * wc.shape[2]} E={wc.shape[0]} epi={epi}")
    abi.mxfp4_mm_grouped(dev(wc), dev(ws), offsets, dev(ac), dev(as_), out, src=src, K=K,
                         out_scales=os_)
    torch.cuda.synchronize()
    untouched(ow, rows)
    if swig:
        untouched(sw, rows)
    return out, os_


def sum_bound(k, s):
    """fp32 sums of k exact products in any order, each addition off by 2^-23 (truncation allowed for)
    of a partial sum that sum |a||w| bounds."""
    return k * 2.0 ** -23 * s


SHAPES = [  # T, K, E, N, k, gather, skew
    (1, 1, 1, 32, 128, False, 0.0), (1, 2, 8, 64, 256, True, 0.0), (3, 1, 2, 96, 384, True, 0.0),
    (5, 3, 40, 160, 2048, True, 0.0), (40, 2, 4, 128, 128, False, 0.0), (33, 1, 1, 224, 640, True, 0.0),
    (130, 4, 16, 256, 512, True, 0.7), (300, 1, 3, 288, 896, False, 1.5), (257, 6, 64, 64, 1024, True, 0.2),
    (64, 8, 2048, 32, 128, True, 0.0), (700, 2, 3, 512, 256, True, 3.0), (1000, 1, 1, 384, 1152, False, 0.0),
    (1600, 4, 16, 320, 384, True, 0.1), (2500, 2, 9, 128, 640, False, 0.4),
    # the wide kernel's tiles (two shapes for each: scale bytes in pieces of 16 and of 4), a last
    # stage of 128 values, columns that end inside a tile
    (1024, 1, 1, 1024, 1024, True, 0.0), (1300, 1, 3, 1056, 128, False, 0.5),
    (900, 2, 40, 512, 512, True, 0.5), (900, 2, 40, 544, 128, False, 0.5),
    (1200, 4, 200, 1024, 512, True, 0.1), (1200, 4, 200, 1056, 640, False, 0.1),
    (1200, 4, 200, 1056, 128, True, 1.0), (2048, 4, 64, 2048, 512, True, 0.3),
    (2051, 4, 64, 2080, 640, False, 0.3), (2047, 4, 16, 2080, 1024, True, 0.5),
    (2048, 4, 16, 2048, 384, True, 2.0)]


@pytest.mark.parametrize("epi", [abi.MX_F32, abi.MX_BF16, abi.MX_SWIGLU_MXFP4])
@pytest.mark.parametrize("T,K,E,N,k,gather,skew", SHAPES)
def test_mm_grouped(T, K, E, N, k, gather, skew, epi):
    rng = np.random.default_rng(T * 131 + N + k)
    idx = routes(rng, T, K, E, skew)
    _, maps = gpu_maps(idx, E, 0)
    R = T * K
    swig = epi == abi.MX_SWIGLU_MXFP4
    wc, ws = weights(rng, E, 2 * N if swig else N, k)
    ac, as_ = mxref.encode(rng.standard_normal((T if gather else R, k)))
    src = maps["src"] if gather else None
    out, os_ = product(wc, ws, maps["offsets"], ac, as_, R, src, K, epi)
    a = mxref.decode(ac, as_)
    if gather:
        a = a[host(maps["src"]) // K]
    y, s = mxref.grouped(a, mxref.decode(wc, ws), host(maps["offsets"]))
    tol = sum_bound(k, s)
    if not swig:
        if epi == abi.MX_BF16:
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(y)
        assert np.all(np.abs(exact_f64(out) - y) <= tol)
        return
    g, u, dg, du = y[:, :N], y[:, N:], tol[:, :N], tol[:, N:]
    # |silu'| < 1.1, |silu(g)| <= |g|; exp within 2 ulp, and one rounding each for the sum, the
    # quotient and the product: 8 * 2^-24 of h
    h = mxref.silu(g) * u
    dh = 1.1 * dg * (np.abs(u) + du) + np.abs(mxref.silu(g)) * du + 2.0 ** -21 * np.abs(h) + 2.0 ** -126
    mxref.check_codes(host(out), host(os_), h, dh)


def test_mm_scales_at_any_4_byte_address():
    """Scales that are 4-byte aligned only: the same bytes come out as with aligned ones."""
    rng = np.random.default_rng(6)
    T, K, E, N, k = 2000, 2, 30, 512, 512
    _, maps = gpu_maps(routes(rng, T, K, E, 0.2), E, 0)
    wc, ws = weights(rng, E, N, k)
    ac, as_ = mxref.encode(rng.standard_normal((T, k)))
    wc, ac = dev(wc), dev(ac)

    def at(a, skip):
        t = torch.empty(a.size + 16, dtype=torch.uint8, device="cuda")[skip:skip + a.size].view(a.shape)
        return t.copy_(dev(a))

    outs = []
    for w_skip, a_skip in ((0, 0), (4, 0), (0, 8), (12, 4)):
        out = empty((T * K, N), torch.float32)
        note(f"mm scales at {w_skip} {a_skip}")
        abi.mxfp4_mm_grouped(wc, at(ws, w_skip), maps["offsets"], ac, at(as_, a_skip), out,
                             src=maps["src"], K=K)
        outs.append(out)
    assert all(torch.equal(outs[0], o) for o in outs[1:])
    for skip in (1, 2):
        with pytest.raises(abi.MoeError):
            abi.mxfp4_mm_grouped(wc, at(ws, skip), maps["offsets"], ac, at(as_, 0), outs[0],
                                 src=maps["src"], K=K)


@pytest.mark.parametrize("T,K,E,N,k", [(50, 3, 6, 64, 256), (3000, 3, 50, 640, 256),
                                       (1200, 4, 200, 1024, 256), (3000, 3, 70, 2048, 256),
                                       (3000, 3, 30, 2048, 256)])
def test_mm_rows_past_the_experts_are_left_alone(T, K, E, N, k):
    """Routes to ids outside [0, E) take rows past offsets[E]: those keep their bytes, in every epilogue."""
    rng = np.random.default_rng(3)
    idx = routes(rng, T, K, E, 0.0)
    idx.reshape(-1)[::7] = np.array([-1, E, 99])[np.arange(len(idx.reshape(-1)[::7])) % 3]
    _, maps = gpu_maps(idx, E, 0)
    end = int(host(maps["offsets"])[E])
    assert end < T * K
    ac, as_ = mxref.encode(rng.standard_normal((T, k)))
    for epi in (abi.MX_F32, abi.MX_BF16, abi.MX_SWIGLU_MXFP4):
        wc, ws = weights(rng, E, 2 * N if epi == abi.MX_SWIGLU_MXFP4 else N, k)
        out, os_ = product(wc, ws, maps["offsets"], ac, as_, T * K, maps["src"], K, epi)
        for t in (out,) if os_ is None else (out, os_):
            assert bool((t[end:].contiguous().view(torch.uint8) == GUARD).all())
        a = mxref.decode(ac, as_)[np.maximum(host(maps["src"]), 0) // K]
        y, s = mxref.grouped(a, mxref.decode(wc, ws), host(maps["offsets"]))
        if epi == abi.MX_F32:
            assert np.all(np.abs(exact_f64(out) - y)[:end] <= sum_bound(k, s)[:end])


@pytest.mark.parametrize("R,N,k", [(40, 64, 256), (1300, 1056, 384), (1100, 1024, 512)])
def test_mm_scales_at_their_ends(R, N, k):
    """Scale bytes at both ends of their range (products of normal size or 0), and NaN ones: a NaN block
    of a weight row makes its column NaN, one of an activation row that row, and nothing else."""
    rng = np.random.default_rng(4)
    wc, ws = weights(rng, 1, N, k)
    ac, as_ = mxref.encode(rng.standard_normal((R, k)))
    ws[0, :8], as_[:5] = 250, 10
    ws[0, 8:16], as_[5:9] = 0, 230
    ws[0, 20, 3], as_[30, 7] = 255, 255
    offsets = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    out, _ = product(wc, ws, offsets, ac, as_, R, None, 1, abi.MX_F32)
    got = exact_f64(out)
    want = np.zeros((R, N), bool)
    want[30, :], want[:, 20] = True, True
    ws[0, 20, 3], as_[30, 7] = 100, 100
    y, s = mxref.grouped(mxref.decode(ac, as_), mxref.decode(wc, ws), [0, R])
    # with sum |a||w| from 2^127 on a partial sum may pass fp32's range, and inf - inf is NaN too
    fits = s < 2.0 ** 127
    assert np.array_equal(np.isnan(got)[fits], want[fits])
    assert np.all(np.isnan(got)[want])
    ok = ~want & fits
    assert ok.sum() > 0.5 * R * N
    assert np.all(np.abs(got - y)[ok] <= (sum_bound(k, s) + 2.0 ** -126)[ok])


def test_mm_src_out_of_range_stays_in_bounds():
    """src entries that name no activation row read the nearest one."""
    rng = np.random.default_rng(5)
    N, k, R = 32, 128, 6
    wc, ws = weights(rng, 1, N, k)
    ac, as_ = mxref.encode(rng.standard_normal((3, k)))
    src = dev(np.array([0, 2, 5, 6, 1 << 30, -5], np.int32))
    offsets = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    out, _ = product(wc, ws, offsets, ac, as_, R, src, 2, abi.MX_F32)
    a = mxref.decode(ac, as_)[[0, 1, 2, 2, 2, 0]]
    y, s = mxref.grouped(a, mxref.decode(wc, ws), [0, R])
    assert np.all(np.abs(exact_f64(out) - y) <= sum_bound(k, s))


def test_mm_offsets_past_31_bits():
    """A matrix and activations of more than 2 GiB of codes each, the last columns and rows among those
    looked at."""
    N, k, n_act = 1_200_000 // 32 * 32, 4096, 1_200_000
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    wc = torch.randint(0, 256, (1, N, k // 2), dtype=torch.uint8, device="cuda", generator=g)
    ws = torch.randint(118, 124, (1, N, k // 32), dtype=torch.uint8, device="cuda", generator=g)
    ac = torch.randint(0, 256, (n_act, k // 2), dtype=torch.uint8, device="cuda", generator=g)
    as_ = torch.randint(118, 124, (n_act, k // 32), dtype=torch.uint8, device="cuda", generator=g)
    assert wc.numel() > 1 << 31 and ac.numel() > 1 << 31
    rows = np.array([n_act - 1, 0, n_act - 12345], np.int32)
    offsets = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    out = empty((3, N), torch.float32)
    note("mm past 31 bits")
    abi.mxfp4_mm_grouped(wc, ws, offsets, ac, as_, out, src=dev(rows), K=1)
    cols = np.concatenate([np.arange(40), np.arange(N // 2, N // 2 + 40), np.arange(N - 40, N)])
    at = torch.from_numpy(cols).cuda()
    a = mxref.decode(host(ac[dev(rows).long()]), host(as_[dev(rows).long()]))
    w = mxref.decode(host(wc[0, at]), host(ws[0, at]))
    y, s = mxref.grouped(a, w[None], [0, 3])
    assert np.all(np.abs(exact_f64(out[:, at]) - y) <= sum_bound(k, s))


def test_binding_refuses_mismatched_tensors():
    u8 = torch.uint8
    w, ws = empty((2, 32, 64), u8), empty((2, 32, 4), u8)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    a, as_, out = empty((4, 64), u8), empty((4, 4), u8), empty((4, 32), torch.float32)
    good = dict(w_codes=w, w_scales=ws, offsets=off, a_codes=a, a_scales=as_, out=out)
    for bad in (dict(w_scales=empty((2, 32, 8), u8)), dict(offsets=off[:2]), dict(offsets=off.long()),
                dict(a_codes=empty((4, 32), u8)), dict(a_scales=empty((3, 4), u8)),
                dict(out=empty((4, 64), torch.float32)), dict(out=out.half()),
                dict(out=empty((4, 64), torch.float32)[:, :32]), dict(out_scales=empty((4, 1), u8)),
                dict(src=off), dict(w_codes=w.cpu())):
        with pytest.raises(ValueError):
            abi.mxfp4_mm_grouped(**{**good, **bad})
    x = empty((4, 128), torch.float32)
    with pytest.raises(ValueError):
        abi.mxfp4_quantize(x.t(), empty((128, 2), u8), empty((128, 0), u8))
    with pytest.raises(ValueError):
        abi.mxfp4_quantize(x.double(), empty((4, 64), u8), empty((4, 4), u8))
    with pytest.raises(ValueError):
        abi.mxfp4_dequantize(empty((4, 64), u8), empty((4, 2), u8), x)
    with pytest.raises(abi.MoeError):                       # one row given to all: rows 0 apart
        abi.mxfp4_quantize(x[:1].expand(4, 128), empty((4, 64), u8), empty((4, 4), u8))


# ---- combine --------------------------------------------------------------------------------
@pytest.mark.parametrize("T,K,H", [(1, 1, 8), (1, 10, 2048), (17, 3, 136), (100, 64, 256),
                                   (1000, 10, 512), (33, 17, 4096), (5, 2, 2056)])
def test_combine_bf16(T, K, H):
    rng = np.random.default_rng(T + H)
    rows = dev(rng.standard_normal((T * K, H)).astype(np.float32)).bfloat16()
    w = rng.random((T, K)).astype(np.float32)
    slot = rng.permutation(T * K).astype(np.int32).reshape(T, K)
    slot.reshape(-1)[3::11] = -1
    slot.reshape(-1)[5::23] = T * K                      # no row either
    whole, out = guarded((T, H), torch.float32)
    note(f"combine_bf16 T={T} K={K} H={H}")
    abi.combine_bf16(rows, dev(slot), dev(w), out)
    r = exact_f64(rows)
    on = (slot >= 0) & (slot < T * K)
    term = np.where(on[..., None], w[..., None].astype(np.float64) * r[np.where(on, slot, 0)], 0.0)
    # K fused multiply-adds, each rounding a partial sum by half an ulp
    assert np.all(np.abs(exact_f64(out) - term.sum(1)) <= K * 2.0 ** -24 * np.abs(term).sum(1))
    untouched(whole, T)


# ---- the path -------------------------------------------------------------------------------
class Path:
    """Router to output over MXFP4 experts, on buffers of its own."""

    def __init__(self, T, H, F, E, K, seed):
        self.rng = np.random.default_rng(seed)
        self.T, self.H, self.F, self.E, self.K = T, H, F, E, K
        rng, R, u8, i32 = self.rng, T * K, torch.uint8, torch.int32
        self.gu_h = mxref.encode(rng.standard_normal((E * 2 * F, H)).astype(np.float32) / np.sqrt(H))
        self.dn_h = mxref.encode(rng.standard_normal((E * H, F)).astype(np.float32) / np.sqrt(F))
        self.gu = [dev(v.reshape(E, 2 * F, -1)) for v in self.gu_h]
        self.dn = [dev(v.reshape(E, H, -1)) for v in self.dn_h]
        self.x = dev(rng.standard_normal((T, H)).astype(np.float32))
        self.logits = dev(rng.standard_normal((T, E)).astype(np.float32))
        self.idx, self.w = empty((T, K), i32), empty((T, K), torch.float32)
        self.maps = dict(counts=empty(E, i32), offsets=empty(E + 1, i32), src=empty(R, i32),
                         slot=empty(R, i32), order=empty(E, i32), n_active=empty(1, i32))
        self.mws = empty(abi.build_maps_workspace_size(T, K, E), u8)
        self.counts, self.prob, self.loss = empty(E + 1, i32), empty(E, torch.float32), empty(1, torch.float32)
        self.grad, self.bws = empty((T, E), torch.float32), empty(abi.balance_workspace_size(T, E), u8)
        self.xc, self.xs = empty((T, H // 2), u8), empty((T, H // 32), u8)
        self.hc, self.hs = empty((R, F // 2), u8), empty((R, F // 32), u8)
        self.rows, self.out = empty((R, H), torch.bfloat16), empty((T, H), torch.float32)
        self.results = [self.idx, self.w, self.maps["src"], self.counts, self.prob, self.loss, self.grad,
                        self.xc, self.xs, self.hc, self.hs, self.rows, self.out]

    def run(self):
        m = self.maps
        abi.route_topk(self.logits, self.K, self.idx, self.w)
        abi.balance_loss(self.logits, self.idx, self.counts, self.prob, self.loss, self.bws)
        abi.balance_loss_backward(self.logits, self.counts, self.K, self.grad)
        abi.build_maps(self.idx, self.E, 0, m["counts"], m["offsets"], m["src"], m["slot"], m["order"],
                       m["n_active"], self.mws)
        abi.mxfp4_quantize(self.x, self.xc, self.xs)
        abi.mxfp4_mm_grouped(*self.gu, m["offsets"], self.xc, self.xs, self.hc, src=m["src"], K=self.K,
                             out_scales=self.hs)
        abi.mxfp4_mm_grouped(*self.dn, m["offsets"], self.hc, self.hs, self.rows)
        abi.combine_bf16(self.rows, m["slot"], self.w, self.out)

    def bytes(self):
        torch.cuda.synchronize()
        return [t.cpu().contiguous().view(torch.uint8).numpy().copy() for t in self.results]


@pytest.mark.parametrize("T,H,F,E,K", [(1, 256, 128, 16, 2), (37, 256, 128, 16, 2),
                                       (300, 512, 256, 12, 3)])
def test_path_against_the_reference(T, H, F, E, K):
    """Each stage against the reference applied to the stage before it as the GPU left it, and the output
    against the reference's own whole path: the roundings that may fall apart there are those of h, at
    most one level (a third of the value, 2 / 6) each, and those rarely, so 1% in the 2-norm."""
    p = Path(T, H, F, E, K, T + E)
    note(f"mxfp4 path T={T} H={H} F={F} E={E} K={K}")
    p.run()
    off, src, slot = (host(p.maps[k]) for k in ("offsets", "src", "slot"))
    idx, w = host(p.idx), host(p.w).astype(np.float64)
    counts = host(p.counts)
    assert np.array_equal(counts[:E], host(p.maps["counts"])) and counts[E] == T
    ec, es = mxref.encode(host(p.x))
    assert np.array_equal(host(p.xc), ec) and np.array_equal(host(p.xs), es)
    gu = mxref.decode(*p.gu_h).reshape(E, 2 * F, H)
    dn = mxref.decode(*p.dn_h).reshape(E, H, F)
    y, s = mxref.grouped(mxref.decode(ec, es)[src // K], gu, off)
    tol = sum_bound(H, s)
    g, u = y[:, :F], y[:, F:]
    h = mxref.silu(g) * u
    dh = 1.1 * tol[:, :F] * (np.abs(u) + tol[:, F:]) + np.abs(mxref.silu(g)) * tol[:, F:] + 2.0 ** -21 * np.abs(h)
    mxref.check_codes(host(p.hc), host(p.hs), h, dh)
    y2, s2 = mxref.grouped(mxref.decode(host(p.hc), host(p.hs)), dn, off)
    rows = exact_f64(p.rows)
    assert np.all(np.abs(rows - y2) <= sum_bound(F, s2) * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(y2))
    own = (w[..., None] * rows[slot.reshape(T, K)])
    out = exact_f64(p.out)
    assert np.all(np.abs(out - own.sum(1)) <= K * 2.0 ** -24 * np.abs(own).sum(1))
    hq = mxref.decode(*mxref.encode(h))
    whole = (w[..., None] * mxref.grouped(hq, dn, off)[0][slot.reshape(T, K)]).sum(1)
    assert np.linalg.norm(out - whole) <= 0.01 * np.linalg.norm(whole)


def test_path_replays_from_a_graph_and_on_two_streams():
    """Two paths with inputs of their own: captured, replayed on changed inputs with eager work between the
    replays, and run at once on two streams, every result equal to the eager one's bytes."""
    ps = [Path(29, 256, 128, 16, 2, 1), Path(150, 512, 128, 8, 3, 2)]
    eager = []
    for p in ps:
        p.run()
        eager.append(p.bytes())
    graphs = []
    for p in ps:
        g = torch.cuda.CUDAGraph()
        note(f"capture T={p.T}")
        with torch.cuda.graph(g):
            p.run()
        graphs.append(g)
    for i in range(4):
        for p, g, want in zip(ps, graphs, eager):
            for t in p.results:
                t.zero_()
            g.replay()
            assert all(np.array_equal(a, b) for a, b in zip(p.bytes(), want)), i
    for p, g in zip(ps, graphs):
        p.x.mul_(1.75)
        p.logits.neg_()
        g.replay()
        got = p.bytes()
        p.run()
        assert all(np.array_equal(a, b) for a, b in zip(p.bytes(), got))
    want = [p.bytes() for p in ps]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for p in ps:
        for t in p.results:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for p, st in zip(ps, streams):
            with torch.cuda.stream(st):
                p.run()
    for p, wt in zip(ps, want):
        assert all(np.array_equal(a, b) for a, b in zip(p.bytes(), wt))


def test_layer_is_the_path():
    """MoeMxfp4Layer's results are the path's bytes, for fewer tokens than its buffers hold, after a call of
    another size, from (codes, scales) and from float weights that those stand for."""
    p = Path(45, 256, 128, 16, 2, 9)
    p.run()
    want = p.bytes()[-1]
    floats = [torch.empty((m[0].shape[0], m[0].shape[1], 2 * m[0].shape[2]), device="cuda") for m in (p.gu, p.dn)]
    for f, m in zip(floats, (p.gu, p.dn)):
        abi.mxfp4_dequantize(m[0].flatten(0, 1), m[1].flatten(0, 1), f.flatten(0, 1))
    for gate_up, down in ((p.gu, p.dn), floats):
        layer = MoeMxfp4Layer(gate_up, down, max_tokens=70, K=2)
        assert (layer.E, layer.H, layer.F) == (16, 256, 128)
        layer.step(torch.randn(70, 256, device="cuda"), torch.randn(70, 16, device="cuda"))
        out = layer.step(p.x, p.logits)
        assert np.array_equal(host(out).view(np.uint8), want)
        idx, _ = layer.route(p.logits)
        for got, ref in zip(layer.balance(p.logits, idx), (p.counts, p.prob, p.loss, p.grad)):
            assert torch.equal(got, ref)
        with pytest.raises(ValueError):
            layer.step(torch.randn(71, 256, device="cuda"), torch.randn(71, 16, device="cuda"))
    with pytest.raises(ValueError):
        MoeMxfp4Layer(p.gu, p.gu, max_tokens=4, K=2)


def test_layer_refuses_what_does_not_fit_it():
    """Routes and logits of other sizes, types, layouts or devices than the layer's are refused before a
    launch: the maps would be written past their buffers, or read through a host address."""
    p = Path(12, 256, 128, 16, 2, 4)
    layer = MoeMxfp4Layer(p.gu, p.dn, max_tokens=12, K=2)
    idx, w = layer.route(p.logits)
    x = p.x
    more = torch.zeros((13, 2), dtype=torch.int32, device="cuda")
    wide = torch.zeros((12, 3), dtype=torch.int32, device="cuda")
    for bad in (more, wide, idx[:11], idx.long(), idx.cpu(), more.repeat(2, 1)[::2][:12], wide[:, :2]):
        with pytest.raises(ValueError):
            layer.forward(x, bad, w)
        with pytest.raises(ValueError):
            layer.balance(p.logits, bad)
    for bad in (w[:11], w.double(), w.cpu(), w.T.contiguous().T):
        with pytest.raises(ValueError):
            layer.forward(x, idx, bad)
    for bad in (p.logits[:, :15], p.logits.bfloat16(), p.logits.cpu(), torch.randn(12, 17, device="cuda")):
        with pytest.raises(ValueError):
            layer.route(bad)
    with pytest.raises(ValueError):
        layer.balance(torch.randn(12, 17, device="cuda"), idx)
    with pytest.raises(ValueError):
        layer.forward(x[:, :128], idx, w)
    with pytest.raises(ValueError):
        layer.forward(x, idx, w, out=torch.empty(12, 255, device="cuda"))
    with pytest.raises(ValueError):
        MoeMxfp4Layer(p.gu, p.dn, max_tokens=0, K=2)
    assert torch.equal(layer.forward(x, idx, w), layer.step(x, p.logits))
