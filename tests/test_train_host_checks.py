"""What the training entry points and MoeTrainLayer refuse before anything is enqueued (CPU only: no call here
reaches a kernel; pointers are made up and never followed)."""
import pytest
import torch

from quantized_expert_grouped_amd import abi
from quantized_expert_grouped_amd.layer import MoeTrainLayer

P = 1 << 20            # 16-byte aligned
EINVAL, EUNSUPPORTED, EWORKSPACE = -1, -2, -3
BIG = 1 << 31


class Call:
    def __init__(self, name, **ok):
        self.fn, self.ok = getattr(abi.lib(), name), ok

    def __call__(self, **kw):
        assert not kw.keys() - self.ok.keys()
        return self.fn(*{**self.ok, **kw}.values())


@pytest.fixture
def calls():
    return {
        "dispatch": Call("moe_dispatch_rows", x=P, dtype=1, ldx=64, T=8, H=64, src=P, K=2, rows=16, out=P, ldo=64,
                         stream=None),
        "combine": Call("moe_combine_rows", rows=P, dtype=1, ldr=64, n_rows=16, slot=P, w=None, T=8, K=2, H=64,
                        residual=None, ldres=0, out=P, odt=1, ldo=64, stream=None),
        "combine_backward": Call("moe_combine_rows_backward", grad=P, gdt=1, ldg=64, slot=P, w=P, T=8, K=2, H=64,
                                 n_rows=16, rows=P, dtype=1, ldr=64, grad_rows=P, ldgr=64, grad_w=P, stream=None),
        "mm": Call("moe_mm_grouped", w=P, dtype=1, n_out=64, k_in=64, offsets=P, E=4, a=P, lda=64, n_act=16, src=None,
                   K=0, rows=16, bias=None, act=0, residual=None, ldres=0, z=None, ldz=0, out=P, odt=1, ldo=64,
                   stream=None),
        "dgrad": Call("moe_mm_grouped_dgrad", w=P, dtype=1, n_out=64, k_in=64, offsets=P, E=4, grad=P, ldg=64, rows=16,
                      z=None, ldz=0, out=P, odt=1, ldo=64, stream=None),
        "wgrad": Call("moe_mm_grouped_wgrad", grad=P, dtype=1, ldg=64, n_out=64, a=P, lda=64, k_in=64, n_act=16,
                      src=None, K=0, offsets=P, E=4, rows=16, grad_w=P, odt=1, grad_bias=None, ws=P, ws_bytes=1 << 40,
                      stream=None),
        "route": Call("moe_route_topk_backward", idx=P, w=P, gw=P, T=8, E=16, K=2, acc=0, grad=P, dtype=0, ld=16,
                      stream=None),
    }


def refused(call, status, cases):
    for kw in cases:
        assert call(**kw) == status, kw


def test_dispatch(calls):
    refused(calls["dispatch"], EINVAL, [dict(x=None), dict(src=None), dict(out=None), dict(T=0), dict(H=0), dict(K=0),
                                        dict(rows=0), dict(rows=-3), dict(ldx=63), dict(ldo=63), dict(x=P + 1),
                                        dict(out=P + 1), dict(dtype=0, x=P + 2), dict(ldx=0)])
    refused(calls["dispatch"], EUNSUPPORTED, [dict(dtype=3), dict(dtype=-1), dict(K=65), dict(T=1 << 30),
                                              dict(rows=(1 << 23) + 1)])


def test_combine(calls):
    refused(calls["combine"], EINVAL, [dict(rows=None), dict(slot=None), dict(out=None), dict(T=0), dict(K=0), dict(H=0),
                                       dict(n_rows=0), dict(ldr=63), dict(ldo=63), dict(residual=P + 64, ldres=63),
                                       dict(residual=P + 1, ldres=64), dict(odt=0, out=P + 2),
                                       dict(out=P, residual=P, ldres=72)])
    refused(calls["combine"], EUNSUPPORTED, [dict(dtype=5), dict(odt=2), dict(dtype=0, odt=1), dict(K=65), dict(T=1 << 29),
                                             dict(n_rows=(1 << 30) + 1)])


def test_combine_backward(calls):
    c = calls["combine_backward"]
    refused(c, EINVAL, [dict(grad=None), dict(slot=None), dict(rows=None), dict(grad_rows=None, grad_w=None), dict(T=0),
                        dict(ldg=63), dict(ldr=63), dict(ldgr=63), dict(grad_rows=P + 1), dict(n_rows=0),
                        dict(grad_rows=P, ldgr=72)])
    refused(c, EUNSUPPORTED, [dict(dtype=3), dict(gdt=2), dict(dtype=0, gdt=1), dict(K=65), dict(T=(1 << 23) + 1)])


def test_product(calls):
    c = calls["mm"]
    refused(c, EINVAL, [dict(w=None), dict(offsets=None), dict(a=None), dict(out=None), dict(n_out=0), dict(k_in=0),
                        dict(E=0), dict(rows=0), dict(act=2), dict(act=-1), dict(n_act=0), dict(n_act=15),
                        dict(src=P, K=0), dict(z=P, ldz=128), dict(act=1, residual=P, ldres=64), dict(w=P + 8),
                        dict(a=P + 8), dict(out=P + 8), dict(lda=68), dict(ldo=68), dict(lda=56), dict(bias=P + 2),
                        dict(residual=P + 64, ldres=60), dict(act=1, z=P, ldz=64), dict(odt=0, ldo=66),
                        dict(residual=P, ldres=72)])
    refused(c, EUNSUPPORTED, [dict(dtype=0), dict(dtype=3), dict(odt=2), dict(act=1, odt=0), dict(n_out=60, ldo=64),
                              dict(k_in=60), dict(E=2049), dict(src=P, K=65), dict(n_out=32768, k_in=32768),
                              dict(act=1, n_out=16384, k_in=32768), dict(k_in=1 << 21, n_out=8),
                              dict(src=P, K=2, n_act=1 << 26), dict(lda=1 << 21), dict(rows=(1 << 30) + 1, n_act=BIG - 1)])


def test_input_gradient(calls):
    c = calls["dgrad"]
    refused(c, EINVAL, [dict(w=None), dict(offsets=None), dict(grad=None), dict(out=None), dict(rows=0), dict(ldg=56),
                        dict(ldg=68), dict(ldo=56), dict(z=P + 64, ldz=64, ldo=128), dict(z=P + 64, ldz=128, ldo=64),
                        dict(z=P, ldz=128, ldo=136), dict(grad=P + 4)])
    refused(c, EUNSUPPORTED, [dict(dtype=0), dict(odt=2), dict(z=P, ldz=128, ldo=128, odt=0), dict(k_in=4), dict(n_out=12),
                              dict(E=4096), dict(ldg=1 << 21), dict(n_out=32768, k_in=32768)])


def test_weight_gradient(calls):
    c = calls["wgrad"]
    refused(c, EINVAL, [dict(grad=None), dict(a=None), dict(offsets=None), dict(grad_w=None), dict(n_act=15), dict(rows=0),
                        dict(src=P, K=-1), dict(ldg=56), dict(lda=68), dict(grad_w=P + 8), dict(grad_bias=P + 4)])
    refused(c, EUNSUPPORTED, [dict(dtype=0), dict(odt=2), dict(k_in=12), dict(E=2049), dict(src=P, K=65), dict(ldg=1 << 21)])
    need = abi.mm_grouped_wgrad_workspace_size(16, 64, 64, 4)
    if need:
        refused(c, EWORKSPACE, [dict(ws_bytes=need - 1)])
        refused(c, EINVAL, [dict(ws=None), dict(ws=P + 8)])


def test_weight_gradient_workspace():
    """Never less for more rows (a layer sizes it by its largest call), 0 for what the call refuses."""
    size = abi.mm_grouped_wgrad_workspace_size
    for N, k, E in ((64, 64, 1), (4096, 4096, 1), (512, 2048, 8), (2048, 512, 512), (264, 520, 3)):
        got = [size(r, N, k, E) for r in (1, 2, 63, 64, 100, 1000, 4096, 8191, 30000, 1 << 20)]
        assert got == sorted(got) and got[-1] < 1 << 30, got
    assert size(0, 64, 64, 1) == size(64, 60, 64, 1) == size(64, 64, 64, 0) == size(64, 64, 64, 4096) == 0


def test_router_gradient(calls):
    c = calls["route"]
    refused(c, EINVAL, [dict(idx=None), dict(w=None), dict(gw=None), dict(grad=None), dict(T=0), dict(K=0), dict(K=17),
                        dict(ld=15), dict(grad=P + 2)])
    refused(c, EUNSUPPORTED, [dict(dtype=3), dict(E=4096, ld=4096), dict(E=100, K=65, ld=100), dict(T=(1 << 23) + 1)])


# ---- the binding ------------------------------------------------------------------------------
def test_the_binding_refuses_what_the_library_cannot_see(monkeypatch):
    monkeypatch.setattr(abi, "_on_current", lambda t: t.get_device())
    monkeypatch.setattr(abi, "_current_stream", lambda stream, device: 0)
    abi._dtypes()
    b16, i32 = torch.bfloat16, torch.int32
    x, src, rows = torch.zeros(4, 64, dtype=b16), torch.zeros(8, dtype=i32), torch.zeros(8, 64, dtype=b16)
    slot, w = torch.zeros(4, 2, dtype=i32), torch.zeros(4, 2)
    off, wt = torch.zeros(4, dtype=i32), torch.zeros(3, 32, 64, dtype=b16)
    out = torch.zeros(8, 32, dtype=b16)
    bad = [
        lambda: abi.dispatch_rows(x, src.long(), rows, K=2), lambda: abi.dispatch_rows(x, src[:7], rows, K=2),
        lambda: abi.dispatch_rows(x, src, rows.half(), K=2), lambda: abi.dispatch_rows(x, src, rows[:, :60], K=2),
        lambda: abi.dispatch_rows(x.double(), src, rows.double(), K=2), lambda: abi.dispatch_rows(x.t(), src, rows, K=2),
        lambda: abi.combine_rows(rows, slot, w.double(), x), lambda: abi.combine_rows(rows, slot, w[:3], x),
        lambda: abi.combine_rows(rows, slot.view(-1)[:7], w, x), lambda: abi.combine_rows(rows, slot.long(), w, x),
        lambda: abi.combine_rows(rows, slot, w, x[:, :32]), lambda: abi.combine_rows(rows, slot, w, x, residual=x.float()),
        lambda: abi.combine_rows(rows, slot.t(), w, x), lambda: abi.combine_rows_backward(x, slot, w),
        lambda: abi.combine_rows_backward(x, slot, w, rows, rows=rows),
        lambda: abi.combine_rows_backward(x, slot, w, rows, grad_w=w),
        lambda: abi.combine_rows_backward(x, slot, w, rows, rows=rows.half(), grad_w=w),
        lambda: abi.mm_grouped(wt, off, rows, out.double()), lambda: abi.mm_grouped(wt, off[:3], rows, out),
        lambda: abi.mm_grouped(wt, off.long(), rows, out), lambda: abi.mm_grouped(wt.transpose(1, 2), off, rows, out),
        lambda: abi.mm_grouped(wt, off, rows.half(), out), lambda: abi.mm_grouped(wt, off, rows, out, swiglu=True),
        lambda: abi.mm_grouped(wt, off, rows, out, bias=torch.zeros(3, 32)),
        lambda: abi.mm_grouped(wt, off, rows, out, residual=out.float()),
        lambda: abi.mm_grouped(wt, off, x, out, src=src[:7], K=2),
        lambda: abi.mm_grouped(wt[:, :31], off, rows, out, swiglu=True),
        lambda: abi.mm_grouped_dgrad(wt, off, out, rows[:, :32]), lambda: abi.mm_grouped_dgrad(wt, off, out, rows, z=rows),
        lambda: abi.mm_grouped_dgrad(wt, off, out.half(), rows),
        lambda: abi.mm_grouped_wgrad(out, off, rows, wt[:, :16]), lambda: abi.mm_grouped_wgrad(out, off, rows, wt.double()),
        lambda: abi.mm_grouped_wgrad(out, off, rows, wt, grad_bias=torch.zeros(3, 32)),
        lambda: abi.route_topk_backward(slot, w, w[:, :1], torch.zeros(4, 8)),
        lambda: abi.route_topk_backward(slot.long(), w, w, torch.zeros(4, 8)),
        lambda: abi.route_topk_backward(slot, w, w, torch.zeros(4, 8).double()),
        lambda: abi.route_topk_backward(slot, w, w, torch.zeros(5, 8)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was taken")
    # and what only the C side sees, through the binding
    for f in (lambda: abi.mm_grouped(wt, off, rows[0].expand(8, 64), out), lambda: abi.dispatch_rows(x, src, rows, K=0),
              lambda: abi.mm_grouped_dgrad(wt, off, out, torch.zeros(8, 66, dtype=b16)[:, :64])):
        with pytest.raises(abi.MoeError):
            f()


# ---- the layer --------------------------------------------------------------------------------
def make(E=3, F=128, H=256, K=2, max_tokens=4, dtype=torch.bfloat16, **kw):
    args = dict(gate_up=torch.zeros(E, 2 * F, H, dtype=dtype), down=torch.zeros(E, H, F, dtype=dtype), max_tokens=max_tokens,
                K=K, device="cpu")
    return MoeTrainLayer(**{**args, **kw})


def test_layer_takes_and_refuses():
    b16 = torch.bfloat16
    la = make(gate_up_bias=torch.zeros(3, 256, dtype=b16), down_bias=torch.zeros(3, 256, dtype=b16))
    assert (la.E, la.H, la.F, la.K) == (3, 256, 128, 2) and la.z.shape == (8, 256) and la.kept is None
    w = torch.zeros(3, 256, 256, dtype=b16)
    assert make(gate_up=w).gate_up.data_ptr() == w.data_ptr()           # held
    wt = w.transpose(1, 2)
    assert make(gate_up=wt).gate_up.is_contiguous()
    for kw in (dict(gate_up=w.float()), dict(gate_up=w[0]), dict(gate_up=w[:, :255]), dict(down=w), dict(down=w.half()),
               dict(gate_up_bias=torch.zeros(3, 256)), dict(gate_up_bias=torch.zeros(3, 128, dtype=b16)),
               dict(down_bias=torch.zeros(256, dtype=b16)), dict(K=0), dict(K=4), dict(max_tokens=0), dict(H=252), dict(F=124),
               dict(E=abi.MAX_E + 1, F=8, H=8), dict(E=80, K=65, F=8, H=8)):
        with pytest.raises(ValueError):
            make(**kw)
    assert make(E=abi.MAX_E, K=abi.MAX_K, F=8, H=8).K == abi.MAX_K
    assert make(dtype=torch.float16).rows.dtype == torch.float16


def test_parameters_that_require_gradients_are_taken():
    w = torch.nn.Parameter(torch.zeros(3, 256, 256, dtype=torch.bfloat16))
    la = make(gate_up=w)
    assert not la.gate_up.requires_grad and la.gate_up.data_ptr() == w.data_ptr()


@pytest.mark.parametrize("N,k,E", [(64, 64, 1), (1024, 1024, 1), (2048, 2048, 1), (512, 512, 4)])
def test_weight_gradient_with_parts_refuses_what_is_no_workspace(calls, N, k, E):
    """Sizes whose rows are taken in parts, which the workspace holds (256 x 256 tiles among them)."""
    kw = dict(n_out=N, ldg=N, k_in=k, lda=k, E=E, rows=8192, n_act=8192)
    need = abi.mm_grouped_wgrad_workspace_size(8192, N, k, E)
    assert need > E * N * k * 4                                 # two parts at least
    refused(calls["wgrad"], EWORKSPACE, [dict(kw, ws_bytes=v) for v in (need - 1, need // 2, 0)])
    refused(calls["wgrad"], EINVAL, [dict(kw, ws=None, ws_bytes=need), dict(kw, ws=P + 8, ws_bytes=need),
                                     dict(kw, ws=None, ws_bytes=0)])
    assert abi.mm_grouped_wgrad_workspace_size(255 * E, N, k, E) == 0   # one part
