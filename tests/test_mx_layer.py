"""What MoeMxfp4Layer takes and refuses when it is made (CPU only: its buffers are host tensors here and no
call reaches a kernel)."""
import os
import re

import numpy as np
import pytest
import torch

from quantized_expert_grouped_amd import abi
from quantized_expert_grouped_amd.layer import MoeMxfp4Layer

E, H, F = 3, 256, 128


def pairs(seed=0):
    g = torch.Generator().manual_seed(seed)

    def rand(*shape):
        return torch.randint(0, 256, shape, dtype=torch.uint8, generator=g)

    return ((rand(E, 2 * F, H // 2), rand(E, 2 * F, H // 32)), (rand(E, H, F // 2), rand(E, H, F // 32)))


def make(gate_up, down, max_tokens=4, K=2):
    return MoeMxfp4Layer(gate_up, down, max_tokens=max_tokens, K=K, device="cpu")


def test_weights_in_bytes_or_in_torchs_types_for_them():
    """float8_e8m0fnu scales and float4_e2m1fn_x2 codes are taken as the bytes they are, in any layout."""
    gate_up, down = pairs()
    want = make(gate_up, down)
    for t, b in zip(want.gate_up + want.down, gate_up + down):
        assert t.dtype == torch.uint8 and torch.equal(t, b)

    def typed(p):
        return p[0].view(torch.float4_e2m1fn_x2), p[1].view(torch.float8_e8m0fnu)

    def turned(p):                                            # the same values, strides the other way
        return tuple(t.transpose(0, 2).contiguous().transpose(0, 2) for t in p)

    def arrays(p):
        return [t.numpy() for t in p]

    for form in (typed, turned, arrays):
        got = make(form(gate_up), form(down))
        for t, b in zip(got.gate_up + got.down, gate_up + down):
            assert t.dtype == torch.uint8 and t.is_contiguous() and torch.equal(t, b), form
    scales = torch.tensor([0.125, 0.5, 1.0, 8.0]).to(torch.float8_e8m0fnu).repeat(E * 2 * F * 2)
    got = make((gate_up[0], scales.view(E, 2 * F, H // 32)), down).gate_up[1]
    assert got[0, 0].tolist() == [124, 126, 127, 130] * 2


def test_weights_that_are_not_bytes_are_refused():
    gate_up, down = pairs()
    (gc, gs), (dc, ds) = gate_up, down
    for bad in ((gc.int(), gs), (gc.view(torch.int8), gs), (gc.float(), gs), (gc, gs.float()),
                (gc, gs.int()), (gc, gs.view(torch.int8)), (gc, gs.bfloat16()),
                (gc, gs.view(torch.float8_e4m3fn)), (gc.view(torch.float8_e8m0fnu), gs),
                (gc, gs.view(torch.float4_e2m1fn_x2)), (gc.numpy().astype(np.int64), gs)):
        with pytest.raises(ValueError):
            make(bad, down)
    with pytest.raises(ValueError):
        make(gate_up, (dc, ds.float()))


def test_weights_whose_scales_do_not_fit_are_refused():
    gate_up, down = pairs()
    (gc, gs), (dc, ds) = gate_up, down
    for bad in ((gc, gs[..., :-1]), (gc, gs[:-1]), (gc, gs[:, :F]), (gc, gs.flatten(1)), (gc[:-1], gs),
                (gc.flatten(1), gs), (gc, gs, gs), (gc[..., :120], gs[..., :7])):
        with pytest.raises(ValueError):
            make(bad, down)
    for bad in ((dc, ds[..., :2]), (dc, ds[:, :-32]), gate_up):
        with pytest.raises(ValueError):
            make(gate_up, bad)


def test_more_experts_or_routes_than_the_library_takes_are_refused():
    text = open(os.path.join(os.path.dirname(__file__), "..", "include", "moe_prefill.h")).read()
    for name, value in (("MOE_MAX_E", abi.MAX_E), ("MOE_MAX_K", abi.MAX_K)):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == value

    def layer(n, K):
        u8 = torch.uint8
        return MoeMxfp4Layer((torch.zeros(n, 256, 64, dtype=u8), torch.zeros(n, 256, 4, dtype=u8)),
                             (torch.zeros(n, 128, 64, dtype=u8), torch.zeros(n, 128, 4, dtype=u8)),
                             max_tokens=2, K=K, device="cpu")

    assert layer(abi.MAX_E, abi.MAX_K).K == abi.MAX_K
    for n, K in ((abi.MAX_E + 1, 2), (80, abi.MAX_K + 1), (3, 4), (3, 0)):
        with pytest.raises(ValueError):
            layer(n, K)


@pytest.mark.parametrize("default", [torch.float32, torch.bfloat16, torch.float64])
def test_balance_makes_its_outputs_in_the_types_the_library_takes(default, monkeypatch):
    """Whatever torch's default type is.  The library's calls are replaced: their arguments are looked at."""
    layer = make(*pairs())
    seen = []
    monkeypatch.setattr(abi, "_on_current", lambda t: t.get_device())
    monkeypatch.setattr(abi, "balance_loss", lambda *a, **k: seen.extend(a))
    monkeypatch.setattr(abi, "balance_loss_backward", lambda *a, **k: seen.extend(a))
    logits, idx = torch.zeros(4, E, dtype=torch.float16), torch.zeros(4, 2, dtype=torch.int32)
    before = torch.get_default_dtype()
    torch.set_default_dtype(default)
    try:
        counts, prob, loss, grad = layer.balance(logits, idx)
    finally:
        torch.set_default_dtype(before)
    assert seen[2] is counts and seen[3] is prob and seen[4] is loss and seen[-1] is grad
    assert (counts.dtype, prob.dtype, loss.dtype) == (torch.int32, torch.float32, torch.float32)
    assert (counts.shape, prob.shape, loss.shape) == ((E + 1,), (E,), (1,))
    assert grad.dtype == torch.float16 and grad.shape == logits.shape


def test_forward_refuses_x_and_out_before_it_enqueues_anything(monkeypatch):
    layer = make(*pairs())
    done = []
    monkeypatch.setattr(abi, "_on_current", lambda t: t.get_device())
    monkeypatch.setattr(abi, "_current_stream", lambda stream, device: 0)
    for name in ("build_maps", "mxfp4_mm_grouped", "combine_bf16"):
        monkeypatch.setattr(abi, name, lambda *a, _name=name, **k: done.append(_name))
    real = abi.mxfp4_quantize
    monkeypatch.setattr(abi, "mxfp4_quantize", lambda *a: (real(*a), done.append("mxfp4_quantize")))
    idx, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    x = torch.zeros(4, H)
    apart = torch.zeros(4 * (H + 8))
    for bad in (x[:, :128], torch.zeros(4, 2 * H), torch.zeros(4, H + 32), torch.zeros(4, H + 1), x.double(),
                x.int(), x.t().contiguous().t(), x[0].expand(4, H), apart[1:1 + 4 * H].view(4, H),
                torch.zeros(4, H + 1)[:, :H]):
        with pytest.raises((ValueError, abi.MoeError)):
            layer.forward(bad, idx, w)
        assert not done
    for bad in (torch.zeros(4, H - 1), torch.zeros(5, H), torch.zeros(4, H).bfloat16(),
                torch.zeros(4, 2 * H)[:, :H], apart[1:1 + 4 * H].view(4, H)):
        with pytest.raises(ValueError):
            layer.forward(x, idx, w, out=bad)
        assert not done


def test_the_current_stream_without_torchs_private_function(monkeypatch):
    class Stream:
        cuda_stream = 0x1230

    abi._dtypes()
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0x4560 + device, raising=False)
    assert abi._current_stream(None, 2) == 0x4562
    assert abi._current_stream(Stream, 0) == 0x1230 and abi._current_stream(7, 0) == 7
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    assert abi._current_stream(None, 0) == 0x1230


def test_the_rows_type_is_the_callers_choice():
    gate_up, down = pairs()
    assert make(gate_up, down).rows.dtype == torch.bfloat16
    for t in (torch.bfloat16, torch.float32):
        layer = MoeMxfp4Layer(gate_up, down, max_tokens=4, K=2, device="cpu", rows_dtype=t)
        assert layer.rows.dtype == t and layer.rows.shape == (8, H)
    for t in (torch.float16, torch.float64, torch.uint8):
        with pytest.raises(ValueError):
            MoeMxfp4Layer(gate_up, down, max_tokens=4, K=2, device="cpu", rows_dtype=t)
