"""What MoeTrainLayer refuses before anything is enqueued (CPU only: the library's calls are recorded, not
made)."""
import numpy as np
import pytest
import torch

from quantized_expert_grouped_amd import abi, layer
from quantized_expert_grouped_amd.layer import MoeTrainLayer

E, F, H, K, T = 3, 128, 256, 2, 6
B16 = torch.bfloat16
CALLS = ("build_maps", "mm_grouped", "mm_grouped_dgrad", "mm_grouped_wgrad", "combine_rows", "combine_rows_backward",
         "route_topk_backward")


@pytest.fixture
def calls(monkeypatch):
    done = []
    monkeypatch.setattr(abi, "_on_current", lambda t: t.get_device())
    abi._dtypes()
    for name in CALLS:
        monkeypatch.setattr(abi, name, lambda *a, name=name, **k: done.append(name))
    return done


def make(**kw):
    args = dict(gate_up=torch.zeros(E, 2 * F, H, dtype=B16), down=torch.zeros(E, H, F, dtype=B16), max_tokens=8, K=K,
                device="cpu")
    return MoeTrainLayer(**{**args, **kw})


def routes():
    return torch.zeros(T, K, dtype=torch.int32), torch.zeros(T, K)


def test_sharing_of_memory_is_exact():
    """Against the bytes themselves, for matrices anywhere in one small buffer."""
    rng = np.random.default_rng(0)
    buf, seen = torch.zeros(200, dtype=torch.uint8), [0, 0]
    for _ in range(4000):
        m = []
        for _ in range(2):
            size = int(rng.choice([1, 2, 4]))
            cols, n = int(rng.integers(1, 6)), int(rng.integers(1, 6))
            ld = cols + int(rng.integers(0, 9))
            room = 200 // size - ((n - 1) * ld + cols)
            if room < 0:
                break
            t = buf.view({1: torch.uint8, 2: B16, 4: torch.float32}[size])
            m.append(t[int(rng.integers(0, room + 1)):].as_strided((n, cols), (ld, 1)))
        if len(m) < 2:
            continue
        bytes_of = [{t.data_ptr() + (r * t.stride(0) + c) * t.element_size() + b for r in range(t.shape[0])
                     for c in range(t.shape[1]) for b in range(t.element_size())} for t in m]
        want = bool(bytes_of[0] & bytes_of[1])
        assert layer._share(*m) == layer._share(*m[::-1]) == want
        seen[want] += 1
    assert min(seen) > 300


def test_out_over_what_backward_reads_is_refused(calls):
    la, (idx, w) = make(), routes()
    both = torch.zeros(2 * T, H, dtype=B16)
    x = both[2:2 + T]
    for kw in (dict(out=x), dict(out=x, residual=x), dict(out=both[:T]), dict(out=both[T:], residual=both[T:]),
               dict(out=both.view(-1)[2 * H + 8:][:T * H].view(T, H))):
        with pytest.raises(ValueError, match="apart from x"):
            la.forward(x, idx, w, **kw)
    buf = torch.zeros(T * H)
    w = buf[H:H + T * K].view(T, K)
    with pytest.raises(ValueError, match="apart from w"):
        la.forward(x, idx, w, out=buf.view(T, H))
    assert not calls and la.kept is None


def test_out_beside_x_is_taken(calls):
    """Columns of one buffer, the buffer's other rows, the residual itself; one token next to another."""
    la, (idx, w) = make(), routes()
    wide, tall = torch.zeros(T, 2 * H, dtype=B16), torch.zeros(2 * T, H, dtype=B16)
    other = torch.zeros(T, H)
    for x, out, residual in ((wide[:, :H], wide[:, H:], None), (tall[:T], tall[T:], tall[T:]), (tall[T:], other, other),
                             (tall[::2], tall[1::2], None)):
        del calls[:]
        assert la.forward(x, idx, w, out=out, residual=residual) is out
        assert calls == ["build_maps", "mm_grouped", "mm_grouped", "combine_rows"]
    la.forward(tall[:1], idx[:1], w[:1], out=tall[1:2])


def test_out_partly_over_residual_is_refused(calls):
    """The same address with other strides, rows or columns further on."""
    la, (idx, w) = make(), routes()
    x, buf = torch.zeros(T, H, dtype=B16), torch.zeros(4 * T * H)
    out = buf.as_strided((T, H), (H, 1))
    for residual in (buf.as_strided((T, H), (2 * H, 1)), buf.as_strided((T, H), (H, 1), H),
                     buf.as_strided((T, H), (H, 1), 8), buf.as_strided((T, H), (2 * H, 1), (T - 1) * H)):
        for kw in (dict(out=out, residual=residual), dict(out=residual, residual=out)):
            with pytest.raises(ValueError, match="residual's very rows"):
                la.forward(x, idx, w, **kw)
    assert not calls and la.kept is None
    la.forward(x, idx, w, out=buf.as_strided((T, H), (2 * H, 1)), residual=buf.as_strided((T, H), (2 * H, 1), H))
    la.forward(x[:1], idx[:1], w[:1], out=buf.as_strided((1, H), (H, 1)), residual=buf.as_strided((1, H), (8, 1)))
    assert calls == 2 * ["build_maps", "mm_grouped", "mm_grouped", "combine_rows"]


def test_what_the_products_do_not_take_is_refused_before_the_maps(calls):
    """Of the layer's weights and sizes when it is made, of x by the forward (no value is touched: the large
    tensors are address space alone)."""
    odd = torch.zeros(E * 2 * F * H + 8, dtype=B16)
    for at in (1, 4, 7):
        with pytest.raises(ValueError, match="gate_up: an address"):
            make(gate_up=odd[at:at + E * 2 * F * H].view(E, 2 * F, H))
    with pytest.raises(ValueError, match="gate_up_bias: an address"):
        make(gate_up_bias=torch.zeros(E * 2 * F + 1, dtype=B16)[1:].view(E, 2 * F))
    assert make(gate_up=odd[8:].view(E, 2 * F, H)).E == E
    for h, f in ((1 << 15, 1 << 14), (1 << 21, 8), (8, 1 << 20)):
        with pytest.raises(ValueError, match="less than 2 GiB"):
            make(gate_up=torch.empty(1, 2 * f, h, dtype=B16), down=torch.empty(1, h, f, dtype=B16), K=1, max_tokens=1)
    with pytest.raises(ValueError, match="max_tokens"):
        make(max_tokens=(1 << 23) + 1)
    la = make(gate_up=torch.zeros(1, 16, 8, dtype=B16), down=torch.zeros(1, 8, 8, dtype=B16), K=1, max_tokens=1 << 12)
    for t, ld in ((2, 1 << 21), (1 << 12, (1 << 18) + 264), ((1 << 11) + 1, 1 << 19)):
        x = torch.empty((t - 1) * ld + 8, dtype=B16).as_strided((t, 8), (ld, 1))
        with pytest.raises(ValueError, match="x: less than 2 GiB"):
            la.forward(x, torch.zeros(t, 1, dtype=torch.int32), torch.zeros(t, 1))
    assert not calls and la.kept is None
    t, ld = 1 << 11, 1 << 19                                     # the largest below
    x = torch.empty((t - 1) * ld + 8, dtype=B16).as_strided((t, 8), (ld, 1))
    la.forward(x, torch.zeros(t, 1, dtype=torch.int32), torch.zeros(t, 1))
    la.forward(x[:1].as_strided((1, 8), (1 << 22, 1)), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 1))
    assert len(calls) == 8


def test_the_librarys_own_limits_are_the_layers():
    """The sizes on both sides of the layer's limits, put to the C entry points (made-up pointers, refused or
    not before anything is followed: a size that is taken is not called)."""
    P, lib = 1 << 20, abi.lib()

    def mm(n_act, lda, k=8, n=8, w=P):
        return lib.moe_mm_grouped(w, 1, n, k, P, 1, P, lda, n_act, P, 1, 1, None, 1, None, 0, None, 0, P, 1, n, None)

    assert mm(2, 1 << 21) == mm(1 << 12, (1 << 18) + 264) == mm((1 << 11) + 1, 1 << 19) == -2
    assert mm(4, 8, k=1 << 15, n=1 << 14) == mm(4, 1 << 21, k=1 << 21) == -2 and mm(4, 8, w=P + 8) == -1
    assert lib.moe_mm_grouped_wgrad_workspace_size(1 << 20, 1 << 21, 8, 1) == 0
    assert lib.moe_combine_rows(P, 1, 8, 8, P, P, (1 << 23) + 1, 1, 8, None, 0, P, 1, 8, None) == -2


def test_router_gradient_of_another_expert_count_is_refused(calls):
    """Routes to the layer's last experts would be lost in fewer columns without a word."""
    la, (idx, w) = make(), routes()
    for shape in ((T, E - 1), (T, E + 1), (T - 1, E), (T * E,)):
        with pytest.raises(ValueError, match="grad_logits"):
            la.route_backward(idx, w, w, torch.zeros(shape))
    assert not calls
    assert la.route_backward(idx, w, w).shape == la.route_backward(idx, w, w, torch.zeros(T, E)).shape == (T, E)
    assert calls == 2 * ["route_topk_backward"]
