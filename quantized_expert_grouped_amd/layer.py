"""A prefill MoE expert layer held on one GPU: the expert pool and the workspace stay resident in
HBM, and each call enqueues routing and the layer on the current torch stream.

Marshalling only -- the computation is libmoe_prefill.so's (see ``abi``).
"""
from __future__ import annotations

import numpy as np
import torch

from . import abi


class MoePrefillLayer:
    def __init__(self, pool, expert_off, H: int, F: int, E: int, wtype: int, max_tokens: int,
                 K: int, group_size: int = 16, ring_start: int = 0, device="cuda"):
        self.H, self.F, self.E, self.K, self.wtype = H, F, E, K, wtype
        self.group_size, self.ring_start = group_size, ring_start
        self.device = torch.device(device)
        self.pool = _to_device(pool, torch.uint8, self.device)
        self.expert_off = _to_device(expert_off, torch.int64, self.device)
        self.expert_bytes = abi.expert_bytes(H, F, wtype)
        self.max_tokens = max_tokens
        nbytes = abi.workspace_size(max_tokens, H, F, E, K, wtype, group_size)
        if nbytes == 0:
            raise ValueError("unsupported layer shape")
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)

    def route(self, logits: torch.Tensor):
        T = logits.shape[0]
        idx = torch.empty((T, self.K), dtype=torch.int32, device=self.device)
        w = torch.empty((T, self.K), dtype=torch.float32, device=self.device)
        abi.route_topk(logits, self.K, idx, w)
        return idx, w

    def forward(self, x: torch.Tensor, idx: torch.Tensor, w: torch.Tensor,
                out: torch.Tensor | None = None, group_size: int | None = None,
                ring_start: int | None = None) -> torch.Tensor:
        T = x.shape[0]
        if T > self.max_tokens:
            raise ValueError(f"T={T} exceeds the workspace's {self.max_tokens} tokens")
        if out is None:
            out = torch.empty((T, self.H), dtype=torch.float32, device=self.device)
        gs = self.group_size if group_size is None else group_size
        rs = self.ring_start if ring_start is None else ring_start
        abi.prefill_layer(x, idx, w, self.wtype, self.pool, self.expert_off, self.F, self.E, gs,
                          rs, self.ws, out)
        return out

    def pack_pool(self) -> torch.Tensor:
        """The pool with every expert put in the MMQ layout at its own offset (one gather launch
        per expert; done once, the experts never change), for forward_packed."""
        off = self.expert_off.cpu().numpy()
        if np.any(off % 16 != 0):
            raise ValueError("the packed layer reads experts at 16-byte aligned offsets only")
        packed = torch.zeros_like(self.pool)
        base, dst = self.pool.data_ptr(), packed.data_ptr()
        for e in range(self.E):
            o = int(off[e])
            abi.gather_group_mmq([base + o], self.wtype, self.H, self.F, dst + o, 0, 0)
        self.packed = packed
        return packed

    def forward_packed(self, x: torch.Tensor, idx: torch.Tensor, w: torch.Tensor,
                       out: torch.Tensor | None = None, ring_start: int | None = None):
        """The layer reading the packed pool in place (no gather); pack_pool() first."""
        T = x.shape[0]
        if T > self.max_tokens:
            raise ValueError(f"T={T} exceeds the workspace's {self.max_tokens} tokens")
        if out is None:
            out = torch.empty((T, self.H), dtype=torch.float32, device=self.device)
        rs = self.ring_start if ring_start is None else ring_start
        abi.prefill_layer_packed(x, idx, w, self.wtype, self.packed, self.expert_off, self.F,
                                 self.E, rs, self.ws, out)
        return out

    def step(self, x: torch.Tensor, logits: torch.Tensor, out: torch.Tensor | None = None):
        """One pass of the whole hot path: routing, then the layer."""
        idx, w = self.route(logits)
        return self.forward(x, idx, w, out)

    def ws_view(self, which: int, T: int, nbytes: int) -> torch.Tensor:
        off = abi.workspace_offset(which, T, self.H, self.F, self.E, self.K, self.wtype,
                                   self.group_size)
        return self.ws[off:off + nbytes]


class MoeMxfp4Layer:
    """The layer over experts in MXFP4, held on one GPU: routing, maps, the tokens quantised once,
    gate/up with SwiGLU and requantisation, down into rows of rows_dtype, combine.  bfloat16 rows
    are half the bytes (at long prompts fp32 ones are more than all weights) and one rounding,
    2^-8 of a value; float32 rows none.  gate_up [E, 2F, H]
    (gate's F rows, then up's) and down [E, H, F]: floating-point tensors, quantised here once, or
    pairs of codes (uint8 or float4_e2m1fn_x2 [E, rows, k / 2]) and scales (uint8 or float8_e8m0fnu
    [E, rows, k / 32]).  H and F: multiples of 128.  A layer's calls share its buffers, so they
    must not overlap."""

    def __init__(self, gate_up, down, max_tokens: int, K: int, device="cuda",
                 rows_dtype: torch.dtype = torch.bfloat16):
        if rows_dtype not in (torch.bfloat16, torch.float32):
            raise ValueError(f"rows_dtype: bfloat16 or float32 is wanted, not {rows_dtype}")
        self.device = torch.device(device)
        self.gate_up, self.down = self._weights(gate_up), self._weights(down)
        self.E, f2, hb = self.gate_up[0].shape
        self.H, self.F = 2 * hb, f2 // 2
        if self.down[0].shape != (self.E, self.H, self.F // 2) or f2 % 2:
            raise ValueError("gate_up [E, 2F, H] and down [E, H, F] do not fit each other")
        if self.H % 128 or self.F % 128 or not 1 <= K <= min(self.E, abi.MAX_K):
            raise ValueError(f"H and F are multiples of 128, K one of 1 .. E, {abi.MAX_K} at most")
        if self.E > abi.MAX_E:
            raise ValueError(f"E={self.E} exceeds {abi.MAX_E}")
        if max_tokens < 1:
            raise ValueError("max_tokens is at least 1")
        self.max_tokens, self.K = max_tokens, K
        R = max_tokens * K
        self.counts, self.offsets = self._i32(self.E), self._i32(self.E + 1)
        self.src, self.slot = self._i32(R), self._i32(R)
        self.order, self.n_active = self._i32(self.E), self._i32(1)
        self.maps_ws = self._u8(abi.build_maps_workspace_size(max_tokens, K, self.E))
        self.x_codes = self._u8(max_tokens, self.H // 2)
        self.x_scales = self._u8(max_tokens, self.H // 32)
        self.h_codes, self.h_scales = self._u8(R, self.F // 2), self._u8(R, self.F // 32)
        self.rows = torch.empty((R, self.H), dtype=rows_dtype, device=self.device)
        self.balance_ws = self._u8(abi.balance_workspace_size(max_tokens, self.E))

    def _u8(self, *shape):
        return torch.empty(shape, dtype=torch.uint8, device=self.device)

    def _i32(self, n: int):
        return torch.empty(n, dtype=torch.int32, device=self.device)

    def _weights(self, w):
        if isinstance(w, (tuple, list)):
            codes, scales = w
            codes = _mx_bytes("codes", codes, torch.float4_e2m1fn_x2, self.device)
            scales = _mx_bytes("scales", scales, torch.float8_e8m0fnu, self.device)
            E, N, kb = codes.shape
            if scales.shape != (E, N, kb // 16) or kb % 16:
                raise ValueError(f"scales: {(E, N, kb // 16)} are wanted for codes {(E, N, kb)}, "
                                 f"not {tuple(scales.shape)}")
            return codes, scales
        w = w.to(self.device).contiguous()
        E, N, k = w.shape
        codes, scales = self._u8(E, N, k // 2), self._u8(E, N, k // 32)
        abi.mxfp4_quantize(w.view(E * N, k), codes.view(E * N, -1), scales.view(E * N, -1))
        return codes, scales

    def _tokens(self, t: torch.Tensor, idx: torch.Tensor) -> int:
        T = t.shape[0]
        if T > self.max_tokens:
            raise ValueError(f"T={T} exceeds the buffers' {self.max_tokens} tokens")
        self._want(("idx", idx, torch.int32, (T, self.K)))
        return T

    def _want(self, *wants):
        """Routing and maps take pointers: what they read and write has to fit the layer."""
        abi._want(abi._on_current(self.src), *wants)

    def route(self, logits: torch.Tensor):
        T = logits.shape[0]
        self._want(("logits", logits, torch.float32, (T, self.E)))
        idx = torch.empty((T, self.K), dtype=torch.int32, device=self.device)
        w = torch.empty((T, self.K), dtype=torch.float32, device=self.device)
        abi.route_topk(logits, self.K, idx, w)
        return idx, w

    def balance(self, logits: torch.Tensor, idx: torch.Tensor, valid: torch.Tensor | None = None,
                grad_loss: torch.Tensor | None = None):
        """The router's counts int32 [E + 1] (the valid tokens last), mean probabilities, balance loss
        and the loss's gradient (times grad_loss) with respect to the logits."""
        self._tokens(logits, idx)
        counts, grad = self._i32(self.E + 1), torch.empty_like(logits)
        prob, loss = (torch.empty(n, dtype=torch.float32, device=self.device) for n in (self.E, 1))
        abi.balance_loss(logits, idx, counts, prob, loss, self.balance_ws, valid=valid)
        abi.balance_loss_backward(logits, counts, self.K, grad, valid=valid, grad_loss=grad_loss)
        return counts, prob, loss, grad

    def forward(self, x: torch.Tensor, idx: torch.Tensor, w: torch.Tensor,
                out: torch.Tensor | None = None) -> torch.Tensor:
        T = self._tokens(x, idx)
        self._want(("w", w, torch.float32, (T, self.K)), ("out", out, torch.float32, (T, self.H)))
        R = T * self.K
        if out is None:
            out = torch.empty((T, self.H), dtype=torch.float32, device=self.device)
        elif out.data_ptr() % 16:
            raise ValueError("out: an address that is a multiple of 16 is wanted")
        src, slot, rows = self.src[:R], self.slot[:R], self.rows[:R]
        x_codes, x_scales = self.x_codes[:T], self.x_scales[:T]
        h_codes, h_scales = self.h_codes[:R], self.h_scales[:R]
        abi.mxfp4_quantize(x, x_codes, x_scales)  # first: it looks x over
        abi.build_maps(idx, self.E, 0, self.counts, self.offsets, src, slot, self.order,
                       self.n_active, self.maps_ws)
        abi.mxfp4_mm_grouped(*self.gate_up, self.offsets, x_codes, x_scales, h_codes, src=src,
                             K=self.K, out_scales=h_scales)
        abi.mxfp4_mm_grouped(*self.down, self.offsets, h_codes, h_scales, rows)
        combine = abi.combine_bf16 if rows.dtype == torch.bfloat16 else abi.combine
        combine(rows, slot, w, out)
        return out

    def step(self, x: torch.Tensor, logits: torch.Tensor, out: torch.Tensor | None = None):
        """One pass of the whole path: routing, then the layer."""
        idx, w = self.route(logits)
        return self.forward(x, idx, w, out)


def _mx_bytes(name: str, a, own, device) -> torch.Tensor:
    """MXFP4's codes or scales as bytes on the device: uint8, or torch's own type for them, whose bytes
    they are.  (A conversion would take a scale of 0.5 for the byte 0.)"""
    t = a if isinstance(a, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(a))
    if t.dtype not in (torch.uint8, own):
        raise ValueError(f"{name}: uint8 or {own} is wanted, not {t.dtype}")
    return t.view(torch.uint8).to(device).contiguous()


def _to_device(a, dtype, device):
    if isinstance(a, torch.Tensor):
        return a.to(device=device, dtype=dtype).contiguous()
    return torch.from_numpy(np.ascontiguousarray(a)).to(device=device, dtype=dtype)
