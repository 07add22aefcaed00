"""Thin Python binding of libmoe_prefill.so (include/moe_prefill.h).

Argument marshalling only: every step runs in the library's HIP kernels.  Tensors are torch
tensors on the GPU; the stream defaults to torch's current stream.  Loading fails loudly when the
library has not been built (``python -m quantized_expert_grouped_amd.build``) -- there is no
fallback.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoe_prefill.so")

Q8_0, Q4_1, Q8_0_D4 = 0, 1, 2
QUANT_PER_ROW, QUANT_D4 = 1, 2
EPI_F32, EPI_SWIGLU_Q8_1, EPI_I32_BLOCKDOTS = 0, 1, 2
F32, BF16, F16 = 0, 1, 2
MX_F32, MX_BF16, MX_SWIGLU_MXFP4 = 0, 1, 2
ACT_NONE, ACT_SWIGLU = 0, 1
MAX_E, MAX_K = 2048, 64
WS_COUNTS, WS_OFFSETS, WS_SRC, WS_SLOT, WS_ORDER, WS_NACTIVE, WS_Q8X, WS_GROUPS, WS_HQ8, WS_DM, \
    WS_GROUP_STRIDE, WS_STATUS = range(12)
N_STAGES = 6
STAGES = ("maps", "quantize", "gather", "gate_up", "down", "combine")

WALK_EVENTS = 64
WALK_GATHER_ONE, WALK_NO_SKIP_FLUSH, WALK_MMQ_PER_GROUP = 1, 2, 4
WALK_NSTATS = 16
WALK_STATS = ("copies", "bytes", "batches", "waits", "copy_waits", "skip_flushes", "slot_flushes",
              "mmq_launches", "routing_syncs", "transfers", "host_experts", "host_rows",
              "host_us", "share_ppm", "gpu_ns_per_expert", "host_ns_per_expert")
OP_COPY, OP_GATHER, OP_MMQ = 1, 2, 3

STATUS = {0: "MOE_OK", -1: "MOE_EINVAL", -2: "MOE_EUNSUPPORTED", -3: "MOE_EWORKSPACE",
          -4: "MOE_EHIP", -5: "MOE_ENOMEM"}

# name -> (restype, argtypes); the order of this table is the header's order
P, I, SZ, L64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_int64
SIGNATURES = {
    "moe_abi_version": (I, []),
    "moe_abi_minor": (I, []),
    "moe_strerror": (ctypes.c_char_p, [I]),
    "moe_block_bytes": (SZ, [I]),
    "moe_expert_bytes": (SZ, [I, I, I]),
    "moe_q8_1_row_bytes": (SZ, [I]),
    "moe_build_maps_workspace_size": (SZ, [I, I, I]),
    "moe_workspace_size": (SZ, [I, I, I, I, I, I, I]),
    "moe_route_topk": (I, [P, I, I, I, P, P, P]),
    "moe_build_maps": (I, [P, I, I, I, I, P, P, P, P, P, P, P, SZ, P]),
    "moe_build_maps_noalloc": (I, [P, I, I, I, I, P, P, P, P, P, P, P, P]),
    "moe_quantize_scatter_q8_1": (I, [P, I, I, I, P, P, I, P, P]),
    "moe_gather_group": (I, [P, I, SZ, P, I, SZ, P]),
    "moe_gather_group_mmq": (I, [P, I, I, I, I, P, I, SZ, P]),
    "moe_mmq_grouped": (I, [I, P, SZ, SZ, I, I, P, I, P, I, P, I, P, P, P]),
    "moe_combine": (I, [P, P, P, I, I, I, P, P]),
    "moe_prefill_layer": (I, [P, I, I, I, I, I, P, P, I, P, P, SZ, I, I, P, SZ, P, P]),
    "moe_prefill_layer_packed": (I, [P, I, I, I, I, I, P, P, I, P, P, SZ, I, P, SZ, P, P]),
    "moe_workspace_offset": (SZ, [I, I, I, I, I, I, I, I]),
    "moe_walk_create": (I, [P, I, SZ, P]),
    "moe_walk_destroy": (I, [P]),
    "moe_prefill_layer_streamed": (I, [P, P, I, I, I, I, I, P, P, I, P, SZ, P, P, I, I, I, P, SZ,
                                       P, P]),
    "moe_walk_stats": (I, [P, P, I]),
    "moe_walk_cpu_share": (I, [P, ctypes.c_double, I, I, I, I, I]),
    "moe_cpu_expert_rows": (I, [I, I, I, P, P, I, P]),
    "moe_cpu_share_isa": (ctypes.c_char_p, []),
    "moe_walk_plan": (I, [P, P, I, I, I, P, I, I, I, P, P, P, P, I]),
    "moe_profile_begin": (I, [I]),
    "moe_profile_end": (I, [P, I]),
    "moe_mxfp4_quantize": (I, [P, I, L64, I, I, P, P, P]),
    "moe_mxfp4_dequantize": (I, [P, P, I, I, P, I, L64, P]),
    "moe_mxfp4_mm_grouped": (I, [P, P, I, I, P, I, P, P, I, P, I, I, I, P, P, P]),
    "moe_combine_bf16": (I, [P, P, P, I, I, I, P, P]),
    "moe_balance_workspace_size": (SZ, [I, I]),
    "moe_balance_loss": (I, [P, I, L64, I, I, P, I, P, P, P, P, P, SZ, P]),
    "moe_balance_loss_backward": (I, [P, I, L64, I, I, P, I, P, P, P, L64, P]),
    "moe_dispatch_rows": (I, [P, I, L64, I, I, P, I, I, P, L64, P]),
    "moe_combine_rows": (I, [P, I, L64, I, P, P, I, I, I, P, L64, P, I, L64, P]),
    "moe_combine_rows_backward": (I, [P, I, L64, P, P, I, I, I, I, P, I, L64, P, L64, P, P]),
    "moe_mm_grouped": (I, [P, I, I, I, P, I, P, L64, I, P, I, I, P, I, P, L64, P, L64, P, I, L64,
                           P]),
    "moe_mm_grouped_dgrad": (I, [P, I, I, I, P, I, P, L64, I, P, L64, P, I, L64, P]),
    "moe_mm_grouped_wgrad_workspace_size": (SZ, [I, I, I, I]),
    "moe_mm_grouped_wgrad": (I, [P, I, L64, I, P, L64, I, I, P, I, P, I, I, P, I, P, P, SZ, P]),
    "moe_route_topk_backward": (I, [P, P, P, I, I, I, I, P, I, L64, P]),
}


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} returned {status} ({STATUS.get(status, 'unknown')})")
        self.status = status


_lib = None


def lib():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m quantized_expert_grouped_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        lacks = [name for name in SIGNATURES if not hasattr(L, name)]
        if lacks:
            raise RuntimeError(f"{LIB_PATH} is older than this binding and lacks {', '.join(lacks)}: "
                               "build it with `python -m quantized_expert_grouped_amd.build`")
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(name: str, rc: int) -> None:
    if rc != 0:
        raise MoeError(name, rc)


# ---- sizes ----------------------------------------------------------------------------------
def abi_version() -> int:
    return lib().moe_abi_version()


def abi_minor() -> int:
    return lib().moe_abi_minor()


def strerror(status: int) -> str:
    return lib().moe_strerror(status).decode()


def block_bytes(wtype: int) -> int:
    return lib().moe_block_bytes(wtype)


def expert_bytes(H: int, F: int, wtype: int) -> int:
    return lib().moe_expert_bytes(H, F, wtype)


def q8_1_row_bytes(n: int) -> int:
    return lib().moe_q8_1_row_bytes(n)


def build_maps_workspace_size(T: int, K: int, E: int) -> int:
    return lib().moe_build_maps_workspace_size(T, K, E)


def workspace_size(T, H, F, E, K, wtype, group_size=16) -> int:
    return lib().moe_workspace_size(T, H, F, E, K, wtype, group_size)


def workspace_offset(which, T, H, F, E, K, wtype, group_size=16) -> int:
    return lib().moe_workspace_offset(which, T, H, F, E, K, wtype, group_size)


# ---- entry points (raise MoeError on a non-zero status; `raw_*` return the status) -------------
def route_topk(logits, K, idx, w, stream=None):
    T, E = logits.shape
    _check("moe_route_topk", lib().moe_route_topk(_ptr(logits), T, E, K, _ptr(idx), _ptr(w),
                                                  _stream(stream)))


def build_maps(topk_idx, E, ring_start, counts, offsets, src, slot, order, n_active, ws,
               stream=None):
    T, K = topk_idx.shape
    _check("moe_build_maps", lib().moe_build_maps(
        _ptr(topk_idx), T, K, E, ring_start, _ptr(counts), _ptr(offsets), _ptr(src), _ptr(slot),
        _ptr(order), _ptr(n_active), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def raw_build_maps_noalloc(topk_idx, E, ring_start, counts, offsets, src, slot, order,
                           n_active, n_invalid=None, stream=None):
    T, K = topk_idx.shape
    return lib().moe_build_maps_noalloc(
        _ptr(topk_idx), T, K, E, ring_start, _ptr(counts), _ptr(offsets), _ptr(src), _ptr(slot),
        _ptr(order), _ptr(n_active), _ptr(n_invalid), _stream(stream))


def build_maps_noalloc(*args, **kw):
    _check("moe_build_maps_noalloc", raw_build_maps_noalloc(*args, **kw))


def quantize_scatter_q8_1(x, K, slot, src, mode, q8, stream=None):
    T, H = x.shape
    _check("moe_quantize_scatter_q8_1", lib().moe_quantize_scatter_q8_1(
        _ptr(x), T, H, K, _ptr(slot), _ptr(src), mode, _ptr(q8), _stream(stream)))


def raw_gather_group(src_ptrs, expert_bytes_, group_buf, first_pos, pos_stride, stream=None):
    n = len(src_ptrs)
    arr = (ctypes.c_void_p * max(n, 1))(*[int(p) for p in src_ptrs])
    return lib().moe_gather_group(ctypes.cast(arr, ctypes.c_void_p) if n else None, n,
                                  expert_bytes_, _ptr(group_buf), first_pos, pos_stride,
                                  _stream(stream))


def gather_group(src_ptrs, expert_bytes_, group_buf, first_pos, pos_stride, stream=None):
    _check("moe_gather_group", raw_gather_group(src_ptrs, expert_bytes_, group_buf, first_pos,
                                                pos_stride, stream))


def raw_gather_group_mmq(src_ptrs, wtype, H, F, group_buf, first_pos, pos_stride, stream=None):
    n = len(src_ptrs)
    arr = (ctypes.c_void_p * max(n, 1))(*[int(p) for p in src_ptrs])
    return lib().moe_gather_group_mmq(ctypes.cast(arr, ctypes.c_void_p) if n else None, n, wtype,
                                      H, F, _ptr(group_buf), first_pos, pos_stride,
                                      _stream(stream))


def gather_group_mmq(src_ptrs, wtype, H, F, group_buf, first_pos, pos_stride, stream=None):
    _check("moe_gather_group_mmq", raw_gather_group_mmq(src_ptrs, wtype, H, F, group_buf,
                                                        first_pos, pos_stride, stream))


def raw_mmq_grouped(wtype, group_buf, pos_stride, mat_offset, n_out, k_in, group_experts,
                    offsets, E, act_q8, epilogue, out, debug_h=None, stream=None):
    ge = np.ascontiguousarray(group_experts, dtype=np.int32)
    return lib().moe_mmq_grouped(
        wtype, _ptr(group_buf), pos_stride, mat_offset, n_out, k_in,
        ge.ctypes.data_as(ctypes.c_void_p), len(ge), _ptr(offsets), E, _ptr(act_q8), epilogue,
        _ptr(out), _ptr(debug_h), _stream(stream))


def mmq_grouped(*args, **kw):
    _check("moe_mmq_grouped", raw_mmq_grouped(*args, **kw))


def combine(Dm, slot, topk_w, out, stream=None):
    T, K = topk_w.shape
    H = Dm.shape[1]
    _check("moe_combine", lib().moe_combine(_ptr(Dm), _ptr(slot), _ptr(topk_w), T, K, H,
                                            _ptr(out), _stream(stream)))


def raw_prefill_layer(x, topk_idx, topk_w, wtype, pool, expert_off, F, E, group_size, ring_start,
                      ws, out, stream=None, ws_bytes=None):
    T, H = x.shape
    K = topk_idx.shape[1]
    eb = expert_bytes(H, F, wtype)
    nbytes = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    return lib().moe_prefill_layer(_ptr(x), T, H, F, E, K, _ptr(topk_idx), _ptr(topk_w), wtype,
                                   _ptr(pool), _ptr(expert_off), eb, group_size, ring_start,
                                   _ptr(ws), nbytes, _ptr(out), _stream(stream))


def prefill_layer(*args, **kw):
    _check("moe_prefill_layer", raw_prefill_layer(*args, **kw))


def raw_prefill_layer_packed(x, topk_idx, topk_w, wtype, packed_pool, expert_off, F, E,
                             ring_start, ws, out, stream=None):
    T, H = x.shape
    K = topk_idx.shape[1]
    eb = expert_bytes(H, F, wtype)
    return lib().moe_prefill_layer_packed(_ptr(x), T, H, F, E, K, _ptr(topk_idx), _ptr(topk_w),
                                          wtype, _ptr(packed_pool), _ptr(expert_off), eb,
                                          ring_start, _ptr(ws), ws.numel() * ws.element_size(),
                                          _ptr(out), _stream(stream))


def prefill_layer_packed(*args, **kw):
    _check("moe_prefill_layer_packed", raw_prefill_layer_packed(*args, **kw))


def profile_begin(n_calls: int) -> None:
    _check("moe_profile_begin", lib().moe_profile_begin(n_calls))


def profile_end(max_calls: int) -> np.ndarray:
    ms = np.zeros((max_calls, N_STAGES), np.float32)
    n = lib().moe_profile_end(ms.ctypes.data_as(ctypes.c_void_p), max_calls)
    if n < 0:
        raise MoeError("moe_profile_end", n)
    return ms[:n]


# ---- streamed walk --------------------------------------------------------------------------
class Walk:
    """A walk's state (copy stream, events, slot map) over a caller-owned device ring of n_slots
    slots of slot_stride bytes (`ring`: a device tensor kept alive by this object)."""

    def __init__(self, ring, n_slots: int, slot_stride: int):
        self.ring = ring
        self.n_slots, self.slot_stride = n_slots, slot_stride
        h = ctypes.c_void_p()
        _check("moe_walk_create", lib().moe_walk_create(_ptr(ring), n_slots, slot_stride,
                                                        ctypes.byref(h)))
        self.handle = h.value

    def close(self) -> None:
        if self.handle:
            lib().moe_walk_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def cpu_share(self, share: float, max_tokens: int, threads: int, max_T: int, H: int,
                  max_rows: int) -> None:
        """The host's share of the walk (share < 0: automatic; 0: off)."""
        _check("moe_walk_cpu_share", lib().moe_walk_cpu_share(self.handle, float(share),
                                                              max_tokens, threads, max_T, H,
                                                              max_rows))

    def stats(self) -> dict:
        a = np.zeros(WALK_NSTATS, np.int64)
        _check("moe_walk_stats", lib().moe_walk_stats(self.handle,
                                                      a.ctypes.data_as(ctypes.c_void_p),
                                                      WALK_NSTATS))
        return dict(zip(WALK_STATS, (int(v) for v in a)))


def raw_prefill_layer_streamed(walk, x, topk_idx, topk_w, wtype, host_arena, host_off, resident,
                               F, E, group_size, ring_start, flags, ws, out, stream=None,
                               arena_bytes=None):
    """host_arena: a pinned host tensor (uint8); host_off: int64 [E]; resident: E device pointers
    (0 = stream the expert from the arena)."""
    T, H = x.shape
    K = topk_idx.shape[1]
    off = np.ascontiguousarray(host_off, dtype=np.int64)
    res = (ctypes.c_void_p * E)(*[int(p) if p else None for p in resident])
    nb = (host_arena.numel() * host_arena.element_size() if arena_bytes is None
          else arena_bytes) if host_arena is not None else 0
    return lib().moe_prefill_layer_streamed(
        walk.handle if isinstance(walk, Walk) else walk, _ptr(x), T, H, F, E, K, _ptr(topk_idx),
        _ptr(topk_w), wtype, _ptr(host_arena), nb, off.ctypes.data_as(ctypes.c_void_p),
        ctypes.cast(res, ctypes.c_void_p), group_size, ring_start, flags, _ptr(ws),
        ws.numel() * ws.element_size(), _ptr(out), _stream(stream))


def prefill_layer_streamed(*args, **kw):
    _check("moe_prefill_layer_streamed", raw_prefill_layer_streamed(*args, **kw))


def cpu_expert_rows(wtype, H, F, expert, x):
    """The host's computation of one expert's unweighted rows (numpy in, numpy out)."""
    expert = np.ascontiguousarray(expert, dtype=np.uint8)
    x = np.ascontiguousarray(x, dtype=np.float32)
    out = np.empty((x.shape[0], H), np.float32)
    vp = ctypes.c_void_p
    _check("moe_cpu_expert_rows", lib().moe_cpu_expert_rows(
        wtype, H, F, expert.ctypes.data_as(vp), x.ctypes.data_as(vp), x.shape[0],
        out.ctypes.data_as(vp)))
    return out


def cpu_share_isa() -> str:
    return lib().moe_cpu_share_isa().decode()


def walk_plan(counts, order, n_active, ring_start, streamed, group_size, n_slots, flags=0,
              state=None, max_ops=None):
    """The walk's schedule (host only).  state: dict with used_of / cursor / next_event, updated
    in place (a fresh one when None).  Returns (status_or_count, ops int32 [n x 6], state)."""
    counts = np.ascontiguousarray(counts, dtype=np.int32)
    E = len(counts)
    order = np.ascontiguousarray(order, dtype=np.int32)
    if len(order) < E:
        order = np.concatenate([order, np.zeros(E - len(order), np.int32)])
    streamed = np.ascontiguousarray(streamed, dtype=np.uint8)
    if state is None:
        state = {"used_of": np.full(n_slots, -1, np.int32), "cursor": 0, "next_event": 0}
    used_of = state["used_of"]
    cur = ctypes.c_int32(state["cursor"])
    nev = ctypes.c_int32(state["next_event"])
    if max_ops is None:
        max_ops = 4 * E + 8
    ops = np.zeros((max(max_ops, 1), 6), np.int32)
    vp = ctypes.c_void_p
    n = lib().moe_walk_plan(counts.ctypes.data_as(vp), order.ctypes.data_as(vp), n_active, E,
                            ring_start, streamed.ctypes.data_as(vp), group_size, n_slots, flags,
                            used_of.ctypes.data_as(vp), ctypes.byref(cur), ctypes.byref(nev),
                            ops.ctypes.data_as(vp), max_ops)
    state["cursor"], state["next_event"] = cur.value, nev.value
    return n, (ops[:n] if n >= 0 else ops[:0]), state


# ---- MXFP4, the bf16 combine and the balance loss ---------------------------------------------
# These take torch tensors whose sizes say the call's, so what the C side cannot see of a tensor is
# checked here (ValueError): its type, its shape, that it is contiguous (rows of x, values, logits and
# gradients may be apart) and that all of a call's tensors are on the current device.  A call on a
# few rows is bound by the host, so the checks are one pass over the tensors.
_torch = None


def _dtypes():
    global _torch, _DT, _current_device
    if _torch is None:
        import torch
        # the private one looks up nothing else: 0.2 us of a call that takes 6
        _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        _torch, _DT = torch, {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
    return _DT


def _dtype(t):
    d = _dtypes().get(t.dtype)
    if d is None:
        raise ValueError(f"float32, bfloat16 or float16 is wanted, not {t.dtype}")
    return d


def _on_current(t) -> int:
    """The current device's number, which has to be the tensor's."""
    _dtypes()
    device = t.get_device()
    if device < 0 or device != _current_device():
        raise ValueError(f"tensors on the current device are wanted, not on {t.device}")
    return device


def _want(device: int, *wants) -> None:
    """wants: (name, tensor or None, dtype, shape), contiguous tensors."""
    for name, t, dtype, shape in wants:
        if t is None:
            continue
        if t.dtype != dtype or t.shape != shape or t.get_device() != device:
            raise ValueError(f"{name}: {dtype} {tuple(shape)} on device {device} is wanted, not "
                             f"{t.dtype} {tuple(t.shape)} on {t.device}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: a contiguous tensor is wanted")


def _row_stride(name: str, t, device: int) -> int:
    """The distance between a matrix's rows, which are contiguous each."""
    if t.get_device() != device or (t.stride(1) != 1 and t.shape[1] != 1):
        raise ValueError(f"{name}: a matrix of contiguous rows on device {device} is wanted")
    return t.stride(0)


def _current_stream(stream, device: int):
    # torch.cuda.current_stream() builds a Stream object, 2.8 us of a call that takes 6; the raw one
    # comes from a private function, which a torch may not have
    if stream is not None:
        return _stream(stream)
    raw = getattr(_torch._C, "_cuda_getCurrentRawStream", None)
    return _stream(None) if raw is None else raw(device)


def mxfp4_quantize(x, codes, scales, stream=None):
    """x [rows, n] -> codes uint8 [rows, n / 2], scales uint8 [rows, n / 32]."""
    dt, dev = _dtype(x), _on_current(x)
    rows, n = x.shape
    u8 = _torch.uint8
    _want(dev, ("codes", codes, u8, (rows, n // 2)), ("scales", scales, u8, (rows, n // 32)))
    _check("moe_mxfp4_quantize", lib().moe_mxfp4_quantize(
        x.data_ptr(), dt, _row_stride("x", x, dev), rows, n, codes.data_ptr(), scales.data_ptr(),
        _current_stream(stream, dev)))


def mxfp4_dequantize(codes, scales, values, stream=None):
    """The values [rows, n] (float32 or bfloat16) that codes and scales stand for."""
    dt, dev = _dtype(values), _on_current(values)
    rows, n = values.shape
    u8 = _torch.uint8
    _want(dev, ("codes", codes, u8, (rows, n // 2)), ("scales", scales, u8, (rows, n // 32)))
    _check("moe_mxfp4_dequantize", lib().moe_mxfp4_dequantize(
        codes.data_ptr(), scales.data_ptr(), rows, n, values.data_ptr(), dt,
        _row_stride("values", values, dev), _current_stream(stream, dev)))


def mxfp4_mm_grouped(w_codes, w_scales, offsets, a_codes, a_scales, out, src=None, K=1,
                     out_scales=None, stream=None):
    """w_codes uint8 [E, N, k / 2], w_scales [E, N, k / 32]; offsets int32 [E + 1]; a_codes
    [n_act, k / 2], a_scales [n_act, k / 32]; src int32 [rows] or None.  out: float32 or bfloat16
    [rows, N]; with out_scales uint8 [rows, N / 64] the codes uint8 [rows, N / 4] of the SwiGLU
    of gate (matrix rows 0 .. N/2 - 1) and up."""
    dev = _on_current(w_codes)
    E, N, kb = w_codes.shape
    n_act, rows = a_codes.shape[0], out.shape[0]
    u8, i32 = _torch.uint8, _torch.int32
    if out_scales is None:
        epi, n_out, dt, shape = MX_F32, N, out.dtype, (rows, N)
        if dt == _torch.bfloat16:
            epi = MX_BF16
        elif dt != _torch.float32:
            raise ValueError(f"out: float32 or bfloat16 is wanted, not {dt}")
    else:
        if N % 2:
            raise ValueError("gate and up have as many rows each: N is even")
        epi, n_out, dt, shape = MX_SWIGLU_MXFP4, N // 2, u8, (rows, N // 4)
    _want(dev, ("w_codes", w_codes, u8, (E, N, kb)), ("w_scales", w_scales, u8, (E, N, kb // 16)),
          ("offsets", offsets, i32, (E + 1,)), ("a_codes", a_codes, u8, (n_act, kb)),
          ("a_scales", a_scales, u8, (n_act, kb // 16)), ("src", src, i32, (rows,)),
          ("out", out, dt, shape), ("out_scales", out_scales, u8, (rows, n_out // 32)))
    _check("moe_mxfp4_mm_grouped", lib().moe_mxfp4_mm_grouped(
        w_codes.data_ptr(), w_scales.data_ptr(), n_out, 2 * kb, offsets.data_ptr(), E,
        a_codes.data_ptr(), a_scales.data_ptr(), n_act, _ptr(src), K, rows, epi, out.data_ptr(),
        _ptr(out_scales), _current_stream(stream, dev)))


def combine_bf16(rows, slot, topk_w, out, stream=None):
    """out float32 [T, H] of rows bfloat16 [T * K, H], slot int32 (T * K values) and topk_w
    float32 [T, K]."""
    dev = _on_current(rows)
    T, K = topk_w.shape
    H = rows.shape[1]
    f32 = _torch.float32
    if slot.numel() != T * K:
        raise ValueError(f"slot: {T * K} values are wanted, not {slot.numel()}")
    _want(dev, ("rows", rows, _torch.bfloat16, (T * K, H)),
          ("slot", slot, _torch.int32, slot.shape), ("topk_w", topk_w, f32, (T, K)),
          ("out", out, f32, (T, H)))
    _check("moe_combine_bf16", lib().moe_combine_bf16(
        rows.data_ptr(), slot.data_ptr(), topk_w.data_ptr(), T, K, H, out.data_ptr(),
        _current_stream(stream, dev)))


def balance_workspace_size(T: int, E: int) -> int:
    return lib().moe_balance_workspace_size(T, E)


def balance_loss(logits, topk_idx, counts, prob_mean, loss, ws, valid=None, stream=None):
    """logits [T, E] and topk_idx int32 [T, K] -> counts int32 [E + 1] (the valid tokens last),
    prob_mean float32 [E], loss float32 [1]; valid uint8 [T] or None; ws: at least
    balance_workspace_size(T, E) bytes."""
    dt, dev = _dtype(logits), _on_current(logits)
    T, E = logits.shape
    K = topk_idx.shape[1]
    i32, f32 = _torch.int32, _torch.float32
    _want(dev, ("topk_idx", topk_idx, i32, (T, K)), ("counts", counts, i32, (E + 1,)),
          ("prob_mean", prob_mean, f32, (E,)), ("loss", loss, f32, (1,)),
          ("ws", ws, ws.dtype, ws.shape), ("valid", valid, _torch.uint8, (T,)))
    _check("moe_balance_loss", lib().moe_balance_loss(
        logits.data_ptr(), dt, _row_stride("logits", logits, dev), T, E, topk_idx.data_ptr(), K,
        _ptr(valid), counts.data_ptr(), prob_mean.data_ptr(), loss.data_ptr(), ws.data_ptr(),
        ws.numel() * ws.element_size(), _current_stream(stream, dev)))


def balance_loss_backward(logits, counts, K, grad_logits, valid=None, grad_loss=None, stream=None):
    """grad_logits [T, E] in logits' type, from balance_loss's counts and grad_loss float32 [1]
    (None: 1)."""
    dt, dev = _dtype(logits), _on_current(logits)
    T, E = logits.shape
    if grad_logits.dtype != logits.dtype or grad_logits.shape != logits.shape:
        raise ValueError(f"grad_logits: {logits.dtype} {(T, E)} is wanted, not "
                         f"{grad_logits.dtype} {tuple(grad_logits.shape)}")
    _want(dev, ("counts", counts, _torch.int32, (E + 1,)),
          ("grad_loss", grad_loss, _torch.float32, (1,)), ("valid", valid, _torch.uint8, (T,)))
    _check("moe_balance_loss_backward", lib().moe_balance_loss_backward(
        logits.data_ptr(), dt, _row_stride("logits", logits, dev), T, E, counts.data_ptr(), K,
        _ptr(valid), _ptr(grad_loss), grad_logits.data_ptr(),
        _row_stride("grad_logits", grad_logits, dev), _current_stream(stream, dev)))


# ---- training the experts in 16 bits -----------------------------------------------------------
# As above; matrices whose rows may be apart are checked for their type and shape here, too.
def _matrix(name: str, t, device: int, dtype, shape) -> int:
    """The row stride of a matrix of this type and shape."""
    strides = t.stride()
    if t.dtype != dtype or t.shape != shape or t.get_device() != device or (
            strides[1] != 1 and shape[1] != 1):
        raise ValueError(f"{name}: {dtype} {tuple(shape)} of contiguous rows on device {device} is "
                         f"wanted, not {t.dtype} {tuple(t.shape)} of strides {strides} on {t.device}")
    return strides[0]


def _slots(slot, K: int, T: int, device: int) -> None:
    if slot.numel() != T * K:
        raise ValueError(f"slot: {T * K} values are wanted, not {slot.numel()}")
    _want(device, ("slot", slot, _torch.int32, slot.shape))


def dispatch_rows(x, src, out, K, stream=None):
    """out [rows, H]: row r is x's row src[r] / K (src int32 [rows]); rows whose src is outside x are
    left as they were."""
    dt, dev = _dtype(x), _on_current(x)
    (T, H), rows = x.shape, out.shape[0]
    _want(dev, ("src", src, _torch.int32, (rows,)))
    ldo = _matrix("out", out, dev, x.dtype, (rows, H))
    _check("moe_dispatch_rows", lib().moe_dispatch_rows(
        x.data_ptr(), dt, _row_stride("x", x, dev), T, H, src.data_ptr(), K, rows, out.data_ptr(),
        ldo, _current_stream(stream, dev)))


def combine_rows(rows, slot, topk_w, out, residual=None, stream=None):
    """out [T, H] (rows' type or float32) = residual + sum over k of topk_w[t, k] rows[slot[t, k]];
    topk_w float32 [T, K], or None for the plain sum (K is then slot's T * K values' over T)."""
    dt, dev = _dtype(rows), _on_current(rows)
    (R, H), T = rows.shape, out.shape[0]
    K = topk_w.shape[1] if topk_w is not None else slot.numel() // max(T, 1)
    _slots(slot, K, T, dev)
    _want(dev, ("topk_w", topk_w, _torch.float32, (T, K)))
    odt, ldo = _dtype(out), _matrix("out", out, dev, out.dtype, (T, H))
    ldres = 0 if residual is None else _matrix("residual", residual, dev, out.dtype, (T, H))
    _check("moe_combine_rows", lib().moe_combine_rows(
        rows.data_ptr(), dt, _row_stride("rows", rows, dev), R, slot.data_ptr(), _ptr(topk_w), T, K,
        H, _ptr(residual), ldres, out.data_ptr(), odt, ldo, _current_stream(stream, dev)))


def combine_rows_backward(grad_out, slot, topk_w, grad_rows=None, rows=None, grad_w=None,
                          stream=None):
    """From grad_out [T, H] (rows' type or float32): grad_rows [n_rows, H], and with rows
    [n_rows, H], which may be grad_rows itself, grad_w float32 [T, K]."""
    gdt, dev = _dtype(grad_out), _on_current(grad_out)
    T, H = grad_out.shape
    K = topk_w.shape[1] if topk_w is not None else slot.numel() // max(T, 1)
    _slots(slot, K, T, dev)
    if (rows is None) != (grad_w is None):
        raise ValueError("rows and grad_w are given together")
    like = rows if rows is not None else grad_rows
    if like is None:
        raise ValueError("grad_rows or grad_w is wanted")
    dt, shape = _dtype(like), (like.shape[0], H)
    ldr = 0 if rows is None else _matrix("rows", rows, dev, like.dtype, shape)
    ldgr = 0 if grad_rows is None else _matrix("grad_rows", grad_rows, dev, like.dtype, shape)
    f32 = _torch.float32
    _want(dev, ("topk_w", topk_w, f32, (T, K)), ("grad_w", grad_w, f32, (T, K)))
    _check("moe_combine_rows_backward", lib().moe_combine_rows_backward(
        grad_out.data_ptr(), gdt, _row_stride("grad_out", grad_out, dev), slot.data_ptr(),
        _ptr(topk_w), T, K, H, shape[0], _ptr(rows), dt, ldr, _ptr(grad_rows), ldgr, _ptr(grad_w),
        _current_stream(stream, dev)))


def mm_grouped(w, offsets, a, out, src=None, K=1, bias=None, swiglu=False, residual=None, z=None,
               stream=None):
    """out [rows, N] = a w^T + bias + residual (w's type or float32), or with swiglu [rows, N / 2]
    the SwiGLU of gate and up, whose values before it go to z [rows, N].  w [E, N, k] bfloat16 or
    float16; offsets int32 [E + 1]; a [n_act, k]; src int32 [rows] or None; bias [E, N]."""
    dt, dev = _dtype(w), _on_current(w)
    (E, N, k), rows, n_act = w.shape, out.shape[0], a.shape[0]
    if swiglu and N % 2:
        raise ValueError("gate and up have as many rows each: N is even")
    n_out = N // 2 if swiglu else N
    _want(dev, ("w", w, w.dtype, (E, N, k)), ("offsets", offsets, _torch.int32, (E + 1,)),
          ("src", src, _torch.int32, (rows,)), ("bias", bias, w.dtype, (E, N)))
    lda = _matrix("a", a, dev, w.dtype, (n_act, k))
    odt, ldo = _dtype(out), _matrix("out", out, dev, out.dtype, (rows, n_out))
    ldres = 0 if residual is None else _matrix("residual", residual, dev, out.dtype, (rows, n_out))
    ldz = 0 if z is None else _matrix("z", z, dev, w.dtype, (rows, N))
    _check("moe_mm_grouped", lib().moe_mm_grouped(
        w.data_ptr(), dt, n_out, k, offsets.data_ptr(), E, a.data_ptr(), lda, n_act, _ptr(src), K,
        rows, _ptr(bias), ACT_SWIGLU if swiglu else ACT_NONE, _ptr(residual), ldres, _ptr(z), ldz,
        out.data_ptr(), odt, ldo, _current_stream(stream, dev)))


def mm_grouped_dgrad(w, offsets, grad, out, z=None, stream=None):
    """out [rows, k] = grad w (w's type or float32); with z [rows, 2 k], whose SwiGLU the product
    read, z's gradient [rows, 2 k].  w [E, N, k], grad [rows, N]."""
    dt, dev = _dtype(w), _on_current(w)
    (E, N, k), rows = w.shape, grad.shape[0]
    _want(dev, ("w", w, w.dtype, (E, N, k)), ("offsets", offsets, _torch.int32, (E + 1,)))
    ldg = _matrix("grad", grad, dev, w.dtype, (rows, N))
    cols = k if z is None else 2 * k
    odt, ldo = _dtype(out), _matrix("out", out, dev, out.dtype, (rows, cols))
    ldz = 0 if z is None else _matrix("z", z, dev, w.dtype, (rows, cols))
    _check("moe_mm_grouped_dgrad", lib().moe_mm_grouped_dgrad(
        w.data_ptr(), dt, N, k, offsets.data_ptr(), E, grad.data_ptr(), ldg, rows, _ptr(z), ldz,
        out.data_ptr(), odt, ldo, _current_stream(stream, dev)))


def mm_grouped_wgrad_workspace_size(rows: int, n_out: int, k_in: int, E: int) -> int:
    return lib().moe_mm_grouped_wgrad_workspace_size(rows, n_out, k_in, E)


def mm_grouped_wgrad(grad, offsets, a, grad_w, ws=None, src=None, K=1, grad_bias=None, stream=None):
    """grad_w [E, N, k] and grad_bias [E, N] (a's type or float32) from grad [rows, N] and a
    [n_act, k]; ws: at least mm_grouped_wgrad_workspace_size(rows, N, k, E) bytes, None where that
    is 0."""
    dt, dev = _dtype(grad), _on_current(grad)
    (E, N, k), rows, n_act = grad_w.shape, grad.shape[0], a.shape[0]
    odt = _dtype(grad_w)
    _want(dev, ("grad_w", grad_w, grad_w.dtype, (E, N, k)),
          ("offsets", offsets, _torch.int32, (E + 1,)), ("src", src, _torch.int32, (rows,)),
          ("grad_bias", grad_bias, grad_w.dtype, (E, N)))
    if ws is not None:
        _want(dev, ("ws", ws, ws.dtype, ws.shape))
    ldg = _matrix("grad", grad, dev, grad.dtype, (rows, N))
    lda = _matrix("a", a, dev, grad.dtype, (n_act, k))
    _check("moe_mm_grouped_wgrad", lib().moe_mm_grouped_wgrad(
        grad.data_ptr(), dt, ldg, N, a.data_ptr(), lda, k, n_act, _ptr(src), K, offsets.data_ptr(),
        E, rows, grad_w.data_ptr(), odt, _ptr(grad_bias), _ptr(ws),
        0 if ws is None else ws.numel() * ws.element_size(), _current_stream(stream, dev)))


def route_topk_backward(topk_idx, topk_w, grad_w, grad_logits, accumulate=False, stream=None):
    """grad_logits [T, E] from topk_idx int32, topk_w and grad_w float32 [T, K]; accumulate adds it to
    what grad_logits holds."""
    dt, dev = _dtype(grad_logits), _on_current(grad_logits)
    T, E = grad_logits.shape
    K = topk_idx.shape[1]
    f32 = _torch.float32
    _want(dev, ("topk_idx", topk_idx, _torch.int32, (T, K)), ("topk_w", topk_w, f32, (T, K)),
          ("grad_w", grad_w, f32, (T, K)))
    _check("moe_route_topk_backward", lib().moe_route_topk_backward(
        topk_idx.data_ptr(), topk_w.data_ptr(), grad_w.data_ptr(), T, E, K, int(accumulate),
        grad_logits.data_ptr(), dt, _row_stride("grad_logits", grad_logits, dev),
        _current_stream(stream, dev)))
