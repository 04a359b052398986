"""Python binding of the C ABI (include/moe_nvfp4.h): argument marshalling only.

Every function takes and returns torch tensors on the current HIP device and
enqueues the library's kernels on torch's current stream.  Outputs (and, unless
given, workspaces) are allocated with torch; all arithmetic runs in the HIP
kernels of libmoe_nvfp4.so.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib
from ._lib import (MOE_ACT_BF16, MOE_ACT_FP8_ROUTED, MOE_ACT_FP8_ROW, MOE_ACT_FP8_SHARED,
                   MOE_OP_EXPERT_FFN, MOE_OP_EXPERT_FFN_COMBINE, MOE_OP_LAYER, MOE_OP_PERMUTE,
                   check)

__all__ = [
    "NVFP4Weights", "moe_init", "moe_route_topk", "moe_permute", "moe_expert_ffn",
    "moe_combine", "moe_layer", "workspace_bytes", "moe_expert_ffn_noalloc", "MOE_ACT_BF16", "MOE_ACT_FP8_ROW",
    "NVFP4Router", "moe_router_topk", "moe_combine_gated", "moe_route_permute",
    "moe_expert_ffn_combine", "MOE_ACT_FP8_ROUTED", "MOE_ACT_FP8_SHARED",
    "moe_dispatch", "moe_dispatch_grad", "moe_combine_grad", "moe_route_topk_grad",
    "moe_block_norm", "moe_block_norm_grad", "FP8Matrix", "FP8Weights", "moe_fp8_quant",
    "moe_fp8_linear", "moe_fp8_expert_ffn",
]


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    # the handle itself: torch.cuda.current_stream() builds a Stream object around
    # it, 3 us where this takes 0.2
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _need(t: torch.Tensor, dtype, shape=None, name="tensor"):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


@dataclass
class NVFP4Weights:
    """A device-resident NVFP4 expert bank in the layout of moe_nvfp4_weights."""
    gu_codes: torch.Tensor   # uint8 [E', 2I, H/2]
    gu_scales: torch.Tensor  # uint8 [E', 2I, H/16]
    dn_codes: torch.Tensor   # uint8 [E', H, I/2]
    dn_scales: torch.Tensor  # uint8 [E', H, I/16]
    scale2: torch.Tensor     # float32 [E', 3]
    E: int
    H: int
    I: int
    has_shared: bool

    @classmethod
    def from_bank(cls, bank, device="cuda") -> "NVFP4Weights":
        def up(a):
            return torch.from_numpy(a).to(device)
        return cls(up(bank.gu_codes), up(bank.gu_scales), up(bank.dn_codes), up(bank.dn_scales),
                   up(bank.scale2), bank.E, bank.H, bank.I, bool(bank.has_shared))

    def struct(self) -> _lib.MoeNvfp4Weights:
        G, H, I = self.E + int(self.has_shared), self.H, self.I
        _need(self.gu_codes, torch.uint8, (G, 2 * I, H // 2), "gu_codes")
        _need(self.gu_scales, torch.uint8, (G, 2 * I, H // 16), "gu_scales")
        _need(self.dn_codes, torch.uint8, (G, H, I // 2), "dn_codes")
        _need(self.dn_scales, torch.uint8, (G, H, I // 16), "dn_scales")
        _need(self.scale2, torch.float32, (G, 3), "scale2")
        return _lib.MoeNvfp4Weights(self.gu_codes.data_ptr(), self.gu_scales.data_ptr(),
                                    self.dn_codes.data_ptr(), self.dn_scales.data_ptr(),
                                    self.scale2.data_ptr(), self.E, H, I, int(self.has_shared))


@dataclass
class NVFP4Router:
    """A device-resident NVFP4 router matrix in the layout of moe_nvfp4_router:
    E expert rows, plus the shared-expert gate row at index E when has_gate."""
    codes: torch.Tensor   # uint8 [E + has_gate, H/2]
    scales: torch.Tensor  # uint8 [E + has_gate, H/16]
    scale2: float
    E: int
    H: int
    has_gate: bool

    @classmethod
    def from_bank(cls, rb, device="cuda") -> "NVFP4Router":
        return cls(torch.from_numpy(rb.codes).to(device), torch.from_numpy(rb.scales).to(device),
                   float(rb.scale2), rb.E, rb.H, bool(rb.has_gate))

    def struct(self) -> _lib.MoeNvfp4Router:
        R = self.E + int(self.has_gate)
        _need(self.codes, torch.uint8, (R, self.H // 2), "router codes")
        _need(self.scales, torch.uint8, (R, self.H // 16), "router scales")
        return _lib.MoeNvfp4Router(self.codes.data_ptr(), self.scales.data_ptr(), self.scale2,
                                   self.E, self.H, int(self.has_gate))


def moe_init() -> None:
    check(_lib.lib().moe_init())


def workspace_bytes(op: int, T: int, E: int, K: int, H: int = 0, I: int = 0,
                    has_shared: bool = False, act_mode: int = MOE_ACT_BF16) -> int:
    return int(_lib.lib().moe_workspace_bytes(op, T, E, K, H, I, int(has_shared), act_mode))


def _workspace(nbytes: int, device, ws: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    if nbytes == 0:
        return ws
    if ws is not None and ws.numel() * ws.element_size() >= nbytes:
        return ws
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def moe_route_topk(logits: torch.Tensor, K: int, ids: Optional[torch.Tensor] = None,
                   w: Optional[torch.Tensor] = None):
    _need(logits, torch.float32, name="logits")
    T, E = logits.shape
    ids = torch.empty((T, K), dtype=torch.int32, device=logits.device) if ids is None else ids
    w = torch.empty((T, K), dtype=torch.float32, device=logits.device) if w is None else w
    _need(ids, torch.int32, (T, K), "ids")
    _need(w, torch.float32, (T, K), "w")
    check(_lib.lib().moe_route_topk(_ptr(logits), T, E, K, _ptr(ids), _ptr(w), _stream()))
    return ids, w


def moe_router_topk(R: NVFP4Router, x: torch.Tensor, K: int,
                    ids: Optional[torch.Tensor] = None, w: Optional[torch.Tensor] = None,
                    logits: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None):
    """Router GEMM + top-K.  Returns (ids, w, logits, gate logits or None)."""
    _need(x, torch.bfloat16, name="x")
    T, H = x.shape
    if H != R.H:
        raise ValueError("x width does not match the router matrix")
    dev = x.device
    ids = torch.empty((T, K), dtype=torch.int32, device=dev) if ids is None else ids
    w = torch.empty((T, K), dtype=torch.float32, device=dev) if w is None else w
    _need(ids, torch.int32, (T, K), "ids")
    _need(w, torch.float32, (T, K), "w")
    logits = torch.empty((T, R.E), dtype=torch.float32, device=dev) if logits is None else logits
    _need(logits, torch.float32, (T, R.E), "logits")
    if R.has_gate and gate is None:
        gate = torch.empty((T,), dtype=torch.float32, device=dev)
    if gate is not None:
        _need(gate, torch.float32, (T,), "gate")
    st = R.struct()
    check(_lib.lib().moe_router_topk(ctypes.byref(st), _ptr(x), T, K, _ptr(ids), _ptr(w),
                                     _ptr(logits), _ptr(gate), _stream()))
    return ids, w, logits, (gate if R.has_gate else None)


def moe_permute(ids: torch.Tensor, E: int, has_shared: bool, ws: Optional[torch.Tensor] = None,
                out=None):
    _need(ids, torch.int32, name="ids")
    T, K = ids.shape
    G = E + int(has_shared)
    dev = ids.device
    if out is None:
        out = (torch.empty(G, dtype=torch.int32, device=dev),
               torch.empty(G + 1, dtype=torch.int32, device=dev),
               torch.empty(T * K + (T if has_shared else 0), dtype=torch.int32, device=dev),
               torch.empty(T * K + (T if has_shared else 0), dtype=torch.int32, device=dev),
               torch.empty(G + 1, dtype=torch.int32, device=dev))
    counts, offsets, sorted_slot, slot_pos, groups = out
    nb = workspace_bytes(MOE_OP_PERMUTE, T, E, K, 0, 0, has_shared)
    ws = _workspace(nb, dev, ws)
    check(_lib.lib().moe_permute(_ptr(ids), T, E, K, int(has_shared), _ptr(counts), _ptr(offsets),
                                 _ptr(sorted_slot), _ptr(slot_pos), _ptr(groups), _ptr(ws), nb,
                                 _stream()))
    return counts, offsets, sorted_slot, slot_pos, groups


def moe_route_permute(logits: torch.Tensor, K: int, has_shared: bool,
                      ws: Optional[torch.Tensor] = None, out=None):
    """moe_route_topk + moe_permute (one kernel for small batches).
    Returns (ids, w, counts, offsets, sorted_slot, slot_pos, groups)."""
    _need(logits, torch.float32, name="logits")
    T, E = logits.shape
    G = E + int(has_shared)
    S = T * K + (T if has_shared else 0)
    dev = logits.device
    i32 = torch.int32
    if out is None:
        out = (torch.empty((T, K), dtype=i32, device=dev),
               torch.empty((T, K), dtype=torch.float32, device=dev),
               torch.empty(G, dtype=i32, device=dev), torch.empty(G + 1, dtype=i32, device=dev),
               torch.empty(S, dtype=i32, device=dev), torch.empty(S, dtype=i32, device=dev),
               torch.empty(G + 1, dtype=i32, device=dev))
    ids, w, counts, offsets, sorted_slot, slot_pos, groups = out
    _need(ids, i32, (T, K), "ids")
    _need(w, torch.float32, (T, K), "w")
    nb = workspace_bytes(MOE_OP_PERMUTE, T, E, K, 0, 0, has_shared)
    ws = _workspace(nb, dev, ws)
    check(_lib.lib().moe_route_permute(_ptr(logits), T, E, K, int(has_shared), _ptr(ids), _ptr(w),
                                       _ptr(counts), _ptr(offsets), _ptr(sorted_slot),
                                       _ptr(slot_pos), _ptr(groups), _ptr(ws), nb, _stream()))
    return ids, w, counts, offsets, sorted_slot, slot_pos, groups


def moe_expert_ffn_combine(W: NVFP4Weights, x: torch.Tensor, K: int, offsets: torch.Tensor,
                           sorted_slot: torch.Tensor, groups: torch.Tensor, w: torch.Tensor,
                           slot_pos: torch.Tensor, act_mode: int = MOE_ACT_BF16,
                           gate: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                           y_slots: Optional[torch.Tensor] = None,
                           out: Optional[torch.Tensor] = None):
    """moe_expert_ffn followed by the combine, one call.  Returns (y_slots, out)."""
    _need(x, torch.bfloat16, name="x")
    T, H = x.shape
    if H != W.H:
        raise ValueError("x width does not match the weight bank")
    S = T * K + (T if W.has_shared else 0)
    dev = x.device
    y_slots = torch.empty((S, H), dtype=torch.bfloat16, device=dev) if y_slots is None else y_slots
    out = torch.empty((T, H), dtype=torch.bfloat16, device=dev) if out is None else out
    _need(y_slots, torch.bfloat16, (S, H), "y_slots")
    _need(out, torch.bfloat16, (T, H), "out")
    _need(w, torch.float32, (T, K), "w")
    _need(slot_pos, torch.int32, (S,), "slot_pos")
    if gate is not None:
        _need(gate, torch.float32, (T,), "gate")
    nb = workspace_bytes(MOE_OP_EXPERT_FFN_COMBINE, T, W.E, K, H, W.I, W.has_shared, act_mode)
    ws = _workspace(nb, dev, ws)
    st = W.struct()
    check(_lib.lib().moe_expert_ffn_combine(ctypes.byref(st), _ptr(x), T, K, _ptr(offsets),
                                            _ptr(sorted_slot), _ptr(groups), act_mode, _ptr(w),
                                            _ptr(slot_pos), _ptr(gate), _ptr(y_slots), _ptr(out),
                                            _ptr(ws), nb, _stream()))
    return y_slots, out


def moe_expert_ffn(W: NVFP4Weights, x: torch.Tensor, K: int, offsets: torch.Tensor,
                   sorted_slot: torch.Tensor, groups: torch.Tensor, act_mode: int = MOE_ACT_BF16,
                   ws: Optional[torch.Tensor] = None, y_slots: Optional[torch.Tensor] = None,
                   return_ws: bool = False):
    _need(x, torch.bfloat16, name="x")
    T, H = x.shape
    if H != W.H:
        raise ValueError("x width does not match the weight bank")
    S = T * K + (T if W.has_shared else 0)
    dev = x.device
    y_slots = torch.empty((S, H), dtype=torch.bfloat16, device=dev) if y_slots is None else y_slots
    _need(y_slots, torch.bfloat16, (S, H), "y_slots")
    _need(offsets, torch.int32, (W.E + int(W.has_shared) + 1,), "offsets")
    _need(sorted_slot, torch.int32, (S,), "sorted_slot")
    _need(groups, torch.int32, (W.E + int(W.has_shared) + 1,), "groups")
    nb = workspace_bytes(MOE_OP_EXPERT_FFN, T, W.E, K, H, W.I, W.has_shared, act_mode)
    ws = _workspace(nb, dev, ws)
    st = W.struct()
    check(_lib.lib().moe_expert_ffn(ctypes.byref(st), _ptr(x), T, K, _ptr(offsets),
                                    _ptr(sorted_slot), _ptr(groups), act_mode, _ptr(y_slots),
                                    _ptr(ws), nb, _stream()))
    return (y_slots, ws) if return_ws else y_slots


def moe_expert_ffn_noalloc(W: NVFP4Weights, x: torch.Tensor, K: int, offsets: torch.Tensor,
                           sorted_slot: torch.Tensor, groups: torch.Tensor,
                           act_mode: int = MOE_ACT_BF16, y_slots: Optional[torch.Tensor] = None):
    """moe_expert_ffn with the library's fixed workspace (no caller workspace);
    pass a preallocated y_slots to allocate nothing at all."""
    _need(x, torch.bfloat16, name="x")
    T, H = x.shape
    if H != W.H:
        raise ValueError("x width does not match the weight bank")
    S = T * K + (T if W.has_shared else 0)
    y_slots = torch.empty((S, H), dtype=torch.bfloat16, device=x.device) if y_slots is None else y_slots
    _need(y_slots, torch.bfloat16, (S, H), "y_slots")
    _need(offsets, torch.int32, (W.E + int(W.has_shared) + 1,), "offsets")
    _need(sorted_slot, torch.int32, (S,), "sorted_slot")
    _need(groups, torch.int32, (W.E + int(W.has_shared) + 1,), "groups")
    st = W.struct()
    check(_lib.lib().moe_expert_ffn_noalloc(ctypes.byref(st), _ptr(x), T, K, _ptr(offsets),
                                            _ptr(sorted_slot), _ptr(groups), act_mode,
                                            _ptr(y_slots), _stream()))
    return y_slots


def moe_combine(y_slots: torch.Tensor, w: torch.Tensor, slot_pos: torch.Tensor, K: int,
                has_shared: bool, out: Optional[torch.Tensor] = None):
    """Weighted sum of each token's rows.  y_slots is bf16, float16 or float32."""
    if y_slots.dtype != torch.bfloat16:
        return _combine_typed(y_slots, w, slot_pos, None, K, has_shared, out)
    _need(y_slots, torch.bfloat16, name="y_slots")
    _need(w, torch.float32, name="w")
    T = w.shape[0]
    H = y_slots.shape[1]
    _need(slot_pos, torch.int32, (T * K + (T if has_shared else 0),), "slot_pos")
    out = torch.empty((T, H), dtype=torch.bfloat16, device=y_slots.device) if out is None else out
    _need(out, torch.bfloat16, (T, H), "out")
    check(_lib.lib().moe_combine(_ptr(y_slots), _ptr(w), _ptr(slot_pos), T, K, H, int(has_shared),
                                 _ptr(out), _stream()))
    return out


def moe_combine_gated(y_slots: torch.Tensor, w: torch.Tensor, slot_pos: torch.Tensor,
                      gate: torch.Tensor, K: int, out: Optional[torch.Tensor] = None):
    """Combine with the shared expert scaled by sigmoid(gate[t]).  y_slots is
    bf16, float16 or float32."""
    if y_slots.dtype != torch.bfloat16:
        return _combine_typed(y_slots, w, slot_pos, gate, K, True, out)
    _need(y_slots, torch.bfloat16, name="y_slots")
    _need(w, torch.float32, name="w")
    T = w.shape[0]
    H = y_slots.shape[1]
    _need(slot_pos, torch.int32, (T * K + T,), "slot_pos")
    _need(gate, torch.float32, (T,), "gate")
    out = torch.empty((T, H), dtype=torch.bfloat16, device=y_slots.device) if out is None else out
    _need(out, torch.bfloat16, (T, H), "out")
    check(_lib.lib().moe_combine_gated(_ptr(y_slots), _ptr(w), _ptr(slot_pos), _ptr(gate), T, K, H,
                                       _ptr(out), _stream()))
    return out


def moe_layer(W: NVFP4Weights, x: torch.Tensor, logits: torch.Tensor, K: int,
              act_mode: int = MOE_ACT_BF16, fused: bool = False,
              gate: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
              perm=None, y_slots: Optional[torch.Tensor] = None,
              out: Optional[torch.Tensor] = None) -> dict:
    """One layer call: route -> permute -> expert FFN -> combine, all on the GPU.
    fused=True is the C entry moe_layer (two or three kernels for decode batches; the
    permutation's outputs in `perm` = (ids, w, counts, offsets, sorted_slot,
    slot_pos, groups) when given); fused=False runs the four separate entry
    points.  Both give the same results."""
    if not fused:
        ids, w = moe_route_topk(logits, K)
        counts, offsets, sorted_slot, slot_pos, groups = moe_permute(ids, W.E, W.has_shared)
        y = moe_expert_ffn(W, x, K, offsets, sorted_slot, groups, act_mode)
        o = (moe_combine(y, w, slot_pos, K, W.has_shared) if gate is None
             else moe_combine_gated(y, w, slot_pos, gate, K))
        return dict(ids=ids, w=w, counts=counts, offsets=offsets, sorted_slot=sorted_slot,
                    slot_pos=slot_pos, groups=groups, y_slots=y, out=o)
    _need(logits, torch.float32, name="logits")
    _need(x, torch.bfloat16, name="x")
    T, E = logits.shape
    H = x.shape[1]
    if H != W.H or E != W.E or x.shape[0] != T:
        raise ValueError("logits / x do not match the weight bank")
    hs = W.has_shared
    G = E + int(hs)
    S = T * K + (T if hs else 0)
    dev = x.device
    i32 = torch.int32
    if perm is None:
        perm = (torch.empty((T, K), dtype=i32, device=dev),
                torch.empty((T, K), dtype=torch.float32, device=dev),
                torch.empty(G, dtype=i32, device=dev), torch.empty(G + 1, dtype=i32, device=dev),
                torch.empty(S, dtype=i32, device=dev), torch.empty(S, dtype=i32, device=dev),
                torch.empty(G + 1, dtype=i32, device=dev))
    ids, w, counts, offsets, sorted_slot, slot_pos, groups = perm
    _need(ids, i32, (T, K), "ids")
    _need(w, torch.float32, (T, K), "w")
    _need(counts, i32, (G,), "counts")
    _need(offsets, i32, (G + 1,), "offsets")
    _need(sorted_slot, i32, (S,), "sorted_slot")
    _need(slot_pos, i32, (S,), "slot_pos")
    _need(groups, i32, (G + 1,), "groups")
    y_slots = torch.empty((S, H), dtype=torch.bfloat16, device=dev) if y_slots is None else y_slots
    out = torch.empty((T, H), dtype=torch.bfloat16, device=dev) if out is None else out
    _need(y_slots, torch.bfloat16, (S, H), "y_slots")
    _need(out, torch.bfloat16, (T, H), "out")
    if gate is not None:
        _need(gate, torch.float32, (T,), "gate")
    nb = workspace_bytes(MOE_OP_LAYER, T, E, K, H, W.I, hs, act_mode)
    ws = _workspace(nb, dev, ws)
    st = W.struct()
    check(_lib.lib().moe_layer(ctypes.byref(st), _ptr(logits), _ptr(x), T, K, act_mode, _ptr(gate),
                               _ptr(ids), _ptr(w), _ptr(counts), _ptr(offsets), _ptr(sorted_slot),
                               _ptr(slot_pos), _ptr(groups), _ptr(y_slots), _ptr(out), _ptr(ws), nb,
                               _stream()))
    return dict(ids=ids, w=w, counts=counts, offsets=offsets, sorted_slot=sorted_slot,
                slot_pos=slot_pos, groups=groups, y_slots=y_slots, out=out)


_DTYPES = {torch.bfloat16: _lib.MOE_DT_BF16, torch.float16: _lib.MOE_DT_F16,
           torch.float32: _lib.MOE_DT_F32}


def _dtype(t: torch.Tensor, name: str) -> int:
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    return dt


def _dev(t: torch.Tensor, name: str) -> torch.device:
    """t's device, which has to be the current one: the kernels go to its stream."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    d = t.device
    if d.index != torch._C._cuda_getDevice():
        raise ValueError(f"{name} is on {d}, not on the current device")
    return d


def _want(t: torch.Tensor, dtype, shape, dev, name: str) -> int:
    """t's pointer, after checks of dtype, shape, device and contiguity."""
    if t.dtype is not dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        if t.device != dev:
            raise ValueError(f"{name} must be on {dev}, got {t.device}")
        _need(t, dtype, shape, name)
    return t.data_ptr()


def _out(t: Optional[torch.Tensor], dtype, shape, dev, name: str) -> torch.Tensor:
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _want(t, dtype, shape, dev, name)
    return t


def _like(t: Optional[torch.Tensor], ref: torch.Tensor, dev, name: str) -> torch.Tensor:
    """Output of ref's type and shape: a new one, or t checked against them."""
    if t is None:
        return torch.empty_like(ref)
    _want(t, ref.dtype, ref.shape, dev, name)
    return t


def _slots(slot_pos: torch.Tensor, K: int, has_shared: bool) -> int:
    """Tokens of a permutation with K routed slots (and a shared one) each."""
    per = K + int(has_shared)
    n = slot_pos.numel()
    if K < 1 or n == 0 or n % per:
        raise ValueError(f"slot_pos has {n} entries, not a positive multiple of {per} slots a token")
    return n // per


def _scratch(ws: Optional[torch.Tensor], nbytes: int, dev) -> torch.Tensor:
    if ws is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    if ws.device != dev or not ws.is_contiguous() or ws.numel() * ws.element_size() < nbytes:
        raise ValueError(f"workspace of {nbytes} contiguous bytes on {dev} needed")
    return ws


def moe_dispatch(x: torch.Tensor, slot_pos: torch.Tensor, K: int, has_shared: bool,
                 xs: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rows of x in expert order: xs[slot_pos[s]] = x[token of s], [T*K (+ T), H].
    Rows that no slot points at stay as they are in xs."""
    dev, dt = _dev(x, "x"), _dtype(x, "x")
    T = _slots(slot_pos, K, has_shared)
    if x.dim() != 2:
        raise ValueError("x must have two dimensions")
    H = x.shape[1]
    _want(x, x.dtype, (T, H), dev, "x")
    S = T * (K + int(has_shared))
    _want(slot_pos, torch.int32, (S,), dev, "slot_pos")
    xs = _out(xs, x.dtype, (S, H), dev, "xs")
    check(_lib.lib().moe_dispatch(x.data_ptr(), slot_pos.data_ptr(), T, K, H, int(has_shared), dt,
                                  xs.data_ptr(), _stream()))
    return xs


def moe_dispatch_grad(dxs: torch.Tensor, slot_pos: torch.Tensor, K: int, has_shared: bool,
                      dx: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of moe_dispatch: dx[t] = sum of dxs over the slots of t (f32 sums)."""
    dev, dt = _dev(dxs, "dxs"), _dtype(dxs, "dxs")
    T = _slots(slot_pos, K, has_shared)
    if dxs.dim() != 2:
        raise ValueError("dxs must have two dimensions")
    H, S = dxs.shape[1], T * (K + int(has_shared))
    _want(dxs, dxs.dtype, (S, H), dev, "dxs")
    _want(slot_pos, torch.int32, (S,), dev, "slot_pos")
    dx = _out(dx, dxs.dtype, (T, H), dev, "dx")
    check(_lib.lib().moe_dispatch_grad(dxs.data_ptr(), slot_pos.data_ptr(), T, K, H,
                                       int(has_shared), dt, dx.data_ptr(), _stream()))
    return dx


def _combine_typed(y_slots, w, slot_pos, gate, K, has_shared, out):
    dev, dt = _dev(y_slots, "y_slots"), _dtype(y_slots, "y_slots")
    T = _slots(slot_pos, K, has_shared)
    if y_slots.dim() != 2:
        raise ValueError("y_slots must have two dimensions")
    H, S = y_slots.shape[1], T * (K + int(has_shared))
    _want(y_slots, y_slots.dtype, (S, H), dev, "y_slots")
    _want(w, torch.float32, (T, K), dev, "w")
    _want(slot_pos, torch.int32, (S,), dev, "slot_pos")
    if gate is not None:
        _want(gate, torch.float32, (T,), dev, "gate")
    out = _out(out, y_slots.dtype, (T, H), dev, "out")
    check(_lib.lib().moe_combine_typed(y_slots.data_ptr(), w.data_ptr(), slot_pos.data_ptr(),
                                       _ptr(gate), T, K, H, int(has_shared), dt, out.data_ptr(),
                                       _stream()))
    return out


def moe_combine_grad(dout: torch.Tensor, y_slots: torch.Tensor, w: torch.Tensor,
                     slot_pos: torch.Tensor, K: int, has_shared: bool,
                     gate: Optional[torch.Tensor] = None,
                     dy_slots: Optional[torch.Tensor] = None, dw: Optional[torch.Tensor] = None,
                     dgate: Optional[torch.Tensor] = None):
    """Gradients of moe_combine (gate None) or moe_combine_gated by the rows, the
    routing weights and the gate logit: (dy_slots, dw, dgate or None).  Rows of
    dy_slots that no slot points at stay as they are; dw is 0 for skipped slots."""
    dev, dt = _dev(dout, "dout"), _dtype(dout, "dout")
    T = _slots(slot_pos, K, has_shared)
    if dout.dim() != 2:
        raise ValueError("dout must have two dimensions")
    H, S = dout.shape[1], T * (K + int(has_shared))
    _want(dout, dout.dtype, (T, H), dev, "dout")
    _want(y_slots, dout.dtype, (S, H), dev, "y_slots")
    _want(w, torch.float32, (T, K), dev, "w")
    _want(slot_pos, torch.int32, (S,), dev, "slot_pos")
    if gate is not None:
        _want(gate, torch.float32, (T,), dev, "gate")
        dgate = _like(dgate, gate, dev, "dgate")
    elif dgate is not None:
        raise ValueError("dgate is given without a gate")
    dy_slots = _like(dy_slots, y_slots, dev, "dy_slots")
    dw = _like(dw, w, dev, "dw")
    check(_lib.lib().moe_combine_grad(dout.data_ptr(), y_slots.data_ptr(), w.data_ptr(),
                                      slot_pos.data_ptr(), _ptr(gate), T, K, H, int(has_shared),
                                      dt, dy_slots.data_ptr(), dw.data_ptr(), _ptr(dgate),
                                      _stream()))
    return dy_slots, dw, dgate


def moe_route_topk_grad(ids: torch.Tensor, w: torch.Tensor, dw: torch.Tensor, E: int,
                        dlogits: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of moe_route_topk's weights by the logits, [T, E] (zero for the
    experts not chosen; the choice itself has no gradient)."""
    dev = _dev(ids, "ids")
    if ids.dim() != 2:
        raise ValueError("ids must have two dimensions")
    T, K = ids.shape
    _want(ids, torch.int32, (T, K), dev, "ids")
    _want(w, torch.float32, (T, K), dev, "w")
    _want(dw, torch.float32, (T, K), dev, "dw")
    dlogits = _out(dlogits, torch.float32, (T, E), dev, "dlogits")
    check(_lib.lib().moe_route_topk_grad(ids.data_ptr(), w.data_ptr(), dw.data_ptr(), T, E, K,
                                         dlogits.data_ptr(), _stream()))
    return dlogits


def _gate_kind(gate, rows: torch.Tensor, dev) -> int:
    if gate is None:
        return _lib.MOE_GATE_NONE
    if gate.dim() == 1:
        _want(gate, torch.float32, (rows.shape[0],), dev, "gate")
        return _lib.MOE_GATE_TOKEN
    _want(gate, rows.dtype, rows.shape, dev, "gate")
    return _lib.MOE_GATE_ELEMENT


def moe_block_norm(residual: torch.Tensor, y: Optional[torch.Tensor] = None,
                   gate: Optional[torch.Tensor] = None, w_post: Optional[torch.Tensor] = None,
                   w_pre: Optional[torch.Tensor] = None, res_scale: float = 1.0,
                   out_scale: float = 1.0, eps: float = 1e-6,
                   r_out: Optional[torch.Tensor] = None, n_out: Optional[torch.Tensor] = None,
                   rstd_post: Optional[torch.Tensor] = None,
                   rstd_pre: Optional[torch.Tensor] = None):
    """The norm after a block, its gate and residual scale, and the norm before
    the next block, in one launch.  Returns (r, n, rstd_post, rstd_pre):

      u = y * rstd(y) * w_post              (y where w_post is None)
      r = res_scale * residual + out_scale * sigmoid(gate) * u
      n = r * rstd(r) * w_pre               (None where w_pre is None)

    residual, y: [T, H] bf16, float16 or float32; w_post, w_pre: float32 [H];
    gate: None, float32 [T] or [T, H] like y.  Without y, r is residual itself
    and only n is computed.  r_out may be residual (an update in place)."""
    dev, dt = _dev(residual, "residual"), _dtype(residual, "residual")
    if residual.dim() != 2:
        raise ValueError("residual must have two dimensions")
    T, H = shape = residual.shape
    _want(residual, residual.dtype, shape, dev, "residual")
    if y is None and (gate is not None or w_post is not None or r_out is not None or w_pre is None):
        raise ValueError("without y only w_pre and n_out are given")
    kind = _gate_kind(gate, residual, dev)
    if y is not None:
        _want(y, residual.dtype, shape, dev, "y")
        r_out = _like(r_out, residual, dev, "r_out")
    if w_post is not None:
        _want(w_post, torch.float32, (H,), dev, "w_post")
        rstd_post = _out(rstd_post, torch.float32, (T,), dev, "rstd_post")
    elif rstd_post is not None:
        raise ValueError("rstd_post is given without w_post")
    if w_pre is not None:
        _want(w_pre, torch.float32, (H,), dev, "w_pre")
        n_out = _like(n_out, residual, dev, "n_out")
        rstd_pre = _out(rstd_pre, torch.float32, (T,), dev, "rstd_pre")
    elif n_out is not None or rstd_pre is not None:
        raise ValueError("n_out or rstd_pre is given without w_pre")
    check(_lib.lib().moe_block_norm(residual.data_ptr(), _ptr(y), _ptr(gate), kind, _ptr(w_post),
                                    _ptr(w_pre), res_scale, out_scale, eps, T, H, dt, _ptr(r_out),
                                    _ptr(n_out), _ptr(rstd_post), _ptr(rstd_pre), _stream()))
    return (residual if y is None else r_out), n_out, rstd_post, rstd_pre


def moe_block_norm_grad(dr: Optional[torch.Tensor], dn: Optional[torch.Tensor], r: torch.Tensor,
                        y: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                        w_post: Optional[torch.Tensor] = None,
                        w_pre: Optional[torch.Tensor] = None,
                        rstd_post: Optional[torch.Tensor] = None,
                        rstd_pre: Optional[torch.Tensor] = None, res_scale: float = 1.0,
                        out_scale: float = 1.0, ws: Optional[torch.Tensor] = None):
    """Gradients of moe_block_norm from those of r (dr, or None for zero) and of
    n (dn; None exactly where w_pre is).  r, y, gate and the statistics are the
    forward call's.  Returns (dresidual, dy, dgate, dw_post, dw_pre), None in
    the place of what was not given; dw_* are float32 sums over the tokens."""
    dev, dt = _dev(r, "r"), _dtype(r, "r")
    if r.dim() != 2:
        raise ValueError("r must have two dimensions")
    T, H = shape = r.shape
    _want(r, r.dtype, shape, dev, "r")
    if dr is None and dn is None:
        raise ValueError("dr and dn are both missing")
    if dr is not None:
        _want(dr, r.dtype, shape, dev, "dr")
    if (dn is None) != (w_pre is None):
        raise ValueError("dn and w_pre are given together")
    dy = dgate = dw_post = dw_pre = None
    if y is None and (gate is not None or w_post is not None):
        raise ValueError("a gate or w_post is given without y")
    kind = _gate_kind(gate, r, dev)
    f32 = torch.float32
    if w_pre is not None:
        _want(dn, r.dtype, shape, dev, "dn")
        _want(w_pre, f32, (H,), dev, "w_pre")
        if rstd_pre is None:
            raise ValueError("w_pre needs rstd_pre")
        _want(rstd_pre, f32, (T,), dev, "rstd_pre")
        dw_pre = torch.empty_like(w_pre)
    if y is not None:
        _want(y, r.dtype, shape, dev, "y")
        dy = torch.empty_like(r)
        if gate is not None:
            dgate = torch.empty_like(gate)
    if w_post is not None:
        _want(w_post, f32, (H,), dev, "w_post")
        if rstd_post is None:
            raise ValueError("w_post needs rstd_post")
        _want(rstd_post, f32, (T,), dev, "rstd_post")
        dw_post = torch.empty_like(w_post)
    dres = torch.empty_like(r)
    L = _lib.lib()
    nb = L.moe_block_norm_workspace_bytes(T, H, dt)
    ws = _scratch(ws, nb, dev)
    check(L.moe_block_norm_grad(_ptr(dr), _ptr(dn), r.data_ptr(), _ptr(y), _ptr(gate), kind,
                                _ptr(w_post), _ptr(w_pre), _ptr(rstd_post), _ptr(rstd_pre),
                                res_scale, out_scale, T, H, dt, dres.data_ptr(), _ptr(dy),
                                _ptr(dgate), _ptr(dw_post), _ptr(dw_pre), ws.data_ptr(), nb,
                                _stream()))
    return dres, dy, dgate, dw_post, dw_pre


_FP8 = torch.float8_e4m3fn
_BLOCK = 128


def _codes(t: torch.Tensor, shape, dev, name: str) -> None:
    _want(t, _FP8 if t.dtype == _FP8 else torch.uint8, shape, dev, name)


@dataclass
class FP8Matrix:
    """A weight matrix in e4m3 with a float32 scale per block of 128 x 128
    (moe_fp8_matrix): W[n][k] = codes[n][k] * scales[n / 128][k / 128]."""
    codes: torch.Tensor   # float8_e4m3fn (or its bytes, uint8) [N, K]
    scales: torch.Tensor  # float32 [ceil(N/128), ceil(K/128)]

    @classmethod
    def from_float(cls, w: torch.Tensor) -> "FP8Matrix":
        """Quantise [N, K]: each block's largest magnitude becomes 448.  Done
        once, when weights are laid out."""
        N, K = w.shape
        nn, nk = -(-N // _BLOCK), -(-K // _BLOCK)
        v = torch.nn.functional.pad(w.float(), (0, nk * _BLOCK - K, 0, nn * _BLOCK - N))
        v = v.reshape(nn, _BLOCK, nk, _BLOCK)
        a = v.abs().amax((1, 3)).clamp_min(2.0 ** -100)
        s = a / 448.0
        q = (v / s[:, None, :, None]).clamp(-448, 448)
        q = q.reshape(nn * _BLOCK, nk * _BLOCK)[:N, :K].to(_FP8).contiguous()
        return cls(q, s.contiguous())

    def transposed(self) -> "FP8Matrix":
        """The transposed matrix, exactly (blocks stay blocks): moe_fp8_linear
        with it on the gradient of the output is the gradient by the input."""
        return FP8Matrix(self.codes.view(torch.uint8).t().contiguous().view(self.codes.dtype),
                         self.scales.t().contiguous())

    def struct(self, dev) -> _lib.MoeFp8Matrix:
        if self.codes.dim() != 2:
            raise ValueError("codes must have two dimensions")
        N, K = self.codes.shape
        _codes(self.codes, (N, K), dev, "codes")
        _want(self.scales, torch.float32, (-(-N // _BLOCK), -(-K // _BLOCK)), dev, "scales")
        return _lib.MoeFp8Matrix(self.codes.data_ptr(), self.scales.data_ptr(), N, K)


@dataclass
class FP8Weights:
    """An expert bank in e4m3 with block scales, in the layout of moe_fp8_weights."""
    gu_codes: torch.Tensor   # float8_e4m3fn or uint8 [E', 2I, H]
    gu_scales: torch.Tensor  # float32 [E', 2I/128, H/128]
    dn_codes: torch.Tensor   # [E', H, I]
    dn_scales: torch.Tensor  # float32 [E', H/128, I/128]
    E: int
    H: int
    I: int
    has_shared: bool

    def struct(self, dev) -> _lib.MoeFp8Weights:
        G, H, I = self.E + int(self.has_shared), self.H, self.I
        _codes(self.gu_codes, (G, 2 * I, H), dev, "gu_codes")
        _want(self.gu_scales, torch.float32, (G, 2 * I // _BLOCK, H // _BLOCK), dev, "gu_scales")
        _codes(self.dn_codes, (G, H, I), dev, "dn_codes")
        _want(self.dn_scales, torch.float32, (G, H // _BLOCK, I // _BLOCK), dev, "dn_scales")
        return _lib.MoeFp8Weights(self.gu_codes.data_ptr(), self.gu_scales.data_ptr(),
                                  self.dn_codes.data_ptr(), self.dn_scales.data_ptr(), self.E, H,
                                  I, int(self.has_shared))


def moe_fp8_quant(x: torch.Tensor, codes: Optional[torch.Tensor] = None,
                  scales: Optional[torch.Tensor] = None):
    """Rows of x (bf16, float16 or float32 [T, K]) as e4m3 codes with a float32
    scale per 128 along K: (codes float8_e4m3fn [T, K], scales [T, ceil(K/128)])."""
    dev, dt = _dev(x, "x"), _dtype(x, "x")
    if x.dim() != 2:
        raise ValueError("x must have two dimensions")
    T, K = x.shape
    _want(x, x.dtype, (T, K), dev, "x")
    codes = _out(codes, _FP8, (T, K), dev, "codes")
    scales = _out(scales, torch.float32, (T, -(-K // _BLOCK)), dev, "scales")
    check(_lib.lib().moe_fp8_quant(x.data_ptr(), T, K, dt, codes.data_ptr(), scales.data_ptr(),
                                   _stream()))
    return codes, scales


def moe_fp8_linear(M: FP8Matrix, x: torch.Tensor, ws: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x [T, K] times the matrix's transpose, [T, N] in x's type: x is quantised
    as by moe_fp8_quant, the product summed in f32."""
    dev, dt = _dev(x, "x"), _dtype(x, "x")
    st = M.struct(dev)
    if x.dim() != 2 or x.shape[1] != st.K:
        raise ValueError(f"x must be [T, {st.K}], got {tuple(x.shape)}")
    T = x.shape[0]
    _want(x, x.dtype, (T, st.K), dev, "x")
    out = _out(out, x.dtype, (T, st.N), dev, "out")
    L = _lib.lib()
    nb = L.moe_fp8_linear_workspace_bytes(T, st.K)
    if nb:
        ws = _scratch(ws, nb, dev)
    check(L.moe_fp8_linear(ctypes.byref(st), x.data_ptr(), T, dt, out.data_ptr(), _ptr(ws), nb,
                           _stream()))
    return out


def moe_fp8_expert_ffn(W: FP8Weights, x: torch.Tensor, K: int, offsets: torch.Tensor,
                       sorted_slot: torch.Tensor, groups: torch.Tensor,
                       ws: Optional[torch.Tensor] = None,
                       y_slots: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_expert_ffn for a bank in e4m3 with block scales: the rows and the
    intermediate are quantised per 128.  Returns y_slots [T*K (+ T), H] bf16."""
    dev = _dev(x, "x")
    if x.dim() != 2 or x.shape[1] != W.H:
        raise ValueError("x width does not match the weight bank")
    T, H = x.shape
    _want(x, torch.bfloat16, (T, H), dev, "x")
    S = T * (K + int(W.has_shared))
    G = W.E + int(W.has_shared)
    _want(offsets, torch.int32, (G + 1,), dev, "offsets")
    _want(sorted_slot, torch.int32, (S,), dev, "sorted_slot")
    _want(groups, torch.int32, (G + 1,), dev, "groups")
    y_slots = _out(y_slots, torch.bfloat16, (S, H), dev, "y_slots")
    st = W.struct(dev)
    L = _lib.lib()
    nb = L.moe_fp8_expert_ffn_workspace_bytes(T, K, H, W.I, int(W.has_shared))
    ws = _scratch(ws, nb, dev)
    check(L.moe_fp8_expert_ffn(ctypes.byref(st), x.data_ptr(), T, K, offsets.data_ptr(),
                               sorted_slot.data_ptr(), groups.data_ptr(), y_slots.data_ptr(),
                               ws.data_ptr(), nb, _stream()))
    return y_slots


def timing_enable(on: bool = True) -> None:
    check(_lib.lib().moe_timing_enable(int(on)))


def timing_reset() -> None:
    check(_lib.lib().moe_timing_reset())


def timing_read(max_names: int = 32) -> dict:
    names = (ctypes.c_char_p * max_names)()
    launches = (ctypes.c_int * max_names)()
    ms = (ctypes.c_double * max_names)()
    dropped = ctypes.c_int(0)
    n = check(_lib.lib().moe_timing_read(names, launches, ms, max_names, ctypes.byref(dropped)))
    res = {names[i].decode(): (launches[i], ms[i]) for i in range(n)}
    if dropped.value:
        res["_dropped"] = (dropped.value, 0.0)
    return res
