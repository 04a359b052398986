"""Python binding of the C ABI (include/moe_nvfp4.h): argument marshalling only
(csrc/binding.cpp does it for the sort, norm, e4m3, dense block, 8-bit integer and
gradient norm operators).

Every function takes and returns torch tensors on the current HIP device and
enqueues the library's kernels on torch's current stream (moe_layer and the
operators of csrc/binding.cpp: on their tensors' device, whichever is current,
and its current stream).  Outputs (and, unless
given, workspaces) are allocated with torch; all arithmetic runs in the HIP
kernels of libmoe_nvfp4.so.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import List, Optional, Sequence

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
    "moe_fp8_linear", "moe_fp8_expert_ffn", "DenseWeights", "moe_dense_ffn", "moe_dense_ffn_grad",
    "Int8Matrix", "moe_int8_quant", "moe_int8_linear", "moe_grad_norm", "moe_grad_clip",
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
    return _lib.binding().combine(y_slots, w, slot_pos, None, K, has_shared, out)


def moe_combine_gated(y_slots: torch.Tensor, w: torch.Tensor, slot_pos: torch.Tensor,
                      gate: torch.Tensor, K: int, out: Optional[torch.Tensor] = None):
    """Combine with the shared expert scaled by sigmoid(gate[t]).  y_slots is
    bf16, float16 or float32."""
    if gate is None:
        raise ValueError("gate is missing")
    return _lib.binding().combine(y_slots, w, slot_pos, gate, K, True, out)


def moe_layer(W: NVFP4Weights, x: torch.Tensor, logits: torch.Tensor, K: int,
              act_mode: int = MOE_ACT_BF16, fused: bool = False,
              gate: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
              perm=None, y_slots: Optional[torch.Tensor] = None,
              out: Optional[torch.Tensor] = None) -> dict:
    """One layer call: route -> permute -> expert FFN -> combine, all on the GPU.
    fused=True is the C entry moe_layer (two or three kernels for decode batches; the
    permutation's outputs in `perm` = (ids, w, counts, offsets, sorted_slot,
    slot_pos, groups) when given); fused=False runs the four separate entry
    points.  Both give the same results.  Runs on x's device."""
    if x.is_cuda and x.get_device() != torch._C._cuda_getDevice():
        with torch.cuda.device(x.device):
            return moe_layer(W, x, logits, K, act_mode, fused, gate, ws, perm, y_slots, out)
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


def moe_dispatch(x: torch.Tensor, slot_pos: torch.Tensor, K: int, has_shared: bool,
                 xs: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rows of x (bf16, float16 or float32 [T, H]) in expert order:
    xs[slot_pos[s]] = x[token of s], [T*K (+ T), H].  Rows that no slot points at
    stay as they are in xs."""
    return _lib.binding().dispatch(x, slot_pos, K, has_shared, xs)


def moe_dispatch_grad(dxs: torch.Tensor, slot_pos: torch.Tensor, K: int, has_shared: bool,
                      dx: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of moe_dispatch: dx[t] = sum of dxs over the slots of t (f32 sums)."""
    return _lib.binding().dispatch_grad(dxs, slot_pos, K, has_shared, dx)


def moe_combine_grad(dout: torch.Tensor, y_slots: torch.Tensor, w: torch.Tensor,
                     slot_pos: torch.Tensor, K: int, has_shared: bool,
                     gate: Optional[torch.Tensor] = None,
                     dy_slots: Optional[torch.Tensor] = None, dw: Optional[torch.Tensor] = None,
                     dgate: Optional[torch.Tensor] = None):
    """Gradients of moe_combine (gate None) or moe_combine_gated by the rows, the
    routing weights and the gate logit: (dy_slots, dw, dgate or None).  Rows of
    dy_slots that no slot points at stay as they are; dw is 0 for skipped slots."""
    return _lib.binding().combine_grad(dout, y_slots, w, slot_pos, K, has_shared, gate, dy_slots,
                                       dw, dgate)


def moe_route_topk_grad(ids: torch.Tensor, w: torch.Tensor, dw: torch.Tensor, E: int,
                        dlogits: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of moe_route_topk's weights by the logits, [T, E] (zero for the
    experts not chosen; the choice itself has no gradient)."""
    return _lib.binding().route_topk_grad(ids, w, dw, E, dlogits)


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
    return _lib.binding().block_norm(residual, y, gate, w_post, w_pre, res_scale, out_scale, eps,
                                     r_out, n_out, rstd_post, rstd_pre)


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
    return _lib.binding().block_norm_grad(dr, dn, r, y, gate, w_post, w_pre, rstd_post, rstd_pre,
                                          res_scale, out_scale, ws)


_FP8 = torch.float8_e4m3fn
_BLOCK = 128


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


def moe_fp8_quant(x: torch.Tensor, codes: Optional[torch.Tensor] = None,
                  scales: Optional[torch.Tensor] = None):
    """Rows of x (bf16, float16 or float32 [T, K]) as e4m3 codes with a float32
    scale per 128 along K: (codes float8_e4m3fn [T, K], scales [T, ceil(K/128)])."""
    return _lib.binding().fp8_quant(x, codes, scales)


def moe_fp8_linear(M: FP8Matrix, x: torch.Tensor, ws: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x [T, K] times the matrix's transpose, [T, N] in x's type: x is quantised
    as by moe_fp8_quant, the product summed in f32."""
    return _lib.binding().fp8_linear(M.codes, M.scales, x, ws, out)


def moe_fp8_expert_ffn(W: FP8Weights, x: torch.Tensor, K: int, offsets: torch.Tensor,
                       sorted_slot: torch.Tensor, groups: torch.Tensor,
                       ws: Optional[torch.Tensor] = None,
                       y_slots: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_expert_ffn for a bank in e4m3 with block scales: the rows and the
    intermediate are quantised per 128.  Returns y_slots [T*K (+ T), H] bf16."""
    return _lib.binding().fp8_expert_ffn(W.gu_codes, W.gu_scales, W.dn_codes, W.dn_scales, W.E, W.H,
                                         W.I, W.has_shared, x, K, offsets, sorted_slot, groups, ws,
                                         y_slots)


@dataclass
class DenseWeights:
    """The weights of a dense gated feed-forward block (moe_dense_weights)."""
    gu: torch.Tensor  # bf16 or float16 [2I, H]: gate rows, then up rows
    dn: torch.Tensor  # the same type, [H, I]


def moe_dense_ffn(W: DenseWeights, x: torch.Tensor, keep: bool = False,
                  ws: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  gu_out: Optional[torch.Tensor] = None):
    """(silu(x Wg^T) * (x Wu^T)) Wd^T for rows x [T, H] of the weights' type: y [T, H],
    or (y, gu) with keep, gu [T, 2I] the projections that moe_dense_ffn_grad reads."""
    return _lib.binding().dense_ffn(W.gu, W.dn, x, keep, ws, out, gu_out)


def moe_dense_ffn_grad(W: DenseWeights, dy: torch.Tensor, x: torch.Tensor, gu: torch.Tensor,
                       ws: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                       dw_gu: Optional[torch.Tensor] = None,
                       dw_dn: Optional[torch.Tensor] = None):
    """Gradients of moe_dense_ffn from that of y, with x and the projections gu of the
    forward call: (dx, dw_gu, dw_dn) like x, W.gu and W.dn."""
    return _lib.binding().dense_ffn_grad(W.gu, W.dn, dy, x, gu, ws, dx, dw_gu, dw_dn)


@dataclass
class Int8Matrix:
    """A weight matrix in 8-bit integers with a float32 scale per row (output channel):
    W[n][k] = codes[n][k] * scales[n]."""
    codes: torch.Tensor   # int8 [N, K]
    scales: torch.Tensor  # float32 [N]

    @classmethod
    def from_float(cls, w: torch.Tensor) -> "Int8Matrix":
        """Quantise [N, K]: each row's largest magnitude becomes 127.  Done once, when
        weights are laid out."""
        v = w.float()
        s = v.abs().amax(1).clamp_min(2.0 ** -100) / 127.0
        return cls(torch.round(v / s[:, None]).clamp(-127, 127).to(torch.int8).contiguous(), s.contiguous())


def moe_int8_quant(x: torch.Tensor, codes: Optional[torch.Tensor] = None,
                   scales: Optional[torch.Tensor] = None):
    """Rows of x (bf16, float16 or float32 [T, K]) as 8-bit integers with a float32
    scale per row: (codes int8 [T, K], scales [T])."""
    return _lib.binding().int8_quant(x, codes, scales)


def moe_int8_linear(M: Int8Matrix, x: torch.Tensor, gated: bool = False,
                    ws: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x [T, K] times the matrix's transpose, [T, N] in x's type: x is quantised as by
    moe_int8_quant, the sums are exact.  gated: the first half of the rows is a gate,
    the result silu(first half) * second half, [T, N/2]."""
    return _lib.binding().int8_linear(M.codes, M.scales, x, gated, ws, out)


def moe_grad_norm(grads: Sequence[torch.Tensor], norm: Optional[torch.Tensor] = None,
                  ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The norm of all gradients together (float32 [1]).  grads: a list of bf16, float16
    or float32 tensors of any shapes, types mixed, on one device."""
    return _lib.binding().grad_norm(grads, norm, ws)


def moe_grad_clip(grads: Sequence[torch.Tensor], norm: torch.Tensor, max_norm: float,
                  out: Optional[Sequence[torch.Tensor]] = None) -> List[torch.Tensor]:
    """Every gradient times min(1, max_norm / (norm + 1e-6)), in place or into the
    tensors of out.  norm is moe_grad_norm's, or one joined over processes; it may not
    stand in a tensor that is written.  Returns the scaled tensors."""
    return _lib.binding().grad_clip(grads, norm, max_norm, out)


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
