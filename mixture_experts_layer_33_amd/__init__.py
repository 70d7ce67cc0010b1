"""Python binding of the MI355X MoE layer library (libmoe.so, include/moe.h).

Argument marshalling only: every step of the layer runs in the library's HIP
kernels.  PyTorch supplies device memory and the current stream.  Functions
with the C names take torch tensors for every buffer (outputs included);
``Layer`` allocates those buffers and chains the calls.
"""
from __future__ import annotations

import math
from dataclasses import dataclass, field
from typing import Dict, Optional

import torch

from ._lib import (DTYPES, MOE_BF16, MOE_F32, MOE_FP8, MOE_MXFP8, OP_BACKWARD, OP_COMBINE,
                   OP_DECODE, OP_DISPATCH, OP_EXPERT_FFN, OP_FORWARD, OP_NORM_BACKWARD, OP_ROUTE,
                   OP_ROUTE_BACKWARD, SCORE_SOFTMAX, SCORES, LIB_PATH, MoeError, MoeRouter, MoeShape, check, lib)

__all__ = ["make_shape", "check_shape", "workspace_bytes", "moe_route", "moe_dispatch", "moe_expert_ffn",
           "moe_expert_ffn_timed",
           "moe_combine", "moe_forward", "moe_decode", "moe_backward", "moe_backward_mx",
           "moe_quantize_mx", "quantize_mx_t_backward_weights", "Layer",
           "make_router", "moe_route_scored", "moe_route_scored_backward", "moe_backward_experts",
           "moe_add_rmsnorm", "moe_add_rmsnorm_backward", "moe_dispatch_q", "quantize_fp8",
           "moe_matmul_fp8", "matmul_fp8_workspace",
           "MoeError",
           "LIB_PATH"]


def make_shape(T: int, d: int, E: int, k: int, f: int, C: Optional[int] = None, fs: int = 0,
               dtype: str = "bf16") -> MoeShape:
    import math
    if C is None:
        C = int(math.ceil(1.25 * T * k))
    return MoeShape(tokens=T, capacity=C, hidden=d, experts=E, top_k=k, ffn=f, shared_ffn=fs,
                    dtype=DTYPES[dtype] if isinstance(dtype, str) else int(dtype))


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libmoe takes device tensors only")
    if not t.is_contiguous():
        raise ValueError("libmoe takes contiguous tensors only")
    return t.data_ptr()


def _s(stream) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def check_shape(shape: MoeShape) -> None:
    """Raise MoeError if the library would reject `shape` (host-side validation only)."""
    check("moe_check_shape", lib().moe_check_shape(shape))


def workspace_bytes(shape: MoeShape, op: int) -> int:
    return int(lib().moe_workspace_bytes(shape, op))


def workspace(shape: MoeShape, op: int, device) -> torch.Tensor:
    """A zero-filled workspace buffer of the size `op` needs (at least 256 bytes)."""
    return torch.zeros(max(workspace_bytes(shape, op), 256), dtype=torch.uint8, device=device)


def moe_route(shape, x, w_router, b_router, topk_idx, topk_gate, expert_count, ws, stream=None):
    check("moe_route", lib().moe_route(shape, _p(x), _p(w_router), _p(b_router), _p(topk_idx),
                                       _p(topk_gate), _p(expert_count), _p(ws), ws.numel(),
                                       _s(stream)))


def moe_dispatch(shape, x, topk_idx, ring_head, ring_x, ring_x_scale, expert_offset, copy_slot,
                 slot_copy, ws, stream=None):
    if shape.dtype == MOE_FP8:
        T, d, E, k, C, dev = (shape.tokens, shape.hidden, shape.experts, shape.top_k, shape.capacity, ring_x.get_device())
        i32 = torch.int32
        args = (_a("x", x, torch.bfloat16, (T, d), dev), _a("topk_idx", topk_idx, i32, (T, k), dev),
                int(ring_head), _a("ring_x", ring_x, torch.uint8, (C, d), dev),
                _a("ring_x_scale", ring_x_scale, *_scale_spec(shape, C), dev),
                _a("expert_offset", expert_offset, i32, (E + 1,), dev),
                _a("copy_slot", copy_slot, i32, (T, k), dev), _a("slot_copy", slot_copy, i32, (C,), dev),
                *_ws_arg("ws", ws, dev))
        return _on(dev, stream, "moe_dispatch", lib().moe_dispatch, shape, *args)
    check("moe_dispatch", lib().moe_dispatch(shape, _p(x), _p(topk_idx), int(ring_head), _p(ring_x),
                                             _p(ring_x_scale), _p(expert_offset), _p(copy_slot),
                                             _p(slot_copy), _p(ws), ws.numel(), _s(stream)))


def moe_expert_ffn(shape, ring_x, ring_x_scale, expert_offset, ring_head, w_gate, w_up, w_down,
                   w_gate_scale, w_up_scale, w_down_scale, ring_y, saved_au, ws, stream=None):
    if shape.dtype == MOE_FP8:
        args = _ffn_fp8_args(shape, ring_x, ring_x_scale, expert_offset, ring_head, w_gate, w_up, w_down,
                             w_gate_scale, w_up_scale, w_down_scale, ring_y, saved_au, ws)
        return _on(ring_x.get_device(), stream, "moe_expert_ffn", lib().moe_expert_ffn, shape, *args)
    check("moe_expert_ffn", lib().moe_expert_ffn(
        shape, _p(ring_x), _p(ring_x_scale), _p(expert_offset), int(ring_head), _p(w_gate),
        _p(w_up), _p(w_down), _p(w_gate_scale), _p(w_up_scale), _p(w_down_scale), _p(ring_y),
        _p(saved_au), _p(ws), ws.numel(), _s(stream)))


def moe_expert_ffn_timed(shape, ring_x, ring_x_scale, expert_offset, ring_head, w_gate, w_up,
                         w_down, w_gate_scale, w_up_scale, w_down_scale, ring_y, saved_au, ws,
                         events, stream=None):
    """moe_expert_ffn that records events[0..2] (torch.cuda.Event) around GEMM-1 and GEMM-2."""
    import ctypes
    for e in events:          # torch creates the HIP event on its first record()
        if e.cuda_event == 0:
            e.record()
    arr = (ctypes.c_void_p * 3)(*[e.cuda_event for e in events])
    if shape.dtype == MOE_FP8:
        args = _ffn_fp8_args(shape, ring_x, ring_x_scale, expert_offset, ring_head, w_gate, w_up, w_down,
                             w_gate_scale, w_up_scale, w_down_scale, ring_y, saved_au, ws)
        return _on(ring_x.get_device(), stream, "moe_expert_ffn_timed", lib().moe_expert_ffn_timed,
                   shape, *args, ctypes.cast(arr, ctypes.c_void_p))
    check("moe_expert_ffn_timed", lib().moe_expert_ffn_timed(
        shape, _p(ring_x), _p(ring_x_scale), _p(expert_offset), int(ring_head), _p(w_gate),
        _p(w_up), _p(w_down), _p(w_gate_scale), _p(w_up_scale), _p(w_down_scale), _p(ring_y),
        _p(saved_au), _p(ws), ws.numel(), ctypes.cast(arr, ctypes.c_void_p), _s(stream)))


def moe_combine(shape, ring_y, copy_slot, topk_gate, y, stream=None):
    check("moe_combine", lib().moe_combine(shape, _p(ring_y), _p(copy_slot), _p(topk_gate), _p(y),
                                           _s(stream)))


def moe_forward(shape, x, w_router, b_router, w_gate, w_up, w_down, ring_head, topk_idx, topk_gate,
                expert_count, ring_x, expert_offset, copy_slot, slot_copy, ring_y, saved_au, y, ws,
                spin_limit=0, stream=None):
    """The whole forward in one cooperative launch (bf16)."""
    check("moe_forward", lib().moe_forward(
        shape, _p(x), _p(w_router), _p(b_router), _p(w_gate), _p(w_up), _p(w_down), int(ring_head),
        _p(topk_idx), _p(topk_gate), _p(expert_count), _p(ring_x), _p(expert_offset), _p(copy_slot),
        _p(slot_copy), _p(ring_y), _p(saved_au), _p(y), int(spin_limit), _p(ws), ws.numel(),
        _s(stream)))


def moe_decode(shape, x, w_router, b_router, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, y,
               topk_idx, topk_gate, ws, stream=None):
    check("moe_decode", lib().moe_decode(shape, _p(x), _p(w_router), _p(b_router), _p(w_gate),
                                         _p(w_up), _p(w_down), _p(ws_gate), _p(ws_up),
                                         _p(ws_down), _p(y), _p(topk_idx), _p(topk_gate), _p(ws),
                                         ws.numel(), _s(stream)))


def moe_backward(shape, dy, x, w_router, topk_idx, topk_gate, ring_x, expert_offset, copy_slot,
                 slot_copy, ring_head, saved_au, w_gate, w_up, w_down, dx, dw_gate, dw_up,
                 dw_down, dw_router, ws, stream=None):
    check("moe_backward", lib().moe_backward(
        shape, _p(dy), _p(x), _p(w_router), _p(topk_idx), _p(topk_gate), _p(ring_x),
        _p(expert_offset), _p(copy_slot), _p(slot_copy), int(ring_head), _p(saved_au),
        _p(w_gate), _p(w_up), _p(w_down), _p(dx), _p(dw_gate), _p(dw_up), _p(dw_down),
        _p(dw_router), _p(ws), ws.numel(), _s(stream)))


def moe_backward_mx(shape, dy, x, w_router, topk_idx, topk_gate, expert_offset, copy_slot,
                    slot_copy, ring_head, saved_au, w_gu_t, w_gu_t_scale, w_down_t, w_down_t_scale,
                    dx, dw_gate, dw_up, dw_down, dw_router, ws, stream=None):
    check("moe_backward_mx", lib().moe_backward_mx(
        shape, _p(dy), _p(x), _p(w_router), _p(topk_idx), _p(topk_gate), _p(expert_offset),
        _p(copy_slot), _p(slot_copy), int(ring_head), _p(saved_au), _p(w_gu_t), _p(w_gu_t_scale),
        _p(w_down_t), _p(w_down_t_scale), _p(dx), _p(dw_gate), _p(dw_up), _p(dw_down),
        _p(dw_router), _p(ws), ws.numel(), _s(stream)))


def quantize_mx_t_backward_weights(w_gate, w_up, w_down, stream=None):
    """The MXFP8 backward's weights from the bf16 ones: (w_gu_t [E,d,2f], its scales,
    w_down_t [E,f,d], its scales), via moe_quantize_mx_t."""
    E, f, d = w_gate.shape
    dev = w_gate.device
    gu = torch.empty((E, d, 2 * f), dtype=torch.uint8, device=dev)
    gus = torch.empty((2 * f // 128, E * d, 4), dtype=torch.uint8, device=dev)
    dn = torch.empty((E, f, d), dtype=torch.uint8, device=dev)
    dns = torch.empty((d // 128, E * f, 4), dtype=torch.uint8, device=dev)
    L = lib()
    s = _s(stream)
    check("moe_quantize_mx_t", L.moe_quantize_mx_t(_p(w_gate), E, f, d, _p(gu), 2 * f, 0, _p(gus), s))
    check("moe_quantize_mx_t", L.moe_quantize_mx_t(_p(w_up), E, f, d, _p(gu), 2 * f, f, _p(gus), s))
    check("moe_quantize_mx_t", L.moe_quantize_mx_t(_p(w_down), E, d, f, _p(dn), d, 0, _p(dns), s))
    return gu, gus, dn, dns


def quantize_mx_training_weights(w_gate, w_up, w_down, stream=None):
    """Every MX weight an MXFP8 training step needs, from the bf16 ones, reading each once
    (moe_quantize_mx_both): ((W_gate, W_up, W_down) codes, (their scales), and the
    backward's w_gu_t, w_gu_t scales, w_down_t, w_down_t scales) -- the outputs of
    quantize_mx on each weight and of quantize_mx_t_backward_weights, bit for bit."""
    E, f, d = w_gate.shape
    dev = w_gate.device
    codes = tuple(torch.empty(w.shape, dtype=torch.uint8, device=dev) for w in (w_gate, w_up, w_down))
    scales = (torch.empty((d // 128, E * f, 4), dtype=torch.uint8, device=dev),
              torch.empty((d // 128, E * f, 4), dtype=torch.uint8, device=dev),
              torch.empty((f // 128, E * d, 4), dtype=torch.uint8, device=dev))
    gu = torch.empty((E, d, 2 * f), dtype=torch.uint8, device=dev)
    gus = torch.empty((2 * f // 128, E * d, 4), dtype=torch.uint8, device=dev)
    dn = torch.empty((E, f, d), dtype=torch.uint8, device=dev)
    dns = torch.empty((d // 128, E * f, 4), dtype=torch.uint8, device=dev)
    L = lib()
    s = _s(stream)
    for w, c, sc, ct, ld, col0, sct, R, Cc in ((w_gate, codes[0], scales[0], gu, 2 * f, 0, gus, f, d),
                                               (w_up, codes[1], scales[1], gu, 2 * f, f, gus, f, d),
                                               (w_down, codes[2], scales[2], dn, d, 0, dns, d, f)):
        check("moe_quantize_mx_both", L.moe_quantize_mx_both(_p(w), E, R, Cc, _p(c), _p(sc), _p(ct),
                                                             ld, col0, _p(sct), s))
    return codes, scales, (gu, gus, dn, dns)


def moe_quantize_mx(src, codes, scales, stream=None):
    rows = src.numel() // src.shape[-1]
    check("moe_quantize_mx", lib().moe_quantize_mx(_p(src), rows, src.shape[-1], _p(codes),
                                                   _p(scales), _s(stream)))


def quantize_mx(src: torch.Tensor, stream=None):
    """(codes uint8, scales uint8) of a bf16 tensor, MX along its last dimension; the
    scales in the library's layout [cols/128][rows][4] (rows = all leading dimensions)."""
    codes = torch.empty(src.shape, dtype=torch.uint8, device=src.device)
    rows = src.numel() // src.shape[-1]
    scales = torch.empty((src.shape[-1] // 128, rows, 4), dtype=torch.uint8, device=src.device)
    moe_quantize_mx(src, codes, scales, stream)
    return codes, scales


# ------------------------------------------------------------------ scored routing, norm, FP8
# These calls check every tensor (type, shape, contiguity, one device) and run on that device,
# on `stream` or its current stream.

try:   # the current device and its stream's raw handle, without building objects (2 us a call)
    _raw_stream, _current = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
except AttributeError:
    _current = torch.cuda.current_device

    def _raw_stream(index: int) -> int:
        return torch.cuda.current_stream(index).cuda_stream


def _on(index: int, stream, fn: str, c_fn, *args):
    """c_fn(*args, raw stream) with device `index` current; raises MoeError on a status."""
    if index < 0:
        raise ValueError("libmoe takes device tensors only")
    if stream is None:
        raw = _raw_stream(index)
    elif stream.device.index == index:
        raw = stream.cuda_stream
    else:
        raise ValueError(f"{fn}: the stream is on {stream.device}, the tensors on device {index}")
    if index == _current():
        st = c_fn(*args, raw)
    else:
        with torch.cuda.device(index):
            st = c_fn(*args, raw)
    if st:
        check(fn, st)


def _a(name: str, t: Optional[torch.Tensor], dtype: torch.dtype, shape: tuple, index: int):
    """The address of an argument after its checks (None for None); index: its device, -1 the host."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name}: needs a contiguous {dtype} tensor {list(shape)} on device {index}, got {t.dtype} {list(t.shape)} on "
                     f"{t.device}{'' if t.is_contiguous() else ', not contiguous'}")


def _act(shape: MoeShape) -> torch.dtype:
    return torch.float32 if shape.dtype == MOE_F32 else torch.bfloat16


def _ws_arg(name: str, ws: Optional[torch.Tensor], index: int):
    if ws is None:
        return None, 0
    if ws.get_device() != index or not ws.is_contiguous():
        raise ValueError(f"{name}: needs a contiguous tensor on device {index}")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def make_router(score: str = "softmax", groups: int = 1, top_groups: Optional[int] = None, group_top: int = 1,
                renormalise: bool = True, scale: float = 1.0) -> MoeRouter:
    """The rule of moe_route_scored: "softmax" or "sigmoid" scores, `groups` groups of experts of
    which a token keeps `top_groups` (default: all) by the sum of their `group_top` best."""
    return MoeRouter(score=SCORES[score] if isinstance(score, str) else int(score), groups=groups,
                     top_groups=groups if top_groups is None else top_groups, group_top=group_top,
                     renormalise=int(renormalise), scale=scale)


def moe_route_scored(shape, router, x, w_router, b_router, balance, topk_idx, topk_gate, expert_count,
                     logits, ws, stream=None):
    T, d, E, k, dev = shape.tokens, shape.hidden, shape.experts, shape.top_k, w_router.get_device()
    f32, i32 = torch.float32, torch.int32
    args = (_a("x", x, _act(shape), (T, d), dev), _a("w_router", w_router, f32, (E, d), dev),
            _a("b_router", b_router, f32, (E,), dev), _a("balance", balance, f32, (E,), dev),
            _a("topk_idx", topk_idx, i32, (T, k), dev), _a("topk_gate", topk_gate, f32, (T, k), dev),
            _a("expert_count", expert_count, i32, (E,), dev), _a("logits", logits, f32, (T, E), dev),
            *_ws_arg("ws", ws, dev))
    _on(dev, stream, "moe_route_scored", lib().moe_route_scored, shape, router, *args)


def moe_route_scored_backward(shape, router, dgate, dlogits, x, w_router, logits, topk_idx, dx_in, dx,
                              dw_router, db_router, ws, stream=None):
    T, d, E, k, dev = shape.tokens, shape.hidden, shape.experts, shape.top_k, w_router.get_device()
    act, f32 = _act(shape), torch.float32
    args = (_a("dgate", dgate, f32, (T, k), dev), _a("dlogits", dlogits, f32, (T, E), dev),
            _a("x", x, act, (T, d), dev), _a("w_router", w_router, f32, (E, d), dev),
            _a("logits", logits, f32, (T, E), dev), _a("topk_idx", topk_idx, torch.int32, (T, k), dev),
            _a("dx_in", dx_in, act, (T, d), dev), _a("dx", dx, act, (T, d), dev),
            _a("dw_router", dw_router, f32, (E, d), dev), _a("db_router", db_router, f32, (E,), dev),
            *_ws_arg("ws", ws, dev))
    _on(dev, stream, "moe_route_scored_backward", lib().moe_route_scored_backward, shape, router, *args)


def moe_backward_experts(shape, dy, topk_idx, topk_gate, ring_x, expert_offset, copy_slot, slot_copy,
                         ring_head, saved_au, w_gate, w_up, w_down, dx, dw_gate, dw_up, dw_down, dgate,
                         ws, stream=None):
    """moe_backward without the router's part: dx of the experts alone, and the gates' gradient."""
    T, d, E, k, f, C = (shape.tokens, shape.hidden, shape.experts, shape.top_k, shape.ffn, shape.capacity)
    dev, bf, f32, i32 = w_gate.get_device(), torch.bfloat16, torch.float32, torch.int32
    args = (_a("dy", dy, bf, (T, d), dev), _a("topk_idx", topk_idx, i32, (T, k), dev),
            _a("topk_gate", topk_gate, f32, (T, k), dev), _a("ring_x", ring_x, bf, (C, d), dev),
            _a("expert_offset", expert_offset, i32, (E + 1,), dev),
            _a("copy_slot", copy_slot, i32, (T, k), dev), _a("slot_copy", slot_copy, i32, (C,), dev),
            int(ring_head), _a("saved_au", saved_au, bf, (C, 2 * f), dev),
            _a("w_gate", w_gate, bf, (E, f, d), dev), _a("w_up", w_up, bf, (E, f, d), dev),
            _a("w_down", w_down, bf, (E, d, f), dev), _a("dx", dx, bf, (T, d), dev),
            _a("dw_gate", dw_gate, bf, (E, f, d), dev), _a("dw_up", dw_up, bf, (E, f, d), dev),
            _a("dw_down", dw_down, bf, (E, d, f), dev), _a("dgate", dgate, f32, (T, k), dev),
            *_ws_arg("ws", ws, dev))
    _on(dev, stream, "moe_backward_experts", lib().moe_backward_experts, shape, *args)


def _scale_spec(shape: MoeShape, rows: int):
    """Type and shape of the scales of 8-bit rows [rows, d]."""
    if shape.dtype == MOE_FP8:
        return torch.float32, (shape.hidden // 128, rows)
    return torch.uint8, (shape.hidden // 128, rows, 4)


def _ffn_fp8_args(shape, ring_x, ring_x_scale, expert_offset, ring_head, w_gate, w_up, w_down,
                  w_gate_scale, w_up_scale, w_down_scale, ring_y, saved_au, ws):
    d, E, f, C, dev = shape.hidden, shape.experts, shape.ffn, shape.capacity, ring_x.get_device()
    u8, f32, bf = torch.uint8, torch.float32, torch.bfloat16
    wide, tall = (E, f // 128, d // 128), (E, d // 128, f // 128)
    return (_a("ring_x", ring_x, u8, (C, d), dev),
            _a("ring_x_scale", ring_x_scale, f32, (d // 128, C), dev),
            _a("expert_offset", expert_offset, torch.int32, (E + 1,), dev), int(ring_head),
            _a("w_gate", w_gate, u8, (E, f, d), dev), _a("w_up", w_up, u8, (E, f, d), dev),
            _a("w_down", w_down, u8, (E, d, f), dev), _a("w_gate_scale", w_gate_scale, f32, wide, dev),
            _a("w_up_scale", w_up_scale, f32, wide, dev), _a("w_down_scale", w_down_scale, f32, tall, dev),
            _a("ring_y", ring_y, bf, (C, d), dev), _a("saved_au", saved_au, bf, (C, 2 * f), dev),
            *_ws_arg("ws", ws, dev))


def moe_add_rmsnorm(shape, x, residual, weight, eps, h, y, y8, y8_scale, rstd, stream=None):
    T, d, dev = shape.tokens, shape.hidden, weight.get_device()
    act, f32 = _act(shape), torch.float32
    sdt, sshape = _scale_spec(shape, T)
    args = (_a("x", x, act, (T, d), dev), _a("residual", residual, act, (T, d), dev),
            _a("weight", weight, f32, (d,), dev), float(eps), _a("h", h, act, (T, d), dev),
            _a("y", y, act, (T, d), dev), _a("y8", y8, torch.uint8, (T, d), dev),
            _a("y8_scale", y8_scale, sdt, sshape, dev), _a("rstd", rstd, f32, (T,), dev))
    _on(dev, stream, "moe_add_rmsnorm", lib().moe_add_rmsnorm, shape, *args)


def moe_add_rmsnorm_backward(shape, dy, dh, h, weight, rstd, dx, dweight, ws, stream=None):
    T, d, dev = shape.tokens, shape.hidden, weight.get_device()
    act, f32 = _act(shape), torch.float32
    args = (_a("dy", dy, act, (T, d), dev), _a("dh", dh, act, (T, d), dev), _a("h", h, act, (T, d), dev),
            _a("weight", weight, f32, (d,), dev), _a("rstd", rstd, f32, (T,), dev),
            _a("dx", dx, act, (T, d), dev), _a("dweight", dweight, f32, (d,), dev),
            *_ws_arg("ws", ws, dev))
    _on(dev, stream, "moe_add_rmsnorm_backward", lib().moe_add_rmsnorm_backward, shape, *args)


def moe_dispatch_q(shape, x8, x8_scale, topk_idx, ring_head, ring_x, ring_x_scale, expert_offset,
                   copy_slot, slot_copy, ws, stream=None):
    """moe_dispatch of 8-bit rows (moe_add_rmsnorm's y8 and its scales)."""
    T, d, E, k, C, dev = (shape.tokens, shape.hidden, shape.experts, shape.top_k, shape.capacity, ring_x.get_device())
    i32, u8 = torch.int32, torch.uint8
    args = (_a("x8", x8, u8, (T, d), dev), _a("x8_scale", x8_scale, *_scale_spec(shape, T), dev),
            _a("topk_idx", topk_idx, i32, (T, k), dev), int(ring_head),
            _a("ring_x", ring_x, u8, (C, d), dev),
            _a("ring_x_scale", ring_x_scale, *_scale_spec(shape, C), dev),
            _a("expert_offset", expert_offset, i32, (E + 1,), dev),
            _a("copy_slot", copy_slot, i32, (T, k), dev), _a("slot_copy", slot_copy, i32, (C,), dev),
            *_ws_arg("ws", ws, dev))
    _on(dev, stream, "moe_dispatch_q", lib().moe_dispatch_q, shape, *args)


def quantize_fp8(src: torch.Tensor, row_block: int = 128, stream=None):
    """(codes uint8, scales f32) of a bf16 tensor [..., cols], E4M3 with one scale per `row_block`
    (1 or 128) rows and 128 columns: scales [cols/128][rows] for rows, and for 128 x 128
    blocks [ceil(rows/128)][cols/128] (an expert stack [E, rows, cols]: [E, rows/128, cols/128],
    its rows a multiple of 128)."""
    if src.dim() < 2:
        raise ValueError("quantize_fp8 takes matrices")
    dev, cols = src.device, src.shape[-1]
    rows = math.prod(src.shape[:-1])
    if row_block == 128 and src.dim() > 2 and src.shape[-2] % 128:
        raise ValueError("the rows of each matrix of a stack must be a multiple of 128")
    if row_block == 1:
        shape = (cols // 128, rows)
    elif src.dim() > 2:
        shape = (*src.shape[:-2], src.shape[-2] // 128, cols // 128)
    else:
        shape = (-(-rows // 128), cols // 128)
    # memory of the stream that writes it: a block that the current stream has freed may still be
    # written by what runs there
    with torch.cuda.stream(stream):
        codes = torch.empty(src.shape, dtype=torch.uint8, device=dev)
        scales = torch.empty(shape, dtype=torch.float32, device=dev)
    at = src.get_device()
    p = _a("src", src, torch.bfloat16, src.shape, at)
    _on(at, stream, "moe_quantize_fp8", lib().moe_quantize_fp8, p, rows, cols, row_block, codes.data_ptr(), scales.data_ptr())
    return codes, scales


def matmul_fp8_workspace(M: int, N: int, K: int, device) -> Optional[torch.Tensor]:
    """The workspace moe_matmul_fp8 needs for these sizes (None if it needs none)."""
    n = int(lib().moe_matmul_fp8_workspace_bytes(M, N, K))
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def moe_matmul_fp8(a, a_scale, w, w_scale, out, ws=None, stream=None):
    """out [M, N] (bf16 or fp32) = A W^T of codes a [M, K], w [N, K] with the scales of
    quantize_fp8: a_scale [K/128, M] (row_block 1), w_scale [ceil(N/128), K/128]."""
    if a.dim() != 2 or w.dim() != 2 or out.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("moe_matmul_fp8: two matrices of codes, and an output in bfloat16 or float32")
    dev, (M, K), N = w.get_device(), a.shape, w.shape[0]
    u8, f32 = torch.uint8, torch.float32
    args = (_a("a", a, u8, (M, K), dev), _a("a_scale", a_scale, f32, (K // 128, M), dev),
            _a("w", w, u8, (N, K), dev), _a("w_scale", w_scale, f32, (-(-N // 128), K // 128), dev),
            M, N, K, MOE_F32 if out.dtype is f32 else MOE_BF16, _a("out", out, out.dtype, (M, N), dev),
            *_ws_arg("ws", ws, dev))
    _on(dev, stream, "moe_matmul_fp8", lib().moe_matmul_fp8, *args)


@dataclass
class Layer:
    """Buffers of one layer shape, and the forward / backward / decode as chained C calls.

    Expert weights are passed per call; for MXFP8 pass their MX codes and scales, for FP8 those of
    quantize_fp8.  With a `router` (make_router) the layer routes by moe_route_scored.

    The layer remembers the rule of the last call that routed (route, forward, forward_fused, decode), and a
    backward of other gates raises ValueError.  A replayed graph's forward is not seen: capture the backward with
    it, or route eagerly last."""
    shape: MoeShape
    device: torch.device
    bufs: Dict[str, torch.Tensor] = field(default_factory=dict)
    # the rule that made topk_gate (and, of a router, logits): the bytes of its MoeRouter, b"" for
    # moe_route's, None as long as no call of this layer has routed
    routed: Optional[bytes] = None

    @classmethod
    def create(cls, T, d, E, k, f, C=None, fs=0, dtype="bf16", device="cuda"):
        return cls(make_shape(T, d, E, k, f, C, fs, dtype), torch.device(device))

    @property
    def act_dtype(self):
        return torch.float32 if self.shape.dtype == MOE_F32 else torch.bfloat16

    def _buf(self, name, shape, dtype):
        b = self.bufs.get(name)
        if b is None or tuple(b.shape) != tuple(shape) or b.dtype != dtype:
            b = torch.zeros(shape, dtype=dtype, device=self.device)
            self.bufs[name] = b
        return b

    def _ws(self, op):
        n = max(workspace_bytes(self.shape, op), 256)
        return self._buf(f"ws{op}", (n,), torch.uint8)

    def _check_rule(self, fn, router=None):
        """Refuse the gradient of gates that another rule than `router` (None: moe_route's) has made."""
        if self.routed is None:
            return
        if router is not None:
            if bytes(router) != self.routed:
                raise ValueError(f"{fn}: the tokens were routed by another router, or by none")
        elif self.routed:
            r = MoeRouter.from_buffer_copy(self.routed)
            if r.score != SCORE_SOFTMAX or not r.renormalise or r.scale != 1.0:
                raise ValueError(f"{fn}: the tokens were routed by a router whose gates have another gradient than moe_route's "
                                 "(renormalised softmax, scale 1)")

    def route(self, x, w_router, b_router=None, router=None, balance=None):
        s = self.shape
        T, k, E = s.tokens, s.top_k, s.experts
        idx = self._buf("topk_idx", (T, k), torch.int32)
        gate = self._buf("topk_gate", (T, k), torch.float32)
        cnt = self._buf("expert_count", (E,), torch.int32)
        if router is not None:
            moe_route_scored(s, router, x, w_router, b_router, balance, idx, gate, cnt,
                             self._buf("logits", (T, E), torch.float32), self._ws(OP_ROUTE))
            self.routed = bytes(router)
            return idx, gate, cnt
        if balance is not None:
            raise ValueError("a balance bias needs a router (make_router)")
        moe_route(s, x, w_router, b_router, idx, gate, cnt, self._ws(OP_ROUTE))
        self.routed = b""
        return idx, gate, cnt

    def add_rmsnorm(self, x, residual, weight, eps=1e-6):
        """h = x + residual and its RMS norm: (h, y, y8, y8_scale); y8 is None in a bf16 or fp32
        layer.  h and rstd are kept for add_rmsnorm_backward."""
        s = self.shape
        T, d = s.tokens, s.hidden
        h, y = self._buf("norm_h", (T, d), self.act_dtype), self._buf("norm_y", (T, d), self.act_dtype)
        rstd = self._buf("norm_rstd", (T,), torch.float32)
        y8 = ys = None
        if s.dtype in (MOE_MXFP8, MOE_FP8):
            sdt, sshape = _scale_spec(s, T)
            y8, ys = self._buf("norm_y8", (T, d), torch.uint8), self._buf("norm_y8_scale", sshape, sdt)
        moe_add_rmsnorm(s, x, residual, weight, eps, h, y, y8, ys, rstd)
        return h, y, y8, ys

    def add_rmsnorm_backward(self, dy, dh, weight):
        """(dx, dweight) after add_rmsnorm with the same buffers; dx belongs to x and residual."""
        s = self.shape
        dx = self._buf("norm_dx", (s.tokens, s.hidden), self.act_dtype)
        dw = self._buf("norm_dw", (s.hidden,), torch.float32)
        moe_add_rmsnorm_backward(s, dy, dh, self.bufs["norm_h"], weight, self.bufs["norm_rstd"], dx, dw,
                                 self._ws(OP_NORM_BACKWARD))
        return dx, dw

    def dispatch(self, x, topk_idx, head=0, x_scale=None):
        """With x_scale: x are 8-bit rows (add_rmsnorm's y8 and y8_scale) in an MXFP8 or FP8 layer."""
        s = self.shape
        mx = s.dtype in (MOE_MXFP8, MOE_FP8)
        if x.dtype is not (self.act_dtype if x_scale is None else torch.uint8):
            raise ValueError("dispatch takes act rows, or 8-bit rows with their scales")
        ring = self._buf("ring_x", (s.capacity, s.hidden), torch.uint8 if mx else self.act_dtype)
        rsc = None
        if mx:
            sdt, sshape = _scale_spec(s, s.capacity)
            rsc = self._buf("ring_x_scale", sshape, sdt)
        off = self._buf("expert_offset", (s.experts + 1,), torch.int32)
        cs = self._buf("copy_slot", (s.tokens, s.top_k), torch.int32)
        sc = self._buf("slot_copy", (s.capacity,), torch.int32)
        if x_scale is not None:
            moe_dispatch_q(s, x, x_scale, topk_idx, head, ring, rsc, off, cs, sc, self._ws(OP_DISPATCH))
        else:
            moe_dispatch(s, x, topk_idx, head, ring, rsc, off, cs, sc, self._ws(OP_DISPATCH))
        return ring, rsc, off, cs, sc

    def expert_ffn(self, ring_x, ring_x_scale, expert_offset, head, w_gate, w_up, w_down,
                   scales=(None, None, None), save_au=False, events=None):
        s = self.shape
        ydt = torch.float32 if s.dtype == MOE_F32 else torch.bfloat16
        ring_y = self._buf("ring_y", (s.capacity, s.hidden), ydt)
        au = self._buf("saved_au", (s.capacity, 2 * s.ffn), torch.bfloat16) if save_au else None
        if events is None:
            moe_expert_ffn(s, ring_x, ring_x_scale, expert_offset, head, w_gate, w_up, w_down,
                           scales[0], scales[1], scales[2], ring_y, au, self._ws(OP_EXPERT_FFN))
        else:
            moe_expert_ffn_timed(s, ring_x, ring_x_scale, expert_offset, head, w_gate, w_up, w_down,
                                 scales[0], scales[1], scales[2], ring_y, au,
                                 self._ws(OP_EXPERT_FFN), events)
        return ring_y, au

    def combine(self, ring_y, copy_slot, topk_gate):
        s = self.shape
        y = self._buf("y", (s.tokens, s.hidden), torch.float32 if s.dtype == MOE_F32 else torch.bfloat16)
        moe_combine(s, ring_y, copy_slot, topk_gate, y)
        return y

    def forward(self, x, w_router, b_router, w_gate, w_up, w_down, scales=(None, None, None),
                head=0, save_au=False, events=None, router=None, balance=None, x8=None, x8_scale=None):
        """x8 and x8_scale: the 8-bit rows of x for the experts (add_rmsnorm), instead of
        quantising x in the dispatch."""
        idx, gate, cnt = self.route(x, w_router, b_router, router, balance)
        ring, rsc, off, cs, sc = self.dispatch(x if x8 is None else x8, idx, head, x8_scale)
        ring_y, au = self.expert_ffn(ring, rsc, off, head, w_gate, w_up, w_down, scales, save_au,
                                     events)
        y = self.combine(ring_y, cs, gate)
        return y

    def forward_fused(self, x, w_router, b_router, w_gate, w_up, w_down, head=0, save_au=False,
                      spin_limit=0):
        """The forward as one kernel launch (moe_forward), into the same buffers as forward()."""
        s = self.shape
        T, k, E, C = s.tokens, s.top_k, s.experts, s.capacity
        b = {"topk_idx": ((T, k), torch.int32), "topk_gate": ((T, k), torch.float32),
             "expert_count": ((E,), torch.int32), "ring_x": ((C, s.hidden), torch.bfloat16),
             "expert_offset": ((E + 1,), torch.int32), "copy_slot": ((T, k), torch.int32),
             "slot_copy": ((C,), torch.int32), "ring_y": ((C, s.hidden), torch.bfloat16),
             "y": ((T, s.hidden), torch.bfloat16)}
        t = {n: self._buf(n, shp, dt) for n, (shp, dt) in b.items()}
        au = self._buf("saved_au", (C, 2 * s.ffn), torch.bfloat16) if save_au else None
        moe_forward(s, x, w_router, b_router, w_gate, w_up, w_down, head, t["topk_idx"],
                    t["topk_gate"], t["expert_count"], t["ring_x"], t["expert_offset"],
                    t["copy_slot"], t["slot_copy"], t["ring_y"], au, t["y"], self._ws(OP_FORWARD),
                    spin_limit)
        self.routed = b""
        return t["y"]

    def forward_status(self) -> int:
        """The fused forward's status word (bit 0: a grid barrier gave up); a host read."""
        ws = self.bufs.get(f"ws{OP_FORWARD}")
        return 0 if ws is None else int(ws[8:12].view(torch.int32).item())

    def decode(self, x, w_router, b_router, w_gate, w_up, w_down, ws_gate=None, ws_up=None,
               ws_down=None):
        s = self.shape
        y = self._buf("y", (s.tokens, s.hidden), torch.bfloat16)
        idx = self._buf("topk_idx", (s.tokens, s.top_k), torch.int32)
        gate = self._buf("topk_gate", (s.tokens, s.top_k), torch.float32)
        moe_decode(s, x, w_router, b_router, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, y, idx,
                   gate, self._ws(OP_DECODE))
        self.routed = b""
        return y, idx, gate

    def backward_mx(self, dy, x, w_router, w_gu_t, w_gu_t_scale, w_down_t, w_down_t_scale, head=0):
        """The MXFP8 layer's gradients after forward(..., save_au=True) with the same buffers.  Its router part is
        that of moe_route's gates: after a forward with another router (sigmoid or plain softmax scores, a scale) it
        raises ValueError."""
        self._check_rule("backward_mx")
        s = self.shape
        b = self.bufs
        dx = self._buf("dx", (s.tokens, s.hidden), torch.bfloat16)
        dwg = self._buf("dw_gate", (s.experts, s.ffn, s.hidden), torch.bfloat16)
        dwu = self._buf("dw_up", (s.experts, s.ffn, s.hidden), torch.bfloat16)
        dwd = self._buf("dw_down", (s.experts, s.hidden, s.ffn), torch.bfloat16)
        dwr = self._buf("dw_router", (s.experts, s.hidden), torch.float32)
        moe_backward_mx(s, dy, x, w_router, b["topk_idx"], b["topk_gate"], b["expert_offset"],
                        b["copy_slot"], b["slot_copy"], head, b["saved_au"], w_gu_t, w_gu_t_scale,
                        w_down_t, w_down_t_scale, dx, dwg, dwu, dwd, dwr, self._ws(OP_BACKWARD))
        return dx, dwg, dwu, dwd, dwr

    def backward(self, dy, x, w_router, w_gate, w_up, w_down, head=0, router=None, dlogits=None):
        """Gradients after a forward(..., save_au=True) with the same buffers (and the same
        `router`, another one raises ValueError; then dlogits is a further gradient of the logits,
        and the bias's gradient is left in bufs["db_router"]).  After an FP8 forward the weights
        are the bf16 ones: the tokens are dispatched again in bf16, and the forward's rounding to
        8 bits counts as the identity."""
        self._check_rule("backward", router)
        s = self.shape
        b = self.bufs
        ring = b.get("ring_x")
        if s.dtype == MOE_FP8:
            s = make_shape(s.tokens, s.hidden, s.experts, s.top_k, s.ffn, s.capacity)
            check_shape(s)
            ring = self._buf("ring_x_bf16", (s.capacity, s.hidden), torch.bfloat16)
            moe_dispatch(s, x, b["topk_idx"], head, ring, None, b["expert_offset"], b["copy_slot"],
                         b["slot_copy"], self._ws(OP_DISPATCH))
        ws = self._buf(f"ws{OP_BACKWARD}", (max(workspace_bytes(s, OP_BACKWARD), 256),), torch.uint8)
        dx = self._buf("dx", (s.tokens, s.hidden), torch.bfloat16)
        dwg = self._buf("dw_gate", (s.experts, s.ffn, s.hidden), torch.bfloat16)
        dwu = self._buf("dw_up", (s.experts, s.ffn, s.hidden), torch.bfloat16)
        dwd = self._buf("dw_down", (s.experts, s.hidden, s.ffn), torch.bfloat16)
        dwr = self._buf("dw_router", (s.experts, s.hidden), torch.float32)
        if router is not None:
            dg = self._buf("dgate", (s.tokens, s.top_k), torch.float32)
            db = self._buf("db_router", (s.experts,), torch.float32)
            moe_backward_experts(s, dy, b["topk_idx"], b["topk_gate"], ring, b["expert_offset"],
                                 b["copy_slot"], b["slot_copy"], head, b["saved_au"], w_gate, w_up,
                                 w_down, dx, dwg, dwu, dwd, dg, ws)
            moe_route_scored_backward(s, router, dg, dlogits, x, w_router, b["logits"], b["topk_idx"],
                                      dx, dx, dwr, db, self._ws(OP_ROUTE_BACKWARD))
            return dx, dwg, dwu, dwd, dwr
        if dlogits is not None:
            raise ValueError("a gradient of the logits needs a router (make_router)")
        moe_backward(s, dy, x, w_router, b["topk_idx"], b["topk_gate"], ring,
                     b["expert_offset"], b["copy_slot"], b["slot_copy"], head, b["saved_au"],
                     w_gate, w_up, w_down, dx, dwg, dwu, dwd, dwr, ws)
        return dx, dwg, dwu, dwd, dwr


class RingStack:
    """L MoE layers of one shape sharing one token ring (dzen.guru page, ring-buffer
    paragraph of "Три решения…": a fixed ring whose head advances layer by layer,
    walked in reverse by the backward).

    Layer l dispatches its n = T*k copies at head_l = (head_0 + l*n) mod C, so the
    ring keeps every layer's dispatched rows and saved [A|U] until the backward,
    which consumes the layers last first (the newest segment first) and, inside a
    layer, experts E-1 -> 0 and rows last slot first: nothing is recomputed.  The
    layers are chained directly (x_{l+1} = y_l).  C >= L*n, so no segment is
    overwritten while it is live; segments may wrap past the end of the ring.
    Every step is one of the library's calls; this class only keeps the buffers."""

    def __init__(self, L, T, d, E, k, f, C=None, device="cuda"):
        n = T * k
        C = C if C is not None else L * int(math.ceil(1.25 * n))
        if C < L * n:
            raise ValueError(f"ring of {C} rows cannot hold {L} layers of {n} copies")
        self.L, self.n = L, n
        self.shape = make_shape(T, d, E, k, f, C)
        check_shape(self.shape)   # e.g. a ring of 4 GiB or more per array is rejected
        self.device = torch.device(device)
        dev = self.device
        z = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype, device=dev)
        self.ring_x = z(C, d, dtype=torch.bfloat16)
        self.saved_au = z(C, 2 * f, dtype=torch.bfloat16)
        self.ring_y = z(C, d, dtype=torch.bfloat16)
        self.slot_copy = z(C)
        self.per = [dict(idx=z(T, k), gate=z(T, k, dtype=torch.float32), cnt=z(E),
                         off=z(E + 1), cs=z(T, k), x=z(T, d, dtype=torch.bfloat16),
                         y=z(T, d, dtype=torch.bfloat16)) for _ in range(L)]
        self.ws = {op: z(max(workspace_bytes(self.shape, op), 256), dtype=torch.uint8)
                   for op in (OP_ROUTE, OP_DISPATCH, OP_EXPERT_FFN, OP_BACKWARD)}
        self.heads = [0] * L

    def forward(self, x, weights, head0=0):
        """weights[l] = (w_router, b_router, w_gate, w_up, w_down).  Returns y_{L-1}."""
        s, C = self.shape, self.shape.capacity
        self.heads = [(head0 + l * self.n) % C for l in range(self.L)]
        cur = x
        for l, (w_r, b_r, w_g, w_u, w_d) in enumerate(weights):
            p, h = self.per[l], self.heads[l]
            p["x"].copy_(cur)
            moe_route(s, p["x"], w_r, b_r, p["idx"], p["gate"], p["cnt"], self.ws[OP_ROUTE])
            moe_dispatch(s, p["x"], p["idx"], h, self.ring_x, None, p["off"], p["cs"],
                         self.slot_copy, self.ws[OP_DISPATCH])
            moe_expert_ffn(s, self.ring_x, None, p["off"], h, w_g, w_u, w_d, None, None, None,
                           self.ring_y, self.saved_au, self.ws[OP_EXPERT_FFN])
            moe_combine(s, self.ring_y, p["cs"], p["gate"], p["y"])
            cur = p["y"]
        return cur

    def backward(self, dy, weights, dw=None):
        """Layers L-1 -> 0 (each layer's input gradient is kept as per[l]["dx"]).  Returns
        dx_0 and, per layer, (dw_gate, dw_up, dw_down, dw_router);
        with `dw` given (one set of gradient buffers) every layer writes into it and the
        list holds that set L times (the caller consumes each layer's before the next)."""
        s = self.shape
        T, d, E, f = s.tokens, s.hidden, s.experts, s.ffn
        dev = self.device
        grads = [None] * self.L
        cur = dy
        for l in reversed(range(self.L)):
            w_r, _, w_g, w_u, w_d = weights[l]
            p = self.per[l]
            g = dw if dw is not None else (
                torch.empty(E, f, d, dtype=torch.bfloat16, device=dev),
                torch.empty(E, f, d, dtype=torch.bfloat16, device=dev),
                torch.empty(E, d, f, dtype=torch.bfloat16, device=dev),
                torch.empty(E, d, dtype=torch.float32, device=dev))
            dx = torch.empty(T, d, dtype=torch.bfloat16, device=dev)
            moe_backward(s, cur, p["x"], w_r, p["idx"], p["gate"], self.ring_x, p["off"],
                         p["cs"], self.slot_copy, self.heads[l], self.saved_au, w_g, w_u, w_d,
                         dx, g[0], g[1], g[2], g[3], self.ws[OP_BACKWARD])
            grads[l] = g
            p["dx"] = dx
            cur = dx
        return cur, grads
