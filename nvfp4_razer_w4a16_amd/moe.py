"""Routing of tokens to experts and the combination of the experts' rows: binding of
``razer_moe_route`` and ``razer_moe_combine`` of ``include/librazer.h``.

What stands before and behind the grouped products::

    r = razer_moe_route(logits, 8, score="sigmoid", bias=bias, renormalise=True)
    gu = razer_i8_gemm_grouped(x, gate_up, r.offsets, r.rows)
    rows = razer_i8_gemm_grouped(razer_i8_quantize_gated(gu), down, r.offsets)
    y = razer_moe_combine(rows, r.slots, r.weights, add=h)

Nothing here waits for the GPU, so a layer of experts can be captured in a graph.
Streams as in ``mx``.  No call has a backward, or takes tangents of forward mode.  The package re-exports every name here.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import NamedTuple, Optional

import torch

from . import _check_buffer, lib
from .mx import (_check, _dtype, _entered, _forward, _grad_enabled, _no_tangents, _on_gpu, _stream, _Tensor,
                 _without_backward)

RAZER_MOE_MAX_EXPERTS, RAZER_MOE_MAX_TOP, RAZER_MOE_MAX_GROUPS = 1024, 32, 64
RAZER_SCORE_SOFTMAX, RAZER_SCORE_SIGMOID = 0, 1
RAZER_ROUTE_RENORM = 1
_SCORES = {"softmax": RAZER_SCORE_SOFTMAX, "sigmoid": RAZER_SCORE_SIGMOID}


class razer_route(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("stride", ctypes.c_int64), ("experts", ctypes.c_int32),
                ("top", ctypes.c_int32), ("groups", ctypes.c_int32), ("groups_kept", ctypes.c_int32),
                ("group_best", ctypes.c_int32), ("score", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("scale", ctypes.c_float), ("logits", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("chosen", ctypes.c_void_p), ("weights", ctypes.c_void_p),
                ("offsets", ctypes.c_void_p), ("rows", ctypes.c_void_p), ("slots", ctypes.c_void_p)]


class razer_combine(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("top", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("y_rows", ctypes.c_int64), ("y_stride", ctypes.c_int64), ("add_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("y", ctypes.c_void_p), ("slots", ctypes.c_void_p),
                ("weights", ctypes.c_void_p), ("add", ctypes.c_void_p), ("out", ctypes.c_void_p)]


# The structs as bytes, which cost a fifth of a ctypes instance to make
_route_bytes = struct.Struct("qqiiiiiiiIf4xPPPPPPP").pack
_combine_bytes = struct.Struct("qqqqqqi4xPPPPP").pack


class MoeRoutes(NamedTuple):
    """experts, weights, slots: [tokens, top]; offsets: [E + 1]; rows: [tokens * top].  All are
    int32 but the weights, float32; offsets, rows and slots are None where no order was asked
    for.  Expert and slot -1: a place that no expert takes (weight 0).  The results of a call
    that was given none are views of one buffer, which its workspace is a part of: to keep
    one of them alone, copy it."""
    experts: torch.Tensor
    weights: torch.Tensor
    offsets: Optional[torch.Tensor]
    rows: Optional[torch.Tensor]
    slots: Optional[torch.Tensor]


def bind(L: ctypes.CDLL):
    """Argument types of the calls bound here."""
    vp, sz, i32, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64
    L.razer_moe_route.restype, L.razer_moe_route.argtypes = i32, [vp, vp, sz, vp]
    L.razer_moe_combine.restype, L.razer_moe_combine.argtypes = i32, [vp, vp]
    L.razer_moe_workspace_bytes.restype, L.razer_moe_workspace_bytes.argtypes = sz, [i64] * 3


def razer_moe_workspace_bytes(tokens: int, experts: int, top: int) -> int:
    return int(lib().razer_moe_workspace_bytes(tokens, experts, top))


# a function of the sizes alone
_workspace_bytes = functools.lru_cache(4096)(razer_moe_workspace_bytes)


def _new_routes(tokens: int, experts: int, top: int, order: bool, space: int, device):
    """(routes, their addresses, that of `space` bytes behind them in the same buffer).  The
    buffer has rows of `top`, so that one split makes most of the views."""
    n = tokens * top
    if not order:
        buf = torch.empty(2 * tokens, top, dtype=torch.int32, device=device)
        chosen, weights = buf.split_with_sizes((tokens, tokens))
        at = buf.data_ptr()
        return MoeRoutes(chosen, weights.view(torch.float32), None, None, None), (at, at + 4 * n, 0, 0, 0), None
    head = 4 * n + experts + 4 & ~3  # the space begins at a multiple of 16 bytes
    lines = (head + (space + 3 >> 2) + top - 1) // top
    buf = torch.empty(lines, top, dtype=torch.int32, device=device)
    chosen, weights, slots, rows, rest = buf.split_with_sizes((tokens, tokens, tokens, tokens, lines - 4 * tokens))
    at = buf.data_ptr()
    return (MoeRoutes(chosen, weights.view(torch.float32), rest.as_strided((experts + 1,), (1,)), rows.view(n), slots),
            (at, at + 4 * n, at + 16 * n, at + 12 * n, at + 8 * n), at + 4 * head)


def _packed_rows(t: torch.Tensor, cols: int):
    """(t, stride) of rows that are not contiguous, or overlap: a copy, but for a lone row,
    whose stride means nothing."""
    if t.shape[0] > 1 or t.stride(1) != 1 and cols > 1:
        t = torch.empty(t.shape, dtype=t.dtype, device=t.device).copy_(t)
    return t, cols


def razer_moe_route(logits: torch.Tensor, top: int, *, score: str = "softmax", bias: torch.Tensor | None = None,
                    groups: int = 1, groups_kept: int | None = None, group_best: int = 1, renormalise: bool = False,
                    scale: float = 1.0, order: bool = True, out: MoeRoutes | None = None, workspace=None,
                    stream=None) -> MoeRoutes:
    """The `top` experts of each token, their weights, and the order of rows that the
    grouped products take.

    logits: [tokens, E] (f32, f16 or bf16).  score: "softmax" or "sigmoid" of the logits.
    bias (f32 [E]) is added to the scores for the choice alone.  groups: the experts are
    this many equal runs, of which the groups_kept (all) best stay, by the sum of their
    group_best (1 or 2) best scores.  Ties go to the lowest index.  weights: scores of
    the chosen times `scale`, divided by their sum with `renormalise`.  Logits of -inf are
    never chosen.  order: also offsets, rows and slots.  out takes the results.  There is
    no backward: one that reaches the weights raises; what is written to out stands
    outside any graph."""
    if stream is not None:
        with _entered(stream):
            return razer_moe_route(logits, top, score=score, bias=bias, groups=groups, groups_kept=groups_kept,
                                   group_best=group_best, renormalise=renormalise, scale=scale, order=order, out=out,
                                   workspace=workspace)
    dev = _on_gpu(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D")
    dt = _dtype(logits.dtype)
    tokens, experts = logits.shape
    kind = _SCORES.get(score)
    if kind is None:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, not {score!r}")
    if not 1 <= top <= experts:
        raise ValueError(f"top {top} of {experts} experts")
    if not 1 <= groups <= experts or experts % groups:
        raise ValueError(f"{groups} groups of {experts} experts")
    kept = groups if groups_kept is None else groups_kept
    if not 1 <= kept <= groups or top > experts // groups * kept:
        raise ValueError(f"{kept} of {groups} groups kept for {top} of {experts} experts")
    ld, inner = logits.stride()
    if inner != 1 or ld < experts:
        logits, ld = _packed_rows(logits, experts)
    index = dev.index
    bias_at = 0
    if bias is not None:
        if (not isinstance(bias, _Tensor) or bias.dtype is not torch.float32 or bias.get_device() != index
                or bias.shape != (experts,) or not bias.is_contiguous()):
            _check_buffer(bias, (experts,), dev, "bias", torch.float32)
        bias_at = bias.data_ptr()
    space, given = _workspace_bytes(tokens, experts, top) if order else 0, out is not None
    ws = None
    if not given:
        out, places, ws = _new_routes(tokens, experts, top, order, 0 if workspace is not None else space, dev)
    else:
        _check_buffer(out.experts, (tokens, top), dev, "out.experts", torch.int32)
        _check_buffer(out.weights, (tokens, top), dev, "out.weights", torch.float32)
        if order:
            _check_buffer(out.offsets, (experts + 1,), dev, "out.offsets", torch.int32)
            _check_buffer(out.rows, (tokens * top,), dev, "out.rows", torch.int32)
            _check_buffer(out.slots, (tokens, top), dev, "out.slots", torch.int32)
        places = [t.data_ptr() for t in out[:5 if order else 2]] + ([] if order else [0, 0, 0])
    if workspace is not None:
        _check_buffer(workspace, None, dev, "workspace")
        ws, space = workspace.data_ptr(), workspace.nbytes
    elif given and space:
        workspace = torch.empty(space, dtype=torch.uint8, device=dev)  # kept until the launch is enqueued
        ws = workspace.data_ptr()
    status = lib().razer_moe_route(
        _route_bytes(tokens, ld, experts, top, groups, kept, group_best, kind, dt,
                     RAZER_ROUTE_RENORM if renormalise else 0, scale, logits.data_ptr(), bias_at,
                     *places),
        ws, space, _stream(index))
    if status:
        _check(status, "razer_moe_route")
    if _forward._current_level >= 0 and not given:
        _no_tangents("razer_moe_route", (logits, bias))
    if not given and _grad_enabled() and (logits.requires_grad or bias is not None and bias.requires_grad):
        out = out._replace(weights=_without_backward("razer_moe_route", (out.weights.clone(),), (logits, bias))[0])
    return out


def razer_moe_combine(y: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor, add: torch.Tensor | None = None,
                      out=None, stream=None) -> torch.Tensor:
    """out[t] = add[t] + sum_j weights[t, j] * y[slots[t, j]], in fp32, rounded once.

    y: [rows, cols], the experts' rows; slots (int32) and weights (float32): [tokens, top];
    add: [tokens, cols] of y's dtype.  A slot outside y stands for zeros.  out may be add.
    There is no backward: one that reaches the result raises; what is written to out
    stands outside any graph."""
    if stream is not None:
        with _entered(stream):
            return razer_moe_combine(y, slots, weights, add, out)
    dev = _on_gpu(y, "y")
    index, kind = dev.index, y.dtype
    dt = _dtype(kind)
    shape = slots.shape if isinstance(slots, _Tensor) else ()
    if y.dim() != 2 or len(shape) != 2:
        raise ValueError("y and slots must be 2-D")
    rows, cols = y.shape
    tokens, top = shape
    if slots.dtype is not torch.int32 or slots.get_device() != index or not slots.is_contiguous():
        _check_buffer(slots, shape, dev, "slots", torch.int32)
    if (not isinstance(weights, _Tensor) or weights.dtype is not torch.float32 or weights.get_device() != index
            or weights.shape != shape or not weights.is_contiguous()):
        _check_buffer(weights, shape, dev, "weights", torch.float32)
    y_stride, inner = y.stride()
    if inner != 1 or y_stride < cols:
        y, y_stride = _packed_rows(y, cols)
    source, add_at, add_stride = add, 0, 0
    if add is not None:
        if (not isinstance(add, _Tensor) or add.get_device() != index or add.shape != (tokens, cols)
                or add.dtype is not kind):
            raise ValueError(f"add must be {tokens}x{cols} of {kind} on {dev}")
        add_stride, inner = add.stride()
        if inner != 1 or add_stride < cols:
            add, add_stride = _packed_rows(add, cols)
        add_at = add.data_ptr()
    given = out is not None
    if not given:
        out = torch.empty(tokens, cols, dtype=kind, device=dev)
    else:
        _check_buffer(out, (tokens, cols), dev, "out", kind)
    status = lib().razer_moe_combine(
        _combine_bytes(tokens, top, cols, rows, y_stride, add_stride, dt, y.data_ptr(), slots.data_ptr(),
                       weights.data_ptr(), add_at, out.data_ptr()), _stream(index))
    if status:
        _check(status, "razer_moe_combine")
    if _forward._current_level >= 0 and not given:
        _no_tangents("razer_moe_combine", (y, weights, source))
    if not given and _grad_enabled() and (y.requires_grad or weights.requires_grad
                                          or source is not None and source.requires_grad):
        out, = _without_backward("razer_moe_combine", (out,), (y, weights, source))
    return out
