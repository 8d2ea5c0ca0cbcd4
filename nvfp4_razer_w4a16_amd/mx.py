"""Microscaled 4-bit tensors (MXFP4) and the block norm: binding of the
``razer_mx_*`` calls and ``razer_block_norm`` of ``include/librazer.h``.

An ``MxTensor`` holds 32-element blocks of FP4-E2M1 codes with one power-of-two
scale byte each.  Both operands of a product are MxTensors::

    h, x = razer_block_norm(y, h, post_weight=p, pre_weight=q, packed=True)
    gu   = razer_mx_gemm(x, gate_up)                  # [M, 2 * I]
    y    = razer_mx_gemm(razer_mx_quantize_gated(gu), down)

Calls run on the current stream; with ``stream`` they run as inside
``torch.cuda.stream(stream)``, and what they return belongs to that stream.  No
call has a backward: the block norm's plain results raise in one, packed tensors and
what they are used in stand outside any graph.  The package re-exports every name here.
"""
from __future__ import annotations

import ctypes
import functools

import torch
from torch.autograd import forward_ad as _forward

from . import _DT, RAZER_OK, RazerError, _check_buffer, lib

# Calls on a few rows take microseconds: the checks below are written to cost
# little beside a launch.
_Tensor, _u8, _grad_enabled = torch.Tensor, torch.uint8, torch.is_grad_enabled
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)

RAZER_NORM_POST = 1
RAZER_MX_MAX_EXPERTS = 4096
MX_BLOCK = 32


class razer_mx(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("codes", ctypes.c_void_p),
                ("scales", ctypes.c_void_p)]


class razer_norm(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("y", ctypes.c_void_p), ("h", ctypes.c_void_p),
                ("y_stride", ctypes.c_int64), ("h_stride", ctypes.c_int64), ("post_weight", ctypes.c_void_p),
                ("pre_weight", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("gate_rows", ctypes.c_int64),
                ("residual_scale", ctypes.c_float), ("eps", ctypes.c_float), ("h_out", ctypes.c_void_p),
                ("x_out", ctypes.c_void_p), ("packed", ctypes.POINTER(razer_mx))]


def bind(L: ctypes.CDLL):
    """Argument types of the calls bound here."""
    vp, sz, i32, i64, P = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64, ctypes.POINTER(razer_mx)
    for name, args in (("razer_mx_quantize", [vp, i32, i64, P, vp]),
                       ("razer_mx_quantize_gated", [vp, i32, i64, P, vp]),
                       ("razer_mx_dequant", [P, vp, i32, vp]),
                       ("razer_mx_gemm", [P, P, vp, i32, vp, sz, vp]),
                       ("razer_mx_gemm_grouped", [P, P, vp, i64, vp, i64, vp, i32, vp, sz, vp]),
                       ("razer_block_norm", [ctypes.POINTER(razer_norm), vp])):
        f = getattr(L, name)
        f.restype, f.argtypes = i32, args
    L.razer_mx_workspace_bytes.restype, L.razer_mx_workspace_bytes.argtypes = sz, [i64] * 4


def _check(status: int, what: str):
    if status != RAZER_OK:
        raise RazerError(status, what)


def _stream(index: int) -> int:
    """The current stream of the tensors' device, which has to be the current
    device: launches go to that one."""
    if index != _current_device():
        raise ValueError(f"tensors are on cuda:{index}, the current device is cuda:{_current_device()}")
    return _raw_stream(index)


def _entered(stream):
    """`stream` (a torch stream or a handle) as the current one: what a call
    allocates or copies on the way is then ordered with its launch."""
    if not isinstance(stream, torch.cuda.Stream):
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _dtype(dt: torch.dtype) -> int:
    code = _DT.get(dt)
    if code is None:
        raise TypeError(f"unsupported dtype {dt}")
    return code


def _on_gpu(t, name: str) -> torch.device:
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU, not {t.device}")
    return t.device


class MxTensor:
    """An MXFP4 tensor in device memory.

    codes: uint8 [rows, cols // 2], the even column in the low half of a byte;
    scales: uint8 [rows, cols // 32].  rows, cols and buffers can be replaced; a call
    refuses a tensor whose buffers do not match its shape, also where buffers that it was
    given were changed in place.  (One that made its own buffer keeps to that, whatever is
    done in place to the shapes or memory of the codes and scales it shows.)"""

    # _index: the GPU, -1 without one; _at, _scales_at: addresses of the buffers it was
    # given, when they were last looked at, and what shapes they had
    __slots__ = ("_rows", "_cols", "_buf", "_codes", "_scales", "_device", "_index", "_at", "_scales_at",
                 "_codes_shape", "_scales_shape")

    def __init__(self, rows: int, cols: int, device):
        if rows < 0 or cols < 0 or cols % MX_BLOCK:
            raise ValueError(f"cols must be a multiple of {MX_BLOCK}")
        self._rows = rows
        self._cols = cols
        # one buffer for both: codes, then scales; their views are made when asked for
        self._buf = buf = torch.empty(rows * cols // 32 * 17, dtype=torch.uint8, device=device)
        self._device, self._index = buf.device, buf.get_device()
        self._codes = self._scales = None

    @classmethod
    def of(cls, codes: torch.Tensor, scales: torch.Tensor) -> "MxTensor":
        """The tensor that these buffers hold (shared, not copied); leading
        dimensions, such as a stack of experts, are rows."""
        t = cls.__new__(cls)
        shape = codes.shape
        if len(shape) != 2:
            codes, scales = codes.view(-1, shape[-1]), scales.view(-1, scales.shape[-1])
            shape = codes.shape
        t._rows, half = shape
        t._cols, t._buf, t._codes, t._scales = 2 * half, None, codes, scales
        t._check_buffers("MxTensor", shape)
        return t

    def _detach(self):
        """From here on the buffers are plain tensors that have to match the shape."""
        self._codes, self._scales, self._buf, self._at = self.codes, self.scales, None, -1

    @property
    def rows(self) -> int:
        return self._rows

    @rows.setter
    def rows(self, rows: int):
        self._detach()
        self._rows = rows

    @property
    def cols(self) -> int:
        return self._cols

    @cols.setter
    def cols(self, cols: int):
        self._detach()
        self._cols = cols

    @property
    def codes(self) -> torch.Tensor:
        if self._codes is None:
            self._codes = self._buf[:self._rows * self._cols // 2].view(self._rows, self._cols // 2)
        return self._codes

    @codes.setter
    def codes(self, t: torch.Tensor):
        self._detach()
        self._codes = t

    @property
    def scales(self) -> torch.Tensor:
        if self._scales is None:
            self._scales = self._buf[self._rows * self._cols // 2:].view(self._rows, self._cols // MX_BLOCK)
        return self._scales

    @scales.setter
    def scales(self, t: torch.Tensor):
        self._detach()
        self._scales = t

    @property
    def device(self) -> torch.device:
        return self._device if self._buf is not None else self._codes.device

    @property
    def shape(self):
        return (self._rows, self._cols)

    def nbytes(self) -> int:
        return self._rows * self._cols // 32 * 17

    def check(self, name: str = "MxTensor") -> torch.device:
        """Its buffers match its shape; returns their device."""
        self._checked(name)
        return self._device

    def _checked(self, name: str) -> razer_mx:
        """The struct of buffers that match the shape.  The owner of buffers that it
        was given may have changed them in place since (`.data =`, `t_`, `resize_`):
        every call looks at them, and at the rest if they are not as they were."""
        rows, cols = self._rows, self._cols
        if self._buf is not None:
            at = self._buf.data_ptr()
            return razer_mx(rows, cols, at, at + (rows * cols >> 1))
        c, s = self._codes, self._scales
        at, scales_at = c.data_ptr(), s.data_ptr()
        if (at != self._at or scales_at != self._scales_at or c.shape != self._codes_shape
                or s.shape != self._scales_shape or c.dtype is not _u8 or s.dtype is not _u8
                or not c.is_contiguous() or not s.is_contiguous()):
            self._check_buffers(name)
        return razer_mx(rows, cols, at, scales_at)

    def _check_buffers(self, name: str, codes_shape=None):
        c, s, rows, cols = self._codes, self._scales, self._rows, self._cols
        index, codes_shape, scales_shape = c.get_device(), codes_shape or c.shape, s.shape
        if (c.dtype is not _u8 or s.dtype is not _u8 or cols & 31 or s.get_device() != index
                or codes_shape != (rows, cols >> 1) or scales_shape != (rows, cols >> 5)
                or not c.is_contiguous() or not s.is_contiguous()):
            raise ValueError(f"{name}: codes {tuple(c.shape)} {c.dtype} on {c.device} and scales {tuple(s.shape)} "
                             f"{s.dtype} on {s.device} are no contiguous uint8 MXFP4 tensor of {rows}x{cols}")
        self._device, self._index, self._at, self._scales_at = c.device, index, c.data_ptr(), s.data_ptr()
        self._codes_shape, self._scales_shape = codes_shape, scales_shape

    def struct(self) -> razer_mx:
        if self._buf is not None:
            p = self._buf.data_ptr()
            return razer_mx(self._rows, self._cols, p, p + self._rows * self._cols // 2)
        return razer_mx(self._rows, self._cols, self._codes.data_ptr(), self._scales.data_ptr())


def _operand(t, name: str) -> razer_mx:
    """The struct of an operand on a GPU."""
    if not isinstance(t, MxTensor):
        raise TypeError(f"{name} must be an MxTensor")
    struct = t._checked(name)
    if t._index < 0:
        raise ValueError(f"{name} must be on a GPU, not {t._device}")
    return struct


def _operands(x, w):
    """Both structs of a product."""
    if not (isinstance(x, MxTensor) and isinstance(w, MxTensor)):
        raise TypeError("x and w must be MxTensors")
    xs, ws, index = x._checked("x"), w._checked("w"), x._index
    if index < 0:
        raise ValueError(f"x must be on a GPU, not {x._device}")
    if w._index != index:
        raise ValueError(f"w must be on {x._device}, not {w._device}")
    if x._cols != w._cols:
        raise ValueError(f"x has {x._cols} columns, w {w._cols}")
    return xs, ws


def _rows_of(x: torch.Tensor, cols: int):
    """(x, address, stride) of x [rows, cols] as the calls take it: contiguous rows
    at any stride of whole 16 bytes; copied where it is not."""
    ptr = x.data_ptr()
    ld, inner = x.stride()
    if inner == 1 and not (ld * x.element_size() | ptr) & 15 and ld >= cols:
        return x, ptr, ld
    # A lone row counts as contiguous whatever its stride, and so do copies of it that
    # keep the stride: below, rows are `cols` apart.
    x = x.contiguous()
    if x.data_ptr() & 15:
        x = x.clone()
    return x, x.data_ptr(), cols


def _packed_out(out, rows: int, cols: int, device) -> razer_mx:
    """The struct of a caller's output, which has to fit."""
    struct = _operand(out, "out")
    if out._device != device:
        raise ValueError(f"out must be on {device}, not {out._device}")
    if out.shape != (rows, cols):
        raise ValueError(f"out is {out.rows}x{out.cols}, expected {rows}x{cols}")
    return struct


def _encode(call, x, parts: int, out, stream) -> MxTensor:
    if stream is not None:
        with _entered(stream):
            return _encode(call, x, parts, out, None)
    dev = _on_gpu(x, "x")
    dt = _dtype(x.dtype)
    if x.dim() != 2:
        raise ValueError("expected a 2-D tensor")
    rows, width = x.shape
    cols = width // parts
    if width % parts or cols % MX_BLOCK:
        raise ValueError(f"columns must be a multiple of {parts * MX_BLOCK}")
    if out is None:
        out = MxTensor(rows, cols, dev)
        packed = out.struct()
    else:
        packed = _packed_out(out, rows, cols, dev)
    x, ptr, ld = _rows_of(x, width)
    st = call(ptr, dt, ld, packed, _stream(dev.index))
    if st:
        _check(st, call.__name__)
    return out


def razer_mx_quantize(x: torch.Tensor, out: MxTensor | None = None, stream=None) -> MxTensor:
    """MXFP4 encoding of x [rows, cols] (f32, f16 or bf16; cols % 32 == 0)."""
    return _encode(lib().razer_mx_quantize, x, 1, out, stream)


def razer_mx_quantize_gated(gu: torch.Tensor, out: MxTensor | None = None, stream=None) -> MxTensor:
    """MXFP4 encoding of silu(g) * u for gu [rows, 2 * cols] = [g | u]."""
    return _encode(lib().razer_mx_quantize_gated, gu, 2, out, stream)


def razer_mx_dequant(t: MxTensor, dtype: torch.dtype = torch.float32, out=None, stream=None) -> torch.Tensor:
    """The values of t [rows, cols] (exact in f32, rounded once to f16 / bf16)."""
    if stream is not None:
        with _entered(stream):
            return razer_mx_dequant(t, dtype, out)
    packed, dev = _operand(t, "t"), t._device
    if out is None:
        out = torch.empty(t._rows, t._cols, dtype=dtype, device=dev)
    else:
        _check_buffer(out, t.shape, dev, "out")
        dtype = out.dtype
    st = lib().razer_mx_dequant(packed, out.data_ptr(), _dtype(dtype), _stream(t._index))
    if st:
        _check(st, "razer_mx_dequant")
    return out


def razer_mx_workspace_bytes(m: int, n: int, k: int, experts: int = 0) -> int:
    return int(lib().razer_mx_workspace_bytes(m, n, k, experts))


@functools.lru_cache(4096)
def _workspace_bytes(m: int, n: int, k: int, device: int) -> int:
    """razer_mx_workspace_bytes on a device: a function of the sizes and its compute units."""
    return razer_mx_workspace_bytes(m, n, k)


def _space(need: int, workspace, dev):
    """(workspace, its address, its bytes): the caller's, or one of `need` bytes.  It is
    kept until the launch is enqueued; from then on the stream's order keeps it."""
    if workspace is not None:
        _check_buffer(workspace, None, dev, "workspace")
    elif need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        return None, None, 0
    return workspace, workspace.data_ptr(), workspace.nbytes


def razer_mx_gemm(x: MxTensor, w: MxTensor, out_dtype: torch.dtype = torch.bfloat16, out=None, workspace=None,
                  stream=None) -> torch.Tensor:
    """y[M, N] = x[M, K] . w[N, K]^T."""
    if stream is not None:
        with _entered(stream):
            return razer_mx_gemm(x, w, out_dtype, out, workspace)
    xs, ws = _operands(x, w)
    m, n, dev, index, space, space_bytes = x._rows, w._rows, x._device, x._index, None, 0
    current = _stream(index)
    if out is None:
        out = torch.empty(m, n, dtype=out_dtype, device=dev)
    else:
        _check_buffer(out, (m, n), dev, "out")
    need = _workspace_bytes(m, n, x._cols, index)
    if need or workspace is not None:
        workspace, space, space_bytes = _space(need, workspace, dev)
    status = lib().razer_mx_gemm(xs, ws, out.data_ptr(), _dtype(out.dtype), space, space_bytes, current)
    if status:
        _check(status, "razer_mx_gemm")
    return out


def razer_mx_gemm_grouped(x: MxTensor, w: MxTensor, offsets: torch.Tensor, x_rows: torch.Tensor | None = None,
                          out_dtype: torch.dtype = torch.bfloat16, out=None, workspace=None,
                          stream=None) -> torch.Tensor:
    """The products of a mixture of experts: w stacks E = offsets.numel() - 1
    weights [N, K]; rows offsets[e] .. offsets[e + 1] - 1 of the result are
    x[x_rows[r]] . w_e^T (x[r] without x_rows).  offsets (int32 [E + 1]) and
    x_rows (int32 [M]) stay on the GPU.  Rows outside every run are not written;
    a row number outside x makes its row zero."""
    if stream is not None:
        with _entered(stream):
            return razer_mx_gemm_grouped(x, w, offsets, x_rows, out_dtype, out, workspace)
    xs, ws = _operands(x, w)
    dev = x._device
    if offsets.dim() != 1:
        raise ValueError("offsets must be 1-D")
    _check_buffer(offsets, tuple(offsets.shape), dev, "offsets", torch.int32)
    experts, m = offsets.numel() - 1, x.rows
    if experts < 1 or w.rows % experts:
        raise ValueError(f"w has {w.rows} rows for {experts} experts")
    rows = None
    if x_rows is not None:
        if x_rows.dim() != 1:
            raise ValueError("x_rows must be 1-D")
        _check_buffer(x_rows, tuple(x_rows.shape), dev, "x_rows", torch.int32)
        m, rows = x_rows.numel(), x_rows.data_ptr()
    n = w.rows // experts
    if out is None:
        out = torch.empty(m, n, dtype=out_dtype, device=dev)
    else:
        _check_buffer(out, (m, n), dev, "out")
    need = 0 if workspace is not None else razer_mx_workspace_bytes(m, n, x.cols, experts)
    workspace, space, space_bytes = _space(need, workspace, dev)
    _check(lib().razer_mx_gemm_grouped(xs, ws, offsets.data_ptr(), experts, rows, m, out.data_ptr(),
                                       _dtype(out.dtype), space, space_bytes, _stream(x._index)),
           "razer_mx_gemm_grouped")
    return out


class _NoBackward(torch.autograd.Function):
    """Puts results into the graph of the inputs they came from, where a backward pass raises."""

    @staticmethod
    def forward(ctx, call, count, *tensors):
        ctx.call = call
        ctx.mark_dirty(*tensors[:count])
        return tensors[:count]

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError(f"{ctx.call} has no backward: call it under torch.no_grad(), or detach its inputs")


def _without_backward(call: str, results, inputs):
    """The results of a call without a backward: those inputs that require a gradient
    would silently get none, so a backward pass that reaches the results raises."""
    return _NoBackward.apply(call, len(results), *results, *(t for t in inputs if t is not None))


def _no_tangents(call: str, inputs):
    """In forward mode a result would lose its inputs' tangents, so one among them raises,
    whether or not gradients are recorded.  (_forward._current_level: -1 outside that mode.)"""
    for t in inputs:
        if t is not None and _forward.unpack_dual(t).tangent is not None:
            raise RuntimeError(f"{call} has no derivative in forward mode: detach its inputs")


def _vector(t, cols: int, dtype, device, index: int, name: str) -> int:
    """Address of a weight [cols] on GPU `index`."""
    if (not isinstance(t, _Tensor) or t.dtype is not dtype or t.get_device() != index or t.shape != (cols,)
            or not t.is_contiguous()):
        _check_buffer(t, (cols,), device, name, dtype)
    return t.data_ptr()


def razer_block_norm(y: torch.Tensor | None, h: torch.Tensor, *, post_weight=None, post_norm: bool | None = None,
                     gate=None, residual_scale: float = 1.0, pre_weight=None, eps: float = 1e-5,
                     packed: bool = False, h_out=None, x_out=None, stream=None):
    """(h', x) of h' = h + residual_scale * gate . N(y; post_weight) and
    x = N(h'; pre_weight), N(v; w) = w * v / sqrt(mean(v^2) + eps).

    y, h: [rows, cols]; y None: h' = h.  The norm of y is taken where post_norm is
    true (by default, where post_weight is given).  gate: [cols] or
    [gate_rows, cols], gate_rows a divisor of rows.  packed: x is an MxTensor, else
    a tensor of h's dtype.  h_out (h itself, if contiguous) and x_out take the
    results.  There is no backward: one that reaches the results raises, as does a
    tangent of forward mode.  What is written to h_out and x_out, and a packed x, stands
    outside any graph."""
    if stream is not None:
        with _entered(stream):
            return razer_block_norm(y, h, post_weight=post_weight, post_norm=post_norm, gate=gate,
                                    residual_scale=residual_scale, pre_weight=pre_weight, eps=eps, packed=packed,
                                    h_out=h_out, x_out=x_out)
    dev = _on_gpu(h, "h")
    if h.dim() != 2:
        raise ValueError("h must be 2-D")
    rows, cols = shape = h.shape
    if cols % MX_BLOCK:
        raise ValueError(f"columns must be a multiple of {MX_BLOCK}")
    kind = h.dtype
    dt = _dtype(kind)
    h, h_ptr, h_stride = _rows_of(h, cols)
    index = dev.index
    flags, y_ptr, y_stride, post, pre, gates, gate_rows = 0, None, 0, None, None, None, 0
    if y is not None:
        if not isinstance(y, _Tensor) or y.get_device() != index or y.shape != shape or y.dtype is not kind:
            raise ValueError(f"y must be {rows}x{cols} of {kind} on {dev}")
        y, y_ptr, y_stride = _rows_of(y, cols)
        if post_norm if post_norm is not None else post_weight is not None:
            flags = RAZER_NORM_POST
    elif post_weight is not None or gate is not None or post_norm:
        raise ValueError("post_weight, post_norm and gate belong to y")
    if post_weight is not None:
        post = _vector(post_weight, cols, kind, dev, index, "post_weight")
    if pre_weight is not None:
        pre = _vector(pre_weight, cols, kind, dev, index, "pre_weight")
    if gate is not None:
        gate_rows = 1 if gate.dim() == 1 else gate.shape[0]
        _check_buffer(gate, (cols,) if gate.dim() == 1 else (gate_rows, cols), dev, "gate", kind)
        gates = gate.data_ptr()
    new_h, new_x = h_out is None, x_out is None and not packed
    if new_h:
        h_out = torch.empty(rows, cols, dtype=kind, device=dev)
    else:
        _check_buffer(h_out, shape, dev, "h_out", kind)
    x_ptr = p_ptr = None
    if packed:
        x = MxTensor(rows, cols, dev) if x_out is None else x_out
        p_ptr = ctypes.pointer(x.struct() if x_out is None else _packed_out(x, rows, cols, dev))
    elif x_out is None:
        x = torch.empty(rows, cols, dtype=kind, device=dev)
        x_ptr = x.data_ptr()
    else:
        x = x_out
        _check_buffer(x, shape, dev, "x_out", kind)
        x_ptr = x.data_ptr()
    a = razer_norm(rows, cols, dt, flags, y_ptr, h_ptr, y_stride, h_stride, post, pre, gates, gate_rows,
                   residual_scale, eps, h_out.data_ptr(), x_ptr, p_ptr)
    status = lib().razer_block_norm(a, _stream(index))
    if status:
        _check(status, "razer_block_norm")
    if _forward._current_level >= 0 and (new_h or new_x):
        _no_tangents("razer_block_norm", (y, h, post_weight, pre_weight, gate))
    if _grad_enabled() and (h.requires_grad or y is not None and y.requires_grad
                            or post_weight is not None and post_weight.requires_grad
                            or pre_weight is not None and pre_weight.requires_grad
                            or gate is not None and gate.requires_grad):
        inputs = y, h, post_weight, pre_weight, gate
        if new_h and new_x:
            return _without_backward("razer_block_norm", (h_out, x), inputs)
        if new_h:
            h_out, = _without_backward("razer_block_norm", (h_out,), inputs)
        elif new_x:
            x, = _without_backward("razer_block_norm", (x,), inputs)
    return h_out, x
