"""8-bit integer tensors with a scale for each row: binding of the ``razer_i8_*`` calls
of ``include/librazer.h``.

An ``I8Tensor`` holds whole numbers from -127 to 127 and one fp32 scale a row: a scale
for each token of an activation, for each output channel of a weight.  Both operands of
a product are I8Tensors::

    x = razer_i8_quantize(h)
    gu = razer_i8_gemm(x, gate_up)                     # [M, 2 * I]
    y = razer_i8_gemm(razer_i8_quantize_gated(gu), down)

Streams as in ``mx``: calls run on the current stream, or on ``stream``.  No call has a
backward: where an input requires a gradient, or an operand's scales do, one that reaches
the result raises; the scales of an encoded tensor stand in its input's graph for that
(what is written to ``out`` stands outside any graph).  A tangent of forward mode raises in
the call.  The package re-exports every name here.
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from . import _check_buffer, lib
from .mx import (_check, _dtype, _entered, _forward, _grad_enabled, _no_tangents, _on_gpu, _rows_of, _space, _stream,
                 _Tensor, _without_backward)

I8_UNIT = 16
RAZER_I8_MAX_K = 131056
_i8, _f32 = torch.int8, torch.float32


class razer_i8(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("codes", ctypes.c_void_p),
                ("scales", ctypes.c_void_p)]


# The struct as bytes, which cost a quarter of a ctypes instance to make
_struct_bytes = struct.Struct("qqPP").pack


def bind(L: ctypes.CDLL):
    """Argument types of the calls bound here."""
    vp, sz, i32, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64
    for name, args in (("razer_i8_quantize", [vp, i32, i64, vp, vp]),
                       ("razer_i8_quantize_gated", [vp, i32, i64, vp, vp]),
                       ("razer_i8_dequant", [vp, vp, i32, vp]),
                       ("razer_i8_gemm", [vp, vp, vp, i32, vp, sz, vp]),
                       ("razer_i8_gemm_grouped", [vp, vp, vp, i64, vp, i64, vp, i32, vp, sz, vp])):
        f = getattr(L, name)
        f.restype, f.argtypes = i32, args
    L.razer_i8_workspace_bytes.restype, L.razer_i8_workspace_bytes.argtypes = sz, [i64] * 4


class I8Tensor:
    """An 8-bit integer tensor in device memory.

    codes: int8 [rows, cols], scales: float32 [rows].  rows, cols and buffers can be
    replaced, or changed in place; a call takes what codes and scales show, and refuses a
    tensor whose buffers do not match its shape."""

    # _index: the GPU, -1 without one; _at, _scales_at: addresses of the buffers when they were
    # last looked at, and what shapes they had; _struct: the razer_i8 as of then
    __slots__ = ("_rows", "_cols", "_buf", "_codes", "_scales", "_device", "_index", "_at", "_scales_at",
                 "_codes_shape", "_scales_shape", "_struct")

    def __init__(self, rows: int, cols: int, device):
        if rows < 0 or cols < 0 or cols % I8_UNIT:
            raise ValueError(f"cols must be a multiple of {I8_UNIT}")
        self._rows, self._cols = rows, cols
        # one buffer for both: codes, then scales; their views are made when asked for
        self._own(torch.empty(rows * (cols + 4), dtype=torch.int8, device=device))

    def _own(self, buf: torch.Tensor):
        self._buf, self._codes, self._scales = buf, None, None
        self._device, self._index, self._at = buf.device, buf.get_device(), buf.data_ptr()
        self._scales_at = self._at + self._rows * self._cols
        self._struct = _struct_bytes(self._rows, self._cols, self._at, self._scales_at)

    @classmethod
    def of(cls, codes: torch.Tensor, scales: torch.Tensor) -> "I8Tensor":
        """The tensor that these buffers hold (shared, not copied); leading
        dimensions, such as a stack of experts, are rows."""
        t = cls.__new__(cls)
        shape = codes.shape
        if len(shape) != 2:
            codes = codes.view(-1, shape[-1])
            shape = codes.shape
        if scales.dim() != 1:
            scales = scales.view(-1)
        t._rows, t._cols = shape
        t._buf, t._codes, t._scales = None, codes, scales
        t._check_buffers("I8Tensor", shape)
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
            self._codes = self._buf[:self._rows * self._cols].view(self._rows, self._cols)
        return self._codes

    @codes.setter
    def codes(self, t: torch.Tensor):
        self._detach()
        self._codes = t

    @property
    def scales(self) -> torch.Tensor:
        if self._scales is None:
            self._scales = self._buf[self._rows * self._cols:].view(torch.float32)
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
        return self._rows * (self._cols + 4)

    def check(self, name: str = "I8Tensor") -> torch.device:
        """Its buffers match its shape; returns their device."""
        self._checked(name)
        return self._device

    def _checked(self, name: str) -> bytes:
        """The razer_i8 of buffers that match the shape.  Whoever holds the codes or scales
        may have changed them in place since (`.data =`, `t_`, `resize_`): every call looks at
        those that anybody has seen, and at the rest if they are not as they were.  (The one
        buffer of its own moves with a copy of the whole, or a load from a file.)"""
        c, s = self._codes, self._scales
        if self._buf is not None:
            if c is None and s is None:
                if self._buf.data_ptr() != self._at:
                    self._own(self._buf)
                return self._struct
            # from here on what is seen counts, not the buffer behind it
            self._detach()
            c, s = self._codes, self._scales
        if (c.data_ptr() != self._at or s.data_ptr() != self._scales_at or c.shape != self._codes_shape
                or s.shape != self._scales_shape or c.dtype is not _i8 or s.dtype is not _f32
                or not c.is_contiguous() or not s.is_contiguous()):
            self._check_buffers(name)
        return self._struct

    def _check_buffers(self, name: str, codes_shape=None):
        c, s, rows, cols = self._codes, self._scales, self._rows, self._cols
        index, codes_shape, scales_shape = c.get_device(), codes_shape or c.shape, s.shape
        if (c.dtype is not _i8 or s.dtype is not _f32 or cols % I8_UNIT or s.get_device() != index
                or codes_shape != (rows, cols) or scales_shape != (rows,)
                or not c.is_contiguous() or not s.is_contiguous()):
            raise ValueError(f"{name}: codes {tuple(c.shape)} {c.dtype} on {c.device} and scales {tuple(s.shape)} "
                             f"{s.dtype} on {s.device} are no contiguous 8-bit tensor of {rows}x{cols}")
        self._device, self._index, self._at, self._scales_at = c.device, index, c.data_ptr(), s.data_ptr()
        self._codes_shape, self._scales_shape = codes_shape, scales_shape
        self._struct = _struct_bytes(rows, cols, self._at, self._scales_at)


def _operand(t, name: str) -> bytes:
    """The struct of an operand on a GPU."""
    if not isinstance(t, I8Tensor):
        raise TypeError(f"{name} must be an I8Tensor")
    struct = t._checked(name)
    if t._index < 0:
        raise ValueError(f"{name} must be on a GPU, not {t._device}")
    return struct


def _operands(x, w):
    """Both structs of a product."""
    if not (isinstance(x, I8Tensor) and isinstance(w, I8Tensor)):
        raise TypeError("x and w must be I8Tensors")
    xs, ws, index = x._checked("x"), w._checked("w"), x._index
    if index < 0:
        raise ValueError(f"x must be on a GPU, not {x._device}")
    if w._index != index:
        raise ValueError(f"w must be on {x._device}, not {w._device}")
    if x._cols != w._cols:
        raise ValueError(f"x has {x._cols} columns, w {w._cols}")
    return xs, ws


def _outside_graph(call: str, out, x, w):
    """out, in the graph of the scales of x and w where they require a gradient."""
    xs, ws = x._scales, w._scales  # None: nobody has seen them
    if _forward._current_level >= 0:
        _no_tangents(call, (xs, ws))
    if (xs is not None and xs.requires_grad or ws is not None and ws.requires_grad) and _grad_enabled():
        return _without_backward(call, (out,), (xs, ws))[0]
    return out


def _encode(call, x, parts: int, out, stream) -> I8Tensor:
    if stream is not None:
        with _entered(stream):
            return _encode(call, x, parts, out, None)
    dev = _on_gpu(x, "x")
    dt = _dtype(x.dtype)
    if x.dim() != 2:
        raise ValueError("expected a 2-D tensor")
    rows, width = x.shape
    cols = width if parts == 1 else width // parts
    if cols * parts != width or cols % I8_UNIT:
        raise ValueError(f"columns must be a multiple of {parts * I8_UNIT}")
    current, source, given = _stream(dev.index), x, out is not None
    if not given:
        out = I8Tensor(rows, cols, dev)
        packed = out._struct
    else:
        packed = _operand(out, "out")
        if out._device != dev:
            raise ValueError(f"out must be on {dev}, not {out._device}")
        if out.shape != (rows, cols):
            raise ValueError(f"out is {out.rows}x{out.cols}, expected {rows}x{cols}")
    x, ptr, ld = _rows_of(x, width)
    st = call(ptr, dt, ld, packed, current)
    if st:
        _check(st, call.__name__)
    if _forward._current_level >= 0 and not given:
        _no_tangents(call.__name__, (source,))
    if not given and source.requires_grad and _grad_enabled():
        # from the scales it reaches what the tensor is used in: whole numbers have no gradient
        _without_backward(call.__name__, (out.scales,), (source,))
    return out


def razer_i8_quantize(x: torch.Tensor, out: I8Tensor | None = None, stream=None) -> I8Tensor:
    """8-bit encoding of x [rows, cols] (f32, f16 or bf16; cols % 16 == 0), a scale a row.
    There is no backward: where x requires a gradient, one that reaches the scales, or what
    the tensor is used in, raises; what is written to out stands outside any graph."""
    return _encode(lib().razer_i8_quantize, x, 1, out, stream)


def razer_i8_quantize_gated(gu: torch.Tensor, out: I8Tensor | None = None, stream=None) -> I8Tensor:
    """8-bit encoding of silu(g) * u for gu [rows, 2 * cols] = [g | u]; gradients as in
    razer_i8_quantize."""
    return _encode(lib().razer_i8_quantize_gated, gu, 2, out, stream)


def razer_i8_dequant(t: I8Tensor, dtype: torch.dtype = torch.float32, out=None, stream=None) -> torch.Tensor:
    """The values code * scale of t [rows, cols] (rounded to f32, then to dtype)."""
    if stream is not None:
        with _entered(stream):
            return razer_i8_dequant(t, dtype, out)
    packed, dev, index, given = _operand(t, "t"), t._device, t._index, out is not None
    current = _stream(index)
    if not given:
        out = torch.empty(t._rows, t._cols, dtype=dtype, device=dev)
    else:
        _check_buffer(out, t.shape, dev, "out")
        dtype = out.dtype
    st = lib().razer_i8_dequant(packed, out.data_ptr(), _dtype(dtype), current)
    if st:
        _check(st, "razer_i8_dequant")
    return out if given else _outside_graph("razer_i8_dequant", out, t, t)


def razer_i8_workspace_bytes(m: int, n: int, k: int, experts: int = 0) -> int:
    return int(lib().razer_i8_workspace_bytes(m, n, k, experts))


@functools.lru_cache(4096)
def _workspace_bytes(m: int, n: int, k: int, experts: int, device: int) -> int:
    """razer_i8_workspace_bytes on a device: a function of the sizes and its compute units."""
    return razer_i8_workspace_bytes(m, n, k, experts)


def razer_i8_gemm(x: I8Tensor, w: I8Tensor, out_dtype: torch.dtype = torch.bfloat16, out=None, workspace=None,
                  stream=None) -> torch.Tensor:
    """y[M, N] = x[M, K] . w[N, K]^T."""
    if stream is not None:
        with _entered(stream):
            return razer_i8_gemm(x, w, out_dtype, out, workspace)
    xs, ws = _operands(x, w)
    m, n, dev, index, space, space_bytes = x._rows, w._rows, x._device, x._index, None, 0
    current, given = _stream(index), out is not None
    if not given:
        out = torch.empty(m, n, dtype=out_dtype, device=dev)
    else:
        _check_buffer(out, (m, n), dev, "out")
        out_dtype = out.dtype
    need = _workspace_bytes(m, n, x._cols, 0, index)
    if need or workspace is not None:
        workspace, space, space_bytes = _space(need, workspace, dev)
    status = lib().razer_i8_gemm(xs, ws, out.data_ptr(), _dtype(out_dtype), space, space_bytes, current)
    if status:
        _check(status, "razer_i8_gemm")
    return out if given else _outside_graph("razer_i8_gemm", out, x, w)


def razer_i8_gemm_grouped(x: I8Tensor, w: I8Tensor, offsets: torch.Tensor, x_rows: torch.Tensor | None = None,
                          out_dtype: torch.dtype = torch.bfloat16, out=None, workspace=None,
                          stream=None) -> torch.Tensor:
    """The products of a mixture of experts: w stacks E = offsets.numel() - 1
    weights [N, K]; rows offsets[e] .. offsets[e + 1] - 1 of the result are
    x[x_rows[r]] . w_e^T (x[r] without x_rows).  offsets (int32 [E + 1]) and
    x_rows (int32 [M]) stay on the GPU.  Rows outside every run are not written;
    a row number outside x makes its row zero."""
    if stream is not None:
        with _entered(stream):
            return razer_i8_gemm_grouped(x, w, offsets, x_rows, out_dtype, out, workspace)
    xs, ws = _operands(x, w)
    dev, index, given = x._device, x._index, out is not None
    current = _stream(index)
    # (the checks in line cost a third of the call that names what is wrong)
    if not (isinstance(offsets, _Tensor) and offsets.dtype is torch.int32 and offsets.get_device() == index
            and offsets.dim() == 1 and offsets.is_contiguous()):
        if offsets.dim() != 1:
            raise ValueError("offsets must be 1-D")
        _check_buffer(offsets, offsets.shape, dev, "offsets", torch.int32)
    experts, m = offsets.numel() - 1, x._rows
    if experts < 1 or w._rows % experts:
        raise ValueError(f"w has {w._rows} rows for {experts} experts")
    rows = None
    if x_rows is not None:
        if not (isinstance(x_rows, _Tensor) and x_rows.dtype is torch.int32 and x_rows.get_device() == index
                and x_rows.dim() == 1 and x_rows.is_contiguous()):
            if x_rows.dim() != 1:
                raise ValueError("x_rows must be 1-D")
            _check_buffer(x_rows, x_rows.shape, dev, "x_rows", torch.int32)
        m, rows = x_rows.numel(), x_rows.data_ptr()
    n = w._rows // experts
    if not given:
        out = torch.empty(m, n, dtype=out_dtype, device=dev)
    else:
        _check_buffer(out, (m, n), dev, "out")
        out_dtype = out.dtype
    space, space_bytes = None, 0
    need = _workspace_bytes(m, n, x._cols, experts, index)
    if need or workspace is not None:
        workspace, space, space_bytes = _space(need, workspace, dev)
    status = lib().razer_i8_gemm_grouped(xs, ws, offsets.data_ptr(), experts, rows, m, out.data_ptr(),
                                         _dtype(out_dtype), space, space_bytes, current)
    if status:
        _check(status, "razer_i8_gemm_grouped")
    return out if given else _outside_graph("razer_i8_gemm_grouped", out, x, w)
