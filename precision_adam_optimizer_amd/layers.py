"""Binding of the layer operators (C ABI in ``include/fp8adam_layer.h``): linear layers on
8-bit operands, with their activations kept in 8 bits for the backward pass.

They join ``Quantizer``, whose codes are the weights, with ``GradClip`` and ``AdamW``, which take
the gradients.  As in the rest of the package, the functions with the C names only marshal arguments
and there is no fallback; those below them take and return torch tensors.

Activations and their gradients are matrices of fp32, bf16 or fp16, or tensors of more dimensions
whose leading ones fold into rows without a copy; a row is contiguous, rows may lie further apart.
Calls go to the current stream of the tensors' device, allocate their results and workspaces with
torch, wait for nothing, and may be captured into a graph.  Nothing is recorded by autograd: a
backward pass calls the functions that end in ``_backward`` or ``_grad8`` itself, and tensors that require a
gradient are refused where autograd records (under ``torch.no_grad()`` and inside a ``torch.autograd.Function`` it does not).
"""
from __future__ import annotations

import ctypes
from struct import Struct
from typing import NamedTuple

import torch

from . import _FORMATS, BLOCK, E4M3, E5M2, _check, _ptr, current_stream, load
from .lists import _DTYPES

ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU = 0, 1, 2, 3
SCALES_E8M0, SCALES_F32 = 0, 1
LAYER_MAX_COLS, LAYER_MAX_LD = 1 << 20, 1 << 21
_ACTS = {"none": ACT_NONE, "relu": ACT_RELU, "silu": ACT_SILU, "gelu": ACT_GELU}
_FP8 = {E4M3: torch.float8_e4m3fn, E5M2: torch.float8_e5m2}
_FP8_FORMATS = {torch.float8_e4m3fn: E4M3, torch.float8_e5m2: E5M2}

LAYER_EXPORTS = ("fp8adam_pack8", "fp8adam_unpack8", "fp8adam_linear8", "fp8adam_gated8", "fp8adam_linear8_backward",
                 "fp8adam_gated8_backward", "fp8adam_weight_grad8", "fp8adam_input_grad8",
                 "fp8adam_linear8_backward_workspace", "fp8adam_weight_grad8_workspace",
                 "fp8adam_input_grad8_workspace")


class MatrixArg(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("ld", ctypes.c_int64), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class Matrix8Arg(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("ld_scale", ctypes.c_int64), ("format", ctypes.c_int32), ("scale_type", ctypes.c_int32)]


class Product8Arg(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("x_in", MatrixArg),
                ("x", Matrix8Arg), ("w", Matrix8Arg), ("w_up", Matrix8Arg), ("bias", MatrixArg), ("residual", MatrixArg),
                ("y", MatrixArg), ("y8", Matrix8Arg), ("keep", Matrix8Arg), ("keep_up", Matrix8Arg),
                ("activation", ctypes.c_int32), ("exact", ctypes.c_int32)]


class ActBackward8Arg(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("rows", ctypes.c_int64), ("dy", MatrixArg), ("keep", Matrix8Arg),
                ("keep_up", Matrix8Arg), ("dz", MatrixArg), ("dup", MatrixArg), ("bias_grad", MatrixArg),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64), ("accumulate", ctypes.c_int32),
                ("activation", ctypes.c_int32)]


class Grad8Arg(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("n", ctypes.c_int32),
                ("accumulate", ctypes.c_int32), ("dy", MatrixArg * 2), ("b", Matrix8Arg * 2), ("out", MatrixArg),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64), ("exact", ctypes.c_int32), ("reserved", ctypes.c_int32)]


# The same structs packed by the calls below: filling nested ctypes structures costs a small call 5 us.
_M, _M8 = "Qqii", "QQqqii"
_PRODUCT8 = Struct("@3q" + _M + 3 * _M8 + 3 * _M + 3 * _M8 + "2i")
_ACT_BACKWARD8 = Struct("@2q" + _M + 2 * _M8 + 3 * _M + "Qq2i")
_GRAD8 = Struct("@3q2i" + 2 * _M + 2 * _M8 + _M + "Qq2i")

_ready = None
_calls: dict = {}  # the functions on packed structs, by name


def _lib() -> ctypes.CDLL:
    """The library with this header's signatures declared."""
    global _ready
    if _ready is None:
        L = load()
        vp, i64, P = ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER
        L.fp8adam_pack8.argtypes = [P(MatrixArg), P(Matrix8Arg), i64, i64, vp]
        L.fp8adam_unpack8.argtypes = [P(Matrix8Arg), P(MatrixArg), i64, i64, vp]
        for name, arg in (("linear8", Product8Arg), ("gated8", Product8Arg), ("linear8_backward", ActBackward8Arg),
                          ("gated8_backward", ActBackward8Arg), ("weight_grad8", Grad8Arg), ("input_grad8", Grad8Arg)):
            getattr(L, "fp8adam_" + name).argtypes = [P(arg), vp]
            if name in ("linear8_backward", "weight_grad8", "input_grad8"):
                fn = getattr(L, f"fp8adam_{name}_workspace")
                fn.argtypes = [P(arg)]
        for name in LAYER_EXPORTS:
            getattr(L, name).restype = ctypes.c_int64 if name.endswith("_workspace") else ctypes.c_int
        for name in LAYER_EXPORTS[2:]:
            fn = _calls[name[8:]] = L[name]  # another function object
            fn.argtypes = [ctypes.c_char_p] if name.endswith("_workspace") else [ctypes.c_char_p, vp]
            fn.restype = getattr(L, name).restype
        _ready = L
    return _ready


# ---------------------------------------------------------------- C names

def fp8adam_pack8(x: MatrixArg, out: Matrix8Arg, rows: int, cols: int, stream: int | None = None) -> None:
    _check(_lib().fp8adam_pack8(ctypes.byref(x), ctypes.byref(out), rows, cols, current_stream() if stream is None else stream))


def fp8adam_unpack8(src: Matrix8Arg, x: MatrixArg, rows: int, cols: int, stream: int | None = None) -> None:
    _check(_lib().fp8adam_unpack8(ctypes.byref(src), ctypes.byref(x), rows, cols, current_stream() if stream is None else stream))


def _call(name: str, args, stream: int | None) -> None:
    _check(getattr(_lib(), name)(ctypes.byref(args), current_stream() if stream is None else stream))


def _bytes(name: str, args) -> int:
    n = getattr(_lib(), name)(ctypes.byref(args))
    if n < 0:
        _check(n)
    return n


def fp8adam_linear8(args: Product8Arg, stream: int | None = None) -> None:
    _call("fp8adam_linear8", args, stream)


def fp8adam_gated8(args: Product8Arg, stream: int | None = None) -> None:
    _call("fp8adam_gated8", args, stream)


def fp8adam_linear8_backward(args: ActBackward8Arg, stream: int | None = None) -> None:
    _call("fp8adam_linear8_backward", args, stream)


def fp8adam_gated8_backward(args: ActBackward8Arg, stream: int | None = None) -> None:
    _call("fp8adam_gated8_backward", args, stream)


def fp8adam_weight_grad8(args: Grad8Arg, stream: int | None = None) -> None:
    _call("fp8adam_weight_grad8", args, stream)


def fp8adam_input_grad8(args: Grad8Arg, stream: int | None = None) -> None:
    _call("fp8adam_input_grad8", args, stream)


def fp8adam_linear8_backward_workspace(args: ActBackward8Arg) -> int:
    return _bytes("fp8adam_linear8_backward_workspace", args)


def fp8adam_weight_grad8_workspace(args: Grad8Arg) -> int:
    return _bytes("fp8adam_weight_grad8_workspace", args)


def fp8adam_input_grad8_workspace(args: Grad8Arg) -> int:
    return _bytes("fp8adam_input_grad8_workspace", args)


# ------------------------------------------------------------ torch wrappers

def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


class Packed8:
    """A matrix in 8 bits: FP8 codes and one power-of-two scale for every 128 columns of a row.

    codes: uint8 (of format ``fmt``) or a float8 tensor, [rows, cols rounded up to 128], with zeros
    behind ``cols``; rows may lie further apart, by a multiple of 16.  scales: [rows, blocks], either
    uint8 or float8_e8m0fnu bytes b that stand for 2^(b - 127), or float32 powers of two, as ``Quantizer``
    writes them.  Scales lie between 2^-126 and 2^127.

    Codes and scales are views: what is written to them later is what later calls read.  Only where rows of
    bytes are not whole dwords (multiples of 4 bytes, apart and in length, from an address that is one) are
    both copied, and the matrix stays as it was when it was made.

    A matrix that ``pack8`` or a product has made of a tensor of more dimensions stands for that tensor: a product
    of it has the tensor's leading dimensions.
    """
    __slots__ = ("_room", "_codes", "_scales", "rows", "cols", "format", "scale_type", "device", "_fields", "_lead")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, cols: int, fmt: str = "e4m3"):
        self.format = _FP8_FORMATS[codes.dtype] if codes.dtype in _FP8_FORMATS else _FORMATS[fmt]
        if codes.dtype in _FP8_FORMATS:
            codes = codes.view(torch.uint8)
        if scales.dtype == torch.float8_e8m0fnu:
            scales = scales.view(torch.uint8)
        _need(codes.dtype == torch.uint8 and codes.dim() == 2, "codes must be a matrix of uint8 or float8")
        _need(cols >= 1, "cols must be positive")
        self.rows, self.cols = codes.shape[0], cols
        blocks = -(-cols // BLOCK)
        _need(codes.shape[1] == BLOCK * blocks, f"codes must have {BLOCK * blocks} columns, zeros behind column {cols}")
        _need(scales.dtype in (torch.uint8, torch.float32) and scales.dim() == 2 and scales.shape[0] == self.rows and
              scales.shape[1] >= blocks, f"scales must be uint8, float8_e8m0fnu or float32, [{self.rows}, {blocks}]")
        _need(codes.device == scales.device, "codes and scales must be on one device")
        _need(codes.numel() == 0 or (codes.stride(1) == 1 and (self.rows == 1 or codes.stride(0) >= codes.shape[1])),
              "rows of codes must be contiguous and lie one after the other")
        _need(scales.numel() == 0 or scales.shape[1] == 1 or scales.stride(1) == 1, "rows of scales must be contiguous")
        self.scale_type = SCALES_F32 if scales.dtype == torch.float32 else SCALES_E8M0
        if self.scale_type == SCALES_E8M0 and (scales.shape[1] % 4 or (scales.stride(0) % 4 and self.rows > 1) or
                                                scales.data_ptr() % 4 or scales.stride(1) != 1):
            # whole dwords per row, as the kernels read them; the codes with them, or codes rewritten later would be
            # multiplied by scales of before
            padded = scales.new_full((self.rows, -(-blocks // 4) * 4), 127)
            padded[:, :blocks] = scales[:, :blocks]
            codes, scales = codes.clone(memory_format=torch.contiguous_format), padded
        self._codes, self._scales, self.device, self._lead = codes, scales, codes.device, (self.rows,)
        many = self.rows > 1
        self._fields = (codes.data_ptr(), scales.data_ptr(), codes.stride(0) if many else codes.shape[1],
                        scales.stride(0) if many else scales.shape[1], self.format, self.scale_type)

    @classmethod
    def _new(cls, rows: int, cols: int, fmt: str, device, lead) -> "Packed8":
        """Room for a matrix, codes and scales in one allocation; its rows stand for the dimensions ``lead``."""
        return cls._several(1, rows, cols, fmt, device, lead)[0]

    @classmethod
    def _several(cls, n: int, rows: int, cols: int, fmt: str, device, lead) -> list:
        """Room for n matrices in one allocation, which lives as long as one of them: an allocation takes a
        small call 3 us."""
        blocks, fmt8 = -(-cols // BLOCK), _FORMATS[fmt]
        ld, ld_scale = BLOCK * blocks, -(-blocks // 4) * 4
        size = -(-rows * (ld + ld_scale) // 256) * 256
        room = torch.empty(n * size, dtype=torch.uint8, device=device)
        first = room.data_ptr()
        made = []
        for i in range(n):
            p = cls.__new__(cls)
            p._room, p._codes = room, None
            p.rows, p.cols, p.format, p.scale_type, p.device, p._lead = rows, cols, fmt8, SCALES_E8M0, device, lead
            at = first + i * size
            p._fields = (at, at + rows * ld, ld, ld_scale, fmt8, SCALES_E8M0)
            made.append(p)
        return made

    def _views(self):
        if self._codes is None:
            at, _, ld, ld_scale = self._fields[:4]
            at -= self._room.data_ptr()
            self._codes = self._room.as_strided((self.rows, ld), (ld, 1), at)
            self._scales = self._room.as_strided((self.rows, ld_scale), (ld_scale, 1), at + self.rows * ld)
        return self._codes, self._scales

    @property
    def codes(self) -> torch.Tensor:
        return self._views()[0]

    @property
    def scales(self) -> torch.Tensor:
        return self._views()[1]

    @classmethod
    def from_quantizer(cls, q, i: int) -> "Packed8":
        """Matrix ``i`` of a ``Quantizer`` with block scales that are powers of two: a view, which
        every ``quantize()`` renews.  Its rows are whole blocks."""
        v = q.values[i]
        _need(q.granularity == "block128" and q.scale_mode == "pow2", "the Quantizer must have block128 scales in mode pow2")
        _need(v.dim() == 2 and v.is_contiguous() and v.shape[1] % BLOCK == 0 and v.numel() > 0,
              f"tensor {i} must be a contiguous matrix with a multiple of {BLOCK} columns")
        rows, cols = v.shape
        n = rows * cols // BLOCK
        return cls(q.codes[i].view(rows, cols), q.scales[i][:n].view(rows, cols // BLOCK), cols, q.formats[i])

    @property
    def fmt(self) -> str:
        return "e4m3" if self.format == E4M3 else "e5m2"

    def values(self):
        """Views of the codes as float8 [rows, cols] and of the scales, [rows, blocks] (float8_e8m0fnu or float32)."""
        c, s = self._views()
        blocks = -(-self.cols // BLOCK)
        if self.cols != c.shape[1]:
            c = c[:, :self.cols]
        if blocks != s.shape[1]:
            s = s[:, :blocks]
        return c.view(_FP8[self.format]), s if self.scale_type == SCALES_F32 else s.view(torch.float8_e8m0fnu)

    def arg(self) -> tuple:
        """The fields of the C struct."""
        return self._fields


_NO_MATRIX = (0, 0, 0, 0)
_NO_MATRIX8 = (0, 0, 0, 0, 0, 0)


def _matrix(t: torch.Tensor, what: str) -> torch.Tensor:
    """A tensor as rows of its last dimension."""
    if t.dim() == 2:
        return t
    _need(t.dim() > 2, f"{what} must have at least two dimensions")
    try:
        return t.view(-1, t.shape[-1]) if t.numel() else t.reshape(-1, t.shape[-1])
    except RuntimeError:
        raise ValueError(f"the leading dimensions of {what} do not fold into rows without a copy") from None


def _recorded(what: str) -> None:
    if torch.is_grad_enabled():
        raise ValueError(f"{what} requires a gradient, which these calls do not record: call them under torch.no_grad() or detach it")


def _arg(t: torch.Tensor, what: str, rows: int, cols: int, device) -> tuple:
    """The fields of the C struct of a matrix [rows, cols]."""
    if t.requires_grad:
        _recorded(what)
    if t.dim() != 2:
        t = _matrix(t, what)
    dtype = _DTYPES.get(t.dtype)
    _need(dtype is not None, f"{what} must be float32, bfloat16 or float16")
    if t.shape[0] != rows or t.shape[1] != cols:
        raise ValueError(f"{what} must have {rows} rows of {cols}")
    _need(t.device == device, "every tensor must be on one device")
    st, last = t.stride()
    if last != 1 and cols > 1:
        raise ValueError(f"rows of {what} must be contiguous")
    return t.data_ptr(), st if rows > 1 else cols, dtype, 0


def _vector(t: torch.Tensor, what: str, n: int, device) -> tuple:
    if t.requires_grad:
        _recorded(what)
    _need(t.dtype in _DTYPES, f"{what} must be float32, bfloat16 or float16")
    _need(t.numel() == n and t.is_contiguous(), f"{what} must be contiguous, with {n} elements")
    _need(t.device == device, "every tensor must be on one device")
    return t.data_ptr(), n, _DTYPES[t.dtype], 0


def _run(fn, args, device: torch.device) -> None:
    """fn(args, stream) on the device's current stream, with the device current."""
    if device.type != "cuda":
        raise ValueError("the tensors must be on a GPU")
    index = device.index
    if torch.cuda.current_device() == index:
        rc = fn(args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(args, torch._C._cuda_getCurrentRawStream(index))
    if rc:
        _check(rc)


def _call_on(name: str, args: bytes, device: torch.device) -> None:
    if _ready is None:
        _lib()
    _run(_calls[name], args, device)


def _room(name: str, args: bytes) -> int:
    """Bytes of workspace that a call needs."""
    if _ready is None:
        _lib()
    n = _calls[name + "_workspace"](args)
    if n < 0:
        _check(n)
    return n


def _act(name: str) -> int:
    if name not in _ACTS:
        raise ValueError(f"activation must be one of {', '.join(_ACTS)}")
    return _ACTS[name]


def _is8(p, what: str, rows: int, cols: int, device) -> Packed8:
    _need(isinstance(p, Packed8), f"{what} must be a Packed8")
    if p.rows != rows or p.cols != cols:
        raise ValueError(f"{what} must have {rows} rows of {cols}")
    _need(p.device == device, "every tensor must be on one device")
    return p


def pack8(x: torch.Tensor, fmt: str = "e4m3") -> Packed8:
    """x in 8 bits, by rows of its last dimension: the operand of a product and the checkpoint of its input."""
    m = _matrix(x, "x")
    rows, cols = m.shape
    out = Packed8._new(rows, cols, fmt, x.device, x.shape[:-1])
    a, b = MatrixArg(*_arg(m, "x", rows, cols, x.device)), Matrix8Arg(*out.arg())
    _run(lambda args, stream: _lib().fp8adam_pack8(*args, rows, cols, stream), (ctypes.byref(a), ctypes.byref(b)), x.device)
    return out


def unpack8(p: Packed8, dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """The values that a matrix in 8 bits stands for, [rows, cols] in fp32, bf16 or fp16 (``out``: written there)."""
    if out is None:
        _need(dtype in _DTYPES, "dtype must be float32, bfloat16 or float16")
        out = torch.empty((p.rows, p.cols), dtype=dtype, device=p.device)
    a, b = Matrix8Arg(*p.arg()), MatrixArg(*_arg(out, "out", p.rows, p.cols, p.device))
    _run(lambda args, stream: _lib().fp8adam_unpack8(*args, p.rows, p.cols, stream), (ctypes.byref(a), ctypes.byref(b)), p.device)
    return out


class Linear8(NamedTuple):
    """What ``linear8`` gives: the output, the input in 8 bits, the sum before the activation in 8
    bits (``keep``) and the output in 8 bits (``pack``)."""
    y: torch.Tensor | None
    x: Packed8
    z: Packed8 | None
    y8: Packed8 | None


class Gated8(NamedTuple):
    """What ``gated8`` gives: the output, the input in 8 bits, both projections in 8 bits (``keep``) and
    the output in 8 bits (``pack``)."""
    y: torch.Tensor | None
    x: Packed8
    gate: Packed8 | None
    up: Packed8 | None
    y8: Packed8 | None


def _product(x, w: Packed8, w_up, bias, act: str, residual, dtype, fmt: str, keep, pack, out, exact: bool):
    gated = w_up is not None
    _need(isinstance(w, Packed8), "the weights must be a Packed8")
    N, K, device = w.rows, w.cols, w.device
    if isinstance(x, Packed8):
        T, lead = x.rows, x._lead
        x8, x_in = _is8(x, "x", T, K, device), _NO_MATRIX
    else:
        m = x if x.dim() == 2 else _matrix(x, "x")
        T, lead = m.shape[0], x.shape[:-1]
        x_in = _arg(m, "x", T, K, device)
        x8 = Packed8._new(T, K, fmt, device, lead)
    _need(out is not None or dtype is not None or pack is not None, "nothing to write: dtype, out and pack are None")
    if out is not None:
        y = _arg(out, "out", T, N, device)
    elif dtype is not None:
        _need(dtype in _DTYPES, "dtype must be float32, bfloat16 or float16")
        out = torch.empty((*lead, N), dtype=dtype, device=device)
        y = (out.data_ptr(), N, _DTYPES[dtype], 0)
    else:
        y = _NO_MATRIX
    y8 = None if pack is None else Packed8._new(T, N, pack, device, lead)
    z = z_up = None
    if keep is not None:
        z, z_up = Packed8._several(2, T, N, keep, device, lead) if gated else (Packed8._new(T, N, keep, device, lead), None)
    args = _PRODUCT8.pack(
        T, N, K, *x_in, *x8._fields, *w._fields, *(_is8(w_up, "w_up", N, K, device)._fields if gated else _NO_MATRIX8),
        *(_NO_MATRIX if bias is None else _vector(bias, "bias", N, device)),
        *(_NO_MATRIX if residual is None else _arg(residual, "residual", T, N, device)), *y,
        *(_NO_MATRIX8 if y8 is None else y8._fields), *(_NO_MATRIX8 if z is None else z._fields),
        *(_NO_MATRIX8 if z_up is None else z_up._fields), _act(act), 1 if exact else 0)
    _call_on("gated8" if gated else "linear8", args, device)
    return out, x8, z, z_up, y8


def linear8(x, w: Packed8, *, bias=None, activation: str = "none", residual=None, dtype=torch.bfloat16, fmt: str = "e4m3",
            keep: str | None = None, pack: str | None = None, out=None, exact: bool = False) -> Linear8:
    """activation(x w^T + bias) + residual, of x and w in 8 bits.

    x: [..., cols], packed in ``fmt`` by the same call, or a ``Packed8`` of it.  w: [rows, cols].  y: [..., rows].
    activation: "none", "relu", "silu" or "gelu" (with erf).  ``keep``: the format in which the sum
    before the activation is kept for ``linear8_backward``.  y goes to ``out`` (which may be the residual
    itself) or a new tensor of ``dtype`` (None: not written); ``pack``: the format in which it is
    also written in 8 bits, for the next layer.

    More than 64 tokens without an fp32 y are summed by the FP8 matrix instruction, which cuts products far below the
    largest of eight (the C header says by how much).  ``exact``: every product is added in fp32 there too, in up to
    twice the time."""
    y, x8, z, _, y8 = _product(x, w, None, bias, activation, residual, dtype, fmt, keep, pack, out, exact)
    return Linear8(y, x8, z, y8)


def gated8(x, w_gate: Packed8, w_up: Packed8, *, activation: str = "silu", dtype=torch.bfloat16, fmt: str = "e4m3",
           keep: str | None = None, pack: str | None = None, out=None, exact: bool = False) -> Gated8:
    """activation(x w_gate^T) * (x w_up^T): both projections, the activation and the product in one kernel.

    Arguments as for ``linear8``; ``keep`` keeps both projections for ``gated8_backward``."""
    _need(isinstance(w_up, Packed8), "the weights must be a Packed8")
    y, x8, gate, up, y8 = _product(x, w_gate, w_up, None, activation, None, dtype, fmt, keep, pack, out, exact)
    return Gated8(y, x8, gate, up, y8)


def gated8_backward(dy: torch.Tensor, gate: Packed8, up: Packed8, *, activation: str = "silu", outs=None):
    """The gradients of both projections, (dgate, dup), in dy's type, from the kept projections.
    ``outs``: the two tensors to write, of which one may be dy itself."""
    T, N, device = gate.rows, gate.cols, gate.device
    dgate, dup = (torch.empty_like(dy, memory_format=torch.contiguous_format) for _ in range(2)) if outs is None else outs
    args = _ACT_BACKWARD8.pack(T, N, *_arg(dy, "dy", T, N, device), *gate._fields, *_is8(up, "up", T, N, device)._fields,
                               *_arg(dgate, "dgate", T, N, device), *_arg(dup, "dup", T, N, device), *_NO_MATRIX, 0, 0, 0, _act(activation))
    _call_on("gated8_backward", args, device)
    return dgate, dup


def linear8_backward(dy: torch.Tensor, z: Packed8 | None = None, *, activation: str = "none", bias_grad=None,
                     accumulate: bool = False, out=None) -> torch.Tensor:
    """The gradient of the sum before the activation, in dy's type, from the kept sum z; dy itself where
    activation is "none" (z is None then).  ``bias_grad``: a vector of any of the three types that takes
    its sum over the tokens (added to what stands there with ``accumulate``).  ``out`` may be dy itself."""
    device = dy.device
    m = _matrix(dy, "dy")
    T, N = m.shape
    act = _act(activation)
    none = act == ACT_NONE
    _need((z is None) == none, "z is given with an activation, and only then")
    if none:
        _need(out is None, "without an activation dz is dy: out must be None")
        if bias_grad is None:
            return dy
        out = dy
    elif out is None:
        out = torch.empty_like(dy, memory_format=torch.contiguous_format)
    fields = (T, N, *_arg(m, "dy", T, N, device), *(_NO_MATRIX8 if none else _is8(z, "z", T, N, device)._fields), *_NO_MATRIX8,
              *(_NO_MATRIX if none else _arg(out, "out", T, N, device)), *_NO_MATRIX,
              *(_NO_MATRIX if bias_grad is None else _vector(bias_grad, "bias_grad", N, device)))
    _with_room("linear8_backward", _ACT_BACKWARD8, fields, (int(accumulate), act), device, bias_grad is not None)
    return out


def _with_room(name: str, struct: Struct, before: tuple, after: tuple, device: torch.device, asks: bool = True) -> None:
    """A call with the workspace it needs, which torch hands out again in the order of the stream."""
    args = struct.pack(*before, 0, 0, *after)
    n = _room(name, args) if asks else 0
    if n:
        space = torch.empty(n, dtype=torch.uint8, device=device)
        args = struct.pack(*before, space.data_ptr(), n, *after)
    _call_on(name, args, device)


def _grad(name: str, dys, bs, out, T: int, N: int, K: int, rows: int, accumulate: bool, exact: bool) -> torch.Tensor:
    device = bs[0].device
    two = len(dys) == 2
    before = (T, N, K, len(dys), int(accumulate), *_arg(dys[0], "dy", T, N, device), *(_arg(dys[1], "dy", T, N, device) if two else _NO_MATRIX),
              *bs[0]._fields, *(bs[1]._fields if two else _NO_MATRIX8), *_arg(out, "out", rows, K, device))
    _with_room(name, _GRAD8, before, (1 if exact else 0, 0), device)
    return out


def weight_grad8(dy: torch.Tensor, x: Packed8, out: torch.Tensor | None = None, *, accumulate: bool = False,
                 dtype=torch.float32, exact: bool = True) -> torch.Tensor:
    """The gradient of a layer's weights, dy^T x [rows, cols], from the kept input: written to ``out`` (or a new
    tensor of ``dtype``), or added to what stands there with ``accumulate``.  An fp32 dy takes part in all of its bits, or
    without ``exact`` in 16 of them, in two thirds of the time."""
    _need(isinstance(x, Packed8), "x must be a Packed8")
    m = _matrix(dy, "dy")
    _need(m.shape[0] == x.rows, f"dy must have {x.rows} rows")
    N = m.shape[1]
    if out is None:
        _need(not accumulate, "accumulate needs out")
        out = torch.empty((N, x.cols), dtype=dtype, device=x.device)
    return _grad("weight_grad8", [m], [x], out, x.rows, N, x.cols, N, accumulate, exact)


def input_grad8(dy, w, out: torch.Tensor | None = None, *, accumulate: bool = False, dtype=torch.bfloat16,
                exact: bool = True) -> torch.Tensor:
    """The gradient of a layer's input, dy w [..., cols]; of two layers with one input (a gated pair) their sum, from
    two gradients and two weights.  Written to ``out`` (or a new tensor of ``dtype``), or added to what stands there.
    ``exact`` as for ``weight_grad8``."""
    dys, ws = (list(dy), list(w)) if isinstance(dy, (list, tuple)) else ([dy], [w])
    _need(len(dys) == len(ws) and len(dys) in (1, 2), "need one gradient per layer, of one or two layers")
    _need(all(isinstance(p, Packed8) for p in ws), "the weights must be a Packed8")
    N, K, device = ws[0].rows, ws[0].cols, ws[0].device
    ms = [_matrix(d, "dy") for d in dys]
    T = ms[0].shape[0]
    if len(ws) == 2:
        _is8(ws[1], "the second weights", N, K, device)
        _need(ws[0].format == ws[1].format and ws[0].scale_type == ws[1].scale_type and dys[0].dtype == dys[1].dtype,
              "both layers must have one format, one type of scales and one type of dy")
    if out is None:
        _need(not accumulate, "accumulate needs out")
        out = torch.empty((*dys[0].shape[:-1], K), dtype=dtype, device=device)
    return _grad("input_grad8", ms, ws, out, T, N, K, T, accumulate, exact)
