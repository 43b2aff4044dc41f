"""4-bit matrices with group scales and their product with 16-bit rows (include/rwkv7.h).

Calls run on the current stream of the device their tensors are on, allocate outputs and
workspaces from torch's allocator on that stream, do not synchronise, but for a device's
first Q4Matrix, which waits for a word of zeros, and may be captured into a graph, with that
matrix made a process's first product too.
"""
from __future__ import annotations

import threading

import torch

from . import EINVAL, ESTATE, ETIMEOUT, RWKV7Error, load_library
from .mx import _ACTIVATIONS, _DTYPES, _MAX_DIM, _call, _capturing, _room, _rows, _word

GROUPS = (32, 64, 128)
FEW_ROWS, FEW_VALUES = 16, 1 << 17  # RWKV7_Q4_FEW_*

_err: dict[int, torch.Tensor] = {}  # per device: the word in which products latch errors
_err_lock = threading.Lock()


def _err_word(dev: int) -> torch.Tensor:
    """Made with the device's first Q4Matrix; not in a capture, which could not wait for it
    and whose memory goes with the graph."""
    w = _err.get(dev)
    if w is None:
        if _capturing(dev):
            raise RWKV7Error(ESTATE, f"make a Q4Matrix on cuda:{dev} before the first capture of a product there")
        with _err_lock:
            w = _err.get(dev)
            if w is None:
                w = _word(f"cuda:{dev}")
                torch.cuda.current_stream(dev).synchronize()  # other streams will use it
                _err[dev] = w
    return w


def _bytes(rows: int, cols: int, group: int, zeros: bool) -> int:
    """rwkv7_q4_bytes, or a refusal."""
    if group not in GROUPS:
        raise RWKV7Error(EINVAL, f"a group of {group} columns: 32, 64 or 128")
    tiles = (rows + 15 >> 4) * (cols + 127 >> 7)
    if not (1 <= rows <= _MAX_DIM and 1 <= cols <= _MAX_DIM) or tiles >= 1 << 31:
        raise RWKV7Error(EINVAL, f"no 4-bit matrix of {rows} rows and {cols} columns")
    return tiles * (1024 + 128 // group * (48 if zeros else 32))


class Q4Matrix:
    """A matrix [rows, cols] of 4-bit codes with a scale, and with zeros a zero, for each
    group of columns, on the device in the order the product reads (rwkv7_q4_bytes)."""

    __slots__ = ("data", "rows", "cols", "group", "zeros")

    def __init__(self, data: torch.Tensor, rows: int, cols: int, group: int, zeros: bool = False):
        size = _bytes(rows, cols, group, zeros)
        if not data.is_cuda or data.dtype != torch.uint8 or not data.is_contiguous():
            raise TypeError("a 4-bit matrix is a contiguous uint8 tensor on a CUDA device")
        if data.numel() != size:
            raise ValueError(f"a 4-bit matrix of {rows} x {cols} in groups of {group} takes {size} bytes, "
                             f"got {data.numel()}")
        self.data, self.rows, self.cols, self.group, self.zeros = data, rows, cols, group, bool(zeros)
        dev = data.get_device()
        if dev not in _err and not _capturing(dev):
            _err_word(dev)

    @property
    def shape(self):
        return self.rows, self.cols

    def dequantize(self, dtype=torch.float32, out=None):
        """The values it stands for, rounded once (rwkv7_q4_dequantize)."""
        if out is None:
            if dtype not in _DTYPES:
                raise TypeError("dtype must be float32, float16 or bfloat16")
            out = torch.empty(self.shape, dtype=dtype, device=self.data.device)
        rows, cols, ld, code = _rows(out, "out")
        if (rows, cols) != self.shape or out.get_device() != self.data.get_device():
            raise ValueError("out must have the matrix's shape and device")
        _call(load_library().rwkv7_q4_dequantize, out.get_device(), self.data.data_ptr(), rows, cols, self.group,
              self.zeros, out.data_ptr(), code, ld)
        return out


def _empty(rows, cols, group, zeros, device):
    return Q4Matrix(torch.empty(_bytes(rows, cols, group, zeros), dtype=torch.uint8, device=device), rows, cols, group,
                    zeros)


def _strided(t, dtype, rows, cols, device, what):
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.device != device:
        raise TypeError(f"{what} must be a {dtype} tensor on {device}")
    if t.shape != (rows, cols):
        raise ValueError(f"{what} must be [{rows}, {cols}], got {tuple(t.shape)}")
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"the rows of {what} must be contiguous (stride 1 along the last dimension)")
    return t.stride(0) if rows > 1 else cols


def q4_pack(values, scales, zeros=None, group: int = 128) -> Q4Matrix:
    """Lay out a matrix from a checkpoint's parts (rwkv7_q4_pack): values [rows, cols] uint8,
    a code 0 .. 15 each; scales float16 and zeros uint8 0 .. 15 (None: all 8) [rows, ceil(cols /
    group)].  Of values and zeros the low four bits count, so that a zero of 16 (of a
    checkpoint that keeps zero - 1) would be 0: such a matrix does not fit.  Row strides are
    free.  The matrix stands for scale * (value - zero)."""
    if not isinstance(values, torch.Tensor) or values.dtype is not torch.uint8 or not values.is_cuda or values.dim() != 2:
        raise TypeError("values must be a two-dimensional uint8 CUDA tensor")
    rows, cols = values.shape
    _bytes(rows, cols, group, zeros is not None)
    ng, dev = -(-cols // group), values.device
    ldv = _strided(values, torch.uint8, rows, cols, dev, "values")
    lds = _strided(scales, torch.float16, rows, ng, dev, "scales")
    ldz = 0 if zeros is None else _strided(zeros, torch.uint8, rows, ng, dev, "zeros")
    out = _empty(rows, cols, group, zeros is not None, dev)
    _call(load_library().rwkv7_q4_pack, dev.index, values.data_ptr(), ldv, scales.data_ptr(), lds,
          None if zeros is None else zeros.data_ptr(), ldz, rows, cols, group, out.data.data_ptr())
    return out


def q4_quantize(x, group: int = 128, zeros: bool = False) -> Q4Matrix:
    """Rows of x [rows, cols] (float32, float16, bfloat16, any row stride) to 4 bits
    (rwkv7_q4_quantize): by the largest value of each group, or with zeros by its range."""
    rows, cols, ld, code = _rows(x, "x")
    out = _empty(rows, cols, group, zeros, x.device)
    _call(load_library().rwkv7_q4_quantize, x.get_device(), x.data_ptr(), code, rows, cols, ld, group, bool(zeros),
          out.data.data_ptr())
    return out


def q4_linear(x, w: Q4Matrix, out=None, out_dtype=None, activation=None):
    """act(x w^T): x [B, K] float16 or bfloat16 at any row stride, w a Q4Matrix [N, K]; fp32
    sums of exact products, the result [B, N] rounded once to out's type, or out_dtype
    (default: x's).  out may overlap neither x nor w.  activation: None or "relu2"
    (max(y, 0)^2).  rwkv7_q4_linear."""
    if not isinstance(w, Q4Matrix):
        raise TypeError("w must be a Q4Matrix")
    act = _ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"unknown activation {activation!r}")
    B, K, ldx, code = _rows(x, "x")
    if not code:
        raise TypeError("x must be float16 or bfloat16")
    dev = w.data.get_device()
    if K != w.cols:
        raise ValueError(f"x has {K} columns, w {w.cols}")
    if x.get_device() != dev:
        raise ValueError(f"x is on cuda:{x.get_device()}, w on cuda:{dev}")
    N = ldy = w.rows
    if out is None:
        out_code = _DTYPES.get(out_dtype or x.dtype)
        if out_code is None:
            raise TypeError("out_dtype must be float32, float16 or bfloat16")
        out = torch.empty((B, N), dtype=out_dtype or x.dtype, device=x.device)
    else:
        if out_dtype is not None and out.dtype != out_dtype:
            raise TypeError(f"out is {out.dtype}, out_dtype {out_dtype}")
        rows, cols, ldy, out_code = _rows(out, "out")
        if rows != B or cols != N or out.get_device() != dev:
            raise ValueError(f"out must be [{B}, {N}] on cuda:{dev}")
    room = None
    if (B > FEW_ROWS or B * K > FEW_VALUES) and (B > 1 and ldx % 8 or x.data_ptr() % 16):  # off the grid: copied first
        room = _room(B * (K + 7 & ~7) * 2, dev)
    _call(load_library().rwkv7_q4_linear, dev, x.data_ptr(), code, ldx, B, w.data.data_ptr(), N, K, w.group, w.zeros,
          out.data_ptr(), out_code, ldy, act, None if room is None else room.data_ptr(), _err_word(dev).data_ptr())
    return out


def q4_check(device=None):
    """Wait for the device's current stream and raise if a product's bounded wait gave up
    since the last check (its output is then undefined)."""
    index = None if device is None else torch.device(device).index
    w = _err_word(torch.cuda.current_device() if index is None else index)
    flags = int(w.item())
    if flags:
        w.zero_()
        raise RWKV7Error(ETIMEOUT, f"a bounded wait inside a 4-bit product gave up (flags 0x{flags:x})")
