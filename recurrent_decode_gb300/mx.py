"""Microscaled formats of librwkv7 (include/rwkv7.h): MXFP4 matrices and their
product, and a cache of slot states in MXINT8 or MXFP4.

Argument marshalling only.  Calls run on the current stream of the device their
tensors are on, allocate outputs and workspaces from torch's allocator on that
stream, and do not synchronise, but for a device's first MX4Matrix and for making a
StateCache, which wait for a word or bytes of zeros.  With that matrix made, calls may
be captured into a graph, a process's first product too.
"""
from __future__ import annotations

import ctypes as C
import threading

import torch

from . import EINVAL, ESTATE, ETIMEOUT, RWKV7Error, load_library

_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_FORMATS = {"mxfp4": 0, "mxint8": 1}
_ACTIVATIONS = {None: 0, "none": 0, "relu2": 1}
_MAX_DIM = 1 << 24  # RWKV7_MX_MAX_DIM

# The handle of a device's current stream and the current device, without the
# objects that torch.cuda.current_stream builds (2 us a call; a small product takes 5).
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_stream_data = torch._C._cuda_getCurrentStream  # (id, ...)
_is_capturing = torch._C._cuda_isCurrentStreamCapturing  # of the current device

_ROOM = 2 << 20  # 128 rows of 30,000 columns
_kept = threading.local()  # (device, stream) -> bytes of _room
_err: dict[int, torch.Tensor] = {}  # per device: the word in which kernels latch errors
_err_lock = threading.Lock()


def _capturing(dev: int) -> bool:
    """Whether the current stream of device `dev` is being captured."""
    if dev == _current_device():
        return _is_capturing()
    with torch.cuda.device(dev):
        return _is_capturing()


def _word(device) -> torch.Tensor:
    """A word of zeros that a check may reset, in inference mode or out of it."""
    with torch.inference_mode(False):
        return torch.zeros(1, dtype=torch.int32, device=device)


def _err_word(dev: int) -> torch.Tensor:
    """Made with the device's first MX4Matrix, or by its first product or check.  Not in a
    capture, which could not wait for it and whose memory goes with the graph."""
    w = _err.get(dev)
    if w is None:
        if _capturing(dev):
            raise RWKV7Error(ESTATE, f"make an MX4Matrix on cuda:{dev} before the first capture of a product there")
        with _err_lock:  # of threads that come at once, the first makes it
            w = _err.get(dev)
            if w is None:
                w = _word(f"cuda:{dev}")
                torch.cuda.current_stream(dev).synchronize()  # other streams will use it
                _err[dev] = w
    return w


def _call(fn, dev: int, *args):
    """The library's fn(*args, stream, &message) on the current stream of device `dev`,
    with it current."""
    msg = C.c_char_p()
    if dev == _current_device():
        rc = fn(*args, _raw_stream(dev), C.byref(msg))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(dev), C.byref(msg))
    if rc:
        raise RWKV7Error(rc, (msg.value or b"").decode())


def _room(n: int, dev: int) -> torch.Tensor:
    """n bytes for x quantised on the way.  Up to _ROOM of them are kept for the next
    call of the same host thread on the same stream, whose kernels run after this
    call's (an allocation between two launches costs 3 us, a small product takes 6):
    2 MB for each of torch's streams that a thread makes products on, until it ends.
    Torch's own streams live as long as the process, so their handles stay theirs: the
    default one, id 0, and those of its pool, whose ids are odd.  One that was made
    elsewhere, whose id is its handle, may be destroyed with a product in flight and the
    handle go to another, so it gets bytes of the call's own; and so does a graph."""
    if n > _ROOM or (_is_capturing() if dev == _current_device() else _capturing(dev)):
        return torch.empty(n, dtype=torch.uint8, device=f"cuda:{dev}")
    key = dev, _raw_stream(dev)
    rooms = _kept.__dict__
    w = rooms.get(key)
    if w is None:
        stream = _stream_data(dev)[0]
        if stream and not stream & 1:
            return torch.empty(n, dtype=torch.uint8, device=f"cuda:{dev}")
        w = rooms[key] = torch.empty(_ROOM, dtype=torch.uint8, device=f"cuda:{dev}")
    return w


def _rows(x, what: str):
    """(rows, cols, row stride, type code) of a 2-D CUDA tensor whose rows are contiguous."""
    dtype = _DTYPES.get(x.dtype) if isinstance(x, torch.Tensor) else None
    if dtype is None or not x.is_cuda:
        raise TypeError(f"{what} must be a CUDA tensor of float32, float16 or bfloat16")
    if x.dim() != 2:
        raise ValueError(f"{what} must be two-dimensional, got {x.dim()} dimensions")
    rows, cols = x.shape
    ld, step = x.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"the rows of {what} must be contiguous (stride 1 along the last dimension)")
    if rows <= 1:
        ld = cols
    elif ld < cols:
        raise ValueError(f"the rows of {what} overlap (row stride {ld} < {cols})")
    return rows, cols, ld, dtype


def _bytes(rows: int, cols: int) -> int:
    """rwkv7_mx4_bytes, or a refusal."""
    if not (0 <= rows <= _MAX_DIM and 1 <= cols <= _MAX_DIM):
        raise RWKV7Error(EINVAL, f"no MXFP4 matrix of {rows} rows and {cols} columns")
    return (rows + 127 >> 7) * (cols + 255 >> 8) * 17408


def _matrix_made(dev: int):
    """The error word for the products to come, so that the first may be captured."""
    if dev not in _err and not _capturing(dev):
        _err_word(dev)


class MX4Matrix:
    """An MXFP4 matrix [rows, cols] on the device, in the tile order the product
    reads (rwkv7_mx4_bytes)."""

    __slots__ = ("data", "rows", "cols")

    def __init__(self, data: torch.Tensor, rows: int, cols: int):
        if not data.is_cuda or data.dtype != torch.uint8 or not data.is_contiguous():
            raise TypeError("an MXFP4 matrix is a contiguous uint8 tensor on a CUDA device")
        if data.numel() != _bytes(rows, cols):
            raise ValueError(f"an MXFP4 matrix of {rows} x {cols} takes {_bytes(rows, cols)} bytes, got {data.numel()}")
        self.data, self.rows, self.cols = data, rows, cols
        _matrix_made(data.get_device())

    @property
    def shape(self):
        return self.rows, self.cols

    def dequantize(self, dtype=torch.float32, out=None):
        """The values it stands for (rwkv7_mx4_dequantize)."""
        if out is None:
            rows, cols, ld, code = self.rows, self.cols, self.cols, _DTYPES.get(dtype)
            if code is None:
                raise TypeError("dtype must be float32, float16 or bfloat16")
            out = torch.empty((rows, cols), dtype=dtype, device=self.data.device)
        else:
            rows, cols, ld, code = _rows(out, "out")
            if rows != self.rows or cols != self.cols or out.get_device() != self.data.get_device():
                raise ValueError("out must have the matrix's shape and device")
        _call(load_library().rwkv7_mx4_dequantize, out.get_device(), self.data.data_ptr(), rows, cols, out.data_ptr(),
              code, ld)
        return out


def mx4_empty(rows: int, cols: int, device) -> MX4Matrix:
    """An MXFP4 matrix whose values are not set yet."""
    m = MX4Matrix.__new__(MX4Matrix)  # (its checks hold by construction, but for the device)
    m.data, m.rows, m.cols = torch.empty(_bytes(rows, cols), dtype=torch.uint8, device=device), rows, cols
    if not m.data.is_cuda:
        raise TypeError("an MXFP4 matrix lies on a CUDA device")
    _matrix_made(m.data.get_device())
    return m


def mx4_quantize(x, out: MX4Matrix | None = None) -> MX4Matrix:
    """Rows of x [rows, cols] to MXFP4 (rwkv7_mx4_quantize).  x may be a view with
    any row stride."""
    rows, cols, ld, code = _rows(x, "x")
    if out is None:
        out = mx4_empty(rows, cols, x.device)
    elif out.shape != (rows, cols) or out.data.device != x.device:
        raise ValueError("out must have x's shape and device")
    _call(load_library().rwkv7_mx4_quantize, x.get_device(), x.data_ptr(), code, rows, cols, ld, out.data.data_ptr())
    return out


def mx4_linear(x, w: MX4Matrix, out=None, out_dtype=None, activation=None):
    """act(q(x) w^T): x [B, K] (float32, float16, bfloat16, any row stride; quantised
    on the way) or an MX4Matrix [B, K], w an MX4Matrix [N, K]; fp32 sums, the
    result [B, N] rounded once to out's type, or out_dtype (default: x's, float32
    for an MX4Matrix).  out may be x or overlap it, but not a matrix.  activation: None
    or "relu2" (max(y, 0)^2).  rwkv7_mx4_linear."""
    if not isinstance(w, MX4Matrix):
        raise TypeError("w must be an MX4Matrix")
    act = _ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"unknown activation {activation!r}")
    dev = w.data.get_device()
    if isinstance(x, MX4Matrix):
        xq, src, code, ldx = x, None, 0, 0
        B, K, x_dev, default = x.rows, x.cols, x.data.get_device(), torch.float32
    else:
        B, K, ldx, code = _rows(x, "x")
        src, x_dev, default = x.data_ptr(), x.get_device(), x.dtype
    if K != w.cols:
        raise ValueError(f"x has {K} columns, w {w.cols}")
    if x_dev != dev:
        raise ValueError(f"x is on cuda:{x_dev}, w on cuda:{dev}")
    device = w.data.device
    data = xq.data if src is None else _room(_bytes(B, K), dev)
    N = ldy = w.rows
    if out is None:
        out_code = _DTYPES.get(out_dtype or default)
        if out_code is None:
            raise TypeError("out_dtype must be float32, float16 or bfloat16")
        out = torch.empty((B, N), dtype=out_dtype or default, device=device)
    else:
        if out_dtype is not None and out.dtype != out_dtype:
            raise TypeError(f"out is {out.dtype}, out_dtype {out_dtype}")
        rows, cols, ldy, out_code = _rows(out, "out")
        if rows != B or cols != N or out.get_device() != dev:
            raise ValueError(f"out must be [{B}, {N}] on cuda:{dev}")
    _call(load_library().rwkv7_mx4_linear, dev, src, code, ldx, data.data_ptr(), B, w.data.data_ptr(), N, K,
          out.data_ptr(), out_code, ldy, act, _err_word(dev).data_ptr())
    return out


def mx4_check(device=None):
    """Wait for the device's current stream and raise if a product's bounded wait
    gave up since the last check (its output is then undefined)."""
    index = None if device is None else torch.device(device).index
    w = _err_word(torch.cuda.current_device() if index is None else index)
    flags = int(w.item())
    if flags:
        w.zero_()
        raise RWKV7Error(ETIMEOUT, f"a bounded wait inside an MXFP4 product gave up (flags 0x{flags:x})")


def _follow(stream, *tensors):
    """For a kernel that `stream` runs on tensors of the current stream: it comes after
    what that has in flight, and their memory is not handed out again before it ends."""
    dev = stream.device.index
    if _raw_stream(dev) != stream.cuda_stream:
        stream.wait_stream(torch.cuda.current_stream(dev))
        for t in tensors:
            t.record_stream(stream)


def _pair_count(slots, entries, dev: torch.device):
    for what, t in (("slots", slots), ("entries", entries)):
        if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or not t.is_contiguous() \
                or t.get_device() != dev.index:
            raise TypeError(f"{what} must be a contiguous int32 tensor on {dev}")
    n = slots.numel()
    if n != entries.numel():
        raise ValueError("slots and entries differ in length")
    return n


class StateCache:
    """Slot states kept in a quarter (MXINT8) or an eighth (MXFP4) of their size:
    n_entries entries for states of n_layer x n_head heads.  Rwkv7.slots_save and
    slots_load move a ctx's slots; save and load a pool the caller owns.

    MXINT8 keeps every value to within 1/127 of the largest of its block of 32 along
    a state row, MXFP4 to within 1/5, where that is a normal number (and in MXFP4 below
    7/8 of fp32's range); token-shift states are kept exactly.  An entry that nothing
    was saved to holds the state of a slot after a reset."""

    def __init__(self, n_layer: int, n_head: int, n_entries: int, format: str = "mxint8", device=None):
        if format not in _FORMATS:
            raise ValueError(f"unknown format {format!r}: mxint8 or mxfp4")
        self.n_layer, self.n_head, self.n_entries = int(n_layer), int(n_head), int(n_entries)
        self.format = _FORMATS[format]
        self.entry_bytes = load_library().rwkv7_state_entry_bytes(self.n_layer, self.n_head, self.format)
        if self.entry_bytes == 0 or self.n_entries < 1:
            raise RWKV7Error(EINVAL, "layers, heads and entries must be >= 1")
        self.data = torch.zeros(self.n_entries * self.entry_bytes, dtype=torch.uint8,
                                device="cuda" if device is None else device)
        if not self.data.is_cuda:
            raise TypeError("a state cache lies on a CUDA device")
        self.err = _word(self.data.device)
        torch.cuda.current_stream(self.data.device).synchronize()  # a ctx may use it on a stream of its own

    def _states(self, fn, states, slots, entries):
        wkv, att, ffn = states
        dev, index, L, H = self.data.device, self.data.get_device(), self.n_layer, self.n_head
        for what, t in (("wkv", wkv), ("shift_att", att), ("shift_ffn", ffn)):
            if not isinstance(t, torch.Tensor) or t.dtype is not torch.float32 or not t.is_contiguous() \
                    or t.get_device() != index:
                raise TypeError(f"{what} must be a contiguous float32 tensor on {dev}")
        shape = wkv.shape
        n_slots = shape[1] if len(shape) == 5 else -1
        shift = (L, n_slots, 64 * H)
        if shape != (L, n_slots, H, 64, 64) or att.shape != shift or ffn.shape != shift:
            raise ValueError(f"states must be wkv [{L}, slots, {H}, 64, 64] and two token shifts "
                             f"[{L}, slots, {64 * H}]")
        n = _pair_count(slots, entries, dev)
        _call(fn, index, wkv.data_ptr(), att.data_ptr(), ffn.data_ptr(), L, H, n_slots, slots.data_ptr(),
              entries.data_ptr(), n, self.data.data_ptr(), self.n_entries, self.format, self.err.data_ptr())

    def save(self, states, slots, entries):
        """Keep the states of `slots` in `entries` (rwkv7_states_save).  states:
        (wkv [L, n_slots, H, 64, 64], shift_att, shift_ffn [L, n_slots, 64 H])."""
        self._states(load_library().rwkv7_states_save, states, slots, entries)

    def load(self, states, entries, slots):
        """Put the kept states of `entries` into `slots` (rwkv7_states_load)."""
        self._states(load_library().rwkv7_states_load, states, slots, entries)

    def check(self):
        """Wait for the stream and raise if a save or load had a bad or repeated index."""
        flags = int(self.err.item())
        if flags:
            self.err.zero_()
            raise RWKV7Error(EINVAL, "slot or entry out of range, or written twice in one call (flags 0x%x)" % flags)
