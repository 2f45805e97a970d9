"""ctypes binding of the products with 4-bit weights (the C ABI declared in include/pi_linear.h).

Argument marshalling only, as in binding.py and kvcache.py: every tensor is checked on the host before its
address is passed, a failed check raises PiError(PI_ERR_INVALID) and nothing is enqueued.  Calls only enqueue
work on the current stream (or the given one).
"""

from __future__ import annotations

import ctypes

import torch

from .binding import LIB, _invalid, check

PI_LINEAR_F16, PI_LINEAR_BF16 = range(2)
LINEAR_ABI_VERSION = 2   # PI_LINEAR_ABI_VERSION of the header this binding follows
LINEAR_ACTS = {"f16": PI_LINEAR_F16, "bf16": PI_LINEAR_BF16}
_ACT_TORCH = {PI_LINEAR_F16: torch.float16, PI_LINEAR_BF16: torch.bfloat16}

LINEAR_EXPORTED = ("pi_linear_abi_version", "pi_linear_packed_bytes", "pi_linear_create", "pi_linear_destroy",
                   "pi_linear_scratch_bytes", "pi_linear_scratch_bytes_upto", "pi_linear_forward")

_vp, _i32, _i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class LinearDesc(ctypes.Structure):
    _fields_ = [(name, _i32) for name in ("d_in", "d_out", "act_dtype")]


class LinearArgs(ctypes.Structure):
    _fields_ = [("x", _vp), ("add", _vp), ("y", _vp), ("x_stride", _i64), ("add_stride", _i64), ("y_stride", _i64),
                ("scratch", _vp), ("scratch_bytes", ctypes.c_size_t), ("rows", _i32)]


def _declare() -> None:
    p = ctypes.POINTER
    sigs = dict(pi_linear_packed_bytes=[p(LinearDesc), p(ctypes.c_size_t)],
                pi_linear_create=[p(LinearDesc), _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp, p(_vp)],
                pi_linear_destroy=[_vp],
                pi_linear_scratch_bytes=[_vp, _i32, p(ctypes.c_size_t)],
                pi_linear_scratch_bytes_upto=[_vp, _i32, p(ctypes.c_size_t)],
                pi_linear_forward=[_vp, p(LinearArgs), _vp])
    for name, args in sigs.items():
        fn = getattr(LIB, name)
        fn.restype, fn.argtypes = ctypes.c_int, args
    LIB.pi_linear_abi_version.restype, LIB.pi_linear_abi_version.argtypes = _i32, []
    got = LIB.pi_linear_abi_version()
    if got != LINEAR_ABI_VERSION:
        raise ImportError(f"the library's 4-bit products have ABI version {got}, this binding expects {LINEAR_ABI_VERSION}; "
                          "rebuild it")


_declare()
_byref = ctypes.byref


def linear_desc(d_in, d_out, act_dtype="f16") -> LinearDesc:
    act = LINEAR_ACTS[act_dtype] if isinstance(act_dtype, str) else int(act_dtype)
    sizes = dict(d_in=int(d_in), d_out=int(d_out), act_dtype=act)
    for name, value in sizes.items():
        if not -0x80000000 <= value <= 0x7fffffff:
            raise _invalid(f"{name}={value} does not fit in 32 bits")
    return LinearDesc(*sizes.values())


def linear_packed_bytes(desc: LinearDesc) -> int:
    out = ctypes.c_size_t(0)
    check(LIB.pi_linear_packed_bytes(_byref(desc), _byref(out)))
    return int(out.value)


class Linear:
    """y = x W^T + bias + add with W [d_out][d_in] in 4 bits: the projections of an attention layer.

        w        uint8 [d_out][d_in / 2]     q4g32 (pi_ffn.h): byte j holds elements 2j and 2j + 1, two's complement
        scales   fp16 [d_out][d_in / 32]     one for 32 consecutive elements of a row
        bias     fp32 [d_out], or None

    The weights are laid out once, here (`packed`, made unless given); w and scales may then be let go of.  Calls may
    run at the same time on several streams.

    Up to 64 rows sums are rounded in fp32 alone.  More rows take code times scale rounded to fp16, so that y is off by up to
    2^-11 of sum |w x| before its own rounding: call with 64 rows at a time where that is too much.  (pi_linear.h has the
    bounds, and what becomes of infinities.)
    """

    def __init__(self, w, scales, act_dtype="f16", bias=None, packed=None, stream=None):
        self.handle = None
        for t, name in ((w, "w"), (scales, "scales")):
            if not isinstance(t, torch.Tensor):
                raise _invalid(f"{name} must be a torch tensor, not {type(t).__name__}")
        if w.dim() != 2:
            raise _invalid(f"w must be [d_out][d_in / 2], got {list(w.shape)}")
        self.device = w.device
        self.desc = d = linear_desc(2 * w.shape[1], w.shape[0], act_dtype)
        need = linear_packed_bytes(d)
        self._act = _ACT_TORCH[d.act_dtype]
        self._dense(w, "w", torch.uint8, (d.d_out, d.d_in // 2))
        self._dense(scales, "scales", torch.float16, (d.d_out, d.d_in // 32))
        if bias is not None:
            self._dense(bias, "bias", torch.float32, (d.d_out,))
        if packed is None:
            packed = torch.empty(need, dtype=torch.uint8, device=self.device)
        if not isinstance(packed, torch.Tensor) or packed.device != self.device or not packed.is_contiguous():
            raise _invalid(f"packed must be a contiguous tensor on {self.device}")
        if self.device.type != "cuda":
            raise _invalid(f"the weights must be on a CUDA device, not {self.device}")
        self.packed, self.bias = packed, bias
        self._met, self._lone = set(), torch.cuda.device_count() == 1
        if stream is not None:   # the weights were made on the current one
            stream.wait_stream(torch.cuda.current_stream(self.device.index))
        handle = _vp()
        self._run(LIB.pi_linear_create, _byref(d), w.data_ptr(), scales.data_ptr(), None if bias is None else bias.data_ptr(),
                  packed.data_ptr(), packed.numel() * packed.element_size(), self._stream(stream, (w, scales)), _byref(handle))
        self.handle = handle

    def close(self) -> None:
        if getattr(self, "handle", None) is not None and self.handle.value:
            check(LIB.pi_linear_destroy(self.handle))
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _dense(self, t, name, dtype, shape) -> None:
        if not isinstance(t, torch.Tensor):
            raise _invalid(f"{name} must be a torch tensor, not {type(t).__name__}")
        if t.device != self.device:
            raise _invalid(f"{name} is on {t.device}, the weights are on {self.device}")
        if t.dtype is not dtype:
            raise _invalid(f"{name} is {t.dtype}, expected {dtype}")
        if t.shape != shape:
            raise _invalid(f"{name} must be {list(shape)}, got {list(t.shape)}")
        if not t.is_contiguous():
            raise _invalid(f"{name} is not contiguous")

    def _rows(self, t, name, width, rows=None) -> int:
        """A tensor [rows][width] of the activations' type, innermost contiguous; returns the rows' stride."""
        if not isinstance(t, torch.Tensor):
            raise _invalid(f"{name} must be a torch tensor, not {type(t).__name__}")
        if t.device != self.device:
            raise _invalid(f"{name} is on {t.device}, the weights are on {self.device}")
        if t.dtype is not self._act:
            raise _invalid(f"{name} is {t.dtype}, expected {self._act}")
        if t.dim() != 2 or t.shape[1] != width or (rows is not None and t.shape[0] != rows):
            raise _invalid(f"{name} must be [{'rows' if rows is None else rows}][{width}], got {list(t.shape)}")
        row, inner = t.stride()
        if inner != 1 and width > 1:
            raise _invalid(f"{name}: the innermost dimension is not contiguous")
        return row

    def _stream(self, stream, tensors) -> int:
        """The stream's handle; memory that is let go of stays reserved until the stream is past the call, as in
        KVCache._stream."""
        if stream is None:
            stream = torch.cuda.current_stream(self.device.index)
        else:
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
        handle = stream.cuda_stream
        if handle not in self._met:
            self._met.add(handle)
            for t in (self.packed, self.bias):
                if t is not None:
                    t.record_stream(stream)
        return handle or None

    def _run(self, fn, *args) -> None:
        """Call the library on the weights' device: kernels start on the current one."""
        if self._lone or torch.cuda.current_device() == self.device.index:
            check(fn(*args))
        else:
            with torch.cuda.device(self.device.index):
                check(fn(*args))

    def scratch_bytes(self, rows, upto=False) -> int:
        """Bytes of scratch that forward takes for `rows` rows.  More rows may take less (their columns are split into fewer
        ranges): with `upto`, the most that any number of rows up to `rows` takes, for a scratch that serves them all."""
        if rows >> 31:
            raise _invalid(f"rows={rows} does not fit in 32 bits")
        out = ctypes.c_size_t(0)
        size = LIB.pi_linear_scratch_bytes_upto if upto else LIB.pi_linear_scratch_bytes
        check(size(self._live(), rows, _byref(out)))
        return int(out.value)

    def _live(self):
        if self.handle is None:
            raise _invalid("the weights are closed")
        return self.handle

    def forward(self, x, y, add=None, scratch=None, stream=None) -> None:
        """y [rows][d_out] = x [rows][d_in] W^T + bias + add [rows][d_out].  Rows may be strided (x's by a multiple of
        8 elements), the innermost dimension is contiguous.  y may be add itself, and else overlaps neither x nor add.
        scratch: scratch_bytes(rows) bytes (0 up to 64 rows), made here unless given; with less, down to what one range of
        columns takes, a call that would split its columns is slower."""
        d, handle = self.desc, self._live()
        xs = self._rows(x, "x", d.d_in)
        rows = x.shape[0]
        ys = self._rows(y, "y", d.d_out, rows)
        if rows > 1 and ys < d.d_out:
            raise _invalid("y: its rows overlap")
        adds = 0 if add is None else self._rows(add, "add", d.d_out, rows)
        if rows >> 31:
            raise _invalid(f"rows={rows} does not fit in 32 bits")
        need = self.scratch_bytes(rows) if scratch is None and rows > 64 else 0
        if need:
            if stream is None:
                scratch = torch.empty(need, dtype=torch.uint8, device=self.device)
            else:   # of the stream that uses it
                with torch.cuda.stream(stream):
                    scratch = torch.empty(need, dtype=torch.uint8, device=self.device)
        size = 0
        if scratch is not None:
            if not isinstance(scratch, torch.Tensor) or scratch.device != self.device or not scratch.is_contiguous():
                raise _invalid(f"scratch must be a contiguous tensor on {self.device}")
            size = scratch.numel() * scratch.element_size()
        args = LinearArgs(x.data_ptr(), None if add is None else add.data_ptr(), y.data_ptr(), xs, adds, ys,
                          None if scratch is None else scratch.data_ptr(), size, rows)
        self._run(LIB.pi_linear_forward, handle, _byref(args), self._stream(stream, (x, y, add, scratch)))
