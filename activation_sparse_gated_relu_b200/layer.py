"""The operators around the sparse FFN over torch tensors: RMS norm, the 8-bit
linear layer and the experts' grouped products (include/sffn.h).

Argument marshalling only, as in binding.py.  Calls run on the device of their
tensors, on that device's current stream or on `stream`; outputs and scratch
that a call makes itself belong to the stream it runs on.  A tensor made on one
stream and used on another is the caller's to order, as with any torch call.
"""
from __future__ import annotations

import ctypes
from contextlib import contextmanager
from typing import Optional

import torch

from .binding import (SFFN_BF16, SFFN_E4M3, SFFN_FP32, SFFN_OK, SffnError, load_library, sffn_grouped_desc,
                      sffn_qlinear_desc, sffn_rmsnorm_desc)

GROUP = 128     # columns that share a scale, and the side of a weight block that shares one
_BF16, _FP32, _FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
_CODE = {_BF16: SFFN_BF16, _FP32: SFFN_FP32, _FP8: SFFN_E4M3}
_OUT = {"bf16": _BF16, "fp32": _FP32}
_VALUES = (_BF16, _FP32)
_raw_stream = torch._C._cuda_getCurrentRawStream


def _groups(d: int) -> int:
    return (d + GROUP - 1) // GROUP


def _bad(t, name: str, dtypes, shape, device) -> None:
    """Raise what is wrong with t (called only when something is)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.layout != torch.strided:
        raise TypeError(f"{name} must be a dense tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, got cuda:{t.get_device()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major)")
    raise ValueError(f"{name} must start on a 16-byte boundary")


def _check(t, name: str, dtypes, shape, device: Optional[int]) -> int:
    """The C ABI sees only a pointer: t's type, shape, device and layout are
    checked here.  Returns the pointer."""
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.layout == torch.strided and t.shape == shape
            and t.is_cuda and (device is None or t.get_device() == device) and t.is_contiguous()):
        p = t.data_ptr()
        if not p & 15:
            return p
    _bad(t, name, dtypes, shape, device)


def _matrix(t, name: str) -> tuple:
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a [rows][columns] tensor")
    return t.shape


def _bytes(t) -> tuple:
    p = t.data_ptr()
    return p, p + t.numel() * t.element_size()


def _apart(out, name: str, *inputs) -> None:
    """An output that several rows' sums are read for must not overlap an input."""
    a, b = _bytes(out)
    for t in inputs:
        c, d = _bytes(t)
        if a < d and c < b:
            raise ValueError(f"{name} must not overlap an input")


def _apart_or_in_place(out, name: str, *inputs) -> None:
    """An output that may replace an input element by element, but not overlap
    one in any other way."""
    for t in inputs:
        if t is not None and not (out.data_ptr() == t.data_ptr() and out.dtype == t.dtype):
            _apart(out, name, t)


def _moved(name: str) -> None:
    raise ValueError(f"{name}'s storage was replaced after the operator was made: make it anew")


def _out_type(out: str):
    if out not in _OUT:
        raise ValueError(f"out must be one of {sorted(_OUT)}, got {out!r}")
    return _OUT[out]


def _ok(status: int, what: str) -> None:
    if status != SFFN_OK:
        raise SffnError(status, what)


@contextmanager
def _both(device: int, stream: Optional[int]):
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device)):
                yield


class _Plain:
    """The calling thread's device and stream are those of the call."""

    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_PLAIN = _Plain()


def _where(device: int, stream: Optional[int]):
    """Context in which a call on `device` and `stream` allocates and launches."""
    if stream is None and torch._C._cuda_getDevice() == device:
        return _PLAIN
    if stream == 0:
        # the legacy default stream, which is also torch's default stream of a device
        return _default(device)
    return _both(device, stream)


@contextmanager
def _default(device: int):
    with torch.cuda.device(device), torch.cuda.stream(torch.cuda.default_stream(device)):
        yield


class RmsNorm:
    """s = residual + x, y = s / sqrt(mean(s^2) + eps) * weight over rows of d
    columns (d % 8 == 0, d <= 16384).  weight [d] is bf16 or fp32 and is read
    at every call."""

    def __init__(self, weight, eps: float = 1e-6):
        if not isinstance(weight, torch.Tensor) or weight.dim() != 1:
            raise ValueError("weight must be a [d] tensor")
        self.d = weight.shape[0]
        ptr = _check(weight, "weight", (_BF16, _FP32), (self.d,), None)
        self.weight, self.eps, self.device = weight, float(eps), weight.get_device()
        self._lib = load_library()
        self._call, self._call_backward = self._lib.sffn_rmsnorm_forward, self._lib.sffn_rmsnorm_backward
        self._desc, self._work, self._place = {}, {}, weight.device
        # refuse a size or an eps here rather than at the first call
        n = ctypes.c_size_t()
        _ok(self._lib.sffn_rmsnorm_workspace_bytes(self.d, 1, ctypes.byref(n)), "RmsNorm")
        if not 0.0 <= self.eps < float("inf"):
            raise ValueError("eps must be finite and not negative")
        self._ptr = ptr

    def _descriptor(self, x, residual, y):
        if self.weight.data_ptr() != self._ptr:
            _moved("weight")
        key = (x, residual, y)
        d = self._desc.get(key)
        if d is None:
            s = sffn_rmsnorm_desc(d=self.d, eps=self.eps, weight=self._ptr, weight_dtype=_CODE[self.weight.dtype],
                                  x_dtype=_CODE[x], residual_dtype=_CODE[residual], y_dtype=_CODE[y])
            d = self._desc[key] = (ctypes.byref(s), s)
        return d[0]

    def _forward(self, x, residual, dtype, y, scale, residual_out, stream):
        T, d = _matrix(x, "x")
        dev = self.device
        shape = (T, self.d)
        xp = _check(x, "x", _VALUES, shape, dev)
        rp = sp = cp = None
        rt = _BF16
        if residual is not None:
            rp = _check(residual, "residual", _VALUES, shape, dev)
            rt = residual.dtype
        elif residual_out is not None:
            raise ValueError("residual_out needs a residual")
        given = y is not None or scale is not None or residual_out is not None
        with _where(dev, stream):
            if y is None:
                y = torch.empty_like(x, dtype=dtype)
            if residual is not None and residual_out is None:
                residual_out = torch.empty_like(residual)
            if dtype is _FP8 and scale is None:
                scale = torch.empty((T, _groups(d)), dtype=_FP32, device=self._place)
            if given:
                self._check_outputs(x, residual, dtype, y, scale, residual_out, shape)
            yp = y.data_ptr()
            if rp is not None:
                sp = residual_out.data_ptr()
            if dtype is _FP8:
                cp = scale.data_ptr()
            s = self._call(self._descriptor(x.dtype, rt, dtype), xp, rp, T, sp, yp, cp, _raw_stream(dev))
            if s:
                raise SffnError(s, "RmsNorm.forward")
        if residual is None and given and T and yp == xp:   # x holds y now
            return y, scale, None
        return y, scale, residual_out if residual is not None else x

    def _check_outputs(self, x, residual, dtype, y, scale, residual_out, shape) -> None:
        """Outputs that the caller gave (or that were made beside them)."""
        dev = self.device
        _check(y, "y", (dtype,), shape, dev)
        made = [(y, "y")]
        if residual is not None:
            _check(residual_out, "residual_out", (residual.dtype,), shape, dev)
            made.append((residual_out, "residual_out"))
        if dtype is _FP8:
            _check(scale, "scale", (_FP32,), (shape[0], _groups(self.d)), dev)
            made.append((scale, "scale"))
        for i, (t, name) in enumerate(made):
            if name == "scale":
                _apart(t, name, x, *(() if residual is None else (residual,)))
            else:
                _apart_or_in_place(t, name, x, residual)
            _apart(t, name, self.weight, *(u for u, _ in made[:i]))

    def forward(self, x, residual=None, *, out: str = "bf16", y=None, residual_out=None, stream: Optional[int] = None):
        """(y, s): x [T][d] bf16 or fp32, residual [T][d] bf16 or fp32 or None,
        y bf16 or fp32 by `out`, s in the residual's type (x itself without a
        residual, or None where y replaces it).  residual_out may be the
        residual, y x or the residual."""
        y, _, s = self._forward(x, residual, _out_type(out), y, None, residual_out, stream)
        return y, s

    __call__ = forward

    def forward_fp8(self, x, residual=None, *, y=None, scale=None, residual_out=None, stream: Optional[int] = None):
        """(codes, scale, s): y as e4m3 codes with an fp32 scale for each 128
        columns, as Fp8Linear takes them."""
        return self._forward(x, residual, _FP8, y, scale, residual_out, stream)

    def _workspace(self, T: int) -> int:
        n = ctypes.c_size_t()
        _ok(self._lib.sffn_rmsnorm_workspace_bytes(self.d, T, ctypes.byref(n)), "RmsNorm.backward")
        if len(self._work) < 1024:
            self._work[T] = n.value
        return n.value

    def backward(self, dy, s, ds=None, *, dx=None, dweight=None, stream: Optional[int] = None) -> dict:
        """{dx, dweight} for upstream dy (bf16 or fp32) and, if given, ds, the
        gradient that reaches s past the norm; dx has s's type, dweight is
        fp32 [d]."""
        T, _ = _matrix(s, "s")
        dev = self.device
        shape = (T, self.d)
        sp = _check(s, "s", (_BF16, _FP32), shape, dev)
        yp = _check(dy, "dy", (_BF16, _FP32), shape, dev)
        gp = None if ds is None else _check(ds, "ds", (s.dtype,), shape, dev)
        n = self._work.get(T) or self._workspace(T)
        with _where(dev, stream):
            if dweight is None:
                dweight = torch.empty(self.d, dtype=_FP32, device=self._place)
                wp = dweight.data_ptr()
            else:
                wp = _check(dweight, "dweight", (_FP32,), (self.d,), dev)
                _apart(dweight, "dweight", s, dy, self.weight, *(() if ds is None else (ds,)))
            if dx is None:
                dx = torch.empty_like(s)
                xp = dx.data_ptr()
            else:
                xp = _check(dx, "dx", (s.dtype,), shape, dev)
                _apart_or_in_place(dx, "dx", s, dy, ds)
                _apart(dx, "dx", self.weight, dweight)
            work = torch.empty(n, dtype=torch.uint8, device=self._place)
            e = self._call_backward(self._descriptor(_BF16, s.dtype, dy.dtype), yp, sp, gp, T, xp, wp, work.data_ptr(), n,
                                    _raw_stream(dev))
            if e:
                raise SffnError(e, "RmsNorm.backward")
        return {"dx": dx, "dweight": dweight}


def quantize_rows(x, *, codes=None, scale=None, stream: Optional[int] = None):
    """(codes, scale) of x [T][d] bf16 or fp32 (d % 8 == 0): e4m3 codes and an
    fp32 scale for each 128 columns of a row."""
    T, d = _matrix(x, "x")
    dev = x.get_device() if x.is_cuda else None
    xp = _check(x, "x", (_BF16, _FP32), (T, d), dev)
    given = codes is not None or scale is not None
    with _where(dev, stream):
        if codes is None:
            codes = torch.empty_like(x, dtype=_FP8)
        if scale is None:
            scale = x.new_empty((T, _groups(d)), dtype=_FP32)
        qp = _check(codes, "codes", (_FP8,), (T, d), dev)
        cp = _check(scale, "scale", (_FP32,), (T, _groups(d)), dev)
        if given:
            _apart(codes, "codes", x, scale)
            _apart(scale, "scale", x)
        _ok(load_library().sffn_quantize_rows(xp, _CODE[x.dtype], T, d, qp, cp, _raw_stream(dev)), "quantize_rows")
    return codes, scale


def quantize_blocks(W, *, codes=None, scale=None, stream: Optional[int] = None):
    """(codes, scale) of a weight W [n][k] bf16 or fp32 (k % 8 == 0): e4m3
    codes and an fp32 scale for each block of 128 x 128."""
    n, k = _matrix(W, "W")
    dev = W.get_device() if W.is_cuda else None
    wp = _check(W, "W", (_BF16, _FP32), (n, k), dev)
    given = codes is not None or scale is not None
    with _where(dev, stream):
        if codes is None:
            codes = torch.empty((n, k), dtype=_FP8, device=W.device)
        if scale is None:
            scale = torch.empty((_groups(n), _groups(k)), dtype=_FP32, device=W.device)
        qp = _check(codes, "codes", (_FP8,), (n, k), dev)
        cp = _check(scale, "scale", (_FP32,), (_groups(n), _groups(k)), dev)
        if given:
            _apart(codes, "codes", W, scale)
            _apart(scale, "scale", W)
        _ok(load_library().sffn_quantize_blocks(wp, _CODE[W.dtype], n, k, qp, cp, _raw_stream(dev)),
            "quantize_blocks")
    return codes, scale


class _Handle:
    """A library handle that belongs to one device.  It has to outlive the
    graphs that its calls were captured into, as its weights have to."""
    _name = ""

    def _create(self, desc, stream: Optional[int]) -> None:
        self.h = None
        self._lib = load_library()
        h = ctypes.c_void_p()
        with _where(self.device, stream):
            _ok(getattr(self._lib, f"sffn_{self._name}_create")(ctypes.byref(desc), _raw_stream(self.device),
                                                                ctypes.byref(h)), f"sffn_{self._name}_create")
        self.h = h

    def read_status(self, stream: Optional[int] = None) -> int:
        """Synchronise the stream, then return and clear the status word."""
        with _where(self.device, stream):
            return getattr(self._lib, f"sffn_{self._name}_read_status")(self.h, _raw_stream(self.device))

    def close(self) -> None:
        if getattr(self, "h", None) is not None and self.h.value:
            getattr(self._lib, f"sffn_{self._name}_destroy")(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Fp8Linear(_Handle):
    """y = x W^T with both operands in e4m3 codes (inference): Wq [d_out][d_in]
    with a scale for each 128 x 128 block, Ws [ceil(d_out/128)]
    [ceil(d_in/128)] fp32.  d_in % 16 == 0, d_out % 8 == 0."""
    _name = "qlinear"

    def __init__(self, Wq, Ws, *, stream: Optional[int] = None):
        self.h = None
        n, k = _matrix(Wq, "Wq")
        wp = _check(Wq, "Wq", (_FP8,), (n, k), None)
        self.device = Wq.get_device()
        cp = _check(Ws, "Ws", (_FP32,), (_groups(n), _groups(k)), self.device)
        self.d_in, self.d_out, self.Wq, self.Ws = k, n, Wq, Ws
        self._wp, self._cp, self._place = wp, cp, Wq.device
        self._create(sffn_qlinear_desc(d_in=k, d_out=n, Wq=wp, Ws=cp), stream)
        self._call, self._call_values = self._lib.sffn_qlinear_forward, self._lib.sffn_qlinear_quantize_forward

    @classmethod
    def from_weight(cls, W, *, stream: Optional[int] = None) -> "Fp8Linear":
        """From a bf16 or fp32 weight [d_out][d_in], quantised here."""
        return cls(*quantize_blocks(W, stream=stream), stream=stream)

    def forward(self, x, scale=None, *, out: str = "bf16", y=None, stream: Optional[int] = None):
        """y [T][d_out] bf16 or fp32 by `out`.  x [T][d_in] is e4m3 codes with
        their scale [T][ceil(d_in/128)], or bf16 or fp32 and is quantised
        first (scale None)."""
        T, _ = _matrix(x, "x")
        dev, k = self.device, self.d_in
        dtype = _out_type(out)
        if self.Wq.data_ptr() != self._wp or self.Ws.data_ptr() != self._cp:
            _moved("Wq or Ws")
        codes = scale is not None
        xp = _check(x, "x", (_FP8,) if codes else _VALUES, (T, k), dev)
        if codes:
            cp = _check(scale, "scale", (_FP32,), (T, _groups(k)), dev)
        with _where(dev, stream):
            if y is None:
                y = torch.empty((T, self.d_out), dtype=dtype, device=self._place)
                yp = y.data_ptr()
            else:
                yp = _check(y, "y", (dtype,), (T, self.d_out), dev)
                _apart(y, "y", x, self.Wq, self.Ws, *((scale,) if codes else ()))
            if codes:
                s = self._call(self.h, xp, cp, T, yp, _CODE[dtype], _raw_stream(dev))
            else:
                n = (T * k + 15) // 16 * 16 + 4 * T * _groups(k)
                work = torch.empty(n, dtype=torch.uint8, device=self._place)
                s = self._call_values(self.h, xp, _CODE[x.dtype], T, yp, _CODE[dtype], work.data_ptr(), n,
                                      _raw_stream(dev))
            if s:
                raise SffnError(s, "Fp8Linear.forward")
        return y

    __call__ = forward


class GroupedLinear(_Handle):
    """Products of rows sorted by expert with their expert's weight, W
    [n_experts][d_out][d_in] bf16 (d_in and d_out multiples of 8).

    offsets is int32 [n_experts + 1] on the device: expert e owns rows
    offsets[e] <= r < offsets[e+1] (possibly none).  From a router's choice
    `sel` [tokens][top_k], for instance:

        order = sel.flatten().argsort(stable=True)
        offsets = torch.searchsorted(sel.flatten()[order], experts).int()   # experts = arange(n_experts + 1)
        x_sorted = x[order // top_k]
    """
    _name = "grouped"

    def __init__(self, W, *, stream: Optional[int] = None):
        self.h = None
        if not isinstance(W, torch.Tensor) or W.dim() != 3:
            raise ValueError("W must be an [n_experts][d_out][d_in] tensor")
        E, n, k = W.shape
        wp = _check(W, "W", (_BF16,), (E, n, k), None)
        self.device = W.get_device()
        self.n_experts, self.d_out, self.d_in, self.W = E, n, k, W
        self._wp, self._place = wp, W.device
        self._create(sffn_grouped_desc(n_experts=E, d_in=k, d_out=n, W=wp), stream)

    def _rows(self, t, name: str, cols: int, offsets):
        R, _ = _matrix(t, name)
        p = _check(t, name, (_BF16,), (R, cols), self.device)
        if self.W.data_ptr() != self._wp:
            _moved("W")
        if not (isinstance(offsets, torch.Tensor) and offsets.dtype is torch.int32 and offsets.is_cuda
                and offsets.get_device() == self.device and offsets.shape == (self.n_experts + 1,)
                and offsets.is_contiguous()):
            raise ValueError(f"offsets must be a contiguous int32 CUDA tensor [{self.n_experts + 1}] on "
                             f"cuda:{self.device}")
        return R, p, offsets.data_ptr()

    def forward(self, x, offsets, *, out: str = "bf16", y=None, stream: Optional[int] = None):
        """y [R][d_out] bf16 or fp32 by `out`, y[r] = W[e(r)] x[r]; rows in no
        group are left as they were (unset in a y made here)."""
        dtype = _out_type(out)
        R, xp, op = self._rows(x, "x", self.d_in, offsets)
        dev = self.device
        with _where(dev, stream):
            if y is None:
                y = torch.empty((R, self.d_out), dtype=dtype, device=self._place)
                yp = y.data_ptr()
            else:
                yp = _check(y, "y", (dtype,), (R, self.d_out), dev)
                _apart(y, "y", x, self.W, offsets)
            _ok(self._lib.sffn_grouped_forward(self.h, xp, op, R, yp, _CODE[dtype], _raw_stream(dev)),
                "GroupedLinear.forward")
        return y

    __call__ = forward

    def backward(self, x, dy, offsets, *, out: str = "bf16", dx=None, dW=None, stream: Optional[int] = None) -> dict:
        """{dx, dW} for upstream dy [R][d_out] bf16: dx [R][d_in] bf16 or fp32
        by `out` (rows in no group left as they were), dW [n_experts][d_out]
        [d_in] fp32 (or bf16 where the dW given is)."""
        dtype = _out_type(out)
        R, xp, op = self._rows(x, "x", self.d_in, offsets)
        dev = self.device
        yp = _check(dy, "dy", (_BF16,), (R, self.d_out), dev)
        with _where(dev, stream):
            if dx is None:
                dx = torch.empty_like(x, dtype=dtype)
                gp = dx.data_ptr()
            else:
                gp = _check(dx, "dx", (dtype,), (R, self.d_in), dev)
                _apart(dx, "dx", x, dy, self.W, offsets)
            shape = (self.n_experts, self.d_out, self.d_in)
            if dW is None:
                dW = torch.empty_like(self.W, dtype=_FP32)
                wp = dW.data_ptr()
            else:
                wp = _check(dW, "dW", (_FP32, _BF16), shape, dev)
                _apart(dW, "dW", x, dy, self.W, offsets, dx)
            st = _raw_stream(dev)
            _ok(self._lib.sffn_grouped_backward_input(self.h, yp, op, R, gp, _CODE[dtype], st),
                "GroupedLinear.backward")
            _ok(self._lib.sffn_grouped_backward_weight(self.h, xp, yp, op, R, wp, _CODE[dW.dtype], st),
                "GroupedLinear.backward")
        return {"dx": dx, "dW": dW}
