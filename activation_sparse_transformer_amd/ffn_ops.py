"""Binding of the operators around the sparse FFN layer (the C ABI in include/ffn_ops.h): the RMS
norm and the layer norm with the residual's sum, their gradients, products with 4-bit weights, the
norm of all gradients and clipping by it, AdamW.

Argument marshalling only, as in ``sparse_ffn``: every step runs in the library's HIP kernels;
PyTorch supplies device memory and the stream.  With ``stream=None`` a call runs on PyTorch's
current stream of the tensors' device; a given ``stream`` is used for the kernels and for what
the call allocates.  Tensors made on another stream have to be ready on it (the caller's events).
Memory is not given away before the call's work is done: that of every tensor of a call with a
given stream, and on whatever stream a call runs that of what an ``Mx4Linear``, ``Mx4Tokens`` or
``AdamW`` holds.
As with PyTorch's own operations, the other tensors of a call on the current stream are the
caller's to keep (``record_stream``) if they were allocated on a different one.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
from operator import attrgetter

import numpy as np

from . import sparse_ffn as _base

SFFN_E4M3 = 2
NORM_MAX_D = 32768
MX4_GROUP = 32
ADAMW_BLOCK = 256

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t


class AdamwTensorC(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("param", "grad", "master", "m", "v", "m_scale", "v_scale")] + \
               [("n", _I64)]


class AdamwHyperC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay")] + \
               [("step", _I64)]


class GradC(ctypes.Structure):
    _fields_ = [("grad", _P), ("out", _P), ("n", _I64), ("dtype", _I32), ("zero", _I32)]


_GRAD_WORD = AdamwTensorC.grad.offset // 8
_SHAPE, _DTYPE = attrgetter("shape"), attrgetter("dtype")

_NORM = [_I32, _I32, _P, _I64, _P, _I64, _P, ctypes.c_float, _I64, _I32, _P, _P, _P, _P]
_LAYER_NORM = _NORM[:7] + [_P] + _NORM[7:]
_GRAD_NORM = [_P, _I32, ctypes.c_double, _P, _P, _P, _SZ, _P]
_PROTOS = {
    "sffn_rms_norm": _NORM,
    "sffn_rms_norm_fp8": _NORM,
    "sffn_rms_norm_backward_workspace": [_I64, _I32, ctypes.POINTER(_SZ)],
    "sffn_rms_norm_backward": [_I32, _I32, _P, _I64, _P, _I64, _P, _P, _P, _I64, _I64, _I32, _P,
                               _P, _P, _SZ, _P],
    "sffn_layer_norm": _LAYER_NORM[:-1] + [_P, _P],
    "sffn_layer_norm_fp8": _LAYER_NORM,
    "sffn_layer_norm_backward_workspace": [_I64, _I32, ctypes.POINTER(_SZ)],
    "sffn_layer_norm_backward": [_I32, _I32, _P, _I64, _P, _I64, _P, _P, _P, _P, _I64, _I64, _I32,
                                 _P, _P, _P, _P, _SZ, _P],
    "sffn_mx4_quantize": [_I32, _P, _I64, _I32, _I32, _P, _P, _P],
    "sffn_mx4_bytes": [_I32, _I32, ctypes.POINTER(_SZ)],
    "sffn_mx4_tile": [_P, _P, _I32, _I32, _P, _P],
    "sffn_mx4_linear": [_P, _I32, _I32, _I32, _P, _I64, _P, _I32, _P, _I32, _I32, _P, _P],
    "sffn_mx4_tokens_bytes": [_I32, _I32, ctypes.POINTER(_SZ)],
    "sffn_mx4_tokens": [_I32, _P, _I64, _I32, _I32, _P, _P],
    "sffn_mx4_matmul": [_P, _I32, _I32, _P, _I32, _P, _I32, _I32, _P, _P],
    "sffn_mx4_quantized_workspace": [_I32, _I32, ctypes.POINTER(_SZ)],
    "sffn_mx4_quantized": [_P, _I32, _I32, _I32, _P, _I64, _I32, _P, _I32, _I32, _P, _P, _SZ, _P],
    "sffn_grad_norm_workspace": [_P, _I32, ctypes.POINTER(_SZ)],
    "sffn_grad_norm": _GRAD_NORM,
    "sffn_grad_clip": _GRAD_NORM,
    "sffn_adamw_step": [ctypes.POINTER(AdamwTensorC), _I32, _I32, _I32, _I32,
                        ctypes.POINTER(AdamwHyperC), _P, _P],
}

_fns = None


class _Fns:
    pass


def _lib():
    """The entry points with their prototypes, looked up once."""
    global _fns
    if _fns is None:
        import torch
        L = _base.lib()
        f = _Fns()
        for name, args in _PROTOS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
            setattr(f, name, fn)
        f.torch = torch
        # the current device's index, and the handle of a device's current stream (without making
        # a Stream object): torch's own quick forms, where it has them
        f.current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        f.stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda i: torch.cuda.current_stream(i).cuda_stream)
        f.code = {torch.float32: _base.SFFN_F32, torch.bfloat16: _base.SFFN_BF16,
                  torch.float8_e4m3fn: SFFN_E4M3}
        _fns = f
    return _fns


def exported_names():
    return list(_PROTOS)


def _fail(status, where):
    raise _base.SffnError(status, where, _base.last_error())


def _elsewhere(f, device, stream):
    """Whether a call has to enter `_on` first: a stream is given, or `device` is not current."""
    i = device.index
    if i is None:
        raise ValueError("device tensors are needed")
    return stream is not None or i != f.current_device()


@contextlib.contextmanager
def _on(device, stream, *tensors):
    """Makes `device`, and `stream` if given, current: what the call allocates belongs to it, and
    the memory of its `tensors` stays theirs until the stream is past the call."""
    import torch
    if device.type != "cuda":
        raise ValueError("device tensors are needed")
    if stream is None:
        with torch.cuda.device(device):
            yield
    else:
        if stream.device != device:
            raise ValueError("stream is not of the tensors' device")
        with torch.cuda.stream(stream):
            yield
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


class _Held:
    """Tensors that an object keeps from call to call: their memory stays theirs until every stream
    that a call ran on is past it, also after the object is gone."""

    def __init__(self, tensors):
        self._tensors = [t.detach() for t in tensors]  # (not a storage that takes their place)
        self._streams = set()

    def used_on(self, f, device, stream):
        """Called with each call's stream handle, which is current."""
        if stream not in self._streams:
            current = f.torch.cuda.current_stream(device)
            for t in self._tensors:
                t.record_stream(current)
            self._streams.add(stream)


def _matrix(t, name, dtype, shape, device):
    """Row stride of a [rows, d] tensor whose rows are contiguous."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device.index:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {list(shape)} on {device}")
    if t.is_contiguous():
        return shape[1]
    s = t.stride()
    if shape[1] > 1 and s[1] != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    if shape[0] > 1 and s[0] < shape[1]:
        raise ValueError(f"the rows of {name} overlap")
    return s[0] if shape[0] > 1 else shape[1]


def _plain(t, name, dtype, shape, device):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() \
            or t.get_device() != device.index:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)} "
                         f"on {device}")
    return t


def _ptr(t):
    return None if t is None else t.data_ptr()


def _norm(fn, fp8, x, gain, residual, eps, y, stat, h, stream):
    f = _lib()
    torch = f.torch
    dev, dt = x.device, x.dtype
    if _elsewhere(f, dev, stream):
        with _on(dev, stream, x, gain, residual, y, stat, h):
            return _norm(fn, fp8, x, gain, residual, eps, y, stat, h, None)
    shape = x.shape
    if len(shape) != 2 or dt not in (torch.float32, torch.bfloat16):
        raise ValueError("x must be a float32 or bfloat16 tensor [rows, d]")
    rows, d = shape
    xs = d if x.is_contiguous() else _matrix(x, "x", dt, shape, dev)
    rs = _matrix(residual, "residual", dt, shape, dev) if residual is not None else 0
    if gain.dtype != dt and gain.dtype != torch.float32:
        raise ValueError("gain must have x's type or float32")
    _plain(gain, "gain", gain.dtype, (d,), dev)
    out_t = torch.float8_e4m3fn if fp8 else dt
    if y is not None:
        _plain(y, "q" if fp8 else "y", out_t, shape, dev)
    else:
        y = x.new_empty(shape, dtype=out_t) if fp8 or xs != d else torch.empty_like(x)
    stat = x.new_empty(rows, dtype=torch.float32) if stat is None else \
        _plain(stat, "scale" if fp8 else "rstd", torch.float32, (rows,), dev)
    if residual is None:
        if h is not None:
            raise ValueError("h is written only with a residual")
    else:
        if h is not None:
            _plain(h, "h", dt, shape, dev)
        else:
            h = torch.empty_like(residual) if rs == d else residual.new_empty(shape)
    st = fn(f.code[dt], f.code[gain.dtype], x.data_ptr(), xs, _ptr(residual), rs,
            gain.data_ptr(), eps, rows, d, y.data_ptr(), stat.data_ptr(), _ptr(h),
            f.stream(dev.index))
    if st:
        _fail(st, "sffn_rms_norm_fp8" if fp8 else "sffn_rms_norm")
    return y, stat, x if residual is None else h


def rms_norm(x, gain, residual=None, eps=1e-6, y=None, h=None, rstd=None, stream=None):
    """h = x + residual, rstd = 1 / sqrt(mean(h^2) + eps), y = h * rstd * gain over the rows of
    x [rows, d] (float32 or bfloat16; rows may be strided).  gain [d] has x's type or float32.
    Returns (y, h, rstd): what rms_norm_backward takes; h is x without a residual.  y, h and
    rstd may be given to be overwritten; y and h may each be the (contiguous) residual or x
    itself, otherwise they may not overlap anything."""
    y, rstd, h = _norm(_lib().sffn_rms_norm, False, x, gain, residual, eps, y, rstd, h, stream)
    return y, h, rstd


def rms_norm_fp8(x, gain, residual=None, eps=1e-6, q=None, scale=None, h=None, stream=None):
    """The norm for serving, its output in 8 bits: q [rows, d] float8_e4m3fn and scale [rows]
    float32 (max |y| / 448 a row) with y ~ q * scale, as Mx4Linear takes them.  Returns
    (q, scale, h)."""
    return _norm(_lib().sffn_rms_norm_fp8, True, x, gain, residual, eps, q, scale, h, stream)


def rms_norm_backward(dy, h, gain, rstd, dres=None, with_dgain=True, dx=None, dgain=None,
                      stream=None):
    """Gradient of rms_norm for dL/dy = dy, with the forward's h and rstd.  dres is the gradient
    that reaches h past the norm (of the residual stream).  Returns (dx, dgain): dx, in h's
    type, is the gradient of both x and the residual; dgain is float32, or None without
    with_dgain.  dx and dgain may be given; dx may be dres itself, otherwise they may not overlap
    anything (dgain's sums read dy and h while dx is written)."""
    f = _lib()
    torch = f.torch
    dev, dt = h.device, h.dtype
    if _elsewhere(f, dev, stream):
        with _on(dev, stream, dy, h, gain, rstd, dres, dx, dgain):
            return rms_norm_backward(dy, h, gain, rstd, dres, with_dgain, dx, dgain)
    shape = h.shape
    if len(shape) != 2 or dt not in (torch.float32, torch.bfloat16):
        raise ValueError("h must be a float32 or bfloat16 tensor [rows, d]")
    rows, d = shape
    hs = d if h.is_contiguous() else _matrix(h, "h", dt, shape, dev)
    ys = _matrix(dy, "dy", dt, shape, dev)
    rs = _matrix(dres, "dres", dt, shape, dev) if dres is not None else 0
    if gain.dtype != dt and gain.dtype != torch.float32:
        raise ValueError("gain must have h's type or float32")
    _plain(gain, "gain", gain.dtype, (d,), dev)
    _plain(rstd, "rstd", torch.float32, (rows,), dev)
    if dx is not None:
        _plain(dx, "dx", dt, shape, dev)
    else:
        dx = torch.empty_like(h) if hs == d else h.new_empty(shape)
    ws, nb = None, 0
    if with_dgain:
        dgain = torch.empty(d, dtype=torch.float32, device=dev) if dgain is None else \
            _plain(dgain, "dgain", torch.float32, (d,), dev)
        nb = _norm_workspace(rows, d)
        if nb:
            ws = torch.empty(nb, dtype=torch.uint8, device=dev)
    else:
        dgain = None
    st = f.sffn_rms_norm_backward(f.code[dt], f.code[gain.dtype], dy.data_ptr(), ys,
                                  h.data_ptr(), hs, gain.data_ptr(), rstd.data_ptr(),
                                  _ptr(dres), rs, rows, d, dx.data_ptr(), _ptr(dgain),
                                  _ptr(ws), nb, f.stream(dev.index))
    if st:
        _fail(st, "sffn_rms_norm_backward")
    return dx, dgain


@functools.lru_cache(maxsize=256)
def _norm_workspace(rows, d):
    n = _SZ()
    st = _lib().sffn_rms_norm_backward_workspace(rows, d, ctypes.byref(n))
    if st:
        _fail(st, "sffn_rms_norm_backward_workspace")
    return n.value


def _layer_norm(fp8, x, gain, bias, residual, eps, y, mean, stat, h, stream):
    f = _lib()
    torch = f.torch
    dev, dt = x.device, x.dtype
    if _elsewhere(f, dev, stream):
        with _on(dev, stream, x, gain, bias, residual, y, mean, stat, h):
            return _layer_norm(fp8, x, gain, bias, residual, eps, y, mean, stat, h, None)
    shape = x.shape
    if len(shape) != 2 or dt not in (torch.float32, torch.bfloat16):
        raise ValueError("x must be a float32 or bfloat16 tensor [rows, d]")
    rows, d = shape
    xs = d if x.is_contiguous() else _matrix(x, "x", dt, shape, dev)
    rs = _matrix(residual, "residual", dt, shape, dev) if residual is not None else 0
    if gain.dtype != dt and gain.dtype != torch.float32:
        raise ValueError("gain must have x's type or float32")
    _plain(gain, "gain", gain.dtype, (d,), dev)
    if bias is not None:
        _plain(bias, "bias", gain.dtype, (d,), dev)
    out_t = torch.float8_e4m3fn if fp8 else dt
    if y is not None:
        _plain(y, "q" if fp8 else "y", out_t, shape, dev)
    else:
        y = x.new_empty(shape, dtype=out_t) if fp8 or xs != d else torch.empty_like(x)
    stat = x.new_empty(rows, dtype=torch.float32) if stat is None else \
        _plain(stat, "scale" if fp8 else "rstd", torch.float32, (rows,), dev)
    if not fp8:
        mean = torch.empty_like(stat) if mean is None else \
            _plain(mean, "mean", torch.float32, (rows,), dev)
    if residual is None:
        if h is not None:
            raise ValueError("h is written only with a residual")
    else:
        if h is not None:
            _plain(h, "h", dt, shape, dev)
        else:
            h = torch.empty_like(residual) if rs == d else residual.new_empty(shape)
    args = (f.code[dt], f.code[gain.dtype], x.data_ptr(), xs, _ptr(residual), rs, gain.data_ptr(),
            _ptr(bias), eps, rows, d, y.data_ptr())
    if fp8:
        st = f.sffn_layer_norm_fp8(*args, stat.data_ptr(), _ptr(h), f.stream(dev.index))
    else:
        st = f.sffn_layer_norm(*args, mean.data_ptr(), stat.data_ptr(), _ptr(h),
                               f.stream(dev.index))
    if st:
        _fail(st, "sffn_layer_norm_fp8" if fp8 else "sffn_layer_norm")
    return y, x if residual is None else h, mean, stat


def layer_norm(x, gain, bias=None, residual=None, eps=1e-5, y=None, h=None, mean=None, rstd=None,
               stream=None):
    """h = x + residual, mean and rstd = 1 / sqrt(var + eps) of its rows, y = (h - mean) * rstd *
    gain + bias over the rows of x [rows, d] (float32 or bfloat16; rows may be strided).  gain [d]
    has x's type or float32, bias [d] gain's type.  Returns (y, h, mean, rstd): what
    layer_norm_backward takes; h is x without a residual.  Outputs may be given as in rms_norm."""
    return _layer_norm(False, x, gain, bias, residual, eps, y, mean, rstd, h, stream)


def layer_norm_fp8(x, gain, bias=None, residual=None, eps=1e-5, q=None, scale=None, h=None,
                   stream=None):
    """The layer norm for serving, its output in 8 bits as rms_norm_fp8 gives it.  Returns
    (q, scale, h)."""
    q, h, _, scale = _layer_norm(True, x, gain, bias, residual, eps, q, None, scale, h, stream)
    return q, scale, h


def layer_norm_backward(dy, h, gain, mean, rstd, dres=None, with_dgain=True, with_dbias=True,
                        dx=None, dgain=None, dbias=None, stream=None):
    """Gradient of layer_norm for dL/dy = dy, with the forward's h, mean and rstd.  Returns
    (dx, dgain, dbias): dx, in h's type, is the gradient of both x and the residual; dgain and
    dbias are float32, or None if they are not wanted.  dres and given outputs are as in
    rms_norm_backward."""
    f = _lib()
    torch = f.torch
    dev, dt = h.device, h.dtype
    if _elsewhere(f, dev, stream):
        with _on(dev, stream, dy, h, gain, mean, rstd, dres, dx, dgain, dbias):
            return layer_norm_backward(dy, h, gain, mean, rstd, dres, with_dgain, with_dbias, dx,
                                       dgain, dbias)
    shape = h.shape
    if len(shape) != 2 or dt not in (torch.float32, torch.bfloat16):
        raise ValueError("h must be a float32 or bfloat16 tensor [rows, d]")
    rows, d = shape
    hs = d if h.is_contiguous() else _matrix(h, "h", dt, shape, dev)
    ys = _matrix(dy, "dy", dt, shape, dev)
    rs = _matrix(dres, "dres", dt, shape, dev) if dres is not None else 0
    if gain.dtype != dt and gain.dtype != torch.float32:
        raise ValueError("gain must have h's type or float32")
    _plain(gain, "gain", gain.dtype, (d,), dev)
    _plain(mean, "mean", torch.float32, (rows,), dev)
    _plain(rstd, "rstd", torch.float32, (rows,), dev)
    if dx is not None:
        _plain(dx, "dx", dt, shape, dev)
    else:
        dx = torch.empty_like(h) if hs == d else h.new_empty(shape)
    ws, nb = None, 0
    if with_dgain or with_dbias:
        nb = _layer_norm_workspace(rows, d)
        if nb:
            ws = torch.empty(nb, dtype=torch.uint8, device=dev)
    outs = []
    for want, t, name in ((with_dgain, dgain, "dgain"), (with_dbias, dbias, "dbias")):
        outs.append(None if not want else torch.empty(d, dtype=torch.float32, device=dev)
                    if t is None else _plain(t, name, torch.float32, (d,), dev))
    dgain, dbias = outs
    st = f.sffn_layer_norm_backward(f.code[dt], f.code[gain.dtype], dy.data_ptr(), ys,
                                    h.data_ptr(), hs, gain.data_ptr(), mean.data_ptr(),
                                    rstd.data_ptr(), _ptr(dres), rs, rows, d, dx.data_ptr(),
                                    _ptr(dgain), _ptr(dbias), _ptr(ws), nb, f.stream(dev.index))
    if st:
        _fail(st, "sffn_layer_norm_backward")
    return dx, dgain, dbias


@functools.lru_cache(maxsize=256)
def _layer_norm_workspace(rows, d):
    n = _SZ()
    st = _lib().sffn_layer_norm_backward_workspace(rows, d, ctypes.byref(n))
    if st:
        _fail(st, "sffn_layer_norm_backward_workspace")
    return n.value


def mx4_quantize(W, stream=None):
    """(codes, scales) of a dense W [N, K] (float32 or bfloat16): uint8 [N, 16 * ceil(K / 32)]
    with two e2m1 codes a byte (even k low) and uint8 [N, ceil(K / 32)] exponents + 127."""
    f = _lib()
    torch = f.torch
    if _elsewhere(f, W.device, stream):
        with _on(W.device, stream, W):
            return mx4_quantize(W)
    if W.dim() != 2 or W.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("W must be a float32 or bfloat16 tensor [N, K]")
    N, K = W.shape
    st_w = _matrix(W, "W", W.dtype, (N, K), W.device)
    G = -(-K // MX4_GROUP)
    codes = torch.empty((N, 16 * G), dtype=torch.uint8, device=W.device)
    scales = torch.empty((N, G), dtype=torch.uint8, device=W.device)
    st = f.sffn_mx4_quantize(f.code[W.dtype], W.data_ptr(), st_w, N, K, codes.data_ptr(),
                             scales.data_ptr(), f.stream(W.device.index))
    if st:
        _fail(st, "sffn_mx4_quantize")
    return codes, scales


@functools.lru_cache(maxsize=256)
def _tokens_bytes(T, K):
    n = _SZ()
    st = _lib().sffn_mx4_tokens_bytes(T, K, ctypes.byref(n))
    if st:
        _fail(st, "sffn_mx4_tokens_bytes")
    return n.value


@functools.lru_cache(maxsize=256)
def _quantized_workspace(T, K):
    n = _SZ()
    st = _lib().sffn_mx4_quantized_workspace(T, K, ctypes.byref(n))
    if st:
        _fail(st, "sffn_mx4_quantized_workspace")
    return n.value


class Mx4Tokens:
    """Tokens x [T, K] (float32 or bfloat16; rows may be strided) rounded to 4 bits as
    mx4_quantize rounds weights, for one or more calls of Mx4Linear.quantized.  On another
    stream than the one they were made on, a call has to wait for them, as for any tensor."""

    def __init__(self, x, stream=None):
        f = _lib()
        torch = f.torch
        dev = x.device
        if _elsewhere(f, dev, stream):
            with _on(dev, stream, x):
                return self.__init__(x)
        if x.dim() != 2 or x.dtype not in (torch.float32, torch.bfloat16):
            raise ValueError("x must be a float32 or bfloat16 tensor [T, K]")
        T, K = x.shape
        xs = _matrix(x, "x", x.dtype, (T, K), dev)
        data = torch.empty(_tokens_bytes(T, K), dtype=torch.uint8, device=dev)
        st = f.sffn_mx4_tokens(f.code[x.dtype], x.data_ptr(), xs, T, K, data.data_ptr(),
                               f.stream(dev.index))
        if st:
            _fail(st, "sffn_mx4_tokens")
        self._shape, self._dtype, self._data = (T, K), x.dtype, data
        self._streams = {f.stream(dev.index)}

    shape = property(lambda self: self._shape)
    dtype = property(lambda self: self._dtype)  # before rounding
    device = property(lambda self: self._data.device)

    def used_on(self, f, device, stream):
        """Called with each product's stream handle, which is current: the memory is kept until every one
        of them is past it, also after the object is gone."""
        if stream not in self._streams:
            self._data.record_stream(f.torch.cuda.current_stream(device))
            self._streams.add(stream)


class Mx4Linear:
    """y = act(x W^T + bias) with 4-bit weights W [N, K], for batches of few tokens (serving).

    codes and scales are as mx4_quantize gives them (MXFP4: e2m1 values, one power of two per 32
    columns); in_features is K where it is not 32 * scales.shape[1].  They are laid out once for
    the kernel, here (a call on another stream has to wait for that), and not kept.  bias [N]
    float32 is borrowed (kept referenced); it and relu may be assigned, and a bias whose storage
    was replaced (bias.data = b) is followed by the next call."""

    def __init__(self, codes, scales, bias=None, relu=False, in_features=None, stream=None):
        f = _lib()
        torch = f.torch
        if scales.dim() != 2 or scales.shape[1] < 1:
            raise ValueError("scales must be [N, ceil(K / 32)]")
        N, G = scales.shape
        K = G * MX4_GROUP if in_features is None else int(in_features)
        if not (G - 1) * MX4_GROUP < K <= G * MX4_GROUP:
            raise ValueError(f"in_features must lie in ({(G - 1) * MX4_GROUP}, {G * MX4_GROUP}]")
        dev = scales.device
        _plain(scales, "scales", torch.uint8, (N, G), dev)
        _plain(codes, "codes", torch.uint8, (N, 16 * G), dev)
        if bias is not None:
            _plain(bias, "bias", torch.float32, (N,), dev)
        n = _SZ()
        st = f.sffn_mx4_bytes(N, K, ctypes.byref(n))
        if st:
            _fail(st, "sffn_mx4_bytes")
        with _on(dev, stream, codes, scales):
            tiled = torch.empty(n.value, dtype=torch.uint8, device=dev)
            st = f.sffn_mx4_tile(codes.data_ptr(), scales.data_ptr(), N, K, tiled.data_ptr(),
                                 f.stream(dev.index))
        if st:
            _fail(st, "sffn_mx4_tile")
        self._n, self._k, self._bytes, self._device = N, K, n.value, dev
        self.relu = bool(relu)
        self._take(tiled, bias)

    in_features = property(lambda self: self._k)
    out_features = property(lambda self: self._n)
    device = property(lambda self: self._device)
    tiled = property(lambda self: self._tiled)
    bias = property(lambda self: self._bias, lambda self, b: self._take(self._tiled, b))

    def _take(self, tiled, bias):
        """Checks the tensors, then takes them and their addresses.  The memory behind those is held,
        so that an address that is still the same is still the same memory."""
        torch = _lib().torch
        _plain(tiled, "tiled", torch.uint8, (self._bytes,), self._device)
        if bias is not None:
            _plain(bias, "bias", torch.float32, (self._n,), self._device)
        self._tiled, self._bias = tiled, bias
        self._tiled_ptr, self._bias_ptr = tiled.data_ptr(), _ptr(bias)
        self._held = _Held([tiled] if bias is None else [tiled, bias])

    @classmethod
    def from_dense(cls, W, bias=None, relu=False, stream=None):
        """The layer of a dense W [N, K], quantised."""
        codes, scales = mx4_quantize(W, stream=stream)
        return cls(codes, scales, bias=bias, relu=relu, in_features=W.shape[1], stream=stream)

    def __call__(self, x, x_scale=None, dtype=None, y=None, stream=None):
        """x [T, K] is bfloat16, float32, or float8_e4m3fn with x_scale [T] float32 (which the
        other types may have too).  y [T, N] is float32 or bfloat16: `dtype`, or that of a given
        y; by default float32 for float32 x, otherwise bfloat16."""
        f = _lib()
        torch = f.torch
        N, K, dev, bias = self._n, self._k, self._device, self._bias
        if _elsewhere(f, dev, stream):
            with _on(dev, stream, x, x_scale, y):
                return self(x, x_scale, dtype, y)
        if self._tiled.data_ptr() != self._tiled_ptr \
                or (bias is not None and bias.data_ptr() != self._bias_ptr):
            self._take(self._tiled, bias)  # a storage was replaced
        shape = x.shape
        xc = f.code.get(x.dtype)
        if len(shape) != 2 or xc is None:
            raise ValueError(f"x must be a float32, bfloat16 or float8_e4m3fn tensor [T, {K}]")
        T = shape[0]
        xs = _matrix(x, "x", x.dtype, (T, K), dev)
        if x_scale is not None:
            _plain(x_scale, "x_scale", torch.float32, (T,), dev)
        elif xc == SFFN_E4M3:
            raise ValueError("float8 x needs x_scale")
        if y is None:
            dt = dtype or (torch.float32 if xc == _base.SFFN_F32 else torch.bfloat16)
            if dt not in (torch.float32, torch.bfloat16):
                raise ValueError("dtype must be float32 or bfloat16")
            y = torch.empty((T, N), dtype=dt, device=dev)
        else:
            dt = y.dtype
            if dt not in (torch.float32, torch.bfloat16) or dtype not in (None, dt):
                raise ValueError("y must be float32 or bfloat16, and of `dtype`")
            _plain(y, "y", dt, (T, N), dev)
        s = f.stream(dev.index)
        self._held.used_on(f, dev, s)
        st = f.sffn_mx4_linear(self._tiled_ptr, N, K, xc, x.data_ptr(), xs, _ptr(x_scale), T,
                               self._bias_ptr, self.relu, f.code[dt], y.data_ptr(), s)
        if st:
            _fail(st, "sffn_mx4_linear")
        return y

    def quantized(self, x, dtype=None, y=None, stream=None):
        """The layer with the tokens in 4 bits too (x [T, K] float32 or bfloat16 is rounded as
        mx4_quantize rounds weights, or Mx4Tokens already are): for prompts, whose products then
        run at the 4-bit rate, and the same function for single tokens.  y [T, N] is as in a
        call; its default type goes by x's."""
        f = _lib()
        torch = f.torch
        N, K, dev, bias = self._n, self._k, self._device, self._bias
        if _elsewhere(f, dev, stream):
            with _on(dev, stream, None if isinstance(x, Mx4Tokens) else x, y):
                return self.quantized(x, dtype, y)
        if self._tiled.data_ptr() != self._tiled_ptr \
                or (bias is not None and bias.data_ptr() != self._bias_ptr):
            self._take(self._tiled, bias)  # a storage was replaced
        tokens = x._data if isinstance(x, Mx4Tokens) else None
        xt = x.dtype
        T = x.shape[0] if len(x.shape) == 2 else -1
        if T < 0 or x.shape[1] != K or x.device != dev or xt not in (torch.float32, torch.bfloat16):
            raise ValueError(f"x must be a float32 or bfloat16 tensor [T, {K}] on {dev}, or "
                             "Mx4Tokens of one")
        if y is None:
            dt = dtype or xt
            if dt not in (torch.float32, torch.bfloat16):
                raise ValueError("dtype must be float32 or bfloat16")
            y = torch.empty((T, N), dtype=dt, device=dev)
        else:
            dt = y.dtype
            if dt not in (torch.float32, torch.bfloat16) or dtype not in (None, dt):
                raise ValueError("y must be float32 or bfloat16, and of `dtype`")
            _plain(y, "y", dt, (T, N), dev)
        s = f.stream(dev.index)
        self._held.used_on(f, dev, s)
        if tokens is not None:
            x.used_on(f, dev, s)
            st = f.sffn_mx4_matmul(self._tiled_ptr, N, K, tokens.data_ptr(), T, self._bias_ptr,
                                   self.relu, f.code[dt], y.data_ptr(), s)
        else:
            xs = _matrix(x, "x", xt, (T, K), dev)
            nb = _quantized_workspace(T, K)
            ws = torch.empty(nb, dtype=torch.uint8, device=dev) if nb else None
            st = f.sffn_mx4_quantized(self._tiled_ptr, N, K, f.code[xt], x.data_ptr(), xs, T,
                                      self._bias_ptr, self.relu, f.code[dt], y.data_ptr(),
                                      _ptr(ws), nb, s)
        if st:
            _fail(st, "sffn_mx4_quantized" if tokens is None else "sffn_mx4_matmul")
        return y


def _grads(grads, max_norm, out, clip, norm, factor, stream):
    if factor is not None and max_norm is None:
        raise ValueError("factor needs max_norm")
    f = _lib()
    torch = f.torch
    T = torch.Tensor
    n = len(grads)
    if not n:
        raise ValueError("no gradients")
    dev = grads[0].device
    if _elsewhere(f, dev, stream):
        with _on(dev, stream, norm, factor, *grads, *(out or ())):
            return _grads(grads, max_norm, out, clip, norm, factor, None)
    types = list(map(_DTYPE, grads))
    kinds = set(types)
    if not kinds <= {torch.float32, torch.bfloat16} or set(map(T.get_device, grads)) != {dev.index} \
            or not all(map(T.is_contiguous, grads)):
        raise ValueError(f"gradients must be contiguous float32 or bfloat16 tensors on {dev}")
    ptrs = list(map(T.data_ptr, grads))
    if out is not None:
        if len(out) != n or list(map(_DTYPE, out)) != types \
                or not all(map(T.is_same_size, out, grads)) \
                or set(map(T.get_device, out)) != {dev.index} or not all(map(T.is_contiguous, out)):
            raise ValueError("out must have a contiguous tensor of each gradient's shape and type, "
                             f"on {dev}")
        outs = list(map(T.data_ptr, out))
    table = np.empty((n, 4), dtype=np.int64)  # an array of GradC
    table[:, 0] = ptrs
    table[:, 1] = table[:, 0] if out is None else outs
    table[:, 2] = list(map(T.numel, grads))
    table[:, 3] = f.code[types[0]] if len(kinds) == 1 else [f.code[t] for t in types]
    if norm is None:
        norm = torch.empty(1, dtype=torch.float32, device=dev)
    else:
        _plain(norm, "norm", torch.float32, (1,), dev)
    if factor is not None:
        _plain(factor, "factor", torch.float32, (1,), dev)
    elif max_norm is not None:
        factor = torch.empty(1, dtype=torch.float32, device=dev)
    nb = 8 * (1024 + n)  # the most that the call asks for
    ws = torch.empty(nb, dtype=torch.uint8, device=dev)
    fn = f.sffn_grad_clip if clip else f.sffn_grad_norm
    st = fn(table.ctypes.data, n, 0.0 if max_norm is None else max_norm, norm.data_ptr(),
            _ptr(factor), ws.data_ptr(), nb, f.stream(dev.index))
    if st:
        _fail(st, "sffn_grad_clip" if clip else "sffn_grad_norm")
    return norm, factor


def grad_norm(grads, max_norm=None, norm=None, factor=None, stream=None):
    """The norm of all gradients (a list of contiguous device tensors, each float32 or bfloat16)
    together, and with max_norm the factor that clips them to it: 1, or max_norm / norm above it.
    Returns (norm, factor), float32 [1] on the device (factor None without max_norm): factor is
    what AdamW.step takes as grad_scale, with no pass over the gradients of its own.  Sums are in
    64 bits.  An infinity among the gradients, or a norm beyond float32, gives the norm infinity
    and the factor 0, a NaN gives NaN.  norm and factor may be given."""
    return _grads(grads, max_norm, None, False, norm, factor, stream)


def clip_grads(grads, max_norm, out=None, norm=None, factor=None, stream=None):
    """The same, and the gradients times the factor: in place, or into `out` (a list of tensors
    like grads, each of which may be its gradient itself).  The tensors written and read may not
    overlap otherwise.  max_norm is required (None is refused).  Returns (norm, factor)."""
    return _grads(grads, max_norm, out, True, norm, factor, stream)


class AdamW:
    """AdamW over a list of tensors, updated in place by one launch (per 48 tensors).

    params: contiguous device tensors, all float32 or all bfloat16.  master: their float32
    copies (for bfloat16 params), the values the step is taken on; params then receive the
    rounded result.  state_bits 32 keeps both moments in float32; 8 keeps the first moment and
    the root of the second as float8_e4m3fn with one float32 scale per 256 elements.  `state`
    continues from given tensors instead of zeros: [m, v] or [m, m_scale, r, r_scale], each a
    list like params; with it, state_bits goes by its length, and `step` is the number of steps
    done.  A step writes all of these tensors: none may overlap another.

    The tensors are in `.params`, `.master` and `.state`, in that order, as tuples: to replace
    some, assign the whole (checked as here); a tensor whose storage was replaced (p.data = q)
    is followed by the next step.  lr, betas, eps, weight_decay and steps may be changed between
    steps; a step recorded in a graph replays with the values and the memory it was recorded
    with, its number among them."""

    def __init__(self, params, master=None, state_bits=32, state=None, lr=1e-3,
                 betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, step=0):
        torch = _lib().torch
        params = list(params)
        if not params:
            raise ValueError("no parameters")
        dev = params[0].device
        if dev.type != "cuda":
            raise ValueError("parameters must be device tensors")
        if state is None:
            if state_bits not in (8, 32):
                raise ValueError("state_bits must be 8 or 32")
            zeros = lambda t, n: [torch.zeros(n(p), dtype=t, device=dev) for p in params]  # noqa: E731
            if state_bits == 32:
                state = [zeros(torch.float32, lambda p: p.shape) for _ in range(2)]
            else:
                state = [zeros(t, n) for _ in range(2) for t, n in (
                    (torch.float8_e4m3fn, lambda p: p.shape),
                    (torch.float32, lambda p: -(-p.numel() // ADAMW_BLOCK)))]
        self._bind(params, master, state)
        self.lr, self.betas, self.eps, self.weight_decay = lr, betas, eps, weight_decay
        self.steps = int(step)

    params = property(lambda self: self._params,
                      lambda self, t: self._bind(t, self._master, self._state))
    master = property(lambda self: self._master,
                      lambda self, t: self._bind(self._params, t, self._state))
    state = property(lambda self: self._state,
                     lambda self, t: self._bind(self._params, self._master, t))
    state_bits = property(lambda self: self._bits)
    device = property(lambda self: self._device)
    dtype = property(lambda self: self._params[0].dtype)

    def _bind(self, params, master, state):
        """Checks the tensors, then takes them and their addresses."""
        f = _lib()
        torch = f.torch
        params = tuple(params)
        if not params:
            raise ValueError("no parameters")
        dt, dev = params[0].dtype, params[0].device
        if dt not in (torch.float32, torch.bfloat16) or dev.type != "cuda":
            raise ValueError("parameters must be float32 or bfloat16 device tensors")
        for p in params:
            _plain(p, "a parameter", dt, p.shape, dev)
        master = None if master is None else tuple(master)
        if master is not None and dt != torch.bfloat16:
            raise ValueError("a master copy needs bfloat16 parameters")
        state = tuple(tuple(k) for k in state)
        if len(state) not in (2, 4):
            raise ValueError("state must be [m, v] or [m, m_scale, r, r_scale]")
        bits = 32 if len(state) == 2 else 8
        for k in state + (() if master is None else (master,)):
            if len(k) != len(params):
                raise ValueError("master and state must have one tensor for each parameter")
        for i, p in enumerate(params):
            if master is not None:
                _plain(master[i], "a master copy", torch.float32, p.shape, dev)
            for j, k in enumerate(state):
                if bits == 32:
                    _plain(k[i], "a state", torch.float32, p.shape, dev)
                elif j % 2 == 0:
                    _plain(k[i], "a state", torch.float8_e4m3fn, p.shape, dev)
                else:
                    _plain(k[i], "a state's scales", torch.float32,
                           (-(-p.numel() // ADAMW_BLOCK),), dev)
        held = [t for k in (params, master or (), *state) for t in k]
        spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size())
                       for t in held if t.numel())
        if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):  # all of them are written
            raise ValueError("two of the tensors (parameters, master copies, states) overlap")
        table = (AdamwTensorC * len(params))()
        for i, p in enumerate(params):
            t = table[i]
            t.param, t.n = p.data_ptr(), p.numel()
            t.master = _ptr(master[i]) if master is not None else None
            if bits == 32:
                t.m, t.v = (k[i].data_ptr() for k in state)
            else:
                t.m, t.m_scale, t.v, t.v_scale = (k[i].data_ptr() for k in state)
        self._params, self._master, self._state = params, master, state
        self._bits, self._device, self._code = bits, dev, f.code[dt]
        self._shapes = [p.shape for p in params]
        # all of them with the addresses in the table, and the memory behind those: held, so that
        # an address that is still the same is still the same memory
        self._tensors, self._ptrs = held, [t.data_ptr() for t in held]
        self._held = _Held(held)
        # the table, and as words, for the column of gradient pointers
        self._t = table
        self._words = np.frombuffer(table, dtype=np.uint64).reshape(len(params), -1)

    def step(self, grads, grad_scale=None, stream=None):
        """One step with grads (contiguous, shaped like params, all float32 or all bfloat16).
        grad_scale, a float32 tensor of one element on the device, multiplies them (a clipping
        or unscaling factor, without a wait for the host)."""
        f = _lib()
        torch = f.torch
        T = torch.Tensor
        dev = self._device
        if _elsewhere(f, dev, stream):
            with _on(dev, stream, grad_scale, *grads):
                return self.step(grads, grad_scale)
        if list(map(T.data_ptr, self._tensors)) != self._ptrs:  # a storage was replaced
            self._bind(self._params, self._master, self._state)
        if len(grads) != len(self._params):
            raise ValueError("one gradient for each parameter is needed")
        gt = grads[0].dtype
        if gt not in (torch.float32, torch.bfloat16):
            raise ValueError("gradients must be float32 or bfloat16")
        if list(map(_SHAPE, grads)) != self._shapes or set(map(_DTYPE, grads)) != {gt} \
                or set(map(T.get_device, grads)) != {dev.index} \
                or not all(map(T.is_contiguous, grads)):
            raise ValueError(f"gradients must be contiguous {gt} tensors of their parameters' "
                             f"shapes on {dev}")
        if grad_scale is not None and (grad_scale.dtype != torch.float32
                                       or grad_scale.numel() != 1 or grad_scale.device != dev):
            raise ValueError(f"grad_scale must be one float32 element on {dev}")
        self._words[:, _GRAD_WORD] = list(map(T.data_ptr, grads))
        b1, b2 = self.betas
        hp = AdamwHyperC(self.lr, b1, b2, self.eps, self.weight_decay, self.steps + 1)
        s = f.stream(dev.index)
        self._held.used_on(f, dev, s)
        st = f.sffn_adamw_step(self._t, len(self._params), self._code, f.code[gt], self._bits,
                               ctypes.byref(hp), _ptr(grad_scale), s)
        if st:
            _fail(st, "sffn_adamw_step")
        self.steps += 1
