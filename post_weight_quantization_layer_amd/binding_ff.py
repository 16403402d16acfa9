"""ctypes binding of the calls of gptq_ff.h (argument marshalling only).

As in ``binding_run``: every function has the name of the C entry point it
wraps, tensors become device pointers, the current torch stream of their device
(or ``stream``) a hipStream_t, a status that is not OK an exception."""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import binding as B
from . import binding_run as R

EXPORTED = (
    "gptq_f8_quantize_tokens", "gptq_f8_quantize_weight", "gptq_f8_layer_bytes",
    "gptq_f8_prepare", "gptq_f8_gemm_ws_bytes", "gptq_f8_linear_ws_bytes", "gptq_f8_gemm",
    "gptq_f8_linear", "gptq_f8_ff_ws_bytes", "gptq_f8_ff_forward", "gptq_ff_saved_bytes",
    "gptq_ff_forward_ws_bytes", "gptq_ff_backward_ws_bytes", "gptq_ff_forward",
    "gptq_ff_backward",
)


class gptq_f8_layer(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("rows_pad", ctypes.c_int64), ("k_pad", ctypes.c_int64),
                ("mem", ctypes.c_void_p), ("mem_bytes", ctypes.c_size_t)]


class gptq_f8_ff(ctypes.Structure):
    _fields_ = [("gate", gptq_f8_layer), ("up", gptq_f8_layer), ("down", gptq_f8_layer)]


class gptq_ff(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int64), ("inner", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("gate", ctypes.c_void_p), ("up", ctypes.c_void_p), ("down", ctypes.c_void_p),
                ("ld_gate", ctypes.c_int64), ("ld_up", ctypes.c_int64),
                ("ld_down", ctypes.c_int64)]


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is not None:
        return _lib
    L = B.lib()
    P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    layer, f8, ff = (ctypes.POINTER(t) for t in (gptq_f8_layer, gptq_f8_ff, gptq_ff))
    for name, res, args in (
            ("gptq_f8_quantize_tokens", I32, [P, I32, I64, I64, I64, P, I64, P, I64, P]),
            ("gptq_f8_quantize_weight", I32, [P, I32, I64, I64, I64, P, P, P]),
            ("gptq_f8_layer_bytes", SZ, [I64, I64]),
            ("gptq_f8_prepare", I32, [P, P, I64, I64, P, SZ, layer, P]),
            ("gptq_f8_gemm_ws_bytes", SZ, [layer, I64]),
            ("gptq_f8_linear_ws_bytes", SZ, [layer, I64]),
            ("gptq_f8_gemm", I32, [layer, P, I64, P, I64, I64, P, I32, I64, P, SZ, P]),
            ("gptq_f8_linear", I32, [layer, P, I32, I64, I64, P, I32, I64, P, SZ, P]),
            ("gptq_f8_ff_ws_bytes", SZ, [f8, I64]),
            ("gptq_f8_ff_forward", I32, [f8, P, I32, I64, I64, P, I32, I64, P, SZ, P]),
            ("gptq_ff_saved_bytes", SZ, [ff, I64]),
            ("gptq_ff_forward_ws_bytes", SZ, [ff, I64]),
            ("gptq_ff_backward_ws_bytes", SZ, [ff, I64]),
            ("gptq_ff_forward", I32, [ff, P, I64, I64, P, I64, P, SZ, P, SZ, P]),
            ("gptq_ff_backward", I32, [ff, P, I64, I64, P, SZ, P, I64, P, I64, P, I64, P, I64, P,
                                       I64, P, SZ, P])):
        f = getattr(L, name)
        f.restype, f.argtypes = res, args
    _lib = L
    return L


_CURRENT = contextlib.nullcontext()


def on_device(t: torch.Tensor):
    """The calls inside launch on t's device."""
    if t.get_device() == torch.cuda.current_device():
        return _CURRENT
    return torch.cuda.device(t.get_device())


def on_index(device: torch.device):
    """The same for a device; "cuda" is the current one."""
    return _CURRENT if device.index is None else torch.cuda.device(device)


def one_device(*tensors: torch.Tensor):
    device = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != device:
            raise ValueError("all tensors of a call must be on one device")


def gptq_f8_quantize_tokens(x, codes, scale, stream=None):
    """x tokens x cols float; codes tokens x ld uint8; scale blocks x tokens (or more) float32."""
    ptr, stride = R.matrix(x, "x")
    tokens, cols = x.shape
    R._check(lib().gptq_f8_quantize_tokens(ptr, R._dtype(x, "x"), tokens, cols, stride,
                                           codes.data_ptr(), R.ld(codes), scale.data_ptr(),
                                           R.ld(scale), R.stream_ptr(x, stream)))


def gptq_f8_quantize_weight(w, codes, scale, stream=None):
    """w rows x cols float; codes rows x cols, scale a value per 128 x 128 block."""
    ptr, stride = R.matrix(w, "w")
    R._check(lib().gptq_f8_quantize_weight(ptr, R._dtype(w, "w"), *w.shape, stride,
                                           codes.data_ptr(), scale.data_ptr(),
                                           R.stream_ptr(w, stream)))


def gptq_f8_layer_bytes(rows: int, cols: int) -> int:
    n = lib().gptq_f8_layer_bytes(rows, cols)
    if n == 0:
        raise B.GptqError(B.GPTQ_ERR_INVALID_ARG,
                          "rows and cols must be in [1, 2^24] x [1, 65536], padded at most 2^35")
    return n


def gptq_f8_prepare(codes, scale, mem, stream=None) -> gptq_f8_layer:
    """``mem`` must stay alive as long as the returned layer is used."""
    layer = gptq_f8_layer()
    R._check(lib().gptq_f8_prepare(codes.data_ptr(), scale.data_ptr(), *codes.shape,
                                   mem.data_ptr(), mem.numel() * mem.element_size(),
                                   ctypes.byref(layer), R.stream_ptr(codes, stream)))
    return layer


def gptq_f8_gemm_ws_bytes(layer: gptq_f8_layer, tokens: int) -> int:
    return lib().gptq_f8_gemm_ws_bytes(layer, tokens)


def gptq_f8_linear_ws_bytes(layer: gptq_f8_layer, tokens: int) -> int:
    return lib().gptq_f8_linear_ws_bytes(layer, tokens)


def gptq_f8_gemm(layer: gptq_f8_layer, codes, scale, y, ws: int | None = None, ws_bytes: int = 0,
                 stream=None):
    """codes, scale of y's tokens; y tokens x rows.  ``ws``: address."""
    ptr, stride = R.matrix(y, "y", None, layer.rows)
    R._check(lib().gptq_f8_gemm(layer, codes.data_ptr(), R.ld(codes), scale.data_ptr(),
                                R.ld(scale), y.shape[0], ptr, R._dtype(y, "y"), stride, ws,
                                ws_bytes, R.stream_ptr(y, stream)))


def gptq_f8_linear(layer: gptq_f8_layer, x, y, ws: int | None = None, ws_bytes: int = 0,
                   stream=None):
    """x tokens x cols, y tokens x rows.  ``ws``: address."""
    ptr, stride = R.matrix(x, "x", None, layer.cols)
    tokens = x.shape[0]
    yptr, ystride = R.matrix(y, "y", tokens, layer.rows)
    R._check(lib().gptq_f8_linear(layer, ptr, R._dtype(x, "x"), stride, tokens, yptr,
                                  R._dtype(y, "y"), ystride, ws, ws_bytes,
                                  R.stream_ptr(x, stream)))


def gptq_f8_ff_ws_bytes(ff: gptq_f8_ff, tokens: int) -> int:
    return lib().gptq_f8_ff_ws_bytes(ff, tokens)


def gptq_f8_ff_forward(ff: gptq_f8_ff, x, y, ws: int | None = None, ws_bytes: int = 0,
                       stream=None):
    """x, y tokens x d.  ``ws``: address."""
    d = ff.down.rows
    ptr, stride = R.matrix(x, "x", None, d)
    tokens = x.shape[0]
    yptr, ystride = R.matrix(y, "y", tokens, d)
    R._check(lib().gptq_f8_ff_forward(ff, ptr, R._dtype(x, "x"), stride, tokens, yptr,
                                      R._dtype(y, "y"), ystride, ws, ws_bytes,
                                      R.stream_ptr(x, stream)))


_KINDS = {code: kind for kind, code in R.DTYPES.items()}


def make_ff(gate, up, down) -> gptq_ff:
    """The weights of a block: gate and up inner x d, down d x inner, of one type."""
    gptr, gld = R.matrix(gate, "gate")
    inner, d = gate.shape
    uptr, uld = R.matrix(up, "up", inner, d, gate.dtype)
    dptr, dld = R.matrix(down, "down", d, inner, gate.dtype)
    return gptq_ff(d, inner, R._dtype(gate, "gate"), gptr, uptr, dptr, gld, uld, dld)


def gptq_ff_saved_bytes(ff: gptq_ff, tokens: int) -> int:
    return lib().gptq_ff_saved_bytes(ff, tokens)


def gptq_ff_forward_ws_bytes(ff: gptq_ff, tokens: int) -> int:
    return lib().gptq_ff_forward_ws_bytes(ff, tokens)


def gptq_ff_backward_ws_bytes(ff: gptq_ff, tokens: int) -> int:
    return lib().gptq_ff_backward_ws_bytes(ff, tokens)


def gptq_ff_forward(ff: gptq_ff, x, y, saved=None, ws=None, stream=None):
    """x tokens x d, of the weights' type; y a new tokens x d matrix; saved, ws: byte tensors or
    None."""
    ptr, stride = R.matrix(x, "x", None, ff.d, _KINDS[ff.dtype])
    R._check((_lib or lib()).gptq_ff_forward(
        ff, ptr, stride, x.shape[0], y.data_ptr(), ff.d, R.address(saved),
        0 if saved is None else saved.numel(), R.address(ws), 0 if ws is None else ws.numel(),
        R.stream_ptr(x, stream)))


def gptq_ff_backward(ff: gptq_ff, x, saved, dy, dx=None, dgate=None, dup=None, ddown=None,
                     ws=None, stream=None):
    """x, dy of the weights' type; dx, dgate, dup, ddown: new matrices to write, or None."""
    ptr, stride = R.matrix(x, "x", None, ff.d, _KINDS[ff.dtype])
    dptr, dstride = R.matrix(dy, "dy", x.shape[0], ff.d, x.dtype)
    d, inner, at = ff.d, ff.inner, R.address
    R._check((_lib or lib()).gptq_ff_backward(
        ff, ptr, stride, x.shape[0], at(saved), 0 if saved is None else saved.numel(), dptr,
        dstride, at(dx), d, at(dgate), d, at(dup), d, at(ddown), inner, at(ws),
        0 if ws is None else ws.numel(), R.stream_ptr(x, stream)))
