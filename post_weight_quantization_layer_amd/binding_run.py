"""ctypes binding of the calls of gptq_run.h (argument marshalling only), and
the buffers the classes on top of them share.

As in ``binding``: every function has the name of the C entry point it wraps,
tensors become device pointers, the current torch stream (or ``stream``) a
hipStream_t, a status that is not OK an exception.
"""
from __future__ import annotations

import contextlib
import ctypes
import threading

import torch

from . import binding as B

GPTQ_DT_F16 = 2
GPTQ_NORM_NONE, GPTQ_NORM_RMS, GPTQ_NORM_LAYER = range(3)
NORMS = {None: GPTQ_NORM_NONE, "none": GPTQ_NORM_NONE, "rms": GPTQ_NORM_RMS,
         "layer": GPTQ_NORM_LAYER}
DTYPES = {torch.float32: B.GPTQ_DT_F32, torch.bfloat16: B.GPTQ_DT_BF16,
          torch.float16: GPTQ_DT_F16}

EXPORTED = (
    "gptq_tokens_ld", "gptq_quantize_tokens", "gptq_silu_mul_quantize",
    "gptq_w8a8_layer_bytes", "gptq_w8a8_prepare", "gptq_w8a8_gemm_ws_bytes",
    "gptq_w8a8_linear_ws_bytes", "gptq_w8a8_gemm", "gptq_w8a8_linear",
    "gptq_norm_block", "gptq_gated_mlp_ws_bytes", "gptq_gated_mlp_forward",
    "gptq_token_logprobs_ws_bytes", "gptq_token_logprobs",
)


class gptq_w8a8_layer(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("rows_pad", ctypes.c_int64), ("k_pad", ctypes.c_int64),
                ("mem", ctypes.c_void_p), ("mem_bytes", ctypes.c_size_t)]


class gptq_norm_params(ctypes.Structure):
    _fields_ = [("post", ctypes.c_int32), ("pre", ctypes.c_int32), ("w_dtype", ctypes.c_int32),
                ("eps", ctypes.c_float), ("weight_offset", ctypes.c_float),
                ("residual_scale", ctypes.c_float), ("block_scale", ctypes.c_float),
                ("post_weight", ctypes.c_void_p), ("post_bias", ctypes.c_void_p),
                ("pre_weight", ctypes.c_void_p), ("pre_bias", ctypes.c_void_p)]


class gptq_gated_mlp(ctypes.Structure):
    _fields_ = [("enter", gptq_norm_params), ("leave", gptq_norm_params),
                ("gate_up", gptq_w8a8_layer), ("down", gptq_w8a8_layer)]


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is not None:
        return _lib
    L = B.lib()
    P, I64, I32, SZ, F = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t,
                          ctypes.c_float)
    layer = ctypes.POINTER(gptq_w8a8_layer)
    for name, res, args in (
            ("gptq_tokens_ld", I64, [I64]),
            ("gptq_quantize_tokens", I32, [P, I32, I64, I64, I64, P, I64, P, P, P]),
            ("gptq_silu_mul_quantize", I32, [P, P, I32, I64, I64, I64, P, I64, P, P, P]),
            ("gptq_w8a8_layer_bytes", SZ, [I64, I64]),
            ("gptq_w8a8_prepare", I32, [P, P, P, I64, I64, P, SZ, layer, P]),
            ("gptq_w8a8_gemm_ws_bytes", SZ, [layer, I64]),
            ("gptq_w8a8_linear_ws_bytes", SZ, [layer, I64]),
            ("gptq_w8a8_gemm", I32, [layer, P, I64, P, P, I64, P, I32, I64, P, SZ, P]),
            ("gptq_w8a8_linear", I32, [layer, P, I32, I64, I64, P, I32, I64, P, SZ, P]),
            ("gptq_norm_block", I32, [ctypes.POINTER(gptq_norm_params), I32, I64, I64, P, I64, P,
                                      I64, P, I64, I64, P, I64, P, I64, P, I64, P, P, P]),
            ("gptq_gated_mlp_ws_bytes", SZ, [ctypes.POINTER(gptq_gated_mlp), I32, I64]),
            ("gptq_gated_mlp_forward", I32, [ctypes.POINTER(gptq_gated_mlp), I32, I64, P, I64, P,
                                             I64, I64, P, I64, P, I64, P, SZ, P]),
            ("gptq_token_logprobs_ws_bytes", SZ, [I64, I64, I32]),
            ("gptq_token_logprobs", I32, [P, I32, I64, I64, I64, P, F, I32, P, P, P, P, P, P, SZ,
                                          P])):
        f = getattr(L, name)
        f.restype, f.argtypes = res, args
    _lib = L
    return L


def _check(status: int):
    if status != B.GPTQ_OK:
        B._check(status)


def _dtype(t: torch.Tensor, what: str) -> int:
    try:
        return DTYPES[t.dtype]
    except KeyError:
        raise TypeError(f"{what} must be float32, bfloat16 or float16, not {t.dtype}") from None


def stream_ptr(t: torch.Tensor, stream=None) -> int:
    """hipStream_t of ``stream``, or of the current stream of t's device."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(t.get_device())
    return getattr(stream, "cuda_stream", stream)


def matrix(t: torch.Tensor, what: str, rows: int | None = None, cols: int | None = None,
           dtype: torch.dtype | None = None) -> tuple[int, int]:
    """(address, row stride) of a device matrix whose rows are contiguous, of the
    given size and type where one is given."""
    if t.is_contiguous() and t.dim() == 2:
        r, c = t.shape
        if (rows is None or r == rows) and (cols is None or c == cols) and t.is_cuda and \
                (dtype is None or t.dtype is dtype):
            return t.data_ptr(), c
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (stride[1] != 1 and shape[1] > 1 and shape[0] > 0):
        raise ValueError(f"{what} must be a matrix with contiguous rows, got shape "
                         f"{tuple(shape)} and strides {stride}")
    r, c = shape
    if (rows is not None and r != rows) or (cols is not None and c != cols):
        raise ValueError(f"{what} must be {'*' if rows is None else rows} x "
                         f"{'*' if cols is None else cols}, got {tuple(shape)}")
    if not t.is_cuda:
        raise ValueError(f"{what} must be on the GPU")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}, not {t.dtype}")
    return t.data_ptr(), stride[0] if r > 1 else c    # torch may report any for one row or none


def on_gpu(device, what: str) -> torch.device:
    """The device of buffers that kernels write."""
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError(f"{what} must be on the GPU, not on {device}")
    return device


def ld(t: torch.Tensor) -> int:
    """Row stride; a single row's is its length (torch may report any)."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def vector(t: torch.Tensor, what: str, n: int, dtype: torch.dtype | None = None):
    if t.numel() != n or not t.is_contiguous() or not t.is_cuda or \
            (dtype is not None and t.dtype != dtype):
        raise ValueError(f"{what} must be {n} contiguous values on the GPU"
                         + (f" of {dtype}" if dtype is not None else ""))
    return t


_CURRENT = contextlib.nullcontext()


def on(stream):
    """Allocations inside belong to ``stream`` (None: the current one)."""
    if stream is None:
        return _CURRENT
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream)
                             else torch.cuda.ExternalStream(stream))


def capturing(stream=None) -> bool:
    """Whether ``stream`` (None: the current one) is being captured into a graph."""
    if stream is None:
        return torch._C._cuda_isCurrentStreamCapturing()
    with on(stream):
        return torch._C._cuda_isCurrentStreamCapturing()


class Scratch:
    """Workspace of an object, one per stream that uses it, so that calls on
    several streams do not share one; grows to the largest request.

    A call that is being captured gets a buffer of its own, from the graph's
    pool: the graph may be replayed after a larger call has replaced the stream's
    buffer, or beside a call that uses it.

    ``lock`` is held from asking for a buffer until the launches that use it are
    issued, so that threads on one stream share its buffer call by call."""

    def __init__(self, device):
        self.device = device
        self.lock = threading.Lock()
        self._by_stream: dict[int, torch.Tensor] = {}

    def __reduce__(self):
        return Scratch, (self.device,)      # a copy has a lock and buffers of its own

    def __call__(self, nbytes: int, like: torch.Tensor, stream=None) -> torch.Tensor | None:
        """At least ``nbytes`` bytes for one call on ``stream`` (None: the current
        stream of ``like``'s device), to be held, like ``lock``, until its launches
        are issued."""
        if nbytes == 0:
            return None
        if capturing(stream):
            return self._new(nbytes, stream)
        ptr = stream_ptr(like, stream)
        t = self._by_stream.get(ptr)
        if t is None or t.numel() < nbytes:
            t = self._by_stream[ptr] = self._new(nbytes, stream)
        return t

    def _new(self, nbytes: int, stream) -> torch.Tensor:
        with on(stream):
            return torch.empty(nbytes, dtype=torch.uint8, device=self.device)


def address(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def gptq_tokens_ld(cols: int) -> int:
    n = lib().gptq_tokens_ld(cols)
    if n == 0:
        raise B.GptqError(B.GPTQ_ERR_INVALID_ARG, "cols must be in [1, 65536]")
    return n


def gptq_quantize_tokens(x, codes, scale, sum, stream=None):
    """x tokens x cols float; codes tokens x ld int8; scale, sum: tokens float32 / int32."""
    ptr, stride = matrix(x, "x")
    _check(lib().gptq_quantize_tokens(ptr, _dtype(x, "x"), *x.shape, stride, codes.data_ptr(),
                                      ld(codes), scale.data_ptr(), sum.data_ptr(),
                                      stream_ptr(x, stream)))


def gptq_silu_mul_quantize(g, u, codes, scale, sum, stream=None):
    """g, u tokens x cols of one type and row stride."""
    ptr, stride = matrix(g, "g")
    uptr, ustride = matrix(u, "u", *g.shape, g.dtype)
    if ustride != stride:
        raise ValueError("g and u must have one row stride")
    _check(lib().gptq_silu_mul_quantize(ptr, uptr, _dtype(g, "g"), *g.shape, stride,
                                        codes.data_ptr(), ld(codes), scale.data_ptr(),
                                        sum.data_ptr(), stream_ptr(g, stream)))


def gptq_w8a8_layer_bytes(rows: int, cols: int) -> int:
    n = lib().gptq_w8a8_layer_bytes(rows, cols)
    if n == 0:
        raise B.GptqError(B.GPTQ_ERR_INVALID_ARG,
                          "rows and cols must be in [1, 2^24] x [1, 65536], padded at most 2^35")
    return n


def gptq_w8a8_prepare(q, scale, zero, mem, stream=None) -> gptq_w8a8_layer:
    """``mem`` must stay alive as long as the returned layer is used."""
    rows, cols = q.shape
    layer = gptq_w8a8_layer()
    _check(lib().gptq_w8a8_prepare(q.data_ptr(), scale.data_ptr(), zero.data_ptr(), rows, cols,
                                   mem.data_ptr(), mem.numel() * mem.element_size(),
                                   ctypes.byref(layer), stream_ptr(q, stream)))
    return layer


def gptq_w8a8_gemm_ws_bytes(layer: gptq_w8a8_layer, tokens: int) -> int:
    return lib().gptq_w8a8_gemm_ws_bytes(layer, tokens)


def gptq_w8a8_linear_ws_bytes(layer: gptq_w8a8_layer, tokens: int) -> int:
    return lib().gptq_w8a8_linear_ws_bytes(layer, tokens)


def gptq_w8a8_gemm(layer: gptq_w8a8_layer, codes, scale, sum, y, ws: int | None = None,
                   ws_bytes: int = 0, stream=None):
    """codes, scale, sum of y's tokens; y tokens x rows.  ``ws``: address."""
    ptr, stride = matrix(y, "y", None, layer.rows)
    _check(lib().gptq_w8a8_gemm(layer, codes.data_ptr(), ld(codes), scale.data_ptr(),
                                sum.data_ptr(), y.shape[0], ptr, _dtype(y, "y"), stride, ws,
                                ws_bytes, stream_ptr(y, stream)))


def gptq_w8a8_linear(layer: gptq_w8a8_layer, x, y, ws: int | None = None, ws_bytes: int = 0,
                     stream=None):
    """x tokens x cols, y tokens x rows.  ``ws``: address."""
    ptr, stride = matrix(x, "x", None, layer.cols)
    tokens = x.shape[0]
    yptr, ystride = matrix(y, "y", tokens, layer.rows)
    _check(lib().gptq_w8a8_linear(layer, ptr, _dtype(x, "x"), stride, tokens, yptr,
                                  _dtype(y, "y"), ystride, ws, ws_bytes, stream_ptr(x, stream)))


_NONE = (None, 0)


def like(t: torch.Tensor | None, what: str, shape: torch.Size, dtype: torch.dtype):
    """matrix() of a tensor that has to be like another; of None: (None, 0)."""
    if t is None:
        return _NONE
    if t.shape == shape and t.is_contiguous() and t.dtype is dtype and t.is_cuda:
        return t.data_ptr(), shape[1]
    return matrix(t, what, *shape, dtype)


def gptq_norm_block(params: gptq_norm_params, r, b=None, gate=None, gate_tokens: int = 1,
                    r_out=None, h=None, codes=None, scale=None, sum=None, stream=None):
    ptr, stride = matrix(r, "r")
    shape, kind = r.shape, r.dtype
    gptr, gstride = _NONE if gate is None else matrix(gate, "gate", None, shape[1], kind)
    bptr, bstride = like(b, "b", shape, kind)
    optr, ostride = like(r_out, "r_out", shape, kind)
    hptr, hstride = like(h, "h", shape, kind)
    c = s = n = None
    ldc = 0
    if codes is not None:
        c, ldc, s, n = codes.data_ptr(), ld(codes), scale.data_ptr(), sum.data_ptr()
    _check((_lib or lib()).gptq_norm_block(
        params, _dtype(r, "r"), *shape, ptr, stride, bptr, bstride, gptr, gstride, gate_tokens,
        optr, ostride, hptr, hstride, c, ldc, s, n, stream_ptr(r, stream)))


def gptq_gated_mlp_ws_bytes(mlp: gptq_gated_mlp, dtype: torch.dtype, tokens: int) -> int:
    return lib().gptq_gated_mlp_ws_bytes(mlp, DTYPES[dtype], tokens)


def gptq_gated_mlp_forward(mlp: gptq_gated_mlp, r, gate=None, gate_tokens: int = 1, r_out=None,
                           h=None, ws: int | None = None, ws_bytes: int = 0, stream=None):
    """``ws``: address."""
    kind = r.dtype
    d = mlp.down.rows
    ptr, stride = matrix(r, "r", None, d)
    shape = r.shape
    _check(lib().gptq_gated_mlp_forward(
        mlp, _dtype(r, "r"), shape[0], ptr, stride,
        *(_NONE if gate is None else matrix(gate, "gate", None, d, kind)), gate_tokens,
        *like(r_out, "r_out", shape, kind), *like(h, "h", shape, kind),
        ws, ws_bytes, stream_ptr(r, stream)))


def gptq_token_logprobs_ws_bytes(rows: int, vocab: int, top_k: int) -> int:
    return lib().gptq_token_logprobs_ws_bytes(rows, vocab, top_k)


def gptq_token_logprobs(logits, ids, scale, top_k, logprob, rank, entropy, top_ids=None,
                        top_logprobs=None, ws: int | None = None, ws_bytes: int = 0, stream=None):
    """``ws``: address."""
    ptr, stride = matrix(logits, "logits")
    _check(lib().gptq_token_logprobs(
        ptr, _dtype(logits, "logits"), *logits.shape, stride, B._ptr(ids), scale, top_k,
        B._ptr(logprob), B._ptr(rank), B._ptr(entropy), B._ptr(top_ids), B._ptr(top_logprobs),
        ws, ws_bytes, stream_ptr(logits, stream)))
