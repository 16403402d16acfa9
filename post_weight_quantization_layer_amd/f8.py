"""A layer of 8-bit floats (e4m3) with a scale per block of 128 x 128 weights, run
as y = x W^T on activations quantized per token and 128 features (gptq_f8_* of
gptq_ff.h), with torch as the allocator.

Unlike the per-row integer layers of ``w8a8`` such a layer needs no calibration:
``F8Linear.from_weight`` rounds a weight as it is.  The classes own device
buffers and sequence the native calls; they do no arithmetic of their own."""
from __future__ import annotations

import torch

from . import binding_ff as F
from . import binding_run as R

BLOCK = 128


def blocks(n: int) -> int:
    return -(-n // BLOCK)


class F8Tokens:
    """Device buffers for activations as 8-bit floats with a scale per block of 128
    features: up to ``tokens`` rows of ``cols`` features."""

    def __init__(self, tokens: int, cols: int, device="cuda", stream=None):
        device = R.on_gpu(device, "token codes")
        self.tokens, self.cols = tokens, cols
        with F.on_index(device), R.on(stream):
            self.codes = torch.empty((tokens, R.gptq_tokens_ld(cols)), dtype=torch.uint8,
                                     device=device)
            self.scale = torch.empty((blocks(cols), tokens), dtype=torch.float32, device=device)

    def values(self) -> torch.Tensor:
        """What the codes stand for, tokens x cols float32."""
        scale = self.scale.t().repeat_interleave(BLOCK, 1)[:, :self.cols]
        return self.codes.view(torch.float8_e4m3fn)[:, :self.cols].float() * scale


def quantize_tokens(x: torch.Tensor, out: F8Tokens | None = None, stream=None) -> F8Tokens:
    """x (tokens x features) as codes: scale max(2^-100, max|x|) / 448 per token and block."""
    if x.dim() != 2 or not x.is_cuda:
        raise ValueError("activations must be a tokens x features matrix on the GPU")
    tokens, cols = x.shape
    if out is None:
        out = F8Tokens(tokens, cols, x.device, stream)
    elif (out.tokens, out.cols) != (tokens, cols):
        raise ValueError(f"buffers for {out.tokens} x {out.cols}, got {tokens} x {cols}")
    F.one_device(x, out.codes)
    with F.on_device(x):
        F.gptq_f8_quantize_tokens(x, out.codes, out.scale, stream)
    return out


def quantize_weight(w: torch.Tensor, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """w (rows x cols) as (codes float8_e4m3fn, scale float32 per 128 x 128 block)."""
    if w.dim() != 2 or not w.is_cuda:
        raise ValueError("a weight must be a rows x cols matrix on the GPU")
    rows, cols = w.shape
    with F.on_device(w):
        with R.on(stream):
            codes = torch.empty((rows, cols), dtype=torch.uint8, device=w.device)
            scale = torch.empty((blocks(rows), blocks(cols)), dtype=torch.float32,
                                device=w.device)
        F.gptq_f8_quantize_weight(w, codes, scale, stream)
    return codes.view(torch.float8_e4m3fn), scale


class F8Linear:
    """A prepared layer.  Calls on different streams may overlap: each stream has its
    own scratch memory.  Threads may share it and a stream."""

    def __init__(self, codes: torch.Tensor, scale: torch.Tensor, stream=None):
        """codes rows x cols float8_e4m3fn (or its bytes, uint8); scale float32, one per
        128 x 128 block: ceil(rows / 128) x ceil(cols / 128)."""
        if codes.dtype not in (torch.float8_e4m3fn, torch.uint8) or codes.dim() != 2 or \
                not codes.is_contiguous():
            raise ValueError("codes must be a contiguous rows x cols float8_e4m3fn matrix")
        R.matrix(codes, "codes")
        self.rows, self.cols = codes.shape
        R.vector(scale, "scale", blocks(self.rows) * blocks(self.cols), torch.float32)
        if scale.shape != (blocks(self.rows), blocks(self.cols)):
            raise ValueError(f"scale must be {blocks(self.rows)} x {blocks(self.cols)}, "
                             f"got {tuple(scale.shape)}")
        F.one_device(codes, scale)
        self.device = codes.device
        with F.on_device(codes):
            with R.on(stream):
                self.mem = torch.empty(F.gptq_f8_layer_bytes(self.rows, self.cols),
                                       dtype=torch.uint8, device=self.device)
            self.layer = F.gptq_f8_prepare(codes, scale, self.mem, stream)
        self.scratch = R.Scratch(self.device)
        self._last: dict = {}

    @classmethod
    def from_weight(cls, w: torch.Tensor, stream=None) -> "F8Linear":
        """From a float weight (rows x cols), rounded to nearest block by block."""
        codes, scale = quantize_weight(w, stream)
        return cls(codes, scale, stream)

    def _new(self, tokens: int, dtype, stream) -> torch.Tensor:
        with R.on(stream):
            return torch.empty((tokens, self.rows), dtype=dtype, device=self.device)

    def _bytes(self, key: str, tokens: int) -> int:
        """Scratch of a call, looked up once per token count in a row."""
        last = self._last.get(key)
        if last is None or last[0] != tokens:
            last = (tokens, getattr(F, key)(self.layer, tokens))
            self._last[key] = last
        return last[1]

    def __call__(self, x: torch.Tensor, y: torch.Tensor | None = None,
                 dtype: torch.dtype | None = None, stream=None):
        """x tokens x cols -> y tokens x rows, float16 or bfloat16: ``dtype``, or x's type."""
        R.matrix(x, "x", None, self.cols)
        tokens = x.shape[0]
        with F.on_device(self.mem):
            if y is None:
                y = self._new(tokens, dtype or x.dtype, stream)
            F.one_device(self.mem, x, y)
            n = self._bytes("gptq_f8_linear_ws_bytes", tokens)
            with self.scratch.lock:
                ws = self.scratch(n, self.mem, stream)
                F.gptq_f8_linear(self.layer, x, y, R.address(ws), n, stream)
        return y

    def product(self, tokens: F8Tokens, y: torch.Tensor | None = None,
                dtype: torch.dtype = torch.float16, stream=None):
        """Token codes -> y tokens x rows (of ``dtype`` unless ``y`` is given)."""
        t = tokens.tokens
        if tokens.cols != self.cols:
            raise ValueError(f"tokens of {tokens.cols} features, the layer takes {self.cols}")
        with F.on_device(self.mem):
            if y is None:
                y = self._new(t, dtype, stream)
            elif y.shape[0] != t:
                raise ValueError(f"y must have {t} rows, got {y.shape[0]}")
            F.one_device(self.mem, tokens.codes, y)
            n = self._bytes("gptq_f8_gemm_ws_bytes", t)
            with self.scratch.lock:
                ws = self.scratch(n, self.mem, stream)
                F.gptq_f8_gemm(self.layer, tokens.codes, tokens.scale, y, R.address(ws), n, stream)
        return y
