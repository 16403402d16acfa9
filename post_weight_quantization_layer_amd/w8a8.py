"""A layer stored at 8 bits per row, run as y = x W^T in 8-bit integers
(gptq_w8a8_* of gptq_run.h), with torch as the allocator.

The layer is what GptqLayer makes with ``bits`` up to 8 and ``group = cols``.
The classes own device buffers and sequence the native calls; they do no
arithmetic of their own."""
from __future__ import annotations

import torch

from . import binding_run as R


class TokenCodes:
    """Device buffers for activations as 8-bit codes with a scale and a code
    sum per token: up to ``tokens`` rows of ``cols`` features."""

    def __init__(self, tokens: int, cols: int, device="cuda", stream=None):
        device = R.on_gpu(device, "token codes")
        self.tokens, self.cols = tokens, cols
        with R.on(stream):
            self.codes = torch.empty((tokens, R.gptq_tokens_ld(cols)), dtype=torch.int8,
                                     device=device)
            self.scale = torch.empty(tokens, dtype=torch.float32, device=device)
            self.sum = torch.empty(tokens, dtype=torch.int32, device=device)

    def head(self, tokens: int) -> "TokenCodes":
        """The first ``tokens`` rows, on the same buffers."""
        if tokens == self.tokens:
            return self
        if not 0 <= tokens <= self.tokens:
            raise ValueError(f"{tokens} tokens asked of buffers for {self.tokens}")
        part = TokenCodes.__new__(TokenCodes)
        part.tokens, part.cols = tokens, self.cols
        part.codes, part.scale, part.sum = (self.codes[:tokens], self.scale[:tokens],
                                            self.sum[:tokens])
        return part

    def values(self) -> torch.Tensor:
        """What the codes stand for, tokens x cols float32."""
        return self.codes[:, :self.cols].float() * self.scale[:, None]


def _for(x: torch.Tensor, out: TokenCodes | None, stream) -> TokenCodes:
    if x.dim() != 2 or not x.is_cuda:
        raise ValueError("activations must be a tokens x features matrix on the GPU")
    tokens, cols = x.shape
    if out is None:
        return TokenCodes(tokens, cols, x.device, stream)
    if out.cols != cols:
        raise ValueError(f"buffers for {out.cols} features, got {cols}")
    return out.head(tokens)


def quantize_tokens(x: torch.Tensor, out: TokenCodes | None = None, stream=None) -> TokenCodes:
    """x (tokens x features) as codes: scale max|x| / 127 per token."""
    out = _for(x, out, stream)
    R.gptq_quantize_tokens(x, out.codes, out.scale, out.sum, stream)
    return out


def silu_mul_quantize(g: torch.Tensor, u: torch.Tensor, out: TokenCodes | None = None,
                      stream=None) -> TokenCodes:
    """silu(g) * u as codes; g and u may be the halves of one matrix."""
    out = _for(g, out, stream)
    R.gptq_silu_mul_quantize(g, u, out.codes, out.scale, out.sum, stream)
    return out


class W8A8Linear:
    """A prepared per-row 8-bit layer.  Calls on different streams may overlap:
    each stream has its own scratch memory.  Threads may share it and a stream."""

    def __init__(self, codes: torch.Tensor, scale: torch.Tensor, zero: torch.Tensor, stream=None):
        """codes rows x cols uint8; scale (float32) and zero (uint8) one per row."""
        if codes.dtype != torch.uint8 or not codes.is_contiguous():
            raise ValueError("codes must be a contiguous rows x cols uint8 matrix")
        R.matrix(codes, "codes")
        self.rows, self.cols = codes.shape
        R.vector(scale, "scale", self.rows, torch.float32)
        R.vector(zero, "zero", self.rows, torch.uint8)
        self.device = codes.device
        with R.on(stream):
            self.mem = torch.empty(R.gptq_w8a8_layer_bytes(self.rows, self.cols),
                                   dtype=torch.uint8, device=self.device)
        self.layer = R.gptq_w8a8_prepare(codes, scale, zero, self.mem, stream)
        self.scratch = R.Scratch(self.device)
        self._last: dict = {}

    @classmethod
    def from_quantized(cls, *layers, stream=None) -> "W8A8Linear":
        """From ``QuantizedLayer``s with one group per row; several are stacked
        (gate and up of a gated MLP as one product)."""
        for q in layers:
            if q.scale is None or q.scale.shape[1] != 1:
                raise ValueError("the 8-bit product takes layers with one scale per row "
                                 "(affine grid, group = cols)")
        with R.on(stream):
            return cls(torch.cat([q.q for q in layers]), torch.cat([q.scale for q in layers]),
                       torch.cat([q.zero for q in layers]), stream)

    def _new(self, tokens: int, dtype, stream) -> torch.Tensor:
        with R.on(stream):
            return torch.empty((tokens, self.rows), dtype=dtype, device=self.device)

    def _bytes(self, key: str, tokens: int) -> int:
        """Scratch of a call, looked up once per token count in a row."""
        last = self._last.get(key)
        if last is None or last[0] != tokens:
            last = (tokens, getattr(R, key)(self.layer, tokens))
            self._last[key] = last
        return last[1]

    def __call__(self, x: torch.Tensor, y: torch.Tensor | None = None, stream=None):
        """x tokens x cols -> y tokens x rows, of x's type unless ``y`` is given."""
        tokens = x.shape[0]
        if y is None:
            y = self._new(tokens, x.dtype, stream)
        n = self._bytes("gptq_w8a8_linear_ws_bytes", tokens)
        with self.scratch.lock:
            ws = self.scratch(n, self.mem, stream)
            R.gptq_w8a8_linear(self.layer, x, y, R.address(ws), n, stream)
        return y

    def product(self, tokens: TokenCodes, y: torch.Tensor | None = None,
                dtype: torch.dtype = torch.float16, stream=None):
        """Token codes -> y tokens x rows (of ``dtype`` unless ``y`` is given)."""
        t = tokens.tokens
        if tokens.cols != self.cols:
            raise ValueError(f"tokens of {tokens.cols} features, the layer takes {self.cols}")
        if y is None:
            y = self._new(t, dtype, stream)
        elif y.shape[0] != t:
            raise ValueError(f"y must have {t} rows, got {y.shape[0]}")
        n = self._bytes("gptq_w8a8_gemm_ws_bytes", t)
        with self.scratch.lock:
            ws = self.scratch(n, self.mem, stream)
            R.gptq_w8a8_gemm(self.layer, tokens.codes, tokens.scale, tokens.sum, y, R.address(ws),
                             n, stream)
        return y
