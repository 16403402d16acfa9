"""A gated MLP block on per-row 8-bit layers: the blocks GatedMLPCalibrator
quantizes, run on token codes.

    codes(N_pre(r)) -> gate|up product -> codes(silu(g) u) -> down product b
    -> r' = alpha r + beta gate * N_post(b),  h = the next block's N_pre(r')

Five launches; only g|u and b are stored in the stream's type."""
from __future__ import annotations

import torch

from .norms import NormBlock
from .w8a8 import TokenCodes, W8A8Linear, silu_mul_quantize


class GatedMLP8:
    """``enter``: the NormBlock before the block; ``gate_up``: gate and up
    stacked along the rows; ``leave``: the NormBlock after it (its ``pre`` norm
    is the next block's)."""

    def __init__(self, enter: NormBlock, gate_up: W8A8Linear, down: W8A8Linear,
                 leave: NormBlock):
        if gate_up.rows != 2 * down.cols:
            raise ValueError("gate_up must hold gate and up: twice down's input features")
        if not enter.d == gate_up.cols == down.rows == leave.d:
            raise ValueError("the norms, gate_up's inputs and down's outputs must agree in width")
        self.enter, self.gate_up, self.down, self.leave = enter, gate_up, down, leave
        self.d, self.inner = down.rows, down.cols
        self._buffers: dict = {}

    def buffers(self, tokens: int, dtype: torch.dtype, device, key: int):
        """Activations of up to ``tokens`` tokens, one set per stream and type."""
        kept = self._buffers.get((key, dtype))
        if kept is None or kept[0].tokens < tokens:
            def empty(cols):
                return torch.empty((tokens, cols), dtype=dtype, device=device)
            kept = (TokenCodes(tokens, self.d, device), empty(2 * self.inner),
                    TokenCodes(tokens, self.inner, device), empty(self.d), empty(self.d),
                    empty(self.d))
            self._buffers[(key, dtype)] = kept
        x, gu, a, b, r_out, h = kept
        if x.tokens == tokens:
            return kept
        return (x.head(tokens), gu[:tokens], a.head(tokens), b[:tokens], r_out[:tokens],
                h[:tokens])

    def __call__(self, r: torch.Tensor, *, gate=None, gate_tokens: int | None = None):
        """r: tokens x d, on the current stream.  Returns (r', h), which the next
        call on this stream overwrites."""
        key = torch.cuda.current_stream().cuda_stream
        x, gu, a, b, r_out, h = self.buffers(r.shape[0], r.dtype, r.device, key)
        self.enter(r, codes=x)
        self.gate_up.product(x, gu)
        silu_mul_quantize(gu[:, :self.inner], gu[:, self.inner:], a)
        self.down.product(a, b)
        return self.leave(r, b, gate=gate, gate_tokens=gate_tokens, r_out=r_out, h=h)
