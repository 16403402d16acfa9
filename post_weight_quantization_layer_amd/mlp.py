"""A gated MLP block on per-row 8-bit layers: the blocks GatedMLPCalibrator
quantizes, run on token codes (gptq_gated_mlp_forward of gptq_run.h).

    codes(N_pre(r)) -> gate|up product -> codes(silu(g) u) -> down product b
    -> r' = alpha r + beta gate * N_post(b),  h = the next block's N_pre(r')

Five launches from one call; only g|u and b are stored in the stream's type."""
from __future__ import annotations

import torch

from . import binding_run as R
from .norms import NormBlock, tokens_per_gate
from .w8a8 import W8A8Linear


class GatedMLP8:
    """``enter``: the NormBlock before the block; ``gate_up``: gate and up
    stacked along the rows; ``leave``: the NormBlock after it (its ``pre`` norm
    is the next block's).  Calls on different streams may overlap: each stream
    has its own scratch memory.  Threads may share it and a stream."""

    def __init__(self, enter: NormBlock, gate_up: W8A8Linear, down: W8A8Linear,
                 leave: NormBlock):
        if gate_up.rows != 2 * down.cols:
            raise ValueError("gate_up must hold gate and up: twice down's input features")
        if not enter.d == gate_up.cols == down.rows == leave.d:
            raise ValueError("the norms, gate_up's inputs and down's outputs must agree in width")
        self.enter, self.gate_up, self.down, self.leave = enter, gate_up, down, leave  # kept alive
        self.d, self.inner = down.rows, down.cols
        self.block = R.gptq_gated_mlp(enter.params, leave.params, gate_up.layer, down.layer)
        self.scratch = R.Scratch(down.device)
        self._last = (-1, None, 0)      # tokens, type, scratch bytes

    def __call__(self, r: torch.Tensor, *, gate=None, gate_tokens: int | None = None,
                 r_out: torch.Tensor | None = None, h: torch.Tensor | None = None, stream=None):
        """r: tokens x d; gate as for ``leave``.  Returns (r', h): ``r_out`` (which
        may be r) and ``h``, or new tensors."""
        if r.dim() != 2 or r.shape[1] != self.d:
            raise ValueError(f"r must be tokens x {self.d}, got {tuple(r.shape)}")
        if not r.is_cuda:
            raise ValueError("r must be on the GPU")
        R._dtype(r, "r")
        t = r.shape[0]
        gate_tokens = 1 if gate is None else tokens_per_gate(gate, gate_tokens, t)
        last = self._last
        if last[0] != t or last[1] is not r.dtype:
            last = self._last = (t, r.dtype, R.gptq_gated_mlp_ws_bytes(self.block, r.dtype, t))
        n = last[2]
        if r_out is None or h is None:
            with R.on(stream):
                r_out = torch.empty_like(r) if r_out is None else r_out
                h = torch.empty_like(r) if h is None else h
        with self.scratch.lock:
            # the struct holds copies: what the norms say now counts
            self.block.enter, self.block.leave = self.enter.params, self.leave.params
            ws = self.scratch(n, r, stream)
            R.gptq_gated_mlp_forward(self.block, r, gate, gate_tokens, r_out, h, R.address(ws), n,
                                     stream)
        return r_out, h
