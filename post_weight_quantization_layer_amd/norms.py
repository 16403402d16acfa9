"""The residual stream between two blocks: the norms after one and before the
next, the block's gate and the residual scales, in one call
(gptq_norm_block of gptq_run.h)."""
from __future__ import annotations

import torch

from . import binding_run as R
from .w8a8 import TokenCodes


def tokens_per_gate(gate: torch.Tensor, gate_tokens: int | None, tokens: int) -> int:
    """Tokens that share a row of ``gate``: ``gate_tokens``, or by default all of
    them for one row and one for several."""
    if gate_tokens is None:
        gate_tokens = max(tokens, 1) if gate.shape[0] == 1 else 1
    if gate_tokens < 1 or gate.shape[0] * gate_tokens < tokens:
        raise ValueError(f"{gate.shape[0]} gate rows of {gate_tokens} tokens do not "
                         f"cover {tokens} tokens")
    return gate_tokens


class NormBlock:
    """r' = residual_scale r + block_scale gate * N_post(b);  h = N_pre(r').

    ``post``, ``pre``: "rms", "layer" or None (no norm).  Weights and biases are
    vectors of d values of one type, or None; a norm multiplies by
    ``weight_offset + weight``."""

    def __init__(self, d: int, *, post: str | None = None, post_weight=None, post_bias=None,
                 pre: str | None = None, pre_weight=None, pre_bias=None,
                 residual_scale: float = 1.0, block_scale: float = 1.0, eps: float = 1e-6,
                 weight_offset: float = 0.0):
        self.d = d
        self.vectors = (post_weight, post_bias, pre_weight, pre_bias)   # kept alive
        given = [v for v in self.vectors if v is not None]
        for v in given:
            R.vector(v, "weights and biases", d, given[0].dtype)
        dtype = R._dtype(given[0], "weights") if given else 0
        self.params = R.gptq_norm_params(
            R.NORMS[post], R.NORMS[pre], dtype, eps, weight_offset, residual_scale, block_scale,
            *(None if v is None else v.data_ptr() for v in self.vectors))

    def __call__(self, r: torch.Tensor, b: torch.Tensor | None = None, *, gate=None,
                 gate_tokens: int | None = None, r_out: torch.Tensor | None = None,
                 h: torch.Tensor | None = None, codes: TokenCodes | None = None, stream=None):
        """r, b: tokens x d.  gate: rows of d, ``gate_tokens`` consecutive tokens
        each (default: one row for all tokens, else one per token).

        Returns (r', h).  r' goes to ``r_out`` (which may be r), or to a new
        tensor if b is given.  With neither, r' is not stored: the first result
        is r itself, not scaled by ``residual_scale`` (h is made from the scaled
        one).  h goes to ``h`` and / or, as codes, to ``codes``; the second result
        is ``codes`` where only that is given, and a new tensor where neither
        is."""
        shape = r.shape
        if len(shape) != 2 or shape[1] != self.d:
            raise ValueError(f"r must be tokens x {self.d}, got {tuple(shape)}")
        t = shape[0]
        gate_tokens = 1 if gate is None else tokens_per_gate(gate, gate_tokens, t)
        if (r_out is None and b is not None) or (h is None and codes is None):
            if not r.is_cuda:
                raise ValueError("r must be on the GPU")
            with R.on(stream):
                if r_out is None and b is not None:
                    r_out = torch.empty((t, self.d), dtype=r.dtype, device=r.device)
                if h is None and codes is None:
                    h = torch.empty((t, self.d), dtype=r.dtype, device=r.device)
        c = s = n = None
        if codes is not None:
            if codes.cols != self.d:
                raise ValueError(f"buffers for {codes.cols} features, got {self.d}")
            codes = codes.head(t)
            c, s, n = codes.codes, codes.scale, codes.sum
        R.gptq_norm_block(self.params, r, b, gate, gate_tokens, r_out, h, c, s, n, stream)
        return r if r_out is None else r_out, codes if h is None else h
