"""Log probabilities of given tokens, their ranks, the entropy and the top
alternatives, from rows of logits (gptq_token_logprobs of gptq_run.h)."""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch

from . import binding_run as R


@dataclass
class TokenLogprobs:
    logprob: torch.Tensor | None        # rows float32 (None without ids)
    rank: torch.Tensor | None           # rows int32, 0: the given token is the top one
    entropy: torch.Tensor               # rows float32
    top_ids: torch.Tensor               # rows x top_k int32, -1 past the last alternative
    top_logprobs: torch.Tensor          # rows x top_k float32

    def perplexity(self) -> float:
        """exp of minus the mean log probability over the rows that have a given
        token (synchronizes)."""
        scored = self.rank >= 0
        n = int(scored.sum())
        if n == 0:
            return math.nan
        return math.exp(-float(self.logprob[scored].double().sum()) / n)


class TokenScorer:
    """Owns the outputs and the scratch memory for up to ``rows`` rows of
    ``vocab`` logits; a call's result is overwritten by the next."""

    def __init__(self, rows: int, vocab: int, top_k: int = 0, device="cuda"):
        if not 0 <= top_k <= min(64, vocab):
            raise ValueError("top_k must be in [0, min(64, vocab)]")
        self.rows, self.vocab, self.top_k = rows, vocab, top_k

        def buffer(dtype, *shape):
            return torch.empty(shape, dtype=dtype, device=device)

        self.logprob = buffer(torch.float32, rows)
        self.rank = buffer(torch.int32, rows)
        self.entropy = buffer(torch.float32, rows)
        self.top_ids = buffer(torch.int32, rows, top_k)
        self.top_logprobs = buffer(torch.float32, rows, top_k)
        self.scratch = R.Scratch(self.logprob.device)

    def __call__(self, logits: torch.Tensor, ids: torch.Tensor | None = None, *,
                 scale: float = 1.0, stream=None) -> TokenLogprobs:
        """logits rows x vocab; ids rows int64 (negative: none given); ``scale``
        multiplies the logits (an inverse temperature)."""
        R.matrix(logits, "logits", None, self.vocab)
        n = logits.shape[0]
        if n > self.rows:
            raise ValueError(f"{n} rows asked of buffers for {self.rows}")
        if ids is not None:
            R.vector(ids, "ids", n, torch.int64)
        whole = n == self.rows

        def part(t):
            return t if whole else t[:n]

        out = TokenLogprobs(None if ids is None else part(self.logprob),
                            None if ids is None else part(self.rank), part(self.entropy),
                            part(self.top_ids), part(self.top_logprobs))
        nbytes = R.lib().gptq_token_logprobs_ws_bytes(n, self.vocab, self.top_k)
        ptr = R.stream_ptr(stream)
        R._check(R.lib().gptq_token_logprobs(
            logits.data_ptr(), R._dtype(logits, "logits"), n, self.vocab, R.ld(logits),
            None if ids is None else ids.data_ptr(), scale, self.top_k,
            None if ids is None else self.logprob.data_ptr(),
            None if ids is None else self.rank.data_ptr(), self.entropy.data_ptr(),
            self.top_ids.data_ptr(), self.top_logprobs.data_ptr(),
            self.scratch(nbytes, ptr, stream), nbytes, ptr))
        return out
