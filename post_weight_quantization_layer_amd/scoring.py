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
    ids: torch.Tensor | None = None     # the given tokens: the caller's tensor itself

    def perplexity(self) -> float:
        """exp of minus the mean log probability over the rows that have a given
        token (id >= 0; synchronizes).  NaN where such a row could not be scored
        (it holds a NaN or +infinity, or its id is past the vocabulary) and where
        no row has a token; infinity where a token is impossible or the mean is
        past exp's range.  Reads ``ids``, which must not have changed."""
        if self.ids is None:
            raise ValueError("no perplexity without ids: the call was given no tokens")
        given = self.ids.view(-1) >= 0
        n = int(given.sum())
        if n == 0:
            return math.nan
        try:
            return math.exp(-float(self.logprob[given].double().sum()) / n)
        except OverflowError:
            return math.inf


class TokenScorer:
    """Owns the outputs and the scratch memory for up to ``rows`` rows of
    ``vocab`` logits; a call's result is overwritten by the next.  So calls of one
    scorer follow each other: on one stream or ordered by events, and from one
    thread at a time."""

    def __init__(self, rows: int, vocab: int, top_k: int = 0, device="cuda"):
        if not 0 <= top_k <= min(64, vocab):
            raise ValueError("top_k must be in [0, min(64, vocab)]")
        device = R.on_gpu(device, "a scorer's outputs")
        self.rows, self.vocab, self.top_k = rows, vocab, top_k

        def buffer(dtype, *shape):
            return torch.empty(shape, dtype=dtype, device=device)

        self.logprob = buffer(torch.float32, rows)
        self.rank = buffer(torch.int32, rows)
        self.entropy = buffer(torch.float32, rows)
        self.top_ids = buffer(torch.int32, rows, top_k)
        self.top_logprobs = buffer(torch.float32, rows, top_k)
        self._out = TokenLogprobs(self.logprob, self.rank, self.entropy, self.top_ids,
                                  self.top_logprobs)
        self.scratch = R.Scratch(self.logprob.device)
        self._last = (-1, 0)       # rows, scratch bytes

    def __call__(self, logits: torch.Tensor, ids: torch.Tensor | None = None, *,
                 scale: float = 1.0, stream=None) -> TokenLogprobs:
        """logits rows x vocab; ids rows int64 (negative: none given); ``scale``
        multiplies the logits (an inverse temperature)."""
        if logits.dim() != 2 or logits.shape[1] != self.vocab:
            raise ValueError(f"logits must be rows x {self.vocab}, got {tuple(logits.shape)}")
        n = logits.shape[0]
        if n > self.rows:
            raise ValueError(f"{n} rows asked of buffers for {self.rows}")
        out = self._out if n == self.rows else TokenLogprobs(
            *(None if t is None else t[:n] for t in (self.logprob, self.rank, self.entropy,
                                                     self.top_ids, self.top_logprobs)))
        if ids is None:
            out = TokenLogprobs(None, None, out.entropy, out.top_ids, out.top_logprobs)
        else:
            R.vector(ids, "ids", n, torch.int64)
            out.ids = ids
        last = self._last
        if last[0] != n:
            last = self._last = (n, R.gptq_token_logprobs_ws_bytes(n, self.vocab, self.top_k))
        nbytes = last[1]
        with self.scratch.lock:
            ws = self.scratch(nbytes, logits, stream)
            R.gptq_token_logprobs(logits, ids, scale, self.top_k, out.logprob, out.rank,
                                  out.entropy, out.top_ids, out.top_logprobs, R.address(ws),
                                  nbytes, stream)
        return out
