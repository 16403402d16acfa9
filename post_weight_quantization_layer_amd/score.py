"""Quantize a gated MLP block and a head at 8 bits per row, run them in 8-bit
integers and score tokens, against the float weights:

    python -m post_weight_quantization_layer_amd.score [--tokens 512 ...]

The model is synthetic (random weights, a stream that leans on the token that
follows): what is shown is the path.  GPTQ quantizes gate, up and down one after the other
(GatedMLPCalibrator, one scale per row) and then the head on the block's
outputs; GatedMLP8 runs the block, W8A8Linear the head, TokenScorer gives the
log probabilities of the next tokens, and their perplexity is compared with
that of the float weights."""
from __future__ import annotations

import argparse
from dataclasses import dataclass

import torch

from .calibrate import GatedMLPCalibrator
from .layer import GptqLayer
from .mlp import GatedMLP8
from .norms import NormBlock
from .scoring import TokenScorer
from .w8a8 import W8A8Linear

EPS = 1e-6


@dataclass
class Report:
    perplexity: float          # of the 8-bit path
    perplexity_float: float    # of the float32 weights
    logprob_difference: float  # mean |difference| of the tokens' log probabilities
    same_top: float            # share of positions with the same most likely token


def _float_logprobs(r, ids, weights, norms):
    def rms(v, w):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS) * w

    gate, up, down, head = weights
    x = rms(r, norms[0])
    g, u = x @ gate.t(), x @ up.t()
    r = r + 0.5 * rms((g / (1 + torch.exp(-g)) * u) @ down.t(), norms[1])
    logp = torch.log_softmax(rms(r, norms[2]) @ head.t(), -1)
    return logp.gather(1, ids.view(-1, 1)).view(-1), logp.argmax(-1)


def _calibration(h: torch.Tensor) -> torch.Tensor:
    """tokens x features -> features x tokens bfloat16, the calibration layout."""
    return h.to(torch.bfloat16).t().contiguous()


def run(d: int = 512, inner: int = 1408, vocab: int = 4000, tokens: int = 512,
        calibration_tokens: int = 4096, seed: int = 0, device="cuda") -> Report:
    """d and inner multiples of 128, tokens a multiple of 8."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device=device) * scale

    gate, up = normal(inner, d, scale=d ** -0.5), normal(inner, d, scale=d ** -0.5)
    down = normal(d, inner, scale=inner ** -0.5)
    embedding = normal(vocab, d)
    head = embedding * (2 * d ** -0.5)
    norms = [1 + 0.1 * normal(d) for _ in range(3)]
    ids = torch.randint(0, vocab, (tokens,), generator=g, device=device)
    target = torch.roll(ids, -1)

    def stream(following):                              # leans on the token that follows
        return 0.2 * embedding[following] + normal(len(following), d)

    r = stream(target)
    target[-1] = -1                                     # no next token
    floats = _float_logprobs(r, target.clamp(min=0), (gate, up, down, head), norms)

    enter = NormBlock(d, pre="rms", pre_weight=norms[0], eps=EPS)
    leave = NormBlock(d, post="rms", post_weight=norms[1], pre="rms", pre_weight=norms[2],
                      block_scale=0.5, eps=EPS)
    sample = stream(torch.randint(0, vocab, (calibration_tokens,), generator=g, device=device))
    cal = GatedMLPCalibrator(d, inner, bits=8, group=None, block=128, act_order=True,
                             device=device)
    q = cal.run(gate.clone(), up.clone(), down.clone(), [_calibration(enter(sample)[1])])
    mlp = GatedMLP8(enter, W8A8Linear.from_quantized(q.gate, q.up),
                    W8A8Linear.from_quantized(q.down), leave)

    head_layer = GptqLayer(vocab, d, bits=8, group=d, block=128, act_order=True, device=device)
    head_layer.reset_hessian()
    head_layer.add_batch(_calibration(mlp(sample)[1]))  # the quantized block's outputs
    head_layer.prepare()
    head8 = W8A8Linear.from_quantized(head_layer.quantize(head.clone()))

    _, h = mlp(r)
    out = TokenScorer(tokens, vocab, 1, device=device)(head8(h), target)
    n = tokens - 1                                      # positions with a next token
    logp = floats[0][:n].double()
    return Report(out.perplexity(), float(torch.exp(-logp.mean())),
                  float((out.logprob[:n].double() - logp).abs().mean()),
                  float((out.top_ids[:, 0] == floats[1]).double().mean()))


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("d", 512), ("inner", 1408), ("vocab", 4000), ("tokens", 512),
                        ("calibration-tokens", 4096), ("seed", 0)):
        p.add_argument("--" + name, type=int, default=value)
    r = run(**vars(p.parse_args()))
    print(f"perplexity {r.perplexity:.3f} in 8 bits, {r.perplexity_float:.3f} in float; "
          f"log probabilities differ by {r.logprob_difference:.4f} on average, "
          f"{100 * r.same_top:.1f} % of positions keep their most likely token")


if __name__ == "__main__":
    main()
