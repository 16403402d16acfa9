"""Outputs of the norm block that overlap its inputs: refused on the host where
rows of different tokens would share memory, taken where they do not."""
import numpy as np
import pytest

from post_weight_quantization_layer_amd import binding as B
from post_weight_quantization_layer_amd import binding_run as R

A, FAR = 0x100000, 0x900000
T, D, F16 = 6, 64, 2
ROW = 2 * D


def status(r=A, ld_r=D, b=FAR, ld_b=D, gate=None, ld_gate=D, gate_tokens=1, r_out=None,
           ld_r_out=D, h=None, ld_h=D, tokens=T):
    p = R.gptq_norm_params(1, 1, F16, 1e-6, 0.0, 1.0, 1.0, None, None, None, None)
    return R.lib().gptq_norm_block(p, F16, tokens, D, r, ld_r, b, ld_b, gate, ld_gate, gate_tokens,
                                   r_out, ld_r_out, h, ld_h, None, 0, None, None, None)


@pytest.mark.parametrize("args", [
    dict(r_out=A + ROW), dict(r_out=A - ROW), dict(h=A + ROW), dict(h=A + 2), dict(r_out=A - 2),
    dict(r_out=FAR + ROW), dict(h=FAR - 3 * ROW), dict(r_out=A, ld_r_out=D + 1),
    dict(r_out=A + ROW, ld_r_out=2 * D),                  # pitches differ
    dict(ld_r=3 * D, r_out=A + 3 * ROW - 2, ld_r_out=3 * D),   # the next row's first element
    dict(ld_r=3 * D, r_out=A + ROW - 2, ld_r_out=3 * D),
    dict(ld_r=4 * D, r_out=A + ROW, ld_r_out=5 * D),      # meet at the fourth row
    dict(gate=2 * FAR, r_out=2 * FAR + ROW), dict(gate=2 * FAR, gate_tokens=T, r_out=2 * FAR),
    dict(gate=2 * FAR, gate_tokens=2, h=2 * FAR), dict(r_out=3 * FAR, h=3 * FAR),
    dict(r_out=3 * FAR, h=3 * FAR + ROW), dict(tokens=1, r_out=A + 2)])
def test_shifted_rows_are_refused(args):
    assert status(**args) == B.GPTQ_ERR_INVALID_ARG
    assert "overlap" in B.gptq_last_error()


@pytest.mark.gpu
def test_rows_that_share_nothing_are_taken():
    """In place, over b, over a gate row for row, beside each other in one matrix,
    and with other pitches in between."""
    import torch
    from post_weight_quantization_layer_amd.norms import NormBlock
    rng = np.random.default_rng(3)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    op = NormBlock(D, post="rms", pre="layer", residual_scale=0.5)

    def fresh():
        m = torch.randn((64, 4 * D), device="cuda", generator=g).half()
        return m[:T, :D], m[:T, D:2 * D], m[:T, 2 * D:3 * D], m[:T, 3 * D:], m
    r, b, gate, other, m = fresh()
    want = op(r.clone(), b.clone(), gate=gate.clone())
    for outs in (dict(r_out=r, h=b), dict(r_out=other, h=gate), dict(r_out=b, h=r),
                 dict(r_out=m[T:2 * T, :D], h=m[T:2 * T, D:2 * D]),
                 dict(r_out=m.view(-1, D)[1 + 4 * T::8][:T], h=m.view(-1, D)[3::8][:T])):
        keep = m.clone()
        got = op(r, b, gate=gate, **outs)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), outs
        m.copy_(keep)
