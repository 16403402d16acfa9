"""The norm block before the first block, without a block output: what comes back
as the stream."""
import numpy as np
import pytest

from tests.test_gpu_run import activations, back, to_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_stream_of_the_first_norm(kind):
    import torch
    from post_weight_quantization_layer_amd.norms import NormBlock
    r = to_gpu(activations(np.random.default_rng(6), 5, 300), kind)
    op = NormBlock(300, pre="rms", residual_scale=1.5, eps=1e-6)
    out = torch.empty_like(r)
    got, h = op(r, r_out=out)
    assert got is out
    want = torch.from_numpy(back(r) * np.float32(1.5)).to(r.dtype)
    assert torch.equal(out.cpu(), want)
    before = r.clone()
    same, h2 = op(r)                              # r' is not stored
    assert same is r and torch.equal(r, before) and torch.equal(h2, h)
    over, h3 = op(r, r_out=r)
    assert over is r and torch.equal(r, out) and torch.equal(h3, h)
