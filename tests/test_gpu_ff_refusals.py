"""Calls of the 16-bit feed-forward block that are refused, with tensors on the GPU."""
import pytest

from tests.test_gpu_ff import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [4, 40])
def test_x_and_dy_of_another_type_than_the_weights(t):
    import torch
    from post_weight_quantization_layer_amd import feed_forward as FF
    x, gate, up, down, dy = make(61, t, 64, 96, "f16")
    _, saved = FF.gated_feed_forward_saved(x, gate, up, down)
    for kind in (torch.bfloat16, torch.float32, torch.uint8):
        with pytest.raises(TypeError):
            FF.gated_feed_forward_backward(dy.to(kind), saved, x.to(kind), gate, up, down)
        with pytest.raises(TypeError):
            FF.gated_feed_forward_backward(dy, saved, x.to(kind), gate, up, down)
        with pytest.raises(TypeError):
            FF.gated_feed_forward_saved(x.to(kind), gate, up, down)


def test_tangents():
    import torch
    from torch.autograd import forward_ad
    from post_weight_quantization_layer_amd.feed_forward import gated_feed_forward
    args = make(62, 4, 64, 96, "bf16")[:4]
    with forward_ad.dual_level():
        gated_feed_forward(*args)
        for i in range(4):
            dual = list(args)
            dual[i] = forward_ad.make_dual(args[i], torch.ones_like(args[i]))
            with pytest.raises(NotImplementedError, match="forward-mode"):
                gated_feed_forward(*dual)
