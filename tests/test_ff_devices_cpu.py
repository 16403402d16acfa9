"""Memory of the floating-point layers and blocks, where a call names its stream by address and
its tensors lie on another device than the current one (no GPU: a stand-in for both).  A bare
address says no device, so it is the current device's at that time that is meant."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

from post_weight_quantization_layer_amd import binding_ff as F
from post_weight_quantization_layer_amd import binding_run as R
from post_weight_quantization_layer_amd import f8
from post_weight_quantization_layer_amd import feed_forward as FF
from tests.test_ff_arguments_cpu import Library, block, on_gpu


@pytest.fixture
def entered(monkeypatch):
    """Streams that were entered, each with whether the tensors' device was current."""
    seen, depth = [], [0]

    @contextlib.contextmanager
    def device(_):
        depth[0] += 1
        yield
        depth[0] -= 1

    def on(stream):
        seen.append(depth[0] > 0)
        return contextlib.nullcontext()
    lib = Library()
    monkeypatch.setattr(F, "_lib", lib)
    monkeypatch.setattr(F, "on_device", device)
    monkeypatch.setattr(F, "on_index", device, raising=False)
    monkeypatch.setattr(R, "on", on)
    monkeypatch.setattr(R, "on_gpu", lambda d, what: torch.device("cpu"))
    monkeypatch.setattr(R, "capturing", lambda stream=None: False)
    monkeypatch.setattr(R, "gptq_tokens_ld", lambda cols: -(-cols // 128) * 128)
    return seen


def test_streams_are_entered_on_the_tensors_device(entered):
    half = on_gpu(8, 64, dtype=torch.float16)
    f8.F8Tokens(4, 64, "cuda", 77)
    f8.quantize_tokens(half, stream=77)
    codes, scale = f8.quantize_weight(half, 77)
    lin = f8.F8Linear(*(t.as_subclass(type(half)) for t in (codes, scale)), 77)
    weights = block()
    _, saved = FF.gated_feed_forward_saved(half, *weights, 77)
    dy = on_gpu(64, 8, dtype=torch.float16).t()
    FF.gated_feed_forward_backward(dy, saved, half, *weights, stream=77)
    assert lin.rows == 8 and len(entered) >= 6 and all(entered)
