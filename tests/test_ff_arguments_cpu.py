"""What the calls of the 16-bit feed-forward block refuse before they reach the library (no
GPU: tensors that say they are on one, and a library that must not be called)."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

from post_weight_quantization_layer_amd import binding_ff as F
from post_weight_quantization_layer_amd import feed_forward as FF


class OnGpu(torch.Tensor):
    is_cuda = True



def on_gpu(*shape, dtype):
    return torch.zeros(shape).to(dtype).as_subclass(OnGpu)


class Library:
    """Sizes that are plausible; calls that are counted."""

    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*args):
            if not name.endswith("_bytes"):
                self.calls += 1
            return 1 << 16 if name.endswith("_bytes") else 0
        return call


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(F, "_lib", lib)
    monkeypatch.setattr(F, "on_device", lambda t: contextlib.nullcontext())
    monkeypatch.setattr(FF.R, "stream_ptr", lambda t, stream=None: 0)
    return lib


def block(kind=torch.float16):
    return (on_gpu(96, 64, dtype=kind), on_gpu(96, 64, dtype=kind), on_gpu(64, 96, dtype=kind))


def test_the_stand_ins_reach_the_library(library):
    x, weights = on_gpu(4, 64, dtype=torch.float16), block()
    _, saved = FF.gated_feed_forward_saved(x, *weights)
    out = FF.gated_feed_forward_backward(x, saved, x, *weights)
    assert len(out) == 4 and library.calls == 2


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32, torch.float64, torch.uint8,
                                  torch.int16])
def test_x_and_dy_of_another_type_than_the_weights(library, kind):
    x, dy = on_gpu(4, 64, dtype=kind), on_gpu(4, 64, dtype=kind)
    saved, weights = torch.zeros(1 << 16, dtype=torch.uint8), block()
    ff = F.make_ff(*weights)
    half = on_gpu(4, 64, dtype=torch.float16)
    for call in (lambda: FF.gated_feed_forward_backward(dy, saved, x, *weights),
                 lambda: FF.gated_feed_forward_backward(dy, saved, half, *weights),
                 lambda: FF.gated_feed_forward_backward(half, saved, x, *weights),
                 lambda: FF.gated_feed_forward_saved(x, *weights),
                 lambda: F.gptq_ff_forward(ff, x, half),
                 lambda: F.gptq_ff_backward(ff, x, saved, dy, half)):
        with pytest.raises(TypeError):
            call()
    assert library.calls == 0


@pytest.mark.parametrize("which", range(4))
def test_tangents(library, which):
    """A result without one would be a derivative of zero."""
    from torch.autograd import forward_ad
    args = [on_gpu(4, 64, dtype=torch.float16), *block()]
    with forward_ad.dual_level():
        FF.gated_feed_forward(*args)
        assert library.calls == 1
        args[which] = forward_ad.make_dual(args[which], torch.ones_like(args[which]))
        for mode in (torch.enable_grad, torch.no_grad):
            with mode(), pytest.raises(NotImplementedError, match="forward-mode"):
                FF.gated_feed_forward(*args)
        args[which].requires_grad_()
        with pytest.raises(NotImplementedError, match="forward-mode"):
            FF.gated_feed_forward(*args)
    assert library.calls == 1


@pytest.mark.parametrize("needed", [(), (True,), (True, True, True), (True,) * 5])
def test_needed_names_four_gradients(library, needed):
    x, weights = on_gpu(4, 64, dtype=torch.float16), block()
    saved = torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="needed"):
        FF.gated_feed_forward_backward(x, saved, x, *weights, needed)
    assert library.calls == 0


def test_tensors_on_the_cpu_with_and_without_gradients():
    """The arguments are looked at before the GPU is."""
    for needs in (False, True):
        args = [torch.zeros(s, dtype=torch.float16, requires_grad=needs)
                for s in ((4, 64), (96, 64), (96, 64), (64, 96))]
        with pytest.raises(ValueError, match="on the GPU"):
            FF.gated_feed_forward(*args)
        with pytest.raises(TypeError, match="one type"):
            FF.gated_feed_forward(args[0].double(), *args[1:])


def test_a_capture_is_looked_for_on_the_tensors_device(library, monkeypatch):
    current = []

    @contextlib.contextmanager
    def on_device(t):
        current.append(True)
        yield
        current.pop()
    asked = []
    monkeypatch.setattr(F, "on_device", on_device)
    monkeypatch.setattr(FF.R, "capturing", lambda: asked.append(bool(current)))
    FF.gated_feed_forward(on_gpu(4, 64, dtype=torch.float16).requires_grad_(), *block())
    assert asked == [True] and library.calls == 1
