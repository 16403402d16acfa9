"""What the classes over gptq_run.h keep between calls, with the streams and the
native calls replaced by stand-ins (no GPU)."""
import contextlib
import threading
import time

import pytest

torch = pytest.importorskip("torch")

from post_weight_quantization_layer_amd import binding_run as R


@pytest.fixture
def streams(monkeypatch):
    """stream: the current one's number; capturing: whether it is being captured."""
    class Now:
        stream, capturing = 1, False
    monkeypatch.setattr(R, "stream_ptr", lambda t, stream=None: Now.stream)
    monkeypatch.setattr(R, "capturing", lambda stream=None: Now.capturing, raising=False)
    return Now


def test_scratch_is_kept_per_stream_and_grows(streams):
    s, like = R.Scratch("cpu"), torch.zeros(1)
    a = s(100, like)
    assert s(50, like) is a and s(100, like) is a and s(0, like) is None
    streams.stream = 2
    b = s(100, like)
    assert b.data_ptr() != a.data_ptr()
    streams.stream = 1
    c = s(200, like)
    assert c.numel() >= 200 and s(100, like) is c


def test_a_captured_call_has_scratch_of_its_own(streams):
    """Warmed up, captured, then called with more and captured again: no buffer
    that a capture was given is kept, replaced or handed out again."""
    s, like = R.Scratch("cpu"), torch.zeros(1)
    warm = s(100, like)
    streams.capturing = True
    first, second = s(100, like), s(100, like)
    streams.capturing = False
    assert s(100, like) is warm
    larger = s(1000, like)
    addresses = {t.data_ptr() for t in (warm, first, second, larger)}
    assert len(addresses) == 4
    assert all(t is not first and t is not second for t in s._by_stream.values())


def gated_mlp(monkeypatch, seen):
    """A GatedMLP8 of width 4 whose native call records its outputs."""
    from types import SimpleNamespace as N
    from post_weight_quantization_layer_amd.mlp import GatedMLP8
    monkeypatch.setattr(R, "gptq_gated_mlp_ws_bytes", lambda block, dtype, t: 256 * t)
    monkeypatch.setattr(R, "gptq_gated_mlp_forward",
                        lambda block, r, gate, each, r_out, h, ws, n, stream: seen(r_out, h, ws, n))
    norm = N(d=4, params=R.gptq_norm_params())
    up, down = (N(rows=r, cols=c, layer=R.gptq_w8a8_layer(), device="cpu", mem=torch.zeros(1))
                for r, c in ((16, 4), (4, 8)))
    return GatedMLP8(norm, up, down, norm)


class OnGpu(torch.Tensor):
    is_cuda = True


def test_a_block_calls_outputs_are_its_own(streams, monkeypatch):
    """The next call, and one of more tokens, leave earlier results alone."""
    mlp = gated_mlp(monkeypatch, lambda r_out, h, ws, n: (r_out.fill_(mark[0]), h.fill_(mark[0])))
    kept = []
    for i, tokens in enumerate((2, 2, 3, 1)):
        mark = [float(i)]
        kept.append(mlp(torch.zeros(tokens, 4).as_subclass(OnGpu)))
    for i, (r, h) in enumerate(kept):
        assert (r == i).all() and (h == i).all() and len(r) == (2, 2, 3, 1)[i]


class Issue:
    """A native call of several launches: notes calls that use the same scratch at
    once, and scratch smaller than asked for."""

    def __init__(self):
        self.busy, self.faults = set(), []

    def __call__(self, ws, n, need):
        if n < need:
            self.faults.append(f"{n} bytes for {need}")
        if ws in self.busy:
            self.faults.append("two calls in one buffer")
        self.busy.add(ws)
        time.sleep(0.002)
        self.busy.discard(ws)


def from_threads(call, n=4, times=6):
    def work(i):
        for k in range(times):
            call(1 + (i + k) % 3)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()


def test_threads_on_one_stream_share_a_layer(streams, monkeypatch):
    from post_weight_quantization_layer_amd.w8a8 import W8A8Linear
    issue = Issue()
    monkeypatch.setattr(R, "gptq_w8a8_linear_ws_bytes", lambda layer, t: 256 * t)
    monkeypatch.setattr(R, "gptq_w8a8_linear",
                        lambda layer, x, y, ws, n, stream: issue(ws, n, 256 * len(x)))
    lin = W8A8Linear.__new__(W8A8Linear)
    lin.rows, lin.cols, lin.device, lin.layer, lin._last = 4, 4, "cpu", None, {}
    lin.mem, lin.scratch = torch.zeros(1), R.Scratch("cpu")
    from_threads(lambda t: lin(torch.zeros(t, 4)))
    assert not issue.faults


def test_threads_on_one_stream_share_a_block(streams, monkeypatch):
    issue = Issue()
    mlp = gated_mlp(monkeypatch, lambda r_out, h, ws, n: issue(ws, n, 256 * len(h)))

    def size(block, dtype, t):
        time.sleep(0.001)
        return 256 * t
    monkeypatch.setattr(R, "gptq_gated_mlp_ws_bytes", size)
    from_threads(lambda t: mlp(torch.zeros(t, 4).as_subclass(OnGpu)))
    assert not issue.faults


def test_a_4_bit_layers_scratch(streams, monkeypatch):
    """Per stream, call by call, and none of a captured call's."""
    from post_weight_quantization_layer_amd import binding as B
    from post_weight_quantization_layer_amd.w4a16 import W4A16Linear
    issue = Issue()
    monkeypatch.setattr(B, "gptq_w4a16_workspace_bytes", lambda layer, t: 256 * t)
    monkeypatch.setattr(B, "gptq_w4a16_gemm", lambda layer, x, y, ws, stream=None:
                        issue(ws.data_ptr(), ws.numel(), 256 * len(x)))
    monkeypatch.setattr(B, "gptq_w4a16_layer_bytes", lambda *a: 256)
    monkeypatch.setattr(B, "gptq_w4a16_prepare", lambda *a: None)
    none = torch.zeros(1)
    lin = W4A16Linear(none, none, none, none, 4, 4, 4)
    from_threads(lambda t: lin(torch.zeros(t, 4)))
    assert not issue.faults
    one = lin.workspace(3)
    streams.stream = 2
    assert lin.workspace(3).data_ptr() != one.data_ptr()
    streams.capturing = True
    caught = lin.workspace(3)
    streams.capturing = False
    assert lin.workspace(3) is not caught
    # the output it allocates belongs to the stream it is written on
    asked = []

    def on(stream):
        asked.append(stream)
        return contextlib.nullcontext()
    monkeypatch.setattr(R, "on", on)
    lin(torch.zeros(3, 4), stream="side")
    assert asked == ["side"]


def test_buffers_off_the_gpu_are_refused():
    """Kernels would write to host addresses."""
    from post_weight_quantization_layer_amd.scoring import TokenScorer
    from post_weight_quantization_layer_amd.w8a8 import TokenCodes
    for device in ("cpu", torch.device("cpu"), "meta"):
        with pytest.raises(ValueError, match="GPU"):
            TokenCodes(4, 8, device)
        with pytest.raises(ValueError, match="GPU"):
            TokenScorer(4, 8, 2, device=device)


def test_a_block_uses_its_norms_as_they_are(streams, monkeypatch):
    """A change of a norm's parameters reaches the block it was made with."""
    mlp = gated_mlp(monkeypatch, None)
    scales = []
    monkeypatch.setattr(R, "gptq_gated_mlp_forward", lambda block, *rest: scales.append(
        (block.enter.residual_scale, block.leave.residual_scale)))
    r = torch.zeros(2, 4).as_subclass(OnGpu)
    for scale in (0.5, 0.75):
        mlp.enter.params.residual_scale = scale
        mlp(r)
    assert scales == [(0.5, 0.5), (0.75, 0.75)]      # one norm object on both sides here


def test_scratch_of_a_copied_object(streams):
    import copy
    import pickle
    s, like = R.Scratch(torch.device("cpu")), torch.zeros(1)
    kept = s(100, like)
    for twin in (copy.deepcopy(s), pickle.loads(pickle.dumps(s))):
        assert twin.device == s.device and twin.lock is not s.lock
        assert twin(100, like).data_ptr() != kept.data_ptr()
    assert s(100, like) is kept
