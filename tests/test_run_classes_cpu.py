"""What the classes over gptq_run.h keep between calls, with the streams and the
native calls replaced by stand-ins (no GPU)."""
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
