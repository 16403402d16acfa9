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
