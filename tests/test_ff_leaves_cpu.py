"""Which graphs share leaves with a call that is captured (no GPU)."""
import gc

import pytest

torch = pytest.importorskip("torch")

from post_weight_quantization_layer_amd import feed_forward as FF


@pytest.fixture
def capturing(monkeypatch):
    now = [False]
    monkeypatch.setattr(FF.R, "capturing", lambda: now[0])
    return now


def leaf(*shape):
    return torch.zeros(shape, requires_grad=True)


MADE = [lambda w: w.chunk(2)[0],                  # gate out of a packed weight
        lambda w: w[1:].t(),
        lambda w: w.to(torch.float16),            # of a master weight
        lambda w: (w * 2).view(-1, 2) + 1,
        lambda w: w]


@pytest.mark.parametrize("then", range(len(MADE)))
@pytest.mark.parametrize("now", range(len(MADE)))
def test_leaves_are_found_behind_views_and_casts(capturing, now, then):
    """The nodes that add up a leaf's gradient are the leaf's, whatever was made of it."""
    w, other = leaf(4, 2), leaf(4, 2)
    graph = FF._graph_of([MADE[then](w)])
    capturing[0] = True
    with pytest.raises(RuntimeError, match="alive"):
        FF._graph_of([MADE[now](other), MADE[now](w)])
    assert FF._graph_of([MADE[now](other)]) is None
    del graph
    gc.collect()
    assert FF._graph_of([MADE[now](w)]) is None


def test_a_graph_of_many_layers(capturing):
    """Inputs that come out of other layers: shared weights anywhere below are found, and a
    graph is walked once although its nodes are reached along many ways."""
    layers = [leaf(1) for _ in range(40)]

    def x(weights):
        out = torch.ones(1)
        for w in weights:
            out = out * w + out * w              # 2^40 ways down
        return out
    graph = FF._graph_of([x(layers)])
    capturing[0] = True
    with pytest.raises(RuntimeError, match="alive"):
        FF._graph_of([x([leaf(1), layers[0]])])
    assert FF._graph_of([x([leaf(1) for _ in range(40)])]) is None
    del graph


def test_a_graph_whose_buffers_are_freed_still_lives(capturing):
    w = leaf(3)
    y = w * 2
    graph = FF._graph_of([y])
    y.sum().backward()
    del y
    capturing[0] = True
    with pytest.raises(RuntimeError, match="alive"):
        FF._graph_of([w])
    del graph
    gc.collect()
    assert FF._graph_of([w]) is None


def test_it_keeps_no_tensor_alive(capturing):
    import weakref
    w = leaf(3)
    gone = weakref.ref(w)
    graph = FF._graph_of([w])
    del w
    gc.collect()
    assert gone() is None
    del graph
