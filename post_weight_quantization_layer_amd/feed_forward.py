"""Gated feed-forward blocks in floating point: on layers of 8-bit floats
(gptq_f8_ff_* of gptq_ff.h), and in 16 bits with gradients (gptq_ff_*).

    y = (silu(x W_gate^T) * (x W_up^T)) W_down^T

The second is the block that GatedMLPCalibrator quantizes: to measure a
quantized block against, and to tune what stays in float around it."""
from __future__ import annotations

import threading
import weakref

import torch
from torch.autograd import forward_ad

from . import binding_ff as F
from . import binding_run as R
from .f8 import F8Linear


class GatedFeedForwardF8:
    """The block on three layers of 8-bit floats.  v = silu(g) u goes from float32 to
    codes; g, u and v are not stored in the activations' type.  Calls on different
    streams may overlap: each stream has its own scratch memory.  Threads may share it
    and a stream."""

    def __init__(self, gate: F8Linear, up: F8Linear, down: F8Linear):
        if (gate.rows, gate.cols) != (up.rows, up.cols) or \
                (down.rows, down.cols) != (gate.cols, gate.rows):
            raise ValueError("gate and up must be inner x d, down d x inner")
        F.one_device(gate.mem, up.mem, down.mem)
        self.gate, self.up, self.down = gate, up, down      # kept alive
        self.d, self.inner = down.rows, down.cols
        self.block = F.gptq_f8_ff(gate.layer, up.layer, down.layer)
        self.scratch = R.Scratch(down.device)
        self._last = (-1, 0)      # tokens, scratch bytes

    @classmethod
    def from_weights(cls, gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor, stream=None):
        """From float weights, rounded to nearest block by block."""
        return cls(*(F8Linear.from_weight(w, stream) for w in (gate, up, down)))

    def __call__(self, x: torch.Tensor, y: torch.Tensor | None = None,
                 dtype: torch.dtype | None = None, stream=None):
        """x tokens x d -> y tokens x d, float16 or bfloat16 (``dtype``, or x's type);
        ``y`` may be x."""
        R.matrix(x, "x", None, self.d)
        t = x.shape[0]
        mem = self.down.mem
        with F.on_device(mem):
            if y is None:
                with R.on(stream):
                    y = torch.empty((t, self.d), dtype=dtype or x.dtype, device=self.down.device)
            F.one_device(mem, x, y)
            last = self._last
            if last[0] != t:
                last = self._last = (t, F.gptq_f8_ff_ws_bytes(self.block, t))
            n = last[1]
            with self.scratch.lock:
                ws = self.scratch(n, mem, stream)
                F.gptq_f8_ff_forward(self.block, x, y, R.address(ws), n, stream)
        return y


def _bytes(n: int, device) -> torch.Tensor | None:
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def _new(t: torch.Tensor) -> torch.Tensor:
    """A contiguous tensor of t's shape and type."""
    return torch.empty_like(t) if t.is_contiguous() else \
        torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _block(x, gate, up, down):
    """The weights of a forward pass whose arguments fit."""
    kind = x.dtype
    if kind is not gate.dtype:
        raise TypeError(f"x and the weights must be of one type, got {kind} and {gate.dtype}")
    if kind is not torch.bfloat16 and kind is not torch.float16:
        raise TypeError(f"the block is in float16 or bfloat16, not {kind}")
    ff = F.make_ff(gate, up, down)
    R.matrix(x, "x", None, ff.d)
    F.one_device(x, gate, up, down)
    return ff


def _forward(ff, x, save: bool, stream=None):
    """(y, saved or None)"""
    t = x.shape[0]
    with F.on_device(x), R.on(stream):
        y = _new(x)
        saved = _bytes(F.gptq_ff_saved_bytes(ff, t), x.device) if save else None
        ws = _bytes(F.gptq_ff_forward_ws_bytes(ff, t), x.device)
        F.gptq_ff_forward(ff, x, y, saved, ws, stream)
    return y, saved


def gated_feed_forward_saved(x: torch.Tensor, gate: torch.Tensor, up: torch.Tensor,
                             down: torch.Tensor, stream=None):
    """(y, saved): the forward pass with what ``gated_feed_forward_backward`` takes (an
    opaque byte tensor, None for no tokens), outside of autograd."""
    with torch.no_grad():
        return _forward(_block(x, gate, up, down), x, True, stream)


def _backward(ff, dy, saved, x, gate, up, down, needed, stream=None):
    with F.on_device(x), R.on(stream):
        if not dy.is_contiguous() and (dy.stride(-1) != 1 or dy.stride(0) < dy.shape[1]):
            dy = dy.contiguous()        # an expanded gradient, as that of a sum
        out = [_new(t) if n else None for t, n in zip((x, gate, up, down), needed)]
        ws = _bytes(F.gptq_ff_backward_ws_bytes(ff, x.shape[0]), x.device)
        F.gptq_ff_backward(ff, x, saved, dy, *out, ws, stream)
    return tuple(out)


def gated_feed_forward_backward(dy: torch.Tensor, saved: torch.Tensor | None, x: torch.Tensor,
                                gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor,
                                needed=(True, True, True, True), stream=None):
    """Gradients of x, gate, up and down (None where not ``needed``) for the gradient
    ``dy`` of y.  x and the weights have to be what the forward pass had."""
    if len(needed) != 4:
        raise ValueError(f"needed says of four gradients whether, got {len(needed)}")
    ff = F.make_ff(gate, up, down)
    F.one_device(x, gate, up, down, dy)
    if saved is not None:
        if saved.dtype is not torch.uint8 or not saved.is_contiguous():
            raise TypeError("saved must be what gated_feed_forward_saved gave")
        F.one_device(x, saved)
    with torch.no_grad():
        return _backward(ff, dy, saved, x, gate, up, down, needed, stream)


class _Eager:
    """Alive as long as a graph made outside of a capture, with where it goes on to its leaves."""
    living: "weakref.WeakSet[_Eager]" = weakref.WeakSet()
    lock = threading.Lock()              # a set may not grow while it is read

    def __init__(self, inputs):
        self.leaves = [weakref.ref(t) for t in inputs if t.grad_fn is None]
        self.nodes = [t.grad_fn for t in inputs if t.grad_fn is not None]
        with self.lock:
            self.living.add(self)


def _leaves_below(nodes, seen: set) -> list:
    """The leaves that the graphs below these nodes end in, without what is below ``seen``."""
    found, stack = [], list(nodes)
    while stack:
        node = stack.pop()
        if node is None or node in seen:
            continue
        seen.add(node)
        leaf = getattr(node, "variable", None)
        if isinstance(leaf, torch.Tensor):
            found.append(leaf)
        stack.extend(n for n, _ in node.next_functions)
    return found


def _graph_of(inputs):
    """A token for the graph that is being made from these inputs.

    The nodes that add up a leaf's gradient belong to the stream of the first living graph
    of it.  A captured backward pass that reached nodes of another stream would make
    that stream wait for the capture, an error in a thread of autograd's that ends the
    process; so it is refused here.  An input may be made of leaves (a view of a packed
    weight, a cast of a master weight, another layer's output): those count, and are looked
    for only in a capture, where a walk costs nothing that is replayed."""
    if not R.capturing():
        return _Eager(inputs)
    with _Eager.lock:
        living = list(_Eager.living)
    seen: set = set()
    theirs = [t for graph in living for t in (r() for r in graph.leaves) if t is not None]
    theirs += _leaves_below((n for graph in living for n in graph.nodes), seen)
    ours = [t for t in inputs if t.grad_fn is None]
    ours += _leaves_below((t.grad_fn for t in inputs), set())
    taken = {id(t) for t in theirs}
    if any(id(t) in taken for t in ours):
        raise RuntimeError("a graph of the same tensors made outside of this capture is alive: "
                           "drop its outputs first, or capture gated_feed_forward_saved and "
                           "gated_feed_forward_backward, which make none")
    return None


class _GatedFeedForward(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, up, down):
        ctx.ff = _block(x, gate, up, down)
        with F.on_device(x):
            ctx.graph = _graph_of([t for t in (x, gate, up, down) if t.requires_grad])
        y, saved = _forward(ctx.ff, x, True)
        ctx.save_for_backward(x, gate, up, down, saved)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, gate, up, down, saved = ctx.saved_tensors
        ff = ctx.ff
        if (gate.data_ptr(), up.data_ptr(), down.data_ptr()) != (ff.gate, ff.up, ff.down):
            ff = F.make_ff(gate, up, down)          # a hook unpacked them elsewhere
        return _backward(ff, dy, saved, x, gate, up, down, ctx.needs_input_grad)


def gated_feed_forward(x: torch.Tensor, gate: torch.Tensor, up: torch.Tensor,
                       down: torch.Tensor) -> torch.Tensor:
    """x tokens x d -> y tokens x d; gate and up inner x d, down d x inner; all
    float16 or all bfloat16.  Differentiable once in all four, on the current stream; not in
    forward mode.

    It may be captured into a CUDA graph, with its backward pass in the same capture, while no
    graph of the same tensors, or of what they are made of, that was made outside of the
    capture is alive (such a call of this function is refused; of other functions it cannot
    know)."""
    if forward_ad._current_level >= 0 and any(forward_ad.unpack_dual(t).tangent is not None
                                              for t in (x, gate, up, down)):
        raise NotImplementedError("gated_feed_forward has no forward-mode derivative")
    if torch.is_grad_enabled() and (x.requires_grad or gate.requires_grad or up.requires_grad or
                                    down.requires_grad):
        return _GatedFeedForward.apply(x, gate, up, down)
    return _forward(_block(x, gate, up, down), x, False)[0]
