"""The floating-point layers and blocks at ends that the other tests leave out: outputs with
strides and at odd places through the C calls, and values so small that they have no leading
one."""
import pytest

from tests.test_gpu_ff import make, run

pytestmark = pytest.mark.gpu


def spread(rows, cols, kind, left, right):
    """A matrix cut out of a wider one filled with 5, and the wider one."""
    import torch
    wide = torch.full((rows + 2, cols + left + right), 5.0, dtype=kind, device="cuda")
    return wide[1:rows + 1, left:left + cols], wide


def margins_kept(cut, wide, left):
    import torch
    mask = torch.ones_like(wide, dtype=torch.bool)
    mask[1:-1, left:left + cut.shape[1]] = False
    return bool((wide[mask] == 5).all())


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("t,d,n", [(0, 72, 136), (3, 72, 136), (16, 65, 259), (40, 72, 136),
                                   (130, 264, 257), (700, 1000, 2731), (2051, 1024, 1408)])
def test_outputs_with_strides_of_their_own(t, d, n, kind):
    """Each output with another stride, so that no two can share a launch: the bits of contiguous
    ones, and nothing around them is written."""
    import torch
    from post_weight_quantization_layer_amd import binding_ff as F
    from post_weight_quantization_layer_amd import binding_run as R
    x, gate, up, down, dy = make(t + d + n, t, d, n, kind)
    want = run(x, gate, up, down, dy)
    ff, L, stream = F.make_ff(gate, up, down), F.lib(), R.stream_ptr(gate)
    outs = {"y": spread(t, d, x.dtype, 3, 5), "dx": spread(t, d, x.dtype, 1, 0),
            "dgate": spread(n, d, x.dtype, 8, 8), "dup": spread(n, d, x.dtype, 5, 6),
            "ddown": spread(d, n, x.dtype, 7, 0)}
    left = {"y": 3, "dx": 1, "dgate": 8, "dup": 5, "ddown": 7}

    def buffer(nbytes):
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device="cuda")
    saved = buffer(L.gptq_ff_saved_bytes(ff, t))
    ws = buffer(max(L.gptq_ff_forward_ws_bytes(ff, t), L.gptq_ff_backward_ws_bytes(ff, t)))

    def at(name):
        cut, wide = outs[name]
        return cut.data_ptr(), wide.stride(0)
    print("strided", t, d, n, kind, flush=True)
    R._check(L.gptq_ff_forward(ff, x.data_ptr(), d, t, *at("y"), saved.data_ptr(), saved.numel(),
                               ws.data_ptr(), ws.numel(), stream))
    R._check(L.gptq_ff_backward(ff, x.data_ptr(), d, t, saved.data_ptr(), saved.numel(),
                                dy.data_ptr(), d, *at("dx"), *at("dgate"), *at("dup"),
                                *at("ddown"), ws.data_ptr(), ws.numel(), stream))
    torch.cuda.synchronize()
    for name, (cut, wide) in outs.items():
        assert torch.equal(cut, want[name]), name
        assert margins_kept(cut, wide, left[name]), name


@pytest.mark.parametrize("t", [2, 40, 600])
def test_small_values_of_16_bits_count(t):
    """Tokens, weights and gradients below float16's smallest normal value, 2^-14, in whole steps
    of 2^-24.  The gate is 32 throughout, whose silu is 32 in float32 and its slope 1; products
    are whole steps and their sums below 2^24 of them, so results are their exact values,
    rounded where the definition does."""
    import torch
    d, n = 136, 264
    g = torch.Generator(device="cuda")
    g.manual_seed(80)

    def ints(*shape, most):
        return torch.randint(-most, most + 1, shape, generator=g, device="cuda").double()

    def half(v):
        assert torch.equal(v.half().double(), v)
        return v.half()
    gate = torch.zeros((n, d), dtype=torch.float64, device="cuda")
    gate[:, 0] = 32
    step = 2.0 ** -24
    # x small, up not; then up small; down small; dy small
    for x_unit, up_unit, down_unit, dy_unit in ((step, 1, 1, 1), (1, step, 1, 1), (1, 1, step, 1),
                                                (1, 1, 1, step)):
        x, up = ints(t, d, most=7) * x_unit, ints(n, d, most=7) * up_unit
        x[:, 0], up[:, 0] = 1, 0
        down, dy = ints(d, n, most=7) * down_unit, ints(t, d, most=7) * dy_unit
        got = {k: v.double() for k, v in run(half(x), half(gate), half(up), half(down),
                                             half(dy)).items()}
        r = lambda v: v.half().double()
        mm = lambda a, b: torch.mm(a.contiguous(), b.contiguous())
        u = mm(x, up.t())
        v, dv = r(32 * u), mm(dy, down)
        dg, du = r(dv * r(u)), r(dv * 32)
        want = {"y": r(mm(v, down.t())), "dx": r(mm(dg, gate) + mm(du, up)),
                "dgate": r(mm(dg.t(), x)), "dup": r(mm(du.t(), x)), "ddown": r(mm(dy.t(), v))}
        for name in want:
            assert want[name].any() or name in ("dx", "dgate"), name
            assert torch.equal(got[name], want[name]), (name, x_unit, up_unit, down_unit, dy_unit)


@pytest.mark.parametrize("t", [1, 9, 40, 300])
@pytest.mark.parametrize("rows,cols", [(200, 300), (4100, 256)])
def test_the_smallest_codes_count(rows, cols, t):
    """Codes 1 to 7 are steps of 2^-9.  Sums of them are whole steps of 2^-18, below 2^24 of
    them, so that the result is their exact value, rounded once."""
    import torch
    from post_weight_quantization_layer_amd.f8 import F8Linear
    g = torch.Generator(device="cuda")
    g.manual_seed(81)

    def codes(*shape):
        return torch.randint(0, 8, shape, generator=g, device="cuda") | \
            torch.randint(0, 2, shape, generator=g, device="cuda") << 7
    w, q = codes(rows, cols), codes(t, cols)
    value = lambda c: ((c & 7) * torch.where(c > 127, -1.0, 1.0)).double()
    lin = F8Linear(w.to(torch.uint8), torch.ones((-(-rows // 128), -(-cols // 128)), device="cuda"))
    from post_weight_quantization_layer_amd.f8 import F8Tokens
    tokens = F8Tokens(t, cols)
    tokens.codes.zero_()
    tokens.codes[:, :cols] = q.to(torch.uint8)
    tokens.scale.fill_(1.0)
    want = torch.mm(value(q), value(w).t().contiguous()) * 2.0 ** -18
    for kind in (torch.float16, torch.bfloat16):
        assert torch.equal(lin.product(tokens, dtype=kind), want.to(kind))


@pytest.mark.parametrize("t", [2, 40, 1030])
def test_the_smallest_codes_count_in_the_block(t):
    """Gate's and up's codes are all of the smallest: were one of them taken for zero, v and y
    would be none."""
    import torch
    from post_weight_quantization_layer_amd.f8 import F8Linear
    from post_weight_quantization_layer_amd.feed_forward import GatedFeedForwardF8
    from tests.test_gpu_f8 import block_reference
    d, n = 130, 8300 if t > 1000 else 300
    g = torch.Generator(device="cuda")
    g.manual_seed(82)
    layers = []
    for rows, cols, scale in ((n, d, 16.0), (n, d, 16.0), (d, n, 1.0)):
        c = torch.randint(1, 8, (rows, cols), generator=g, device="cuda") | \
            torch.randint(0, 2, (rows, cols), generator=g, device="cuda") << 7
        s = torch.full((-(-rows // 128), -(-cols // 128)), scale, device="cuda")
        w = ((c & 7) * torch.where(c > 127, -1.0, 1.0)).double() * 2.0 ** -9 * scale
        layers.append((c.to(torch.uint8), s, w))
    block = GatedFeedForwardF8(*(F8Linear(c, s) for c, s, _ in layers))
    x = torch.randn((t, d), generator=g, device="cuda").half()
    want = block_reference(x, layers)
    off = (block(x).double() - want).norm() / want.norm()
    assert off <= 2.0 ** -11 + 7e-4 + 4e-5     # as test_gpu_f8's blocks
