"""Captured calls of the classes that run layers beside other calls of the same
objects: a graph's replays give its results and write nothing else."""
import numpy as np
import pytest

from tests.test_gpu_run import activations, layer_on_gpu, small_mlp, stored_layer, to_gpu

pytestmark = pytest.mark.gpu


def linear(rng):
    """Few tokens (rows kernel) and more (k in several parts): codes, scales, parts."""
    lin = layer_on_gpu(*stored_layer(rng, 300, 4100))

    def step(x):
        return (lin(x),)
    return step, 4100


def scorer(rng):
    import torch
    from post_weight_quantization_layer_amd.scoring import TokenScorer
    sc = TokenScorer(64, 30000, 7)

    def step(x):
        out = sc(x, torch.full((x.shape[0],), 5, device="cuda"))
        return out.logprob, out.rank, out.entropy, out.top_ids, out.top_logprobs
    return step, 30000


def gated_mlp(rng):
    return small_mlp(rng)[0], 256


def w4a16(rng):
    """Columns stored out of order: x is gathered into scratch before the product."""
    import torch
    from post_weight_quantization_layer_amd import inputs as I
    from post_weight_quantization_layer_amd.w4a16 import W4A16Linear
    st = I.stored_int4_layer(512, 2048, 128, True, seed=7)
    lin = W4A16Linear.from_codes(*(torch.from_numpy(a).cuda()
                                   for a in (st.codes, st.g_idx, st.scale, st.zero)), 128)
    assert lin.workspace(2) is not None

    def step(x):
        return (lin(x),)
    return step, 2048


MAKERS = [linear, scorer, gated_mlp, w4a16]


@pytest.mark.parametrize("make", MAKERS)
def test_replays_after_larger_calls_on_the_stream(make):
    """Warm up and capture 2 tokens, then 40 and 64 on the same stream, then memory
    for other tensors: the replays leave those as they are."""
    import torch
    rng = np.random.default_rng(41)
    step, width = make(rng)
    x = to_gpu(activations(rng, 2, width), "f16")
    more = [to_gpu(activations(rng, t, width), "f16") for t in (40, 64)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [t.clone() for t in step(x)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step(x)
        large = [[t.clone() for t in step(m)] for m in more]
        # takes up whatever the stream's allocator has been given back
        other = [torch.full((n,), 77, dtype=torch.uint8, device="cuda")
                 for n in (512, 4096, 20000, 100000, 600000, 1 << 20) for _ in range(20)]
    torch.cuda.synchronize()
    for i in range(4):
        for t in got:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
        assert all(bool((t == 77).all()) for t in other), i
        with torch.cuda.stream(side):                  # eager calls go on as before
            for m, w in zip(more, large):
                assert all(torch.equal(a, b) for a, b in zip(step(m), w)), i
        torch.cuda.synchronize()


def test_gated_mlp_takes_its_own_outputs_and_others():
    """An output goes on as an input, whole, in part or shifted by a row; outputs
    of the caller's are written and returned, r' over r among them."""
    import torch
    rng = np.random.default_rng(43)
    mlp, *_ = small_mlp(rng)
    r0 = to_gpu(activations(rng, 30, 256), "f16")
    r, h = mlp(r0)
    kept = r.clone(), h.clone()
    for part in (r, r[1:], r[3:20], h[2:]):
        copy = part.clone()
        got, want = mlp(part), mlp(copy)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(part, copy)
    assert torch.equal(r, kept[0]) and torch.equal(h, kept[1])
    out, hout = torch.empty_like(r0), torch.empty((30, 300), dtype=r0.dtype, device="cuda")[:, 7:263]
    got = mlp(r0, r_out=out, h=hout)
    assert got[0] is out and got[1] is hout
    assert torch.equal(out, kept[0]) and torch.equal(hout, kept[1])
    got = mlp(r0, r_out=r0)
    assert got[0] is r0 and torch.equal(r0, kept[0]) and torch.equal(got[1], kept[1])
    with pytest.raises(ValueError):
        mlp(r0, h=hout[1:])
    with pytest.raises(TypeError):
        mlp(r0, r_out=out.float())


@pytest.mark.parametrize("make", [linear, gated_mlp, w4a16])
def test_threads_that_share_an_object_and_a_stream(make):
    """Each thread's results are those of its own inputs."""
    import threading
    import torch
    rng = np.random.default_rng(47)
    step, width = make(rng)
    xs = [to_gpu(activations(rng, t, width), "f16") for t in (1, 3, 20, 40)]
    want = [[t.clone() for t in step(x)] for x in xs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        for _ in range(40):
            if not all(torch.equal(a, b) for a, b in zip(step(xs[i]), want[i])):
                wrong.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
