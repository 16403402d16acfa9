"""Every kernel of the 8-bit product, exactly, at sizes that reach it: the name
of what was launched is checked, so a change of the launch rule cannot leave a
kernel without its test.  Sizes are ragged in rows, tokens and k."""
import numpy as np
import pytest

from oracle import run_oracle as R
from tests.test_gpu_run import (activations, back, expected_product, layer_on_gpu, stored_layer,
                                to_gpu)

pytestmark = pytest.mark.gpu

KERNELS = ("w8a8_rows", "w8a8_gemm_256x256", "w8a8_gemm_128x256", "w8a8_gemm_128x128",
           "w8a8_gemm_128x64", "w8a8_gemm_128x128_split", "w8a8_gemm_128x64_split", "w8a8_join")

# tokens, rows, cols for 256 compute units
SIZES = [
    ("256x256", 900, 15001, 532), ("256x256", 392, 24917, 1036), ("256x256", 1025, 12300, 900),
    ("128x256", 2047, 4091, 1030), ("128x256", 129, 22646, 2120), ("128x256", 3900, 2047, 1100),
    ("128x128", 1023, 4090, 515), ("128x128", 66, 16479, 5), ("128x128", 8402, 135, 129),
    ("128x128", 8450, 130, 316),
    ("128x64", 33, 1, 1), ("128x64", 33, 5, 137), ("128x64", 34, 301, 263), ("128x64", 333, 1031, 1100),
    ("128x128_split", 4025, 16, 43581), ("128x128_split", 6551, 3, 15377),
    ("128x64_split", 35, 19, 2361), ("128x64_split", 200, 601, 4000), ("128x64_split", 2738, 7, 4191),
    ("rows", 1, 33, 700), ("rows", 16, 515, 2000), ("rows", 32, 515, 300)]


def launched(call):
    """The product kernels that a call launches."""
    import torch
    from post_weight_quantization_layer_amd import binding as B
    B.gptq_profile_reset()
    B.gptq_profile_enable(True)
    try:
        call()
        torch.cuda.synchronize()
    finally:
        B.gptq_profile_enable(False)
    got = {k for k in KERNELS if B.gptq_profile_query(k)[0]}
    B.gptq_profile_reset()
    return got


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tile,t,rows,cols", SIZES)
def test_every_product_kernel_is_exact(kind, tile, t, rows, cols):
    import torch
    from post_weight_quantization_layer_amd.w8a8 import quantize_tokens
    if torch.cuda.get_device_properties(0).multi_processor_count != 256:
        pytest.skip("sizes chosen for 256 compute units")
    rng = np.random.default_rng(t + 3 * rows + 5 * cols)
    codes, scale, zero = stored_layer(rng, rows, cols)
    lin = layer_on_gpu(codes, scale, zero)
    x = to_gpu(activations(rng, t, cols), kind)
    # an output with a margin on every side, which stays as it is
    wide = torch.full((t + 2, rows + 5), 5.0, dtype=x.dtype, device="cuda")
    y = wide[1:t + 1, 3:rows + 3]
    tokens = quantize_tokens(x)
    name = "w8a8_rows" if tile == "rows" else "w8a8_gemm_" + tile
    ran = launched(lambda: lin.product(tokens, y))
    assert ran == ({name, "w8a8_join"} if "split" in tile else {name})
    q, s, _ = R.token_codes(back(x))
    np.testing.assert_array_equal(back(y), expected_product(q, s, codes, scale, zero, kind))
    keep = wide.clone()
    keep[1:t + 1, 3:rows + 3] = 5
    assert (keep == 5).all()


def test_every_kernel_has_a_size():
    assert {("w8a8_" if k[0] == "rows" else "w8a8_gemm_") + k[0] for k in SIZES} | {"w8a8_join"} == \
        set(KERNELS)
