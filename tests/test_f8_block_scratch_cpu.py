"""The scratch of the block on 8-bit floats holds what its two halves keep and the down
product's own (no GPU is touched: sizes only)."""
import pytest

from post_weight_quantization_layer_amd import binding_ff as F

A = 0x10000          # a plausible address, 256-byte aligned

WIDTHS = (64, 4096, 8192, 26112, 26240, 28672, 32768, 32784, 32896, 33000, 36864, 40960, 49040,
          54400, 65535, 65536)
INNER = (64, 1408, 4096, 11008, 14336, 28672, 49152, 65536)


def layer(rows, cols):
    return F.gptq_f8_layer(rows, cols, -(-rows // 16) * 16, -(-cols // 128) * 128, A,
                           F.lib().gptq_f8_layer_bytes(rows, cols))


def up256(n):
    return -(-n // 256) * 256


def codes(tokens, cols):
    blocks = -(-cols // 128)
    return up256(tokens * blocks * 128) + up256(tokens * blocks * 4)


@pytest.mark.parametrize("inner", INNER)
@pytest.mark.parametrize("d", WIDTHS)
def test_room_for_the_codes_and_the_down_product(d, inner):
    down = layer(d, inner)
    block = F.gptq_f8_ff(layer(inner, d), layer(inner, d), down)
    for tokens in (*range(1, 41), 64, 100, 333):
        need = codes(tokens, d) + codes(tokens, inner) + F.gptq_f8_gemm_ws_bytes(down, tokens)
        if tokens <= 16:                 # v in float32 between the halves
            need += tokens * inner * 4
        assert F.gptq_f8_ff_ws_bytes(block, tokens) >= need, tokens
