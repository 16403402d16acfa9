"""Which matrices of a call of gptq_ff.h share memory: compared with their bytes one by one
(no GPU is touched: a call that is not refused for that lacks its scratch)."""
import random

import pytest

from post_weight_quantization_layer_amd import binding as B
from post_weight_quantization_layer_amd import binding_ff as F
from tests.test_ff_abi_cpu import FAR, ff, layer, said

BASE = 1 << 32
F32, BF16, F16 = 0, 1, 2
SIZE = {F32: 4, BF16: 2, F16: 2}


def linear(x, x_dtype, ld_x, tokens, y, ld_y):
    """Whether gptq_f8_linear takes x and y for matrices that overlap."""
    st = F.lib().gptq_f8_linear(layer(), x, x_dtype, ld_x, tokens, y, F16, ld_y, None, 0, None)
    assert st == (B.GPTQ_ERR_INVALID_ARG if said("overlap") else B.GPTQ_ERR_WORKSPACE)
    return said("overlap")


def bytes_of(at, rows, width, pitch):
    return {at + r * pitch + i for r in range(rows) for i in range(width)}


@pytest.mark.parametrize("x,x_dtype,ld_x,y,ld_y,meet", [
    (BASE, F16, 400, BASE + 2 * 300, 400, False),            # columns 0 .. 299 and 300 .. 363
    (BASE, F16, 400, BASE + 2 * 299, 400, True),
    (BASE + 2 * 64, F16, 400, BASE, 400, False),             # y before x
    (BASE + 2 * 63, F16, 400, BASE, 400, True),
    (BASE, F16, 364, BASE + 2 * 300, 364, False),            # y ends where x's next row starts
    (BASE, F16, 363, BASE + 2 * 300, 363, True),
    (BASE, F32, 400, BASE + 4 * 300, 800, False),            # y in float32 rows' tails
    (BASE, F32, 400, BASE + 4 * 299, 800, True),
    (BASE, F16, 600, BASE + 2 * 300, 600, False),            # rows by turns
    (BASE, F16, 500, BASE + 2 * 400, 1000, False),           # y behind every second row
    (BASE, F16, 500, BASE + 2 * 400, 900, True),             # at other steps they meet
    (BASE, F16, 300, BASE + 2 * 300 * 100, 64, False),       # one after the other
    (BASE, F16, 300, BASE + 2 * 300 * 100 - 2, 64, True)])
def test_columns_and_rows_of_one_matrix(x, x_dtype, ld_x, y, ld_y, meet):
    assert linear(x, x_dtype, ld_x, 100, y, ld_y) == meet


def test_against_bytes_one_by_one():
    rng = random.Random(5)
    met = 0
    for _ in range(400):
        dt, tokens = rng.choice([F32, F16]), rng.choice([17, 17, 20, 33])
        ld_x, ld_y = 300 + rng.randrange(0, 200), 64 + rng.randrange(0, 700)
        if rng.random() < 0.5:
            ld_y = ld_x * SIZE[dt] // 2
        y = BASE + 2 * rng.randrange(-700, 12000)
        pitch = ld_x * SIZE[dt]
        want = bool(bytes_of(BASE, tokens, 300 * SIZE[dt], pitch) &
                    bytes_of(y, tokens, 128, 2 * ld_y))
        assert linear(BASE, dt, ld_x, tokens, y, ld_y) == want, (dt, tokens, ld_x, ld_y, y - BASE)
        met += want
    assert 50 < met < 380


def test_the_16_bit_block_takes_columns_of_one_matrix():
    """y beside x, gradients beside each other and beside the inputs."""
    L = F.lib()
    st = L.gptq_ff_forward(ff(), FAR, 128, 100, FAR + 128, 128, None, 0, None, 0, None)
    assert st == B.GPTQ_ERR_WORKSPACE, B.gptq_last_error()

    def backward(dup, dx=5 * FAR):
        return L.gptq_ff_backward(ff(), FAR, 128, 100, 2 * FAR, 1 << 30, 4 * FAR, 64, dx, 128, 6 * FAR,
                                  128, dup, 128, 8 * FAR, 304, None, 0, None)
    assert backward(6 * FAR + 128, FAR + 128) == B.GPTQ_ERR_WORKSPACE, B.gptq_last_error()
    assert backward(6 * FAR + 126) == B.GPTQ_ERR_INVALID_ARG and said("overlap each other")
    assert backward(7 * FAR, FAR + 126) == B.GPTQ_ERR_INVALID_ARG and said("overlap the inputs")
