"""Scoring rows whose masks are large finite values, and rows far from zero,
against the float64 definition, within the bounds of the other scoring tests."""
import numpy as np
import pytest

from tests.test_gpu_run import check_scores

pytestmark = pytest.mark.gpu


def masked_rows(rng, vocab, mask):
    """Masked by a value rather than by -infinity: a few tokens allowed, a tenth,
    none, all but the first tile's, one, and alternating halves of a lane's eight."""
    x = rng.standard_normal((7, vocab)).astype(np.float32) * 3
    x[0, 10:] = mask
    x[1, rng.random(vocab) < 0.9] = mask
    x[2] = mask
    x[3, :4096] = mask
    x[4] = mask
    x[4, vocab // 2] = 1.5
    x[5, np.arange(vocab) % 8 < 4] = mask
    x[6] += np.float32(mask)                      # an added mask, values apart where they can be
    return x


@pytest.mark.parametrize("vocab", [9000, 130001])
@pytest.mark.parametrize("mask", [-1e4, -1e6, -3e6, -1e8, -1e9, -1e10, -1e12, -1e20, -1e30, -1e38])
def test_scores_masked_by_finite_values(vocab, mask):
    rng = np.random.default_rng(vocab)
    x = masked_rows(rng, vocab, mask)
    ids = rng.integers(0, vocab, 7)
    ids[0] = 3
    for scale in (1.0, 0.8, 2.0):
        check_scores(x, ids, "f32", scale, 5, "plain", f"mask {mask} scale {scale}")
    check_scores(x, ids, "bf16", 1.25, 20, "odd", f"mask {mask} bf16")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("power", [12, 16, 20, 21, 22, 23, 26, 31, 40, 70, 100])
def test_scores_of_rows_far_from_zero(kind, sign, power):
    """Rows around one large value, whose lanes' maxima differ by a few steps of
    the type, and rows that run from -2^power to 2^power."""
    rng = np.random.default_rng(power)
    base = np.float32(sign * 2.0 ** power)
    step = np.spacing(np.abs(base)) * (1 if kind == "f32" else 2 ** 16)
    x = (base + step * rng.integers(-9, 9, (4, 20000))).astype(np.float32)
    x[2, rng.random(20000) < 0.5] = 0
    x[3] = np.linspace(-base, base, 20000)
    ids = rng.integers(0, 20000, 4)
    for scale in (1.0, 0.7 / float(step), 1.0 / float(abs(base))):
        check_scores(x, ids, kind, max(scale, 1e-30), 7, "plain", f"2^{power} scale {scale:.2e}")
