"""silu(g) u over the whole range of g, through the scale of rows of one feature:
scale = |silu(g) u| / 127.

Bound, in units of u = 2^-24 of the value: 2^t is within 1 ulp (2), its argument's
rounding error put back with one operation (1), the sum with 1 adds 1, the
reciprocal is within 1 ulp (2), the product with g adds 1: 7.  For g < -83 two
exponentials of 2 and two products make 6.  The product with u and the division
by 127 add 1 each: 9 in all; below float32's normal range the last steps round to
multiples of 2^-149."""
import numpy as np
import pytest

from tests.test_gpu_run import U32, to_gpu

pytestmark = pytest.mark.gpu


def scales(g, u):
    from post_weight_quantization_layer_amd.w8a8 import silu_mul_quantize
    out = silu_mul_quantize(to_gpu(g[:, None]), to_gpu(u[:, None]))
    return (out.scale.cpu().numpy().astype(np.float64), out.codes[:, 0].cpu().numpy(),
            out.sum.cpu().numpy())


def test_silu_over_its_range():
    rng = np.random.default_rng(1)
    n = 1 << 18
    g = np.concatenate([np.linspace(-104, 104, n), rng.uniform(-92, -80, n), rng.uniform(80, 92, n),
                        rng.standard_normal(n), np.exp(rng.uniform(-80, 5, n)),
                        -np.exp(rng.uniform(-80, 4.6, n)), [0.0, -0.0, 1e38, -1e38, 1e-45, -1e-45]])
    g = g.astype(np.float32)
    u = (rng.uniform(0.5, 2, len(g)) * rng.choice([-1, 1], len(g))).astype(np.float32)
    s, q, total = scales(g, u)
    g64, u64 = g.astype(np.float64), u.astype(np.float64)
    with np.errstate(over="ignore"):
        a = g64 / (1 + np.exp(-g64)) * u64
    a[np.abs(g) > 1e37] = np.where(g64 > 0, g64, 0)[np.abs(g) > 1e37] * u64[np.abs(g) > 1e37]
    want = np.abs(a) / 127
    err = np.abs(s - want)
    tol = 9.01 * U32 * want + 2.0 ** -149
    worst = int(np.argmax(err / tol))
    assert err[worst] <= tol[worst], (g[worst], s[worst], want[worst])
    sure = want > 2.0 ** -141           # a scale below this is off by more than a 254th
    assert (q[sure] == 127 * np.sign(a[sure])).all() and (total == q).all()


def test_silu_of_infinities_and_nan():
    """The quotient's own values: infinity, -infinity / infinity, NaN.  All mark the row."""
    g = np.array([np.inf, -np.inf, np.nan, 1.0], np.float32)
    s, q, total = scales(g, np.ones(4, np.float32))
    assert np.isnan(s[:3]).all() and np.isfinite(s[3])
    assert (q[:3] == 0).all() and q[3] == 127 and (total == q).all()
