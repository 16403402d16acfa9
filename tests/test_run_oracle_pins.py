"""Pins of the float64 definitions behind the 8-bit product, the norm block
and the token scoring: values derived by hand, brute force, invariances."""
import math

import numpy as np
import pytest

from oracle import run_oracle as R


def test_token_codes_worked():
    # scale 2 = 254 / 127; 3 / 2 = 1.5 and 1 / 2 = 0.5 are ties, to even
    q, s, n = R.token_codes([[254.0, -254.0, 3.0, 1.0, -5.0, 0.0]])
    assert s[0] == 2.0
    np.testing.assert_array_equal(q[0], [127, -127, 2, 0, -2, 0])
    assert n[0] == 0


def test_token_codes_special_rows():
    q, s, n = R.token_codes([[0, 0, 0], [1, np.nan, 2], [np.inf, 1, 2], [1e-45, 0, 0]])
    assert s[0] == 0 and np.isnan(s[1]) and np.isnan(s[2]) and s[3] == 0
    assert not q.any() and not n.any()


def test_product_sums_brute_force():
    rng = np.random.default_rng(0)
    q = rng.integers(-127, 128, (3, 9)).astype(np.int8)
    c = rng.integers(0, 256, (4, 9)).astype(np.uint8)
    z = rng.integers(0, 256, 4).astype(np.uint8)
    got = R.product_sums(q, c, z)
    for t in range(3):
        for r in range(4):
            assert got[t, r] == sum(int(q[t, k]) * (int(c[r, k]) - int(z[r])) for k in range(9))


def test_norms_worked():
    v = [[3.0, -4.0]]
    rms = math.sqrt(12.5)
    np.testing.assert_allclose(R.norm(v, "rms"), [[3 / rms, -4 / rms]], rtol=1e-15)
    np.testing.assert_allclose(R.norm(v, "layer"), [[1, -1]], rtol=1e-15)
    np.testing.assert_allclose(R.norm(v, "rms", [1, 2], [10, 20], 0.0, 1.0),
                               [[10 + 6 / rms, 20 - 12 / rms]], rtol=1e-15)
    np.testing.assert_allclose(R.norm(v, "rms", eps=12.5), [[3 / 5, -4 / 5]], rtol=1e-15)


def test_norm_block_worked_and_invariant():
    r, h = R.norm_block([[1.0, 1.0]], [[3.0, -4.0]], [[0.5, 2.0]], post="layer", pre="rms",
                        residual_scale=2.0, block_scale=4.0)
    np.testing.assert_allclose(r, [[2 + 4 * 0.5, 2 - 4 * 2.0]], rtol=1e-15)
    np.testing.assert_allclose(h, np.array([[4.0, -6.0]]) / math.sqrt(26), rtol=1e-15)
    rng = np.random.default_rng(1)
    b = rng.standard_normal((4, 32))
    a = R.norm_block(np.zeros((4, 32)), b, post="rms")[0]
    np.testing.assert_allclose(R.norm_block(np.zeros((4, 32)), 7 * b, post="rms")[0], a, rtol=1e-12)
    c = R.norm_block(np.zeros((4, 32)), b + 5, post="layer")[0]
    np.testing.assert_allclose(c, R.norm_block(np.zeros((4, 32)), b, post="layer")[0], rtol=1e-10)


def test_logprobs_worked():
    # probabilities 1/2, 1/4, 1/4 in two layouts, and a temperature
    x = np.log([[2.0, 1.0, 1.0], [1.0, 2.0, 1.0]])
    lp, rank, ent, ids, tlp = R.token_logprobs(x, [2, 0], 1.0, 3)
    np.testing.assert_allclose(lp, [-math.log(4), -math.log(4)], rtol=1e-14)
    np.testing.assert_array_equal(rank, [2, 1])
    np.testing.assert_allclose(ent, [1.5 * math.log(2)] * 2, rtol=1e-14)
    np.testing.assert_array_equal(ids, [[0, 1, 2], [1, 0, 2]])
    np.testing.assert_allclose(tlp[0], [-math.log(2), -math.log(4), -math.log(4)], rtol=1e-14)
    lp, *_ = R.token_logprobs(x, [0, 1], 2.0)
    np.testing.assert_allclose(lp, [math.log(4 / 6)] * 2, rtol=1e-14)


@pytest.mark.parametrize("fill,want_lp,want_ids", [
    (-np.inf, -np.inf, -1), (np.nan, np.nan, -1), (np.inf, np.nan, -1)])
def test_logprobs_special_rows(fill, want_lp, want_ids):
    lp, rank, ent, ids, tlp = R.token_logprobs(np.full((1, 4), fill), [1], 1.0, 2)
    np.testing.assert_array_equal(lp, [want_lp])
    assert (ids == want_ids).all() and tlp.shape == (1, 2)
    assert rank[0] == (1 if np.isneginf(fill) else -1)
    assert (ent[0] == 0) if np.isneginf(fill) else np.isnan(ent[0])


def test_logprobs_missing_and_outside_tokens():
    lp, rank, *_ = R.token_logprobs(np.zeros((2, 3)), [-1, 3], 1.0)
    assert lp[0] == 0 and np.isnan(lp[1]) and (rank == -1).all()


def test_logprobs_agree_with_differences():
    """d logprob / d l_v = scale (1[v = id] - p_v), against central differences."""
    rng = np.random.default_rng(2)
    x, h = rng.standard_normal((1, 6)), 1e-6
    base = R.token_logprobs(x, [3], 0.7, 6)
    p = np.zeros(6)
    p[base[3][0]] = np.exp(base[4][0])
    for v in range(6):
        up, dn = x.copy(), x.copy()
        up[0, v] += h
        dn[0, v] -= h
        diff = (R.token_logprobs(up, [3], 0.7)[0] - R.token_logprobs(dn, [3], 0.7)[0]) / (2 * h)
        assert abs(diff[0] - 0.7 * ((v == 3) - p[v])) < 1e-8
