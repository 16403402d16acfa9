"""TokenLogprobs.perplexity: over every row that has a given token, whatever
the row holds (no GPU)."""
import math

import pytest

torch = pytest.importorskip("torch")

from post_weight_quantization_layer_amd.scoring import TokenLogprobs


def result(logprob, rank, ids):
    n = len(logprob)
    return TokenLogprobs(torch.tensor(logprob), torch.tensor(rank, dtype=torch.int32),
                         torch.zeros(n), torch.zeros((n, 0), dtype=torch.int32),
                         torch.zeros((n, 0)), torch.tensor(ids))


def test_mean_over_given_tokens():
    got = result([-1.0, 0.0, -3.0], [2, -1, 0], [5, -1, 7]).perplexity()
    assert got == pytest.approx(math.exp(2.0), rel=1e-12)


def test_rows_that_could_not_be_scored_count():
    """A NaN or +infinity in the row, or a token outside the vocabulary."""
    assert math.isnan(result([-1.0, math.nan, -1.0], [0, -1, 3], [5, 6, 7]).perplexity())
    assert math.isnan(result([math.nan], [-1], [10 ** 6]).perplexity())


def test_rows_without_a_token_do_not_count_even_if_bad():
    got = result([-2.0, math.nan, 0.0], [1, -1, -1], [3, -1, -100]).perplexity()
    assert got == pytest.approx(math.exp(2.0), rel=1e-12)
    assert math.isnan(result([0.0], [-1], [-1]).perplexity())        # nothing to score


def test_impossible_and_nearly_impossible_tokens():
    assert result([-math.inf, -1.0], [9, 0], [1, 2]).perplexity() == math.inf
    assert result([-3.4e38, -1.0], [9, 0], [1, 2]).perplexity() == math.inf   # past float64's exp
    assert result([-700.0], [9], [1]).perplexity() == pytest.approx(math.exp(700.0))


def test_without_ids():
    empty = TokenLogprobs(None, None, torch.zeros(2), torch.zeros((2, 0)), torch.zeros((2, 0)))
    with pytest.raises(ValueError, match="ids"):
        empty.perplexity()
