"""Scoring of rows so wide that a group of tiles with one maximum holds several
tiles: unsplit rows of more than 32 tiles of 4096."""
import numpy as np
import pytest

from oracle import run_oracle as R
from tests.test_gpu_run import score_bounds, to_gpu, U32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,vocab,k", [(256, 135201, 20), (300, 200003, 64), (257, 262144, 5)])
def test_scores_of_unsplit_wide_rows(kind, rows, vocab, k):
    """Picked rows against the definition: alternatives in the last, partial
    group, in each tile of a group, tied across tiles and groups, and plain rows."""
    import torch
    from post_weight_quantization_layer_amd.scoring import TokenScorer
    rng = np.random.default_rng(vocab)
    x = to_gpu(rng.standard_normal((rows, vocab), dtype=np.float32), kind)
    at = [1, 2, 3, 4, 5, 6, 7, rows // 2, rows - 1]
    tiles = np.arange(0, vocab, 4096)
    with torch.no_grad():
        x[1, vocab - 3:] = 9.0                                  # the very end
        x[2, torch.from_numpy(tiles + 5 - 5 * (tiles + 5 >= vocab)).cuda()] = 8.0   # one in every tile
        x[3, 4096 + 7::8192] = 7.0                              # second tiles of pairs
        x[4, 8192 - 40:8192 + 40] = 6.5                         # a tie across a boundary
        x[5] = 1.0                                              # ties everywhere
        x[6, :vocab - 4000] = -np.inf                           # the last tiles only
        x[7, 100:] = -np.inf
    ids = rng.integers(0, vocab, rows)
    ids[1], ids[6], ids[7] = vocab - 2, vocab - 1, vocab - 1
    got = TokenScorer(rows, vocab, k)(x, torch.from_numpy(ids).cuda())
    seen = x[at].double().cpu().numpy()
    with np.errstate(all="ignore"):
        want = R.token_logprobs(seen, ids[at], 1.0, k)
        log_s, ent = score_bounds(seen, want, 1.0)
    np.testing.assert_array_equal(got.rank.cpu().numpy()[at], want[1])
    np.testing.assert_array_equal(got.top_ids.cpu().numpy()[at], want[3])
    for a, b, tol in ((got.logprob, want[0], log_s), (got.top_logprobs, want[4], log_s[:, None]),
                      (got.entropy, want[2], ent)):
        a = a.double().cpu().numpy()[at]
        fin = np.isfinite(b)
        np.testing.assert_array_equal(np.where(fin, 0, a), np.where(fin, 0, b))
        # a log probability's own difference and last sum, as for narrower rows
        own = 6 * U32 * (np.abs(np.where(fin, b, 0)) + 2 * np.log(vocab + 1.0)) + 1e-30
        err = np.abs(np.where(fin, a, 0) - np.where(fin, b, 0))
        assert (err <= tol + own).all(), float((err / (tol + own)).max())
