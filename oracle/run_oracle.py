"""Float64 definitions of the operators that run and score a per-row 8-bit
layer (shares no code with the HIP path).

Integer decisions (token codes) are taken in float32 with the IEEE quotient,
as the definition states them, so they can be compared exactly; everything
else is float64."""
import numpy as np


def token_codes(x):
    """x: tokens x cols float32 (exactly the stored activations).

    Returns (codes int8, scale float32, sum int32): scale = max|x| / 127 and
    codes = clamp(rint(x / scale)) in float32; a zero row has codes 0; a row
    with a NaN or an infinity has scale NaN and codes 0."""
    x = np.asarray(x, np.float32)
    bad = ~np.isfinite(x).all(axis=1)
    amax = np.where(bad, np.float32(0), np.abs(np.where(np.isfinite(x), x, 0)).max(axis=1))
    scale = (amax.astype(np.float32) / np.float32(127)).astype(np.float32)
    q = np.zeros(x.shape, np.int8)
    for t in np.nonzero(~bad & (scale > 0))[0]:
        q[t] = np.clip(np.rint(x[t] / scale[t]), -127, 127).astype(np.int8)
    scale[bad] = np.nan
    return q, scale, q.astype(np.int64).sum(axis=1).astype(np.int32)


def silu_mul(g, u):
    g, u = np.asarray(g, np.float64), np.asarray(u, np.float64)
    return g / (1 + np.exp(-g)) * u


def product_sums(q, codes, zero):
    """sum_k q[t][k] (codes[r][k] - zero[r]), exact, tokens x rows int64."""
    w = codes.astype(np.int64) - zero.astype(np.int64).reshape(-1, 1)
    # exact in float64: |sum| <= 127 * 255 * 65536 < 2^53
    return (q.astype(np.float64) @ w.T.astype(np.float64)).astype(np.int64)


def norm(v, kind, weight=None, bias=None, eps=0.0, offset=0.0):
    v = np.asarray(v, np.float64)
    if kind in (None, "none"):
        return v
    if kind == "layer":
        v = v - v.mean(axis=1, keepdims=True)
    y = v / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)
    if weight is not None:
        y = y * (offset + np.asarray(weight, np.float64))
    return y if bias is None else y + np.asarray(bias, np.float64)


def norm_block(r, b=None, gate=None, *, post=None, post_weight=None, post_bias=None, pre=None,
               pre_weight=None, pre_bias=None, residual_scale=1.0, block_scale=1.0, eps=0.0,
               weight_offset=0.0):
    """gate: tokens x d (already one row per token) or None.  Returns (r', h)."""
    out = residual_scale * np.asarray(r, np.float64)
    if b is not None:
        p = norm(b, post, post_weight, post_bias, eps, weight_offset)
        out = out + block_scale * (p if gate is None else np.asarray(gate, np.float64) * p)
    return out, norm(out, pre, pre_weight, pre_bias, eps, weight_offset)


def token_logprobs(logits, ids, scale=1.0, top_k=0):
    """Row by row from the definition.  Returns logprob, rank, entropy, top_ids, top_logprobs."""
    rows, vocab = logits.shape
    logprob, entropy = np.zeros(rows), np.zeros(rows)
    rank = np.full(rows, -1, np.int32)
    top_ids = np.full((rows, top_k), -1, np.int32)
    top_lp = np.full((rows, top_k), -np.inf)
    for t in range(rows):
        x = logits[t].astype(np.float64)
        i = int(ids[t])
        if np.isnan(x).any() or np.isposinf(x).any():
            logprob[t], entropy[t], top_lp[t] = np.nan, np.nan, np.nan
            continue
        order = np.lexsort((np.arange(vocab), -x))
        m = x.max()
        if np.isneginf(m):
            lp = np.full(vocab, -np.inf)
        else:
            e = np.exp(scale * (x - m))
            lp = scale * (x - m) - np.log(e.sum())
            seen = e > 0
            entropy[t] = -(e[seen] / e.sum() * lp[seen]).sum()
        if i >= vocab:
            logprob[t] = np.nan
        elif i >= 0:
            logprob[t] = lp[i]
            rank[t] = int(np.nonzero(order == i)[0][0])
        best = [v for v in order[:top_k] if np.isfinite(x[v])]
        top_ids[t, :len(best)] = best
        top_lp[t, :len(best)] = lp[best]
    return logprob, rank, entropy, top_ids, top_lp
