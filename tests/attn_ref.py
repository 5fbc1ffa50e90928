"""Plain 64-bit forms of the per-head norms with rotation, the 4-bit cache's rounding and
the attention over it, with error bounds that follow from the formulas and the kernels' number of
roundings.  CPU, numpy, no code of the library."""
from __future__ import annotations

import math

import numpy as np

F24 = 2.0 ** -24
HALF_STEP = {"bf16": 2.0 ** -8, "f32": F24}  # of a value, when it is rounded to the type
LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
GROUP, E_MIN, E_MAX = 32, -22, 13


# ---- norms and rotation

def norm_rope(x, norm, weight, bias, eps, rope, cos, sin, rot):
    """(y, size): the result of rows x (tokens, heads, D) in 64 bits and, for each value, the sum of the
    magnitudes that were added up to it.  cos, sin: (tokens, rot/2)."""
    x = np.asarray(x, np.float64)
    size = np.abs(x)
    if norm == "layer":
        size = size + size.mean(-1, keepdims=True)
        x = x - x.mean(-1, keepdims=True)
    if norm != "none":
        r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        x, size = x * r, size * r
    if weight is not None:
        x, size = x * weight, size * np.abs(weight)
    if bias is not None:
        x, size = x + bias, size + np.abs(bias)
    if rope == "none":
        return x, size
    i, j = pairs(rope, rot)
    c, s = np.asarray(cos, np.float64)[:, None], np.asarray(sin, np.float64)[:, None]
    y, t = x.copy(), size.copy()
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., j] * c + x[..., i] * s
    t[..., i] = t[..., j] = size[..., i] + size[..., j]
    return y, t


def pairs(rope, rot):
    p = np.arange(rot // 2)
    return (2 * p, 2 * p + 1) if rope == "interleaved" else (p, p + rot // 2)


def norm_rope_bound(y, size, dtype):
    """Half a step of the type, and the fp32 roundings before it: a lane adds 8 squares, lanes
    at most 32 (5 more sums), the mean likewise, then root, reciprocal, and five products and
    sums: under 64 roundings of quantities no larger than `size`."""
    return HALF_STEP[dtype] * np.abs(y) + 64 * F24 * size


# ---- the cache's rounding

def quantize(x):
    """The values that rows x (..., D) have in the cache: the nearest level by distance, ties to the
    level of even index."""
    x = np.asarray(x, np.float64)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    with np.errstate(all="ignore"):
        top = np.abs(g).max(-1, keepdims=True)
        bad = ~np.isfinite(top)
        e = np.full(top.shape, E_MIN)
        for k in range(E_MIN, E_MAX):  # the least e with top <= 6 * 2^e
            e = np.where(top > 6.0 * 2.0 ** k, k + 1, e)
        y = np.minimum(np.abs(g) / 2.0 ** e, 8)  # 6 is the nearest to all above
        d = np.abs(y[..., None] - LEVELS)
        d = np.where(np.isnan(d), 0, d)
        d[..., 1::2] += 1e-12  # a tie goes to the even index; levels are at least 2^-1 apart, ties exact
        out = LEVELS[d.argmin(-1)] * 2.0 ** e * np.where(np.signbit(g), -1, 1)
    return np.where(bad, np.nan, out).reshape(x.shape)


# ---- attention

def attention(q, k, v, n_q, scale, causal, window):
    """(out, lse, bound of out without the last rounding, bound of lse) for one sequence: q (n, Hq, D),
    k, v (len, Hk, D)."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n, hq, d = q.shape
    length, hk = k.shape[:2]
    share = hq // hk
    out, lse = np.zeros((n, hq, d)), np.full((n, hq), -np.inf)
    b_out, b_lse = np.zeros((n, hq, d)), np.zeros((n, hq))
    keys = np.arange(length)
    for i in range(n):
        at = length - n_q + i
        see = np.ones(length, bool) if not causal else keys <= at
        if causal and window:
            see &= keys > at - window
        if not see.any():
            continue
        for h in range(hq):
            kk, vv = k[see, h // share], v[see, h // share]
            s = kk @ q[i, h] * scale
            m = s.max() if not np.isnan(s).any() else np.nan
            p = np.exp(s - m)
            total = p.sum()
            out[i, h] = p @ vv / total
            lse[i, h] = m + math.log(total) if total == total else np.nan
            # a score is a sum of d exact products and is then scaled, shifted and raised: d + 8
            # roundings of at most its terms' magnitudes, or of the shift
            err = (d + 8) * F24 * (np.abs(kk) @ np.abs(q[i, h]) * scale + abs(m))
            w = p / total
            many = (len(s) + 64) * F24  # roundings of a sum over the keys and of joining parts
            b_out[i, h] = (w * 2 * err) @ np.abs(vv) + (w @ err + many) * (w @ np.abs(vv))
            b_lse[i, h] = (w * err).sum() * 2 + many + 4 * F24 * abs(lse[i, h])
    return out, lse, b_out, b_lse


# Half a step of a probability, relative to it: fp16 for bf16 queries, a sum of two fp16 for fp32.
P_STEP = {"bf16": 2.0 ** -11, "f32": 2.0 ** -22}


def out_bound(out, b_out, k_len, v, dtype, q_heads):
    """b_out with the rounding of the probabilities (of weights that sum to one, so of at most the largest
    |v| of the channel) and the last rounding."""
    top = np.nan_to_num(np.abs(np.asarray(v, np.float64))).max(0) if k_len else np.zeros(v.shape[1:])
    top = np.repeat(top, q_heads // top.shape[0], 0)
    return b_out + P_STEP[dtype] * top + HALF_STEP[dtype] * np.abs(out)
