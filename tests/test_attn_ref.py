"""The 64-bit forms that the GPU tests of the attention operators compare with, checked on the CPU against
definitions written another way, and planted mistakes that their bounds have to see."""
from __future__ import annotations

import math

import numpy as np
import pytest

import attn_ref as ref


def test_quantize_takes_the_nearest_level_and_the_least_scale():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((200, 32)) * np.exp(3 * rng.standard_normal((200, 1)))
    x[0], x[1, 3:] = 0, 0
    got = ref.quantize(x)
    for row, out in zip(x, got):
        top = np.abs(row).max()
        e = ref.E_MIN if top == 0 else min(max(math.ceil(math.log2(top / 6) - 1e-12), ref.E_MIN), ref.E_MAX)
        grid = np.concatenate([ref.LEVELS, -ref.LEVELS]) * 2.0 ** e
        assert np.allclose(np.abs(row - out), np.abs(row[:, None] - grid).min(1), rtol=0, atol=0)
        assert (np.abs(row - out) <= 2.0 ** e).all()


def test_quantize_ties_range_and_non_finite():
    x = np.zeros((5, 32))
    x[0, :9] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5]
    x[1, 0], x[2, 0], x[3, 5], x[4, 5] = 1e9, 1e-12, np.nan, -np.inf
    q = ref.quantize(x)
    assert q[0, :9].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -4]
    assert q[1, 0] == 6 * 2.0 ** 13 and q[2, 0] == 0
    assert np.isnan(q[3]).all() and np.isnan(q[4]).all()


@pytest.mark.parametrize("rope", ["interleaved", "half"])
def test_rotation_keeps_lengths_and_adds_angles(rope):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 2, 16))
    a, b = rng.standard_normal((2, 3, 4))
    once = lambda v, t: ref.norm_rope(v, "none", None, None, 0, rope, np.cos(t), np.sin(t), 8)[0]
    i, j = ref.pairs(rope, 8)
    y = once(x, a)
    assert np.allclose(y[..., i] ** 2 + y[..., j] ** 2, x[..., i] ** 2 + x[..., j] ** 2)
    assert np.array_equal(y[..., 8:], x[..., 8:])
    assert np.allclose(once(y, b), once(x, a + b))


def test_norms():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((4, 1, 64)) * 5 + 3
    y, _ = ref.norm_rope(x, "layer", None, None, 0, "none", None, None, 0)
    assert np.allclose(y.mean(-1), 0) and np.allclose(y.std(-1), 1)
    y, _ = ref.norm_rope(x, "rms", np.full(64, 2.0), None, 0, "none", None, None, 0)
    assert np.allclose((y ** 2).mean(-1), 4)


def _case():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((5, 4, 32)), rng.standard_normal((40, 2, 32)), rng.standard_normal((40, 2, 32))
    return q, k, v, 32 ** -0.5


def test_attention_against_whole_matrices():
    q, k, v, scale = _case()
    for causal, window in ((False, 0), (True, 0), (True, 7)):
        out, lse, _, _ = ref.attention(q, k, v, 5, scale, causal, window)
        for h in range(4):
            s = q[:, h] @ k[:, h // 2].T * scale
            at, key = 35 + np.arange(5)[:, None], np.arange(40)[None]
            if causal:
                s = np.where((key <= at) & ((key > at - window) if window else True), s, -np.inf)
            p = np.exp(s)
            assert np.allclose(out[:, h], p @ v[:, h // 2] / p.sum(1, keepdims=True))
            assert np.allclose(lse[:, h], np.log(p.sum(1)))


@pytest.mark.parametrize("mistake", ["a key too many", "a key too few", "heads in another order", "half the scale", "no rounding step"])
def test_bounds_see_mistakes(mistake):
    q, k, v, scale = _case()
    o, _, b, _ = ref.attention(q, k, v, 5, scale, True, 0)
    bound = ref.out_bound(o, b, 40, v, "bf16", 4)
    if mistake == "a key too many":
        wrong = ref.attention(q, k, v, 4, scale, True, 0)[0]
    elif mistake == "a key too few":
        wrong = ref.attention(q, k[1:], v[1:], 5, scale, True, 0)[0]
    elif mistake == "heads in another order":
        wrong = ref.attention(q, k[:, ::-1], v[:, ::-1], 5, scale, True, 0)[0]
    elif mistake == "half the scale":
        wrong = ref.attention(q, k, v, 5, scale / 2, True, 0)[0]
    else:  # 4-bit values where the cache holds others: an error of an eighth of a step
        wrong = ref.attention(q, k, v * (1 + 2.0 ** -5), 5, scale, True, 0)[0]
    assert (np.abs(wrong - o) > bound).mean() > 0.2
