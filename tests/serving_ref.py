"""Plain forms of the 8-bit cache's writer, of attention over rows and over that cache (64 bits, with bounds that follow
from the formulas and the kernels' roundings), and of the operations on pages (lists).  CPU, numpy, no code of the
library."""
from __future__ import annotations

import numpy as np

import attn_ref

BLOCK, E_MIN, E_MAX = 16, -15, 7
# magnitudes of codes 0 .. 126
LEVELS = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)])


def round_e4m3(x, e):
    """What is held of x at the scale 2^e: the nearest level by distance, ties to the level of even index; NaN for
    what is not finite."""
    x = np.asarray(x, np.float64)
    unit = 2.0 ** np.asarray(e, np.float64)
    with np.errstate(all="ignore"):
        y = np.minimum(np.abs(x) / unit, 448.0)
    y = np.where(np.isfinite(x), y, 0)
    hi = np.clip(np.searchsorted(LEVELS, y), 1, 126)
    a, b = y - LEVELS[hi - 1], LEVELS[hi] - y
    low = (a < b) | ((a == b) & (hi % 2 == 1))
    return np.where(np.isfinite(x), np.copysign(np.where(low, LEVELS[hi - 1], LEVELS[hi]), x) * unit, np.nan)


def exponent(top):
    """The least e with top <= 448 * 2^e, within its limits."""
    e = np.full(np.shape(top), E_MIN)
    for k in range(E_MIN, E_MAX):
        e = np.where(np.asarray(top) > 448.0 * 2.0 ** k, k + 1, e)
    return e


class Held:
    """What one sequence holds of K or V: rows (tokens, heads, D) and the exponents of each 16 of them."""

    def __init__(self, heads, dim):
        self.x = np.zeros((0, heads, dim))
        self.e = np.zeros((0, heads), int)

    def append(self, rows):
        rows = np.asarray(rows, np.float64)
        while len(rows):
            at = len(self.x) % BLOCK
            new, rows = rows[:BLOCK - at], rows[BLOCK - at:]
            e = exponent(np.where(np.isfinite(new), np.abs(new), 0).max((0, 2)))
            if at:
                e = np.maximum(e, self.e[-1])
                grown = (e > self.e[-1])[None, :, None]
                self.x[-at:] = np.where(grown, round_e4m3(self.x[-at:], e[:, None]), self.x[-at:])
                self.e[-1] = e
            else:
                self.e = np.concatenate([self.e, e[None]])
            self.x = np.concatenate([self.x, round_e4m3(new, e[:, None])])

    def cut(self, tokens):
        """Forgets what is behind; the scale of the last 16 stays."""
        self.x, self.e = self.x[:tokens].copy(), self.e[:-(-tokens // BLOCK)].copy()


# ---- attention

# Half a step of a probability relative to it: in bf16, in fp16, as bf16 parts that add up to it (rounded in fp32).
P_BF16, P_FP16, P_PARTS = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24


def attention(q, k, v, scale, causal, window, p_step, products=1, kind="bf16"):
    """(out, lse, bound of out, bound of lse) for one sequence.  p_step: rounding of a probability; products: how many
    products of parts make one of the formula's (their sum has so many times the roundings, and leaves out 2^-24 of each
    factor pair where it is more than one); kind: the type of the result."""
    n = len(q)
    o, l, b, bl = attn_ref.attention(q, k, v, n, scale, causal, window)
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    share = q.shape[1] // max(k.shape[1], 1)
    # weights sum to one, so an error of p_step of each is at most that of the mean of |v| under them
    size = np.zeros_like(o)
    more = np.zeros(o.shape[:2])
    keys = np.arange(len(k))
    for i in range(n):
        at = len(k) - n + i
        see = np.ones(len(k), bool) if not causal else keys <= at
        if causal and window:
            see &= keys > at - window
        for h in range(q.shape[1]):
            if not see.any():
                continue
            kk, vv = k[see, h // share], v[see, h // share]
            w = np.exp(kk @ q[i, h] * scale - l[i, h])
            size[i, h] = w @ np.abs(vv)
            if products > 1:  # of a score, and so of a weight and of lse
                more[i, h] = ((products - 1) * q.shape[2] + 1) * attn_ref.F24 * (w @ (np.abs(kk) @ np.abs(q[i, h]))) * scale
                b[i, h] += (2 * more[i, h] + (products * len(kk) + 1) * attn_ref.F24) * size[i, h] \
                    + ((products - 1) * q.shape[2] + 1) * attn_ref.F24 * scale * ((w * (np.abs(kk) @ np.abs(q[i, h]))) @ np.abs(vv))
    # a probability's parts below 2^-126, fp32's smallest normal number, may count as nothing; the largest is at least one
    least = 3 * len(k) * 2.0 ** -126 * (np.nan_to_num(np.abs(v)).max() if v.size else 0)
    return o, l, b + p_step * size + attn_ref.HALF_STEP[kind] * np.abs(o) + least, bl + 2 * more


# ---- pages

def count_refs(pages, table, lens, page):
    refs = [0] * pages
    for row, n in zip(table, lens):
        for p in row[:-(-n // page)]:
            if 0 <= p < pages:
                refs[p] += 1
    return refs


def resize(refs, table, lens, page, want):
    """(refs, table, lens, missing), row by row with a list of the free pages."""
    refs, width = list(refs), len(table[0])
    held = [list(t[:-(-n // page)]) for t, n in zip(table, lens)]
    lens = list(lens)
    for r, w in enumerate(want):
        if 0 <= w <= width * page:
            for p in held[r][-(-w // page):]:
                if 0 <= p < len(refs):
                    refs[p] -= 1
            if w < lens[r]:
                held[r], lens[r] = held[r][:-(-w // page)], w
    free = [p for p, c in enumerate(refs) if c == 0]
    asked = missing = 0
    for r, w in enumerate(want):
        if w < 0:
            continue
        if w > width * page:
            missing += 1
            continue
        need = -(-w // page) - len(held[r])
        if need > 0:
            asked += need
            if asked > len(free):
                missing += 1
                continue
            for p in free[asked - need:asked]:
                held[r].append(p)
                refs[p] = 1
        lens[r] = w
    return refs, [h + [-1] * (width - len(h)) for h in held], lens, missing


def fork(refs, table, lens, page, parents):
    """(refs, table, lens, src, dst, missing)."""
    refs, rows, width = list(refs), len(table), len(table[0])
    held = [list(t[:-(-n // page)]) for t, n in zip(table, lens)]
    par = [p if 0 <= p < rows else -1 for p in parents]
    keeper = {}
    for r in range(rows):
        if par[r] >= 0:
            keeper.setdefault(par[r], r)
    for r in range(rows):
        if par[r] == r:
            keeper[r] = r
    for h in held:
        for p in h:
            if 0 <= p < len(refs):
                refs[p] -= 1
    new, asks = [], []
    for r in range(rows):
        h = list(held[par[r]]) if par[r] >= 0 else []
        if par[r] >= 0 and lens[par[r]] % page and keeper[par[r]] != r and 0 <= h[-1] < len(refs):
            asks.append((r, h.pop()))
        new.append(h)
        for p in h:
            if 0 <= p < len(refs):
                refs[p] += 1
    size = [lens[p] if p >= 0 else 0 for p in par]
    src, dst, missing = [-1] * rows, [-1] * rows, 0
    free = [p for p, c in enumerate(refs) if c == 0]
    for i, (r, p) in enumerate(asks):
        if i >= len(free):
            size[r] = size[r] // page * page
            missing += 1
            continue
        src[r], dst[r] = p, free[i]
        new[r].append(free[i])
        refs[free[i]] = 1
    return refs, [h + [-1] * (width - len(h)) for h in new], size, src, dst, missing


def compact(refs, table):
    """(refs, table, pairs)."""
    used = [p for p, c in enumerate(refs) if c]
    pairs = list(zip([p for p in used if p >= len(used)], [p for p, c in enumerate(refs) if not c]))
    to = dict(pairs)
    out = [0] * len(refs)
    for p in used:
        out[to.get(p, p)] = refs[p]
    return out, [[to.get(p, p) for p in row] for row in table], pairs


def fork_own(refs, table, lens, page, parents):
    """The fork after which a last, partly filled page is one row's alone: (refs, table, lens, src, dst, missing)."""
    pages, rows, width = len(refs), len(table), len(table[0])
    held = [list(t[:-(-n // page)]) for t, n in zip(table, lens)]
    par = [p if 0 <= p < rows else -1 for p in parents]
    new, size = [list(held[p]) if p >= 0 else [] for p in par], [lens[p] if p >= 0 else 0 for p in par]
    whole, claims = set(), {}
    for r, h in enumerate(new):
        for j, p in enumerate(h):
            if 0 <= p < pages:
                if (j + 1) * page > size[r]:
                    claims.setdefault(p, []).append(r)
                else:
                    whole.add(p)
    asks = {}
    for p, of in claims.items():
        stay = [r for r in of if par[r] == r] or of
        for r in of:
            if p in whole or r != stay[0]:
                asks[r] = p
                new[r].pop()
    refs = [0] * pages
    for h in new:
        for p in h:
            if 0 <= p < pages:
                refs[p] += 1
    free = [p for p, c in enumerate(refs) if c == 0]
    src, dst, missing = [-1] * rows, [-1] * rows, 0
    for r in sorted(asks):
        if free:
            src[r], dst[r] = asks[r], free.pop(0)
            new[r].append(dst[r])
            refs[dst[r]] = 1
        else:
            size[r] = size[r] // page * page
            missing += 1
    return refs, [h + [-1] * (width - len(h)) for h in new], size, src, dst, missing


# ---- rounding by rounding

def one_key(q, k, v, scale):
    """(out, lse, bound of out, bound of lse) of rows (n, D) that see one key each, fp32 operands of which q and k have one
    channel that is not zero, |score| at least 64 and scale a power of two: few roundings, so that products of
    parts that are left out show.  In units of 2^-24 of the value:
      score: 1 of what six products leave out, 2 of the last sum (the sums before it are 2^-8 of it), 2 of scale * log2 e
      lse: the score, 1 of m + log2 p, 2 of the product with ln 2, and 8 of a unit (p's exponent below one, exp2 and log2 within 2 of
           their last places each), an eighth of one of 64
      out: 1 of what is left out, 2 of the last sum, 2 of the reciprocal of p, 1 of the product with it"""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    lse = (q * k).sum(-1) * scale
    assert (np.abs(lse) >= 64).all()
    return v, lse, 6 * attn_ref.F24 * np.abs(v), 9 * attn_ref.F24 * np.abs(lse)


def one_key_rows(rng, n, dim):
    """q, k, v (n, dim) fp32 for it, with a score of 64 to 256 at a scale of 1/4 whose parts are all there."""
    q, k = (np.zeros((n, dim), np.float32) for _ in range(2))
    at = np.arange(n), np.arange(n) % dim
    q[at], k[at] = (rng.uniform(16, 32, n).astype(np.float32) * rng.choice([-1, 1], n).astype(np.float32) for _ in range(2))
    return q, k, (rng.uniform(1, 2, (n, dim)) * rng.choice([-1, 1], (n, dim))).astype(np.float32)


def two_keys(x, p_step):
    """(out, bound) of rows of bf16 that see a key of score 0 and value 1 and one of score x, at most an eighth, and value -1:
    the values all but cancel, so that the probabilities' rounding shows beside the result's.  A probability is off by at
    most p_step of the larger of the two."""
    x = np.asarray(x, np.float64)
    assert (np.abs(x) <= 0.125).all()
    w = 1 / (1 + np.exp(-np.abs(x)))
    out = -np.tanh(x / 2)
    # fp32: a handful of roundings of numbers up to one
    return out, 2 * w * p_step + attn_ref.HALF_STEP["bf16"] * np.abs(out) + 16 * attn_ref.F24
