"""The plain forms that the serving operators' GPU tests use, checked by other means, and planted mistakes that those
checks see."""
import numpy as np
import pytest

import serving_ref as ref


def test_levels_are_e4m3():
    assert len(ref.LEVELS) == 127 and (np.diff(ref.LEVELS) > 0).all()
    assert ref.LEVELS[1] == 2.0 ** -9 and ref.LEVELS[8] == 2.0 ** -6 and ref.LEVELS[126] == 448
    import torch

    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, ref.LEVELS)


def test_rounding_is_to_the_nearest_with_ties_to_even():
    import torch

    rng = np.random.default_rng(0)
    mid = (ref.LEVELS[1:] + ref.LEVELS[:-1]) / 2
    x = np.concatenate([ref.LEVELS, mid, np.nextafter(mid, 0), np.nextafter(mid, 1e9), rng.uniform(0, 448, 5000), 2.0 ** rng.uniform(-12, 8, 5000)])
    x = np.concatenate([x, -x])
    want = torch.from_numpy(x).float()
    keep = want.double().numpy() == x  # the other rounding starts from fp32
    assert np.array_equal(ref.round_e4m3(x[keep], 0), want[keep].to(torch.float8_e4m3fn).double().numpy())
    assert ref.round_e4m3(1e9, 0) == 448 and ref.round_e4m3(-460.0, 0) == -448
    assert np.isnan(ref.round_e4m3(np.array([np.nan, np.inf, -np.inf]), 3)).all()
    assert np.array_equal(ref.round_e4m3(x * 2.0 ** 5, 5), ref.round_e4m3(x, 0) * 2.0 ** 5)


def test_exponents():
    for top, e in ((0, -15), (448, 0), (448.0001, 1), (224, -1), (1e-30, -15), (1e30, 7), (448 * 128, 7), (448 * 64, 6)):
        assert ref.exponent(top) == e, top


def test_held_tokens_keep_or_raise_their_scale():
    h = ref.Held(1, 4)
    h.append(np.full((3, 1, 4), 1.0))
    assert h.e.tolist() == [[-8]] and (h.x == 1).all()
    h.append(np.full((1, 1, 4), 300.0))
    assert h.e.tolist() == [[0]] and (h.x[:3] == 1).all() and (h.x[3] == ref.round_e4m3(300.0, 0)).all()
    h.append(np.full((13, 1, 4), 2.0 ** -11))  # below half of the least level
    assert h.e.tolist() == [[0], [ref.exponent(2.0 ** -11)]] and (h.x[4:16] == 0).all() and h.x[16, 0, 0] == 2.0 ** -11
    # what is already held is rounded again when the scale grows, and not before
    h = ref.Held(1, 1)
    h.append(np.array([[[2.0 ** -20]]]))
    assert h.x[0, 0, 0] == 2.0 ** -20
    h.append(np.array([[[448.0]]]))
    assert h.x[0, 0, 0] == 0
    h.cut(1)
    h.append(np.array([[[1.0]]]))
    assert h.e.tolist() == [[0]]


def random_state(rng, pages, rows, width, page):
    lens = [int(rng.integers(0, width * page + 1)) for _ in range(rows)]
    table = [[-1] * width for _ in range(rows)]
    order = rng.permutation(pages).tolist()
    for r in range(rows):
        for j in range(-(-lens[r] // page)):
            share = [t[j] for t in table[:r] if t[j] >= 0]
            table[r][j] = share[0] if share and rng.random() < 0.3 else order.pop() if order else -1
        if -1 in table[r][:-(-lens[r] // page)]:
            lens[r] = table[r].index(-1) * page
            table[r][lens[r] // page:] = [-1] * (width - lens[r] // page)
    return ref.count_refs(pages, table, lens, page), table, lens


@pytest.mark.parametrize("seed", range(30))
def test_pages_stay_counted(seed):
    rng = np.random.default_rng(seed)
    page, rows, width = int(rng.choice([1, 3, 16])), int(rng.integers(1, 9)), int(rng.integers(1, 7))
    pages = int(rng.integers(1, rows * width + 5))
    refs, table, lens = random_state(rng, pages, rows, width, page)
    for _ in range(6):
        want = [int(rng.integers(-1, width * page + 2)) for _ in range(rows)]
        was = lens
        refs, table, lens, missing = ref.resize(refs, table, lens, page, want)
        assert refs == ref.count_refs(pages, table, lens, page)
        assert sum(1 for w, n, o in zip(want, lens, was) if w >= 0 and n != w) == missing
        parents = [int(rng.integers(-1, rows)) for _ in range(rows)]
        old = [list(t) for t in table]
        o_lens = lens
        refs, table, lens, src, dst, missing = ref.fork(refs, table, lens, page, parents)
        assert refs == ref.count_refs(pages, table, lens, page)
        back = {d: s for s, d in zip(src, dst) if d >= 0}
        for r, p in enumerate(parents):
            n = -(-lens[r] // page)
            assert lens[r] <= (o_lens[p] if p >= 0 else 0)
            assert [back.get(x, x) for x in table[r][:n]] == old[p][:n] if p >= 0 else n == 0
        refs, table, pairs = ref.compact(refs, table)
        assert refs == ref.count_refs(pages, table, lens, page)
        assert all(c > 0 for c in refs[:sum(1 for c in refs if c)])


def last_pages(table, lens, page):
    """(row, page) of the last, partly filled ones."""
    return [(r, t[n // page]) for r, (t, n) in enumerate(zip(table, lens)) if n % page]


@pytest.mark.parametrize("seed", range(30))
def test_a_fork_parts_rows_that_shrank_into_a_page(seed):
    rng = np.random.default_rng(1000 + seed)
    page, rows, width = int(rng.choice([1, 3, 16])), int(rng.integers(1, 9)), int(rng.integers(1, 7))
    pages = int(rng.integers(1, rows * width + 5))
    refs, table, lens = random_state(rng, pages, rows, width, page)
    for _ in range(6):
        want = [int(rng.integers(-1, width * page + 2)) for _ in range(rows)]
        refs, table, lens, _ = ref.resize(refs, table, lens, page, want)
        parents = [int(rng.integers(-1, rows)) if rng.random() < 0.5 else r for r in range(rows)]
        old, o_lens = [list(t) for t in table], lens
        refs, table, lens, src, dst, missing = ref.fork_own(refs, table, lens, page, parents)
        assert refs == ref.count_refs(pages, table, lens, page)
        assert all(refs[p] == 1 for _, p in last_pages(table, lens, page))
        assert not set(dst) & set(src) - {-1} and all(refs[s] > 0 for s in src if s >= 0)
        back = {d: s for s, d in zip(src, dst) if d >= 0}
        for r, p in enumerate(parents):
            n = -(-lens[r] // page)
            assert lens[r] == (o_lens[p] if p >= 0 else 0) or lens[r] == o_lens[p] // page * page
            assert [back.get(x, x) for x in table[r][:n]] == old[p][:n] if p >= 0 else n == 0
        assert missing == sum(1 for n, p in zip(lens, parents) if p >= 0 and n != o_lens[p])


def test_rows_that_shrank_share_a_page_until_they_are_parted():
    # two beams of 48 tokens, all pages shared, go back to 20 and 25 tokens
    refs, table, lens = [2, 2, 2, 0, 0], [[0, 1, 2], [0, 1, 2]], [48, 48]
    refs, table, lens, _ = ref.resize(refs, table, lens, 16, [20, 25])
    same = ref.fork(refs, table, lens, 16, [0, 1])
    assert last_pages(same[1], same[2], 16) == [(0, 1), (1, 1)]  # both would write into page 1
    refs, table, lens, src, dst, missing = ref.fork_own(refs, table, lens, 16, [0, 1])
    assert (refs, table, lens, src, dst, missing) == ([2, 1, 1, 0, 0], [[0, 1, -1], [0, 2, -1]], [20, 25], [-1, 1], [-1, 2], 0)
    # where a third row goes on past the page, both get another
    refs, table, lens, _ = ref.resize([3, 3, 3, 0, 0], [[0, 1, 2]] * 3, [48] * 3, 16, [20, 25, -1])
    refs, table, lens, src, dst, missing = ref.fork_own(refs, table, lens, 16, [0, 1, 2])
    assert (refs, table, src, dst, missing) == ([3, 1, 1, 1, 1], [[0, 3, -1], [0, 4, -1], [0, 1, 2]], [1, 1, -1], [3, 4, -1], 0)


def bf16(x):
    import torch

    return torch.from_numpy(np.array(x, np.float32)).bfloat16().float().numpy()


def parts(x):
    x = np.asarray(x, np.float32)
    a = bf16(x)
    b = bf16(x - a)
    return a, b, bf16(x - a - b)


SIX = ((1, 1), (0, 2), (2, 0), (0, 1), (1, 0), (0, 0))


def by_parts(x, y, products):
    x, y, total = parts(x), parts(y), np.float32(0)
    for i, j in products:
        total = total + x[i] * y[j]  # a product of two bf16 numbers is one of fp32
    return total


@pytest.mark.parametrize("score,value,fits", [
    (SIX, SIX, True),
    (SIX[1:], SIX, False), (SIX, SIX[1:], False),                # without the product of the second parts
    (SIX[:1] + SIX[2:], SIX, False), (SIX, SIX[:2] + SIX[3:], False),
    (SIX[3:], SIX, False), (SIX, SIX[3:], False), (SIX[5:], SIX[5:], False)])
def test_products_that_are_left_out_show(score, value, fits):
    """The kernels' arithmetic for fp32 rows that see one key, in numpy's fp32, with all of the products and fewer."""
    q, k, v = ref.one_key_rows(np.random.default_rng(3), 400, 64)
    out, lse, b_out, b_lse = ref.one_key(q, k, v, 0.25)
    f = np.float32
    s = np.stack([by_parts(q[:, c], k[:, c], score) for c in range(64)], 1).sum(1, dtype=f)
    log2e = f(0.25) * f(1.44269504088896341)
    m = np.ceil(s * log2e)
    p = np.exp2((s.astype(np.float64) * log2e - m).astype(f)).astype(f)
    got_lse = (m + np.log2(p)) * f(0.693147180559945309)
    got = by_parts(np.broadcast_to(p[:, None], v.shape), v, value) * (f(1) / p)[:, None]
    assert got.dtype == got_lse.dtype == f
    off_lse, off = np.abs(got_lse - lse) / b_lse, np.abs(got - out) / b_out
    assert ((off_lse <= 1).all() and (off <= 1).all()) == fits
    if score != SIX:
        assert off_lse.max() > 4
    if value != SIX:
        assert off.max() > 4


def test_probabilities_in_bf16_show():
    x = bf16(np.random.default_rng(4).uniform(-0.125, 0.125, 300))
    out, bound = ref.two_keys(x, ref.P_FP16)
    p = np.exp(np.stack([0 * x, x]) - np.maximum(x, 0)).astype(np.float32) * 128
    for rounded, fits in ((p.astype(np.float16).astype(np.float32), True), (bf16(p), False)):
        got = bf16((rounded[0] - rounded[1]) / p.sum(0))
        assert (np.abs(got - out) <= bound).all() == fits


@pytest.mark.parametrize("seed", range(6))
def test_what_is_held_is_within_the_stated_error(seed):
    """At most 2^-4 of a value or 2^(e - 10) at the scale that it came at; raises add less than 2^(e - 9) at the last."""
    rng = np.random.default_rng(seed)
    raised = again = 0
    for _ in range(200):
        h, x, first = ref.Held(1, 8), [], []
        while len(x) < ref.BLOCK:
            n = min(int(rng.integers(1, 4)), ref.BLOCK - len(x))
            new = rng.standard_normal((n, 1, 8)) * 2.0 ** rng.uniform(-10, -8 + len(x))
            h.append(new)
            x += list(new)
            first += [int(h.e[0, 0])] * n
        x, first, last = np.array(x), np.array(first)[:, None, None], int(h.e[0, 0])
        far = np.abs(h.x - x)
        once = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** (first - 10))
        assert (far <= once + np.where(first < last, 2.0 ** (last - 9), 0)).all()
        raised += (first < last).sum()
        again += (far > np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** (last - 10))).sum()
    assert raised and again  # the last scale alone does not bound it


def test_a_raise_adds_to_the_error():
    u = 2.0 ** -9  # the last scale's smallest step
    h = ref.Held(1, 1)
    h.append(np.array([[[448 / 2]], [[3.3 * u]]]))
    assert h.e[0, 0] == -1 and h.x[1, 0, 0] == 3.5 * u
    h.append(np.array([[[448.0]]]))
    assert h.e[0, 0] == 0 and h.x[1, 0, 0] == 4 * u  # 0.7 steps off
