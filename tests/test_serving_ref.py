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
