"""The operations on pages against lists, word for word: sequences that grow, shrink and end, forks with shared and
copied pages, shortage, compaction, one launch and several, in place and not, copies in layers, streams and graphs, and
a serving loop of forks and appends over caches of 4 and 8 bits."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import attn_ref
import serving_ref as ref
from gpu_util import host, say
from test_serving_ref import random_state

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cf():
    from activation_residual_compression_cf_amd import cf as _cf

    return _cf


@pytest.fixture(scope="module")
def dev(cf):
    return cf.require_device()


def ints(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


def put(cf, dev, refs, table, lens, page):
    return cf.PageTable(ints(refs, dev), ints(table, dev), ints(lens, dev), page)


def same(t, refs, table, lens):
    torch.cuda.synchronize()
    assert host(t.refs).tolist() == list(refs), "refs"
    assert host(t.table).tolist() == [list(r) for r in table], "table"
    assert host(t.lens).tolist() == list(lens), "lens"


@pytest.mark.parametrize("seed", range(12))
@pytest.mark.parametrize("in_place", [True, False])
def test_small(cf, dev, seed, in_place):
    """Random steps of all of them, on states that one workgroup works on."""
    rng = np.random.default_rng(100 + seed)
    page, rows, width = int(rng.choice([1, 16, 24, 256])), int(rng.choice([1, 5, 70])), int(rng.choice([1, 3, 40]))
    pages = int(rng.integers(1, rows * width + 20))
    say(f"pages rows={rows} width={width} pages={pages} page={page} in_place={in_place}")
    refs, table, lens = random_state(rng, pages, rows, width, page)
    t = put(cf, dev, refs, table, lens, page)
    for _ in range(5):
        want = [int(rng.integers(-1, width * page + 2)) for _ in range(rows)]
        keep = [x.clone() for x in (t.refs, t.table, t.lens)]
        new, missing = cf.pages_resize(t, ints(want, dev), out=t if in_place else None)
        if not in_place:
            assert all(torch.equal(a, b) for a, b in zip(keep, (t.refs, t.table, t.lens)))
        t = new
        refs, table, lens, m = ref.resize(refs, table, lens, page, want)
        same(t, refs, table, lens)
        assert missing.item() == m
        parents = [int(rng.integers(-1, rows + 1)) for _ in range(rows)]
        out = cf.PageTable(t.refs, torch.empty_like(t.table), torch.empty_like(t.lens), page) if in_place else None
        t, src, dst, missing = cf.pages_fork(t, ints(parents, dev), out=out)
        refs, table, lens, s, d, m = ref.fork(refs, table, lens, page, parents)
        same(t, refs, table, lens)
        assert host(src).tolist() == s and host(dst).tolist() == d and missing.item() == m
        t, src, dst, count = cf.pages_compact(t, out=t if in_place else None)
        refs, table, pairs = ref.compact(refs, table)
        same(t, refs, table, lens)
        pad = [-1] * (pages // 2 - len(pairs))
        assert count.item() == len(pairs)
        assert host(src).tolist() == [a for a, _ in pairs] + pad and host(dst).tolist() == [b for _, b in pairs] + pad


@pytest.mark.parametrize("pages,rows,width", [(40000, 300, 100), (5000, 700, 60), (32768, 8, 4096), (32769, 1, 3), (4096, 2, 20000), (12288, 3000, 11)])
def test_large(cf, dev, pages, rows, width):
    """More pages or entries than one workgroup takes, and chunks that are full and not."""
    say(f"pages rows={rows} width={width} pages={pages}")
    rng = np.random.default_rng(pages)
    page = 16
    share = max(1, min(width, 2 * pages // (3 * rows)))
    lens = rng.integers(0, share * page + 1, rows).tolist()
    order = rng.permutation(pages)
    table, at = np.full((rows, width), -1), 0
    for r in range(rows):
        n = -(-lens[r] // page)
        table[r, :n] = order[at:at + n]
        at += n
    refs, table = ref.count_refs(pages, table.tolist(), lens, page), table.tolist()
    t = put(cf, dev, refs, table, lens, page)
    for i in range(2):
        want = rng.integers(0, 2 * share * page, rows).tolist()
        t, missing = cf.pages_resize(t, ints(want, dev))
        refs, table, lens, m = ref.resize(refs, table, lens, page, want)
        same(t, refs, table, lens)
        assert missing.item() == m
        parents = rng.integers(0, rows, rows).tolist()
        t, src, dst, missing = cf.pages_fork(t, ints(parents, dev))
        refs, table, lens, s, d, m = ref.fork(refs, table, lens, page, parents)
        same(t, refs, table, lens)
        assert host(src).tolist() == s and host(dst).tolist() == d and missing.item() == m
        t, src, dst, count = cf.pages_compact(t, out=t if i else None)
        refs, table, pairs = ref.compact(refs, table)
        same(t, refs, table, lens)
        assert count.item() == len(pairs) and host(src)[:len(pairs)].tolist() == [a for a, _ in pairs]
        assert host(dst)[:len(pairs)].tolist() == [b for _, b in pairs] and (host(src)[len(pairs):] == -1).all()


def test_one_row_takes_many(cf, dev):
    say("pages: one row of 20000 pages, and one of all but one")
    t = cf.PageTable.create(20001, 3, 20000, 16)
    # 4 + 20000 + 3 pages: the second finds too few, and so does what comes behind it
    t, missing = cf.pages_resize(t, ints([50, 20000 * 16, 40], dev))
    torch.cuda.synchronize()
    assert missing.item() == 2 and host(t.lens).tolist() == [50, 0, 0]
    t, missing = cf.pages_resize(t, ints([5, 20000 * 16, 0], dev), out=t)
    torch.cuda.synchronize()
    assert missing.item() == 0 and host(t.table[1]).tolist() == list(range(1, 20001)) and (t.refs == 1).all()


def test_entries_that_are_no_page(cf, dev):
    """Tables with numbers outside the cache inside the lengths: handed on, counted nowhere."""
    say("pages: entries outside the cache")
    page, pages = 16, 8
    table, lens, refs = [[0, 99, 3], [-5, 2, -1], [2 ** 31 - 1, -2 ** 31, 1]], [40, 20, 48], [1, 1, 1, 1, 0, 0, 0, 0]
    for parents in ([0, 0, 0], [2, 1, 1], [1, 2, 0]):
        t = put(cf, dev, refs, table, lens, page)
        t, src, dst, missing = cf.pages_fork(t, ints(parents, dev))
        r, ta, le, s, d, m = ref.fork(refs, table, lens, page, parents)
        same(t, r, ta, le)
        assert host(src).tolist() == s and host(dst).tolist() == d
    t = put(cf, dev, refs, table, lens, page)
    t, _ = cf.pages_resize(t, ints([0, 48, 17], dev))
    r, ta, le, m = ref.resize(refs, table, lens, page, [0, 48, 17])
    same(t, r, ta, le)
    t, src, dst, count = cf.pages_compact(put(cf, dev, [0, 1, 1, 1, 0, 0, 0, 1], table, lens, page))
    r, ta, pairs = ref.compact([0, 1, 1, 1, 0, 0, 0, 1], table)
    same(t, r, ta, lens)
    # lengths outside [0, width * page_size] are taken within
    t = put(cf, dev, refs, table, [1000, -3, 48], page)
    t, _ = cf.pages_resize(t, ints([-1, -1, -1], dev))
    same(t, refs, [table[0], [-1, -1, -1], table[2]], [48, 0, 48])


@pytest.mark.parametrize("page_bytes", [16, 4352, 16384, 16400, 70000])
@pytest.mark.parametrize("layers", [1, 3])
def test_copies(cf, dev, page_bytes, layers):
    say(f"pages copy page_bytes={page_bytes} layers={layers}")
    rng = np.random.default_rng(page_bytes)
    pages, n = 60, 20
    whole = torch.from_numpy(rng.integers(0, 256, (layers, pages + 2, page_bytes)).astype(np.uint8)).to(dev)
    data = whole[:, :pages]
    order = rng.permutation(pages)
    src, dst = order[:n].astype(np.int32), order[n:2 * n].astype(np.int32)
    src[3], dst[5], src[7], dst[9] = -1, pages, 2 ** 31 - 1, -2 ** 31
    dst[11] = src[11]
    src[12] = src[13]  # one page to two
    for count in (None, 0, 6, 20, 10 ** 6, -1):
        want = whole.clone()
        for i in range(n if count is None else max(0, min(n, count))):
            if 0 <= src[i] < pages and 0 <= dst[i] < pages:
                want[:, dst[i]] = whole[:, src[i]]
        got = whole.clone()
        c = None if count is None else ints([count], dev)
        cf.pages_copy(got[:, :pages], ints(src, dev), ints(dst, dev), c)
        torch.cuda.synchronize()
        assert torch.equal(got, want), f"count {count}"


def test_copies_past_32_bits(cf, dev):
    say("pages copy past 4 GiB")
    pages, size = 70, 1 << 26
    data = torch.empty(1, pages, size, dtype=torch.uint8, device=dev)
    data[0, 2], data[0, 69] = 7, 9
    data[0, 69, -5:] = 3
    cf.pages_copy(data, ints([69, 2], dev), ints([0, 68], dev))
    torch.cuda.synchronize()
    assert torch.equal(data[0, 0], data[0, 69]) and (data[0, 68] == 7).all()


def test_graph_and_side_stream(cf, dev):
    say("pages in a graph and on a side stream")
    rng = np.random.default_rng(3)
    page, rows, width, pages = 16, 12, 9, 90
    refs, table, lens = random_state(rng, pages, rows, width, page)
    t = put(cf, dev, refs, table, lens, page)
    out = cf.PageTable(*(torch.empty_like(x) for x in (t.refs, t.table, t.lens)), page)
    parents, want = ints([0] * rows, dev), ints([0] * rows, dev)
    data = torch.from_numpy(rng.integers(0, 256, (2, pages, 64)).astype(np.uint8)).to(dev)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        _, src, dst, m1 = cf.pages_fork(t, parents, out=out)
        _, m2 = cf.pages_resize(out, want, out=t)
        cf.pages_copy(data, src, dst)
    for i in range(5):
        p = [int(rng.integers(-1, rows)) for _ in range(rows)]
        parents.copy_(ints(p, dev))
        r, ta, le, s, d, m = ref.fork(refs, table, lens, page, p)
        w = [min(n + int(rng.integers(0, 20)), width * page) for n in le]
        want.copy_(ints(w, dev))
        expect = data.clone()
        for a, b in zip(s, d):
            if b >= 0:
                expect[:, b] = data[:, a]
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(data, expect) and m1.item() == m
        refs, table, lens, m = ref.resize(r, ta, le, page, w)
        same(t, refs, table, lens)
        assert m2.item() == m
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, src, dst, count = cf.pages_compact(t, stream=side)
    torch.empty(1 << 20, device=dev).fill_(7)  # what the call freed must not be handed out yet
    side.synchronize()
    r, ta, pairs = ref.compact(refs, table)
    same(got, r, ta, lens)
    assert count.item() == len(pairs)


def test_search_with_beams(cf, dev):
    """Beams that fork, grow and end over an 8-bit and a 4-bit cache with one table: each beam's attention is that over
    its own history."""
    say("pages: a search with beams")
    rng = np.random.default_rng(11)
    rows, width, page, heads, dim, pages = 6, 8, 16, 2, 64, 40
    t = cf.PageTable.create(pages, rows, width, page)
    c8, c4 = cf.KV8Cache.create(pages, page, heads, dim), cf.KV4Cache.create(pages, page, heads, dim)
    k8, v8 = ([ref.Held(heads, dim) for _ in range(rows)] for _ in range(2))
    k4, v4 = ([np.zeros((0, heads, dim)) for _ in range(rows)] for _ in range(2))
    lens = [0] * rows

    def grow(new):
        nonlocal t, lens
        lens = [a + b for a, b in zip(lens, new)]
        t, missing = cf.pages_resize(t, ints(lens, dev), out=t)
        k, v = (torch.from_numpy(rng.standard_normal((sum(new), heads, dim)).astype(np.float32)).to(dev) for _ in range(2))
        starts = np.concatenate([[0], np.cumsum(new)])
        cf.kv8_append(c8, k, v, t.lens, table=t.table, starts=ints(starts, dev))
        row = np.repeat(np.arange(rows), new)
        pos = torch.from_numpy(np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)])).to(dev)
        slots = t.table[torch.from_numpy(row).to(dev), pos // page].long() * page + pos % page
        cf.kv4_append(c4, k, v, slots)
        torch.cuda.synchronize()
        assert missing.item() == 0
        for r in np.flatnonzero(new):
            part = slice(starts[r], starts[r + 1])
            for x, h8, h4 in ((k, k8, k4), (v, v8, v4)):
                h8[r].append(host(x[part].double()))
                h4[r] = np.concatenate([h4[r], attn_ref.quantize(host(x[part]))])

    def fork(parents):
        nonlocal t, lens, k8, v8, k4, v4
        t, src, dst, missing = cf.pages_fork(t, ints(parents, dev))
        for c in (c8, c4):
            cf.pages_copy(c.data.flatten(1)[None], src, dst)
        torch.cuda.synchronize()
        assert missing.item() == 0

        def copy(h):
            n = ref.Held(heads, dim)
            if h is not None:
                n.x, n.e = h.x.copy(), h.e.copy()
            return n

        k8, v8 = ([copy(h[p] if p >= 0 else None) for p in parents] for h in (k8, v8))
        k4, v4 = ([h[p] if p >= 0 else h[0][:0] for p in parents] for h in (k4, v4))
        lens = [lens[p] if p >= 0 else 0 for p in parents]

    def check():
        q = torch.from_numpy(rng.standard_normal((rows, heads, dim)).astype(np.float32)).to(dev)
        for c, call, ks, vs in ((c8, cf.kv8_attention, [h.x for h in k8], [h.x for h in v8]), (c4, cf.kv4_attention, k4, v4)):
            lse = torch.empty(rows, heads, device=dev)
            out = call(q, c, t.lens, table=t.table, lse=lse)
            torch.cuda.synchronize()
            for r in range(rows):
                o, l, b, bl = ref.attention(host(q[r:r + 1].double()), ks[r], vs[r], dim ** -0.5, False, 0, ref.P_PARTS, kind="f32")
                assert (np.abs(host(out[r:r + 1].double()) - o) <= b).all(), f"row {r}"

    grow([37, 0, 0, 20, 0, 0])
    fork([0, 0, 0, 3, 3, 3])
    check()
    for parents in ([0, 0, 2, 3, 4, 4], [2, 1, 2, 5, 5, 5], [1, 1, 1, -1, 3, 3], [0, 1, 2, 3, 4, 5]):
        for _ in range(5):
            grow([1] * rows)
        fork(parents)
        check()
    t, src, dst, count = cf.pages_compact(t, out=t)
    for c in (c8, c4):
        cf.pages_copy(c.data.flatten(1)[None], src, dst, count)
    check()
    t, _ = cf.pages_resize(t, ints([0] * rows, dev), out=t)
    torch.cuda.synchronize()
    assert not t.refs.any() and not t.lens.any() and (t.table == -1).all()


@pytest.mark.parametrize("page,width", [(10 ** 9, 2), (1500000000, 1), (2 ** 31 - 257, 1), (2 ** 30 + 3, 1), (715827797, 2), (1000, 2147483), (1, 50)])
def test_page_sizes_up_to_the_largest(cf, dev, page, width):
    """Rows that end near 2^31 tokens, where tokens and a page's together are more than that."""
    say(f"pages of {page} tokens, width={width}")
    most = width * page
    rows, pages = (3, 3 * width + 2) if width < 100 else (1, width + 5)
    t = cf.PageTable.create(pages, rows, width, page)
    refs, table, lens = [0] * pages, [[-1] * width for _ in range(rows)], [0] * rows
    for want in ([most, 1, most - page + 1], [most - 1, most, page - 1], [most + 1, 0, most], [1, page, 0])[:None if rows > 1 else 3]:
        want = want[:rows]
        t, missing = cf.pages_resize(t, ints(want, dev))
        refs, table, lens, m = ref.resize(refs, table, lens, page, want)
        same(t, refs, table, lens)
        assert missing.item() == m
        if rows > 1:
            t, src, dst, missing = cf.pages_fork(t, ints([0, 0, 2], dev))
            refs, table, lens, s, d, m = ref.fork(refs, table, lens, page, [0, 0, 2])
            same(t, refs, table, lens)
            assert host(src).tolist() == s and host(dst).tolist() == d and missing.item() == m


@pytest.mark.parametrize("starts", [True, False])
def test_appends_where_pages_run_out(cf, dev, starts):
    """A serving loop without a host wait, with too few pages and with rows that want more than the table holds: rows
    that were not served keep every token, those that were get theirs, and later pages serve them all."""
    say("pages: appends with too few pages")
    rng = np.random.default_rng(21)
    rows, width, page, heads, dim, pages = 5, 3, 16, 2, 64, 9
    t = cf.PageTable.create(pages, rows, width, page)
    cache = cf.KV8Cache.create(pages, page, heads, dim)
    held = [[ref.Held(heads, dim) for _ in range(rows)] for _ in range(2)]
    refs, table, lens = [0] * pages, [[-1] * width for _ in range(rows)], [0] * rows
    short = 0

    def step(want, new):
        """Rows want so many tokens and bring `new`."""
        nonlocal t, refs, table, lens, short
        was = lens
        refs, table, lens, m = ref.resize(refs, table, lens, page, want)
        short += m
        x = torch.from_numpy(rng.standard_normal((2, sum(new), heads, dim)).astype(np.float32)).to(dev)
        w = ints(want, dev)
        t, missing = cf.pages_resize(t, w, out=t)
        cf.kv8_append(cache, x[0], x[1], t.append_lens(w), table=t.table, starts=ints(np.concatenate([[0], np.cumsum(new)]), dev) if starts else None)
        at = 0
        for r in range(rows):
            for y, h in zip(x, held):
                if lens[r] < was[r]:
                    h[r].cut(lens[r])
                if want[r] == lens[r] and 0 < new[r] <= lens[r]:
                    h[r].append(host(y[at:at + new[r]].double()))
            at += new[r]
        same(t, refs, table, lens)
        assert missing.item() == m
        for r in range(rows):
            if lens[r]:
                pos = np.arange(lens[r])
                slots = torch.from_numpy(np.asarray(table[r])[pos // page] * page + pos % page).to(dev)
                for got, h in zip(cf.kv8_read(cache, slots, torch.float32), held):
                    assert np.array_equal(host(got.double()), h[r].x), f"row {r}"

    n = [16] * rows
    step([16] * rows, n)
    step([32] * rows, n)  # four rows find a page
    for _ in range(3):
        step([x + 1 for x in lens], [1] * rows)  # no page is left
    assert lens == [32, 32, 32, 32, 16] and short == 16
    step([0, -1, 33, 48 + 1, 17], [0, 0, 1, 1, 1] if starts else [1] * rows)
    assert lens == [0, 32, 33, 32, 17]
    if starts:
        step([0, 0, 33 + 7, 10 ** 9, 17 + 20], [0, 0, 7, 5, 20])
        assert lens == [0, 0, 40, 32, 37]


@pytest.mark.parametrize("seed", range(12))
def test_forks_that_part_rows(cf, dev, seed):
    """Random resizes and forks of rows that share pages in any way, on states that one workgroup works on."""
    rng = np.random.default_rng(300 + seed)
    page, rows, width = int(rng.choice([1, 16, 24, 256])), int(rng.choice([1, 5, 70, 1100])), int(rng.choice([1, 3, 20]))
    pages = int(rng.integers(1, rows * width + 20))
    say(f"pages fork own rows={rows} width={width} pages={pages} page={page}")
    refs, table, lens = random_state(rng, pages, rows, width, page)
    t = put(cf, dev, refs, table, lens, page)
    for i in range(5):
        want = [int(rng.integers(-1, width * page + 2)) for _ in range(rows)]
        t, _ = cf.pages_resize(t, ints(want, dev), out=t)
        refs, table, lens, _ = ref.resize(refs, table, lens, page, want)
        parents = [int(rng.integers(-1, rows + 1)) if rng.random() < (0, 0.3, 1)[i % 3] else r for r in range(rows)]
        keep = [x.clone() for x in (t.table, t.lens)]
        out = cf.PageTable(t.refs, torch.empty_like(t.table), torch.empty_like(t.lens), page) if i % 2 else None
        new, src, dst, missing = cf.pages_fork(t, ints(parents, dev), out=out, own=True)
        assert torch.equal(keep[0], t.table) and torch.equal(keep[1], t.lens)
        t = new
        refs, table, lens, s, d, m = ref.fork_own(refs, table, lens, page, parents)
        same(t, refs, table, lens)
        assert host(src).tolist() == s and host(dst).tolist() == d and missing.item() == m


@pytest.mark.parametrize("pages,rows,width", [(40000, 300, 100), (5000, 700, 60), (32769, 1, 3), (12288, 3000, 11)])
def test_forks_that_part_rows_large(cf, dev, pages, rows, width):
    say(f"pages fork own rows={rows} width={width} pages={pages}")
    rng = np.random.default_rng(pages)
    page = 16
    refs, table, lens = [0] * pages, [[-1] * width for _ in range(rows)], [0] * rows
    t = put(cf, dev, refs, table, lens, page)
    share = max(1, min(width, pages // rows))
    for i in range(3):
        want = rng.integers(0, share * page + 1, rows).tolist()
        t, _ = cf.pages_resize(t, ints(want, dev))
        refs, table, lens, _ = ref.resize(refs, table, lens, page, want)
        parents = rng.integers(0, rows, rows).tolist() if i < 2 else list(range(rows))
        t, src, dst, missing = cf.pages_fork(t, ints(parents, dev), own=True)
        refs, table, lens, s, d, m = ref.fork_own(refs, table, lens, page, parents)
        same(t, refs, table, lens)
        assert host(src).tolist() == s and host(dst).tolist() == d and missing.item() == m


def test_entries_that_are_no_page_own(cf, dev):
    say("pages fork own: entries outside the cache")
    page = 16
    table, lens, refs = [[0, 99, 3], [-5, 2, -1], [2 ** 31 - 1, -2 ** 31, 1]], [40, 20, 40], [1, 1, 1, 1, 0, 0, 0, 0]
    for parents in ([0, 0, 0], [2, 1, 1], [1, 2, 0], [0, 1, 2]):
        t, src, dst, missing = cf.pages_fork(put(cf, dev, refs, table, lens, page), ints(parents, dev), own=True)
        r, ta, le, s, d, m = ref.fork_own(refs, table, lens, page, parents)
        same(t, r, ta, le)
        assert host(src).tolist() == s and host(dst).tolist() == d and missing.item() == m


def test_beams_that_go_back(cf, dev):
    """Beams that share pages of a prompt go back to inside of it, are parted and grow on over an 8-bit cache: each reads its own
    tokens, in a captured step too."""
    say("pages: beams that go back")
    rng = np.random.default_rng(31)
    rows, width, page, heads, dim, pages = 4, 6, 16, 2, 64, 30
    t = cf.PageTable.create(pages, rows, width, page)
    cache = cf.KV8Cache.create(pages, page, heads, dim)
    held = [[ref.Held(heads, dim) for _ in range(rows)] for _ in range(2)]

    def rows_of(n):
        return torch.from_numpy(rng.standard_normal((2, n, heads, dim)).astype(np.float32)).to(dev)

    def check():
        table, lens = host(t.table), host(t.lens)
        for r in range(rows):
            pos = np.arange(lens[r])
            slots = torch.from_numpy(table[r][pos // page].astype(np.int64) * page + pos % page).to(dev)
            for got, h in zip(cf.kv8_read(cache, slots, torch.float32), held):
                assert np.array_equal(host(got.double()), h[r].x), f"row {r}"

    x = rows_of(64)
    t, _ = cf.pages_resize(t, ints([64, 0, 0, 0], dev))
    cf.kv8_append(cache, x[0], x[1], t.lens, table=t.table, starts=ints([0, 64, 64, 64, 64], dev))
    t, src, dst, _ = cf.pages_fork(t, ints([0] * rows, dev))
    for h, y in zip(held, x):
        for r in range(rows):
            h[r].append(host(y.double()))
    check()
    back, want = ints([0] * rows, dev), ints([0] * rows, dev)
    x = rows_of(rows)
    stay = ints(range(rows), dev)
    a, b, c = (cf.PageTable(*(y.clone() for y in (t.refs, t.table, t.lens)), page) for _ in range(3))
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        cf.pages_resize(a, back, out=b)
        _, src, dst, m1 = cf.pages_fork(b, stay, out=c, own=True)
        cf.pages_copy(cache.data.flatten(1)[None], src, dst)
        _, m2 = cf.pages_resize(c, want, out=a)
        cf.kv8_append(cache, x[0], x[1], a.append_lens(want), table=a.table)
    for lens in ([50, 47, 64, 33], [51, 20, 36, 34], [20, 20, 37, 35], [21, 21, 17, 17]):
        back.copy_(ints(lens, dev)), want.copy_(ints([n + 1 for n in lens], dev))
        x.copy_(rows_of(rows))
        for h, y in zip(held, x):
            for r, n in enumerate(lens):
                n0 = len(h[r].x)
                if n < n0:
                    h[r].cut(n)
                h[r].append(host(y[r:r + 1].double()))
        g.replay()
        torch.cuda.synchronize()
        assert m1.item() == 0 and m2.item() == 0
        t = a
        check()
        assert all(host(t.refs)[p] == 1 for p in host(t.table)[np.arange(rows), (host(t.lens) - 1) // page])


@pytest.mark.parametrize("in_place", [True, False])
def test_compact_renumbers_entries_behind_the_last_page(cf, dev, in_place):
    """Entries that a length has left behind, of pages that move, that are free and of none, and lengths of any size."""
    say("pages compact: stale entries")
    refs = [0, 1, 0, 0, 2, 0, 1, 1]
    table, lens = [[4, 7, 1], [4, 6, 3], [1, -1, 8], [7, 0, 5]], [16, 32, 10 ** 6, -4]
    t = put(cf, dev, refs, table, lens, 16)
    got, src, dst, count = cf.pages_compact(t, out=t if in_place else None)
    r, ta, pairs = ref.compact(refs, table)
    assert pairs == [(4, 0), (6, 2), (7, 3)] and ta == [[0, 3, 1], [0, 2, 3], [1, -1, 8], [3, 0, 5]]
    same(got, r, ta, lens)
    assert count.item() == 3
