"""The 8-bit cache's writer and reader against the format's definition in 64 bits, value for value: lengths from
none, pages of every size, tokens one by one and in prompts, scales that grow, both ends of the scales' exponents, NaN and
infinities, strides, padding, rows of no sequence, streams and graphs."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import serving_ref as ref
from gpu_util import host, say

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def cf():
    from activation_residual_compression_cf_amd import cf as _cf

    return _cf


@pytest.fixture(scope="module")
def dev(cf):
    return cf.require_device()


class Sequences:
    """Sequences of a cache and what each should hold."""

    def __init__(self, cf, dev, batch, heads, dim, page, width, seed=0, table=True, fill=0x5A):
        rng = np.random.default_rng(seed)
        self.cf, self.dev, self.page, self.heads, self.dim = cf, dev, page, heads, dim
        pages = batch * width + (3 if table else 0)
        data = torch.full((pages, heads, 2 * page * dim + max(16, page // 8)), fill, dtype=torch.uint8, device=dev)
        self.cache = cf.KV8Cache(data, page, dim)
        self.pages = rng.permutation(pages)[:batch * width].reshape(batch, width) if table else np.arange(pages).reshape(batch, width)
        self.table = torch.from_numpy(self.pages.astype(np.int32)).to(dev) if table else None
        self.width = width
        self.lens = np.zeros(batch, int)
        self.k, self.v = ([ref.Held(heads, dim) for _ in range(batch)] for _ in range(2))

    def rows(self, new, dtype, rng, scale=1.0):
        x = rng.standard_normal((2, int(sum(new)), self.heads, self.dim)) * scale * np.exp(rng.standard_normal((2, 1, self.heads, self.dim)))
        return torch.from_numpy(x.astype(np.float32)).to(DT[dtype]).to(self.dev)

    def append(self, new, k, v, starts=True, **kw):
        kh, vh = host(k.double()), host(v.double())
        at = 0
        for b, n in enumerate(new):
            self.k[b].append(kh[at:at + n])
            self.v[b].append(vh[at:at + n])
            at += n
        self.lens += np.asarray(new)
        lens = torch.from_numpy(self.lens.astype(np.int32)).to(self.dev)
        st = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).to(self.dev) if starts else None
        self.cf.kv8_append(self.cache, k, v, lens, table=self.table, starts=st, table_width=self.width, **kw)

    def slots(self, b):
        t = np.arange(self.lens[b])
        return torch.from_numpy(self.pages[b][t // self.page] * self.page + t % self.page).to(self.dev)

    def check(self, dtype="f32"):
        for b in range(len(self.lens)):
            k, v = self.cf.kv8_read(self.cache, self.slots(b), DT[dtype])
            torch.cuda.synchronize()
            for name, got, held in (("k", k, self.k[b]), ("v", v, self.v[b])):
                got = host(got.double())
                assert np.array_equal(got, held.x, equal_nan=True), \
                    f"{name} of sequence {b}: {(~((got == held.x) | (np.isnan(got) & np.isnan(held.x)))).sum()} differ"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_ragged_appends(cf, dev, dtype, dim, page):
    say(f"kv8 append ragged {dtype} dim={dim} page={page}")
    rng = np.random.default_rng(dim + page)
    s = Sequences(cf, dev, 6, 3, dim, page, 512 // page, seed=page)
    for new in ([17, 0, 1, 16, 15, 33], [1, 1, 1, 1, 1, 1], [100, 3, 0, 64, 47, 5], [1, 0, 1, 0, 1, 0], [2, 31, 14, 16, 1, 200]):
        k, v = s.rows(new, dtype, rng, 2.0 ** rng.integers(-6, 7))
        s.append(new, k, v)
    s.check("f32")
    s.check("bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads", [1, 4, 7])
def test_one_token_each(cf, dev, dtype, heads):
    """Token by token, with scales that grow and shrink, through three blocks."""
    say(f"kv8 append single tokens {dtype} heads={heads}")
    rng = np.random.default_rng(heads)
    s = Sequences(cf, dev, 5, heads, 128, 16, 3, seed=2, table=heads != 4)
    for i in range(40):
        k, v = s.rows([1] * 5, dtype, rng, 2.0 ** rng.integers(-12, 6))
        s.append([1] * 5, k, v, starts=i % 2 == 0)
    s.check()


def test_ends_of_the_formats(cf, dev):
    say("kv8 append ends of the formats")
    rng = np.random.default_rng(4)
    mid = np.concatenate([(ref.LEVELS[1:] + ref.LEVELS[:-1]) / 2, ref.LEVELS])
    for scale in (2.0 ** -15, 2.0 ** -16, 2.0 ** -30, 1.0, 2.0 ** 7, 2.0 ** 8, 2.0 ** 100, 2.0 ** -140):
        s = Sequences(cf, dev, 3, 2, 64, 16, 4, fill=0xFF)
        for n in (16, 5, 20):
            x = rng.choice(mid, (2, 3 * n, 2, 64)) * rng.choice([-1, 1], (2, 3 * n, 2, 64)) * scale
            x = x.astype(np.float32)
            x[0, 0, 0, 3], x[1, 1, 1, 0], x[0, 2, 0, 63] = np.nan, np.inf, -np.inf
            x[0, 3, 1, 5] = x[1, 4, 0, 6] = -0.0
            x[0, 5] = 0
            k, v = torch.from_numpy(x).to(dev)
            s.append([n] * 3, k, v)
        s.check()
    # rows without a finite value, and of zeros
    s = Sequences(cf, dev, 1, 1, 64, 16, 2)
    x = torch.full((3, 1, 64), float("nan"), device=dev)
    s.append([3], x, torch.zeros_like(x))
    s.append([3], torch.ones_like(x), x)
    s.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [[16, 1, 0, 9], [40, 17, 0, 70]])
def test_single_numbers_that_are_cut_off(cf, dev, dtype, dim, new):
    """One value past the largest scale's last number, an infinity or NaN, in a call of few and of many tokens."""
    say(f"kv8 append of large numbers {dtype} dim={dim} {new}")
    rng = np.random.default_rng(dim)
    s = Sequences(cf, dev, 4, 5, dim, 32, 8, seed=dim)
    for big in (57344.0, -57344.0, 57856.0, 65536.0, -3e38, np.inf, -np.inf, np.nan, 1.0):
        k, v = s.rows(new, dtype, rng, 2.0)
        for x in (k, v):
            x[rng.integers(len(x)), rng.integers(5), rng.integers(dim)] = big
        s.append(new, k, v)
        if s.lens.max() > 100:
            s.check(dtype)
            s = Sequences(cf, dev, 4, 5, dim, 32, 8, seed=dim)
    s.check(dtype)


def test_rolled_back_tokens_are_written_again(cf, dev):
    """A shorter length and other tokens in the places behind it: the block's scale stays, a block begun anew
    forgets its own."""
    say("kv8 append after a rollback")
    rng = np.random.default_rng(5)
    s = Sequences(cf, dev, 2, 2, 128, 32, 2)
    k, v = s.rows([40, 21], "f32", rng, 30.0)
    s.append([40, 21], k, v)
    for cut in (37, 32, 19):
        for b, n in enumerate((cut, 19)):
            s.lens[b] = n
            s.k[b].cut(n), s.v[b].cut(n)
        k, v = s.rows([3, 2], "f32", rng, 0.01)
        s.append([3, 2], k, v)
        s.check()


def test_strides(cf, dev):
    say("kv8 append strides")
    rng = np.random.default_rng(6)
    for dtype in ("bf16", "f32"):
        s = Sequences(cf, dev, 3, 4, 64, 16, 4, seed=1)
        packed = torch.from_numpy(rng.standard_normal((50, 12, 64)).astype(np.float32)).to(DT[dtype]).to(dev)
        s.append([20, 0, 30], packed[:, 4:8], packed[:, 8:])
        heads = torch.from_numpy(rng.standard_normal((2, 4, 9, 64)).astype(np.float32)).to(DT[dtype]).to(dev)
        s.append([3, 5, 1], heads[0].transpose(0, 1), heads[1].transpose(0, 1))
        one = torch.randn(1, 1, 64, device=dev).to(DT[dtype]).expand(6, 4, 64)  # the same row everywhere
        s.append([2, 2, 2], one, one, starts=False)
        s.check()
        # into rows with strides, and from slots that name nothing
        out = torch.full((2, 60, 12, 64), 7.0, device=dev, dtype=DT[dtype])
        slots = torch.cat([s.slots(0), torch.tensor([-1, 1 << 40, s.cache.data.shape[0] * 16], device=dev)])
        cf.kv8_read(s.cache, slots, k=out[0, :len(slots), 2:6], v=out[1, :len(slots), 2:6])
        torch.cuda.synchronize()
        assert np.array_equal(host(out[0, :25, 2:6].double()), s.k[0].x) and np.array_equal(host(out[1, :25, 2:6].double()), s.v[0].x)
        assert (out[:, 25:28, 2:6] == 0).all() and (out[:, 28:] == 7).all() and (out[:, :, :2] == 7).all() and (out[:, :, 6:] == 7).all()


def test_rows_without_a_place(cf, dev):
    """Padding: lengths below the new tokens, pages outside the cache, rows of no sequence; nothing else is written."""
    say("kv8 append padding")
    rng = np.random.default_rng(7)
    for new in ([1, 1, 1, 1], [18, 18, 18, 18]):
        n = new[0]
        s = Sequences(cf, dev, 4, 2, 128, 16, 3, seed=3, fill=0x11)
        k, v = s.rows([n] * 4, "bf16", rng)
        before = s.cache.data.clone()
        table = s.table.clone()
        table[1] = torch.tensor([-1, s.cache.data.shape[0], 2 ** 31 - 1], dtype=torch.int32)
        lens = torch.tensor([n, n, 0, n - 1], dtype=torch.int32, device=dev)
        starts = torch.tensor([0, n, 2 * n, 3 * n, 4 * n], dtype=torch.int32, device=dev)
        cf.kv8_append(s.cache, k, v, lens, table=table, starts=starts)
        torch.cuda.synchronize()
        touched = set(int(p) for p in s.pages[0][:-(-n // 16)]) | set(int(p) for p in s.pages[3][:-(-(n - 1) // 16)])
        for p in range(s.cache.data.shape[0]):
            assert torch.equal(s.cache.data[p], before[p]) == (p not in touched), f"page {p}"
        for b, rows in ((0, slice(0, n)), (3, slice(3 * n + 1, 4 * n))):
            s.lens[b] = rows.stop - rows.start
            s.k[b].append(host(k[rows].double())), s.v[b].append(host(v[rows].double()))
        s.check()
        # rows before the first sequence and behind the last
        before = s.cache.data.clone()
        cf.kv8_append(s.cache, k, v, torch.full((4,), 48, dtype=torch.int32, device=dev), table=s.table,
                      starts=torch.tensor([2 * n] * 5, dtype=torch.int32, device=dev))
        torch.cuda.synchronize()
        assert torch.equal(s.cache.data, before)


def test_lengths_are_cut_to_the_table(cf, dev):
    say("kv8 append lengths past the table")
    s = Sequences(cf, dev, 1, 1, 64, 16, 2)
    k = torch.randn(20, 1, 64, device=dev)
    cf.kv8_append(s.cache, k, k, torch.tensor([10 ** 9], dtype=torch.int32, device=dev), table=s.table)
    # places 12 .. 31: what the first block's scale was before is not known here
    got, _ = cf.kv8_read(s.cache, torch.from_numpy(s.pages[0][1] * 16 + np.arange(16)).to(dev), torch.float32)
    torch.cuda.synchronize()
    want = ref.Held(1, 64)
    want.append(host(k.double()[4:]))
    assert np.array_equal(host(got.double()), want.x)


def test_nothing_to_do(cf, dev):
    say("kv8 append and read of nothing")
    s = Sequences(cf, dev, 2, 2, 64, 16, 1)
    before = s.cache.data.clone()
    z = torch.zeros(0, 2, 64, device=dev)
    cf.kv8_append(s.cache, z, z, torch.zeros(2, dtype=torch.int32, device=dev), table=s.table)
    k, v = cf.kv8_read(s.cache, torch.zeros(0, dtype=torch.int64, device=dev))
    torch.cuda.synchronize()
    assert k.shape == v.shape == (0, 2, 64) and torch.equal(s.cache.data, before)


def test_many_sequences(cf, dev):
    say("kv8 append of 700 sequences")
    rng = np.random.default_rng(8)
    s = Sequences(cf, dev, 700, 1, 64, 16, 4, seed=9)
    for i in range(2):
        new = [int(x) for x in rng.integers(0, 25, 700)]
        k, v = s.rows(new, "bf16", rng)
        s.append(new, k, v)
    order = rng.permutation(700)[:40]
    s.lens, s.k, s.v, s.pages = s.lens[order], [s.k[i] for i in order], [s.v[i] for i in order], s.pages[order]
    s.check()


def test_offsets_past_32_bits(cf, dev):
    """Pages behind 4 GiB of others."""
    say("kv8 append past 4 GiB")
    heads, dim, page = 8, 128, 256
    size = 2 * page * dim + 32
    pages = (1 << 32) // (heads * size) + 40
    cache = cf.KV8Cache(torch.empty((pages, heads, size), dtype=torch.uint8, device=dev), page, dim)
    table = torch.tensor([[pages - 1, 0], [pages - 2, pages - 3]], dtype=torch.int32, device=dev)
    x = torch.randn(2, 600, heads, dim, device=dev)
    starts = torch.tensor([0, 300, 600], dtype=torch.int32, device=dev)
    cf.kv8_append(cache, x[0], x[1], torch.tensor([300, 300], dtype=torch.int32, device=dev), table=table, starts=starts)
    t = torch.arange(300, device=dev)
    for b in range(2):
        slots = table[b, t // page].long() * page + t % page
        got = cf.kv8_read(cache, slots, torch.float32)
        torch.cuda.synchronize()
        for g, y in zip(got, x):
            h = ref.Held(heads, dim)
            h.append(host(y[300 * b:300 * b + 300].double()))
            assert np.array_equal(host(g.double()), h.x)


def test_side_stream_and_graph(cf, dev):
    say("kv8 append on a side stream and in a graph")
    rng = np.random.default_rng(10)
    s = Sequences(cf, dev, 3, 2, 64, 16, 8)
    side = torch.cuda.Stream()
    k, v = s.rows([5, 20, 1], "bf16", rng)
    side.wait_stream(torch.cuda.current_stream())
    s.append([5, 20, 1], k, v, stream=side)
    side.synchronize()
    s.check()
    k, v = (torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=dev) for _ in range(2))
    lens = torch.zeros(3, dtype=torch.int32, device=dev)
    outs = [torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    slots = torch.zeros(3, dtype=torch.int64, device=dev)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        cf.kv8_append(s.cache, k, v, lens, table=s.table)
        cf.kv8_read(s.cache, slots, k=outs[0], v=outs[1])
    for i in range(20):
        x = s.rows([1, 1, 1], "bf16", rng, 2.0 ** (i % 5))
        k.copy_(x[0]), v.copy_(x[1])
        for b in range(3):
            s.k[b].append(host(k[b:b + 1].double())), s.v[b].append(host(v[b:b + 1].double()))
        s.lens += 1
        lens.copy_(torch.from_numpy(s.lens.astype(np.int32)))
        at = s.lens - 1
        slots.copy_(torch.from_numpy(s.pages[np.arange(3), at // 16] * 16 + at % 16))
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(outs[0].double()), np.stack([h.x[-1] for h in s.k])), f"replay {i}"
        assert np.array_equal(host(outs[1].double()), np.stack([h.x[-1] for h in s.v])), f"replay {i}"
    s.check()
