"""cf_kv8_attention against softmax(scale Q K^T) V in 64 bits over the values the cache holds: ragged lengths from none
to thousands, shared heads, causal and windowed rows, empty rows, pages in any order, bytes of earlier owners, NaN in
hidden and in seen places, splits, strides, streams, graphs that share a workspace, and the chain of append and attention."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import serving_ref as ref
from gpu_util import host, say

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CANARY = 99.0


@pytest.fixture(scope="module")
def cf():
    from activation_residual_compression_cf_amd import cf as _cf

    return _cf


@pytest.fixture(scope="module")
def dev(cf):
    return cf.require_device()


class Case:
    """Sequences of `kv` keys and `nq` queries in a cache whose other bytes are all `stale`."""

    def __init__(self, cf, dev, kv, nq, hq, hk, dim, dtype, page=16, seed=0, spread=1.0, table=True, stale=0xFF, mean=0.2):
        rng = np.random.default_rng(seed)
        self.cf, self.kv, self.nq, self.dtype = cf, list(kv), nq, dtype
        per = [-(-n // page) for n in kv]
        self.width = max(per + [1]) + 1
        pages = sum(per) + 2 if table else len(kv) * self.width
        data = torch.full((pages, hk, 2 * page * dim + max(16, page // 8)), stale, dtype=torch.uint8, device=dev)
        self.cache = cf.KV8Cache(data, page, dim)
        order = rng.permutation(pages)
        tab = np.full((len(kv), self.width), -7, np.int32)
        self.k, self.v, rows = [], [], []
        at = 0
        for i, n in enumerate(kv):
            tab[i, :per[i]] = order[at:at + per[i]] if table else i * self.width + np.arange(per[i])
            at += per[i]
            k = (rng.standard_normal((n, hk, dim)) * spread).astype(np.float32)
            v = (rng.standard_normal((n, hk, dim)) + mean).astype(np.float32)
            rows.append((k, v))
            for x, to in ((k, self.k), (v, self.v)):
                h = ref.Held(hk, dim)
                h.append(x)
                to.append(h.x)
        self.q = torch.from_numpy(rng.standard_normal((sum(nq), hq, dim)).astype(np.float32)).to(DT[dtype]).to(dev)
        self.starts = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
        self.table = torch.from_numpy(tab).to(dev) if table else None
        self.lens = torch.tensor(kv, dtype=torch.int32, device=dev)
        self.q_starts = torch.from_numpy(self.starts).to(dev)
        self.put(dev, [r[0] for r in rows], [r[1] for r in rows])

    def put(self, dev, k, v):
        lens = [len(x) for x in k]
        if sum(lens):
            k, v = (torch.from_numpy(np.concatenate(x)).to(dev) for x in (k, v))
            starts = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).to(dev)
            self.cf.kv8_append(self.cache, k, v, self.lens, table=self.table, starts=starts, table_width=self.width)

    def run(self, **kw):
        lse = torch.full(self.q.shape[:2], CANARY, dtype=torch.float32, device=self.q.device)
        kw = {"table": self.table, "q_starts": self.q_starts, "table_width": self.width, **kw}
        out = self.cf.kv8_attention(self.q, self.cache, self.lens, lse=lse, **kw)
        torch.cuda.synchronize()
        return out, lse

    def check(self, out, lse, causal=False, window=0, scale=None):
        out, lse = host(out.double()), host(lse.double())
        q = host(self.q.double())
        # what a probability is rounded to depends on the kernel that the bound of queries chose: the coarser
        step = ref.P_BF16 if self.dtype == "bf16" else ref.P_PARTS
        for i in range(len(self.nq)):
            a, b = self.starts[i], self.starts[i + 1]
            o, l, bo, bl = ref.attention(q[a:b], self.k[i], self.v[i], scale or q.shape[2] ** -0.5, causal, window, step, kind=self.dtype)
            compare(out[a:b], lse[a:b], o, l, bo, bl, f"sequence {i}")


def compare(out, lse, o, l, bo, bl, name):
    empty = np.isneginf(l)
    assert np.array_equal(np.isneginf(lse), empty), f"{name}: empty rows"
    assert (out[empty] == 0).all()
    nan = np.isnan(o)
    assert np.array_equal(np.isnan(out), nan), f"{name}: NaN"
    far = np.abs(out - o)
    assert (far[~nan] <= bo[~nan]).all(), f"{name}: {np.nanmax(far[~nan] / (bo[~nan] + 1e-30)):.3g} of the bound"
    ok = ~empty & ~np.isnan(l)
    far = np.abs(lse[ok] - l[ok])
    assert (far <= bl[ok]).all(), f"{name}: lse {(far / bl[ok]).max():.3g} of the bound"
    assert np.array_equal(np.isnan(lse), np.isnan(l))


LENGTHS = [0, 1, 7, 8, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 300]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 4), (8, 2), (6, 2), (16, 1), (24, 1), (40, 1)])
def test_one_query_each(cf, dev, dtype, dim, hq, hk):
    say(f"kv8 attention single queries {dtype} dim={dim} heads={hq}/{hk}")
    c = Case(cf, dev, LENGTHS, [1] * len(LENGTHS), hq, hk, dim, dtype, seed=dim + hq)
    c.check(*c.run(max_q=1, causal=True), causal=True)
    # all queries of one size need no starts; without the mask one query sees the same keys
    c.check(*c.run(q_starts=None))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 1), (True, 40)])
@pytest.mark.parametrize("hq,hk,kv,nq", [
    (2, 1, [40, 0, 33, 90], [5, 3, 0, 8]),          # 16 rows at most
    (4, 2, [100, 1, 70, 16], [16, 1, 9, 16]),       # up to 32
    (3, 1, [301, 64, 20], [100, 64, 31]),           # more: rows of their own for each wave; more queries than keys
    (1, 1, [530], [521]),
    (8, 1, [77, 0, 200], [70, 5, 37])])
def test_many_queries(cf, dev, dtype, dim, causal, window, hq, hk, kv, nq):
    say(f"kv8 attention {dtype} dim={dim} causal={causal} window={window} heads={hq}/{hk} kv={kv} nq={nq}")
    c = Case(cf, dev, kv, nq, hq, hk, dim, dtype, page=32, seed=sum(kv))
    c.check(*c.run(max_q=max(nq), causal=causal, window=window), causal, window)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("table", [True, False])
@pytest.mark.parametrize("nq", [[1, 2, 3, 1, 1], [30, 40, 1, 65, 2]])
def test_pages(cf, dev, page, table, nq):
    say(f"kv8 attention page={page} table={table} nq={nq}")
    for dim in (64, 128):
        c = Case(cf, dev, [page - 1, page, page + 1, 3 * page + 5, 0], nq, 4, 2, dim, "bf16", page=page, table=table)
        c.check(*c.run(causal=True), causal=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 20, 300])
def test_split_over_workgroups(cf, dev, dtype, nq):
    """Few rows over many keys: an item's keys are spread over the chip and joined."""
    say(f"kv8 attention split {dtype} nq={nq}")
    kv = {1: 20000, 20: 6000, 300: 2500}[nq]
    c = Case(cf, dev, [kv, 70], [nq, 1], 2, 1, 128, dtype, page=64, seed=nq, spread=2.0)
    a = c.run(max_q=nq, causal=True)
    c.check(*a, causal=True)
    b = c.run(max_q=nq, causal=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), "two calls differ"


def test_peaked_rows(cf, dev):
    """Scores over hundreds: the reference moves, and one key may outweigh the rest."""
    say("kv8 attention peaked rows")
    for dtype in ("bf16", "f32"):
        c = Case(cf, dev, [700, 513], [3, 40], 2, 2, 64, dtype, spread=30.0, seed=9)
        c.check(*c.run(scale=0.5), scale=0.5)
        c.check(*c.run(scale=1e-4), scale=1e-4)


@pytest.mark.parametrize("nq", [1, 70])
def test_what_follows_a_key_that_outweighs_the_rest(cf, dev, nq):
    """Its V is zero, so the result is the tail's, e^-12 to e^-40 of the sum: relative to that, as exact as any, but for the 31
    keys taken with it where few rows' probabilities are fp16: its own is 2^7 there, and half a step of the least is 2^-25."""
    say(f"kv8 attention tails nq={nq}")
    for dtype in ("bf16", "f32"):
        for low in (12.0, 22.0, 30.0, 40.0):
            c = Case(cf, dev, [400], [nq], 1, 1, 64, dtype, seed=3, spread=0.0, mean=1.0)
            k, v = np.zeros((400, 1, 64), np.float32), host(torch.from_numpy(c.v[0])).astype(np.float32)
            k[37, 0, 0], v[37] = 4.0, 0.0
            c.q.zero_()
            c.q[:, :, 0] = 2.0
            c.put(dev, [k], [v])
            for x, to in ((k, c.k), (v, c.v)):
                h = ref.Held(1, 64)
                h.append(x)
                to[0] = h.x
            out, lse = c.run(scale=low / 8)
            o, l, bo, bl = ref.attention(host(c.q.double()), c.k[0], c.v[0], low / 8, False, 0, 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24, kind=dtype)
            beside = 31 * 2.0 ** -32 * np.abs(c.v[0]).max() if dtype == "bf16" and nq == 1 else 0.0
            assert (np.abs(host(out.double()) - o) <= bo + beside).all(), f"{dtype} {low}"


def test_wrong_bound_of_queries_is_only_slow(cf, dev):
    say("kv8 attention max_q below the longest")
    c = Case(cf, dev, [90, 40], [70, 3], 4, 2, 64, "bf16")
    for m in (1, 9, 0, 73):
        c.check(*c.run(max_q=m, causal=True), causal=True)


@pytest.mark.parametrize("nq", [1, 9, 70])
def test_pages_outside_the_cache_hold_nothing(cf, dev, nq):
    say(f"kv8 attention pages outside the cache nq={nq}")
    c = Case(cf, dev, [100], [nq], 2, 1, 128, "bf16", page=16)
    c.check(*c.run())
    for bad in (-1, c.cache.data.shape[0], 2 ** 31 - 1, -2 ** 31):
        keep = c.table.clone()
        c.table[0, 2] = bad
        out, lse = c.run()
        c.table = keep
        k, v = c.k[0], c.v[0]
        c.k[0], c.v[0] = (np.delete(x, np.arange(32, 48), 0) for x in (k, v))
        c.check(out, lse)
        c.k[0], c.v[0] = k, v
    c.table.fill_(-1)
    out, lse = c.run()
    assert not out.any() and lse.isneginf().all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("nq", [4, 30, 120])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_reaches_only_rows_that_see_it(cf, dev, dim, nq, dtype):
    say(f"kv8 attention NaN keys and values dim={dim} nq={nq} {dtype}")
    for what in ("k", "v", "both"):
        c = Case(cf, dev, [150], [nq], 2, 1, dim, dtype, page=16, seed=4)
        rng = np.random.default_rng(5)
        k, v = (rng.standard_normal((150, 1, dim)).astype(np.float32) for _ in range(2))
        at = 150 - nq // 2  # seen by the later half of the rows only
        if what != "v":
            k[at, 0, 3] = np.nan
        if what != "k":
            v[at, 0, dim - 40] = np.inf
            v[at - 1, 0, 1] = np.nan
        c.put(dev, [k], [v])
        for x, to in ((k, c.k), (v, c.v)):
            h = ref.Held(1, dim)
            h.append(x)
            to[0] = h.x
        c.check(*c.run(causal=True), causal=True)
        c.check(*c.run(causal=True, window=5), causal=True, window=5)
        c.check(*c.run())


def test_nan_query_stays_in_its_row(cf, dev):
    say("kv8 attention NaN query")
    for nq in (3, 100):
        c = Case(cf, dev, [90], [nq], 2, 2, 64, "bf16")
        want, wl = c.run()
        c.q[1, 1, 5] = float("nan")
        out, lse = c.run()
        assert out[1, 1].isnan().all() and lse[1, 1].isnan()
        out[1, 1], lse[1, 1] = want[1, 1], wl[1, 1]
        assert torch.equal(out, want) and torch.equal(lse, wl)


def test_stale_bytes_do_not_matter(cf, dev):
    say("kv8 attention stale bytes")
    for nq in (1, 60):
        for dtype in ("bf16", "f32"):
            got = [Case(cf, dev, [37, 5], [nq, nq], 4, 1, 64, dtype, page=64, stale=s).run() for s in (0, 0x7F, 0xFF, 0xC3)]
            for g in got[1:]:
                assert torch.equal(g[0], got[0][0]) and torch.equal(g[1], got[0][1])


@pytest.mark.parametrize("nq", [2, 40])
def test_strides_and_rows_of_no_sequence(cf, dev, nq):
    say(f"kv8 attention strides and rows behind the last sequence nq={nq}")
    c = Case(cf, dev, [50, 60], [nq, nq], 4, 2, 128, "bf16")
    total = 2 * nq
    want, wl = c.run()
    qh = torch.zeros(4, total + 3, 128, dtype=torch.bfloat16, device=dev)
    packed = torch.full((total + 3, 12, 128), CANARY, dtype=torch.bfloat16, device=dev)
    lse = torch.full((total + 3, 4), CANARY, device=dev)
    for gap in (0, 1):
        lse.fill_(CANARY), packed.fill_(CANARY)
        qh[:, gap:total + gap] = c.q.transpose(0, 1)
        cf.kv8_attention(qh.transpose(0, 1), c.cache, c.lens, table=c.table, q_starts=c.q_starts + gap, max_q=nq, out=packed[:, 4:8], lse=lse)
        torch.cuda.synchronize()
        assert torch.equal(packed[gap:total + gap, 4:8], want) and torch.equal(lse[gap:total + gap], wl)
        assert (packed[:, :4] == CANARY).all() and (packed[:, 8:] == CANARY).all() and (packed[:gap] == CANARY).all()
        assert (packed[total + gap:] == CANARY).all() and (lse[total + gap:] == CANARY).all()


def test_nothing_to_do(cf, dev):
    say("kv8 attention no queries")
    c = Case(cf, dev, [20], [1], 2, 2, 64, "bf16")
    assert cf.kv8_attention(c.q[:0], c.cache, c.lens, table=c.table).shape == (0, 2, 64)
    c = Case(cf, dev, [20, 0], [0, 0], 2, 2, 64, "bf16")
    q = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=dev)
    out = torch.full_like(q, CANARY)
    cf.kv8_attention(q, c.cache, c.lens, table=c.table, q_starts=c.q_starts, out=out)
    torch.cuda.synchronize()
    assert (out == CANARY).all()


@pytest.mark.parametrize("most", [2, 45])
def test_many_sequences(cf, dev, most):
    say(f"kv8 attention 500 sequences of up to {most} queries")
    rng = np.random.default_rng(2)
    kv, nq = ([int(x) for x in rng.integers(0, n, 500)] for n in (40, most + 1))
    kv[333], nq[3] = 3000, most
    c = Case(cf, dev, kv, nq, 2, 1, 64, "bf16", seed=3)
    c.check(*c.run(max_q=most, causal=True), causal=True)


def test_workspace_needs_nothing_and_is_not_overrun(cf, dev):
    say("kv8 attention workspace")
    for nq, dtype in ((1, "bf16"), (10, "f32"), (130, "bf16"), (130, "f32")):
        c = Case(cf, dev, [900, 31], [nq, nq], 2, 2, 128, dtype)
        need = cf.kv8_attention_workspace_bytes(DT[dtype], nq, 2, 2, 128)
        want = c.run(max_q=nq)
        for fill in (0xFF, 0x00, 0x7F):
            buf = torch.full((need + 8192,), fill, dtype=torch.uint8, device=dev)
            got = c.run(max_q=nq, workspace=buf[4096:4096 + need])
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            assert (buf[:4096] == fill).all() and (buf[4096 + need:] == fill).all()


def test_offsets_past_32_bits(cf, dev):
    say("kv8 attention past 4 GiB")
    heads, dim, page = 4, 128, 256
    size = 2 * page * dim + 32
    pages = (1 << 32) // (heads * size) + 40
    cache = cf.KV8Cache(torch.empty((pages, heads, size), dtype=torch.uint8, device=dev), page, dim)
    table = torch.tensor([[pages - 1, 3], [0, pages - 3]], dtype=torch.int32, device=dev)
    x = torch.randn(2, 600, heads, dim, device=dev)
    starts, lens = torch.tensor([0, 300, 600], dtype=torch.int32, device=dev), torch.tensor([300, 300], dtype=torch.int32, device=dev)
    cf.kv8_append(cache, x[0], x[1], lens, table=table, starts=starts)
    held = []
    for y in x:
        held.append([])
        for b in range(2):
            h = ref.Held(heads, dim)
            h.append(host(y[300 * b:300 * b + 300].double()))
            held[-1].append(h.x)
    for nq in (1, 50):
        q = torch.randn(2 * nq, heads, dim, device=dev).bfloat16()
        lse = torch.empty(2 * nq, heads, device=dev)
        out = cf.kv8_attention(q, cache, lens, table=table, causal=True, lse=lse)
        torch.cuda.synchronize()
        for b in range(2):
            rows = slice(b * nq, b * nq + nq)
            want = ref.attention(host(q[rows].double()), held[0][b], held[1][b], dim ** -0.5, True, 0, ref.P_BF16)
            compare(host(out[rows].double()), host(lse[rows].double()), *want, f"sequence {b}")


def test_side_stream(cf, dev):
    say("kv8 attention on a side stream")
    c = Case(cf, dev, [600, 50], [1, 1], 8, 2, 128, "bf16")
    want, _ = c.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        out = cf.kv8_attention(c.q, c.cache, c.lens, table=c.table, q_starts=c.q_starts, stream=side)
        torch.empty(1 << 20, device=dev).fill_(7)  # the freed workspace must not be handed out yet
        side.synchronize()
        assert torch.equal(out, want)


def test_two_graphs_share_a_workspace(cf, dev):
    say("kv8 attention, two graphs, one workspace")
    a = Case(cf, dev, [500, 33], [1, 1], 8, 2, 128, "bf16", seed=1)
    b = Case(cf, dev, [260], [50], 8, 2, 128, "bf16", seed=2)
    ws = torch.empty(max(cf.kv8_attention_workspace_bytes(torch.bfloat16, n, 8, 2, 128) for n in (1, 50)), dtype=torch.uint8, device=dev)
    side = torch.cuda.Stream()
    graphs, outs = [], []
    for c, n in ((a, 1), (b, 50)):
        o = torch.zeros_like(c.q)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=side):
            cf.kv8_attention(c.q, c.cache, c.lens, table=c.table, q_starts=c.q_starts, max_q=n, causal=True, out=o, workspace=ws)
        graphs.append(g), outs.append(o)
    for i in range(4):
        for c, g in zip((a, b), graphs):
            c.q.copy_(torch.randn_like(c.q))
            if i == 2:  # lengths are read at every replay
                c.lens.sub_(7)
            g.replay()
        torch.cuda.synchronize()
        for c, o, n in zip((a, b), outs, (1, 50)):
            want = cf.kv8_attention(c.q, c.cache, c.lens, table=c.table, q_starts=c.q_starts, max_q=n, causal=True)
            torch.cuda.synchronize()
            assert torch.equal(o, want), f"replay {i}"


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("max_q", [1, 17, 33])  # each kernel
def test_fp32_queries_and_probabilities_are_whole(cf, dev, dim, max_q):
    """Sequences of one key, which the cache holds exactly: every part of a query and of a probability shows."""
    say(f"kv8 attention fp32, one key a row, dim={dim} max_q={max_q}")
    rng = np.random.default_rng(dim + max_q)
    n = 300
    q, k, v = ref.one_key_rows(rng, n, dim)
    k = np.sign(k) * (16 + 2 * rng.integers(0, 8, (n, 1))).astype(np.float32)  # numbers of three binary places
    v = np.sign(v) * (1 + rng.integers(0, 8, v.shape) / 8).astype(np.float32)
    want = ref.one_key(q, k, v, 0.25)
    cache = cf.KV8Cache.create(n, 16, 1, dim)
    lens = torch.ones(n, dtype=torch.int32, device=dev)
    q, k, v = (torch.from_numpy(x).to(dev)[:, None] for x in (q, k, v))
    cf.kv8_append(cache, k, v, lens, table_width=1)
    kk, vv = cf.kv8_read(cache, torch.arange(n, device=dev) * 16, torch.float32)
    starts = torch.arange(n + 1, dtype=torch.int32, device=dev)
    lse = torch.full((n, 1), CANARY, device=dev)
    out = cf.kv8_attention(q, cache, lens, q_starts=starts, max_q=max_q, scale=0.25, table_width=1, lse=lse)
    torch.cuda.synchronize()
    assert torch.equal(kk, k) and torch.equal(vv, v)
    for got, y, b in ((host(out[:, 0].double()), want[0], want[2]), (host(lse[:, 0].double()), want[1], want[3])):
        assert (np.abs(got - y) <= b).all(), f"{(np.abs(got - y) / b).max():.3g} of the bound"


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("max_q,p_step", [(1, ref.P_FP16), (17, ref.P_FP16), (33, ref.P_BF16)])
def test_probabilities_are_as_exact_as_stated(cf, dev, dim, max_q, p_step):
    """bf16 rows whose two values all but cancel: fp16 probabilities in calls of at most 32 rows."""
    say(f"kv8 attention bf16, two keys a row, dim={dim} max_q={max_q}")
    n = 300
    x = torch.from_numpy(np.random.default_rng(dim).uniform(-0.125, 0.125, n)).to(torch.bfloat16)
    want, bound = ref.two_keys(x.double().numpy(), p_step)
    k, v = torch.zeros(2, n, 2, 1, dim, device=dev)
    k[:, 1, 0, 0] = 1
    v[:, 0], v[:, 1] = 1, -1
    cache = cf.KV8Cache.create(n, 16, 1, dim)
    lens = torch.full((n,), 2, dtype=torch.int32, device=dev)
    cf.kv8_append(cache, k.flatten(0, 1), v.flatten(0, 1), lens, table_width=1)
    q = torch.zeros(n, 1, dim, dtype=torch.bfloat16, device=dev)
    q[:, 0, 0] = x.to(dev)
    starts = torch.arange(n + 1, dtype=torch.int32, device=dev)
    out = cf.kv8_attention(q, cache, lens, q_starts=starts, max_q=max_q, scale=1.0, table_width=1)
    torch.cuda.synchronize()
    far = np.abs(host(out[:, 0].double()) - want[:, None])
    assert (far <= bound[:, None]).all(), f"{(far / bound[:, None]).max():.3g} of the bound"
