"""cf_kv4_attention against softmax(scale Q K^T) V in 64 bits over the values the cache holds: ragged
lengths from none to thousands, shared heads, causal and windowed rows, empty rows, pages in any order,
bytes of earlier owners, NaN and infinities in hidden and in seen places, strides, streams, graphs that
share a workspace, and the chain of norms, cache and attention."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import attn_ref as ref
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
    """Sequences of `kv` keys and `nq` queries in a cache whose other bytes are all 0xFF."""

    def __init__(self, cf, dev, kv, nq, hq, hk, dim, dtype, page=16, seed=0, spread=1.0, table=True, stale=0xFF):
        rng = np.random.default_rng(seed)
        self.kv, self.nq, self.dtype = kv, nq, dtype
        per = [-(-n // page) for n in kv]
        width = max(per + [1]) + 1
        pages = sum(per) + 2 if table else len(kv) * width
        data = torch.full((pages, hk, page * dim * 17 // 16), stale, dtype=torch.uint8, device=dev)
        self.cache = cf.KV4Cache(data, page, dim)
        order = rng.permutation(pages)
        tab = np.full((len(kv), width), -7, np.int32)
        self.k, self.v, self.slots = [], [], []
        at = 0
        for i, n in enumerate(kv):
            mine = order[at:at + per[i]] if table else i * width + np.arange(per[i])
            at += per[i]
            tab[i, :per[i]] = mine
            slots = (mine[:, None] * page + np.arange(page)).reshape(-1)[:n]
            k = (rng.standard_normal((n, hk, dim)) * spread).astype(np.float32)
            v = (rng.standard_normal((n, hk, dim)) + 0.2).astype(np.float32)
            if n:
                s = torch.from_numpy(slots.astype(np.int64)).to(dev)
                cf.kv4_append(self.cache, torch.from_numpy(k).to(dev), torch.from_numpy(v).to(dev), s)
            self.k.append(ref.quantize(k) if n else k)
            self.v.append(ref.quantize(v) if n else v)
            self.slots.append(slots)
        self.q = torch.from_numpy(rng.standard_normal((sum(nq), hq, dim)).astype(np.float32)).to(DT[dtype]).to(dev)
        self.starts = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
        self.table = torch.from_numpy(tab).to(dev) if table else None
        self.width = width
        self.lens = torch.tensor(kv, dtype=torch.int32, device=dev)
        self.q_starts = torch.from_numpy(self.starts).to(dev)

    def run(self, cf, **kw):
        lse = torch.full(self.q.shape[:2], CANARY, dtype=torch.float32, device=self.q.device)
        kw = {"table": self.table, "q_starts": self.q_starts, "table_width": self.width, **kw}
        out = cf.kv4_attention(self.q, self.cache, self.lens, lse=lse, **kw)
        torch.cuda.synchronize()
        return out, lse

    def check(self, out, lse, causal=False, window=0, scale=None):
        d = self.q.shape[2]
        out, lse = host(out.float()).astype(np.float64), host(lse).astype(np.float64)
        q = self.q.double().cpu().numpy()
        for i, n in enumerate(self.nq):
            a, b = self.starts[i], self.starts[i + 1]
            o, l, bo, bl = ref.attention(q[a:b], self.k[i], self.v[i], n, scale or d ** -0.5, causal, window)
            bound = ref.out_bound(o, bo, self.kv[i], self.v[i], self.dtype, q.shape[1])
            empty = np.isneginf(l)
            assert np.array_equal(np.isneginf(lse[a:b]), empty), f"sequence {i}: empty rows"
            assert (out[a:b][empty] == 0).all()
            nan = np.isnan(o)
            assert np.array_equal(np.isnan(out[a:b]), nan), f"sequence {i}: NaN"
            far = np.abs(out[a:b] - o)
            assert (far[~nan] <= bound[~nan]).all(), f"sequence {i}: {np.nanmax(far / (bound + 1e-30)):.3g} of the bound"
            ok = ~empty & ~np.isnan(l)
            far = np.abs(lse[a:b][ok] - l[ok])
            assert (far <= bl[ok]).all(), f"sequence {i}: lse {(far / bl[ok]).max():.3g} of the bound"
            assert np.array_equal(np.isnan(lse[a:b]), np.isnan(l))


LENGTHS = [0, 1, 7, 8, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 300]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 4), (8, 2), (6, 2), (16, 1), (24, 1)])
def test_one_query_each(cf, dev, dtype, dim, hq, hk):
    say(f"kv4 attention single queries {dtype} dim={dim} heads={hq}/{hk}")
    c = Case(cf, dev, LENGTHS, [1] * len(LENGTHS), hq, hk, dim, dtype, seed=dim + hq)
    c.check(*c.run(cf, max_q=1, causal=True), causal=True)
    # all queries of one size need no starts; without the mask one query sees the same keys
    a, b = c.run(cf, q_starts=None)
    c.check(a, b)


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
    say(f"kv4 attention {dtype} dim={dim} causal={causal} window={window} heads={hq}/{hk} kv={kv} nq={nq}")
    c = Case(cf, dev, kv, nq, hq, hk, dim, dtype, page=32, seed=sum(kv))
    c.check(*c.run(cf, max_q=max(nq), causal=causal, window=window), causal, window)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("table", [True, False])
@pytest.mark.parametrize("dim", [64, 128])
def test_pages(cf, dev, page, table, dim):
    say(f"kv4 attention page={page} table={table} dim={dim}")
    c = Case(cf, dev, [page - 1, page, page + 1, 3 * page + 5, 0], [1, 2, 3, 1, 1], 4, 2, dim, "bf16", page=page, table=table)
    c.check(*c.run(cf, causal=True), causal=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 20, 300])
def test_split_over_workgroups(cf, dev, dtype, nq):
    """Few rows over many keys: an item's keys are spread over the chip and joined."""
    say(f"kv4 attention split {dtype} nq={nq}")
    kv = {1: 20000, 20: 6000, 300: 2500}[nq]
    c = Case(cf, dev, [kv, 70], [nq, 1], 2, 1, 128, dtype, page=64, seed=nq, spread=2.0)
    a = c.run(cf, max_q=nq, causal=True)
    c.check(*a, causal=True)
    b = c.run(cf, max_q=nq, causal=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), "two calls differ"


def test_peaked_rows(cf, dev):
    """Scores over hundreds: the reference moves, and one key may outweigh the rest."""
    say("kv4 attention peaked rows")
    for dtype in ("bf16", "f32"):
        c = Case(cf, dev, [700, 513], [3, 40], 2, 2, 64, dtype, spread=30.0, seed=9)
        c.check(*c.run(cf, scale=0.5), scale=0.5)
        c.check(*c.run(cf, scale=1e-4), scale=1e-4)


def test_rising_scores(cf, dev):
    """Each unit of keys beats the last by a little or a lot."""
    say("kv4 attention rising scores")
    for step in (0.01, 0.3, 4.0):
        c = Case(cf, dev, [640], [17], 1, 1, 128, "f32", seed=1)
        k = np.zeros((640, 1, 128), np.float32)
        k[:, 0, 0] = step * (np.arange(640) // 8)
        cf.kv4_append(c.cache, torch.from_numpy(k).to(dev), torch.from_numpy(c.v[0].astype(np.float32)).to(dev),
                      torch.from_numpy(c.slots[0]).to(dev))
        c.k[0] = ref.quantize(k)
        c.q[:, :, 0] = torch.linspace(-8, 8, 17, device=dev)[:, None]
        c.check(*c.run(cf, scale=1.0), scale=1.0)


def test_wrong_bound_of_queries_is_only_slow(cf, dev):
    say("kv4 attention max_q below the longest")
    c = Case(cf, dev, [90, 40], [70, 3], 4, 2, 64, "bf16")
    for m in (1, 9, 0, 73):
        c.check(*c.run(cf, max_q=m, causal=True), causal=True)


@pytest.mark.parametrize("nq", [1, 9, 70])
def test_pages_outside_the_cache_hold_nothing(cf, dev, nq):
    say(f"kv4 attention pages outside the cache nq={nq}")
    c = Case(cf, dev, [100], [nq], 2, 1, 128, "bf16", page=16)
    whole = c.run(cf)
    c.check(*whole)
    for bad in (-1, c.cache.data.shape[0], 2 ** 31 - 1, -2 ** 31):
        keep = c.table.clone()
        c.table[0, 2] = bad
        out, lse = c.run(cf)
        c.table = keep
        k, v = c.k[0], c.v[0]
        c.k[0], c.v[0] = (np.delete(x, np.arange(32, 48), 0) for x in (k, v))
        c.kv[0] = 84
        c.check(out, lse)
        c.k[0], c.v[0], c.kv[0] = k, v, 100
    c.table.fill_(-1)
    out, lse = c.run(cf)
    assert not out.any() and lse.isneginf().all()


def test_lengths_are_cut_to_the_table(cf, dev):
    say("kv4 attention lengths past the table")
    c = Case(cf, dev, [32, 48], [1, 1], 1, 1, 64, "bf16", page=16)
    c.table[0, 2:] = c.table[1, :2]  # a length of 64 is what two more pages hold
    c.lens = torch.tensor([10 ** 9, -5], dtype=torch.int32, device=dev)
    out, lse = c.run(cf)
    c.k[0], c.v[0] = np.concatenate([c.k[0], c.k[1][:32]]), np.concatenate([c.v[0], c.v[1][:32]])
    c.k[1], c.v[1] = c.k[1][:0], c.v[1][:0]
    c.kv = [64, 0]
    c.check(out, lse)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("nq", [4, 30, 120])
def test_nan_reaches_only_rows_that_see_it(cf, dev, dim, nq):
    say(f"kv4 attention NaN keys and values dim={dim} nq={nq}")
    for what in ("k", "v", "both"):
        c = Case(cf, dev, [150], [nq], 2, 1, dim, "bf16", page=16, seed=4)
        at = 150 - nq // 2  # seen by the later half of the rows only
        k, v = np.zeros((1, 1, dim), np.float32), np.ones((1, 1, dim), np.float32)
        if what != "v":
            k[0, 0, 3] = np.nan
        if what != "k":
            v[0, 0, dim - 40] = np.inf
        cf.kv4_append(c.cache, torch.from_numpy(k).to(dev), torch.from_numpy(v).to(dev),
                      torch.from_numpy(c.slots[0][at:at + 1].copy()).to(dev))
        c.k[0][at], c.v[0][at] = ref.quantize(k)[0], ref.quantize(v)[0]
        c.check(*c.run(cf, causal=True), causal=True)
        c.check(*c.run(cf, causal=True, window=5), causal=True, window=5)


def test_nan_query_stays_in_its_row(cf, dev):
    say("kv4 attention NaN query")
    for nq in (3, 100):
        c = Case(cf, dev, [90], [nq], 2, 2, 64, "bf16")
        want, wl = c.run(cf)
        c.q[1, 1, 5] = float("nan")
        out, lse = c.run(cf)
        assert out[1, 1].isnan().all() and lse[1, 1].isnan()
        out[1, 1], lse[1, 1] = want[1, 1], wl[1, 1]
        assert torch.equal(out, want) and torch.equal(lse, wl)


def test_stale_bytes_do_not_matter(cf, dev):
    say("kv4 attention stale bytes")
    for nq in (1, 60):
        got = [Case(cf, dev, [37, 5], [nq, nq], 4, 1, 64, "bf16", page=64, stale=s).run(cf) for s in (0, 0x7F, 0xFF, 0xC3)]
        for g in got[1:]:
            assert torch.equal(g[0], got[0][0]) and torch.equal(g[1], got[0][1])


@pytest.mark.parametrize("nq", [2, 40])
def test_strides_and_rows_of_no_sequence(cf, dev, nq):
    say(f"kv4 attention strides and rows behind the last sequence nq={nq}")
    c = Case(cf, dev, [50, 60], [nq, nq], 4, 2, 128, "bf16")
    total = 2 * nq
    want, wl = c.run(cf)
    # head-major queries with three rows more, which belong to no sequence; a packed output
    qh = torch.zeros(4, total + 3, 128, dtype=torch.bfloat16, device=dev)
    qh[:, :total] = c.q.transpose(0, 1)
    packed = torch.full((total + 3, 12, 128), CANARY, dtype=torch.bfloat16, device=dev)
    lse = torch.full((total + 3, 4), CANARY, device=dev)
    cf.kv4_attention(qh.transpose(0, 1), c.cache, c.lens, table=c.table, q_starts=c.q_starts, max_q=nq,
                     out=packed[:, 4:8], lse=lse)
    torch.cuda.synchronize()
    assert torch.equal(packed[:total, 4:8], want) and torch.equal(lse[:total], wl)
    assert (packed[:, :4] == CANARY).all() and (packed[:, 8:] == CANARY).all()
    assert (packed[total:] == CANARY).all() and (lse[total:] == CANARY).all()
    # a gap before the first sequence
    c.q_starts = c.q_starts + 1
    lse.fill_(CANARY), packed.fill_(CANARY)
    qh[:, 1:total + 1] = c.q.transpose(0, 1)
    cf.kv4_attention(qh.transpose(0, 1), c.cache, c.lens, table=c.table, q_starts=c.q_starts, max_q=nq,
                     out=packed[:, 4:8], lse=lse)
    torch.cuda.synchronize()
    assert torch.equal(packed[1:total + 1, 4:8], want) and (packed[0] == CANARY).all() and (lse[0] == CANARY).all()


def test_nothing_to_do(cf, dev):
    say("kv4 attention no queries")
    c = Case(cf, dev, [20], [1], 2, 2, 64, "bf16")
    out = cf.kv4_attention(c.q[:0], c.cache, c.lens, table=c.table)
    assert out.shape == (0, 2, 64)
    c = Case(cf, dev, [20, 0], [0, 0], 2, 2, 64, "bf16")
    q = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=dev)
    out = torch.full_like(q, CANARY)
    cf.kv4_attention(q, c.cache, c.lens, table=c.table, q_starts=c.q_starts, out=out)
    torch.cuda.synchronize()
    assert (out == CANARY).all()


def test_many_sequences(cf, dev):
    """More sequences than a workgroup has threads, most of them short, some without queries."""
    say("kv4 attention 700 sequences")
    rng = np.random.default_rng(2)
    kv = [int(x) for x in rng.integers(0, 40, 700)]
    nq = [int(x) for x in rng.integers(0, 3, 700)]
    kv[333] = 3000
    c = Case(cf, dev, kv, nq, 2, 1, 64, "bf16", seed=3)
    c.check(*c.run(cf, max_q=2, causal=True), causal=True)


@pytest.mark.parametrize("batch", [33, 64, 65, 130])
def test_many_sequences_of_many_rows(cf, dev, batch):
    say(f"kv4 attention {batch} sequences of up to 45 queries")
    rng = np.random.default_rng(batch)
    kv = [int(x) for x in rng.integers(0, 90, batch)]
    nq = [int(x) for x in rng.integers(0, 46, batch)]
    nq[3] = 45
    c = Case(cf, dev, kv, nq, 2, 1, 64, "bf16", seed=3)
    c.check(*c.run(cf, max_q=45, causal=True), causal=True)


def test_largest_window(cf, dev):
    say("kv4 attention with a window past every length")
    for nq in (3, 90):
        c = Case(cf, dev, [70, 5], [nq, nq], 2, 2, 64, "bf16")
        want = c.run(cf, causal=True)
        got = c.run(cf, causal=True, window=2 ** 31 - 1)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rows_do_not_depend_on_the_tile_they_are_in(cf, dev):
    """The same query at several places of a batch: results agree to the bound, whatever kernel and
    split they meet."""
    say("kv4 attention, one query in many places")
    c = Case(cf, dev, [2000] * 3, [1, 20, 200], 4, 1, 128, "f32", seed=7)
    c.q[:] = c.q[0]
    for i in (1, 2):  # three times the same keys
        c.table[i] = c.table[0]
        c.k[i], c.v[i] = c.k[0], c.v[0]
    out, lse = c.run(cf)
    c.check(out, lse)
    for m in (1, 8, 0):
        c.check(*c.run(cf, max_q=m))


def test_workspace_needs_nothing_and_is_not_overrun(cf, dev):
    say("kv4 attention workspace")
    for nq, dtype in ((1, "bf16"), (10, "f32"), (130, "bf16")):
        c = Case(cf, dev, [900, 31], [nq, nq], 2, 2, 128, dtype)
        need = cf.kv4_attention_workspace_bytes(DT[dtype], nq, 2, 2, 128)
        want = c.run(cf, max_q=nq)
        for fill in (0xFF, 0x00, 0x7F):
            buf = torch.full((need + 8192,), fill, dtype=torch.uint8, device=dev)
            got = c.run(cf, max_q=nq, workspace=buf[4096:4096 + need])
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            assert (buf[:4096] == fill).all() and (buf[4096 + need:] == fill).all()


def test_side_stream(cf, dev):
    say("kv4 attention on a side stream")
    c = Case(cf, dev, [600, 50], [1, 1], 8, 2, 128, "bf16")
    want, _ = c.run(cf)
    side = torch.cuda.Stream()
    for _ in range(3):
        out = cf.kv4_attention(c.q, c.cache, c.lens, table=c.table, q_starts=c.q_starts, stream=side)
        torch.empty(1 << 20, device=dev).fill_(7)  # the freed workspace must not be handed out yet
        side.synchronize()
        assert torch.equal(out, want)


def test_two_graphs_share_a_workspace(cf, dev):
    say("kv4 attention, two graphs, one workspace")
    a = Case(cf, dev, [500, 33], [1, 1], 8, 2, 128, "bf16", seed=1)
    b = Case(cf, dev, [260], [50], 8, 2, 128, "bf16", seed=2)
    ws = torch.empty(max(cf.kv4_attention_workspace_bytes(torch.bfloat16, n, 8, 2, 128) for n in (1, 50)), dtype=torch.uint8, device=dev)
    side = torch.cuda.Stream()
    graphs, outs = [], []
    for c, n in ((a, 1), (b, 50)):
        o = torch.zeros_like(c.q)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=side):
            cf.kv4_attention(c.q, c.cache, c.lens, table=c.table, q_starts=c.q_starts, max_q=n, causal=True, out=o, workspace=ws)
        graphs.append(g), outs.append(o)
    for i in range(4):
        for c, g, o in zip((a, b), graphs, outs):
            c.q.copy_(torch.randn_like(c.q))
            if i == 2:  # lengths are read at every replay
                c.lens.sub_(7)
            g.replay()
        torch.cuda.synchronize()
        for c, o, n in zip((a, b), outs, (1, 50)):
            want = cf.kv4_attention(c.q, c.cache, c.lens, table=c.table, q_starts=c.q_starts, max_q=n, causal=True)
            torch.cuda.synchronize()
            assert torch.equal(o, want), f"replay {i}"


@pytest.mark.parametrize("dim,hq,hk", [(128, 8, 2), (64, 6, 6)])
def test_serving_chain(cf, dev, dim, hq, hk):
    """A prompt in two chunks and then single tokens: norms and rotation, append, attention; against
    the formulas over everything so far."""
    say(f"kv4 serving chain dim={dim} heads={hq}/{hk}")
    rng = np.random.default_rng(8)
    page, n_pos = 16, 200
    cache = cf.KV4Cache.create(16, page, hk, dim)
    table = torch.from_numpy(rng.permutation(16).astype(np.int32)).to(dev)[None]
    ang = np.arange(n_pos)[:, None] * 50.0 ** (-np.arange(dim // 2) / (dim // 2))
    cos, sin = (torch.from_numpy(f(ang).astype(np.float32)).to(dev) for f in (np.cos, np.sin))
    keys, values, done = [], [], 0
    for n in (45, 50, 1, 1, 1):
        x = torch.randn(n, hq + 2 * hk, dim, device=dev, dtype=torch.bfloat16)
        pos = torch.arange(done, done + n, device=dev, dtype=torch.int32)
        slots = table[0, (pos // page).long()].long() * page + pos % page
        q, k = cf.qk_norm_rope(x[:, :hq], x[:, hq:hq + hk], rope=cf.CF_ROPE_HALF, cos=cos, sin=sin, positions=pos)
        cf.kv4_append(cache, k, x[:, hq + hk:], slots)
        done += n
        lens = torch.tensor([done], dtype=torch.int32, device=dev)
        lse = torch.empty(n, hq, device=dev)
        out = cf.kv4_attention(q, cache, lens, table=table, causal=True, lse=lse)
        torch.cuda.synchronize()
        keys.append(ref.quantize(host(k.float())))
        values.append(ref.quantize(host(x[:, hq + hk:].float())))
        kk, vv = np.concatenate(keys), np.concatenate(values)
        o, l, bo, bl = ref.attention(host(q.double()), kk, vv, n, dim ** -0.5, True, 0)
        bound = ref.out_bound(o, bo, done, vv, "bf16", hq)
        assert (np.abs(host(out.double()) - o) <= bound).all()
        assert (np.abs(host(lse.double()) - l) <= bl).all()


def test_receiver_shards(cf, dev):
    """A receiver's reconstructions (fp32, decoded from peers' codes) go into the cache and queries of
    the own shard attend to all of them: what the compressors are for."""
    say("kv4 attention over decoded shards")
    t, h, d = 64, 2, 64
    peers = 3
    g = torch.Generator().manual_seed(6)
    cache = cf.KV4Cache.create(peers * t // 16, 16, h, d)
    keep = []
    for p in range(peers):
        pair = []
        for _ in range(2):
            a0, a1 = (torch.randn(t * h * d, generator=g).to(torch.bfloat16).to(dev) for _ in range(2))
            tx, rx = (torch.empty(t * h * d, device=dev) for _ in range(2))
            cf.init_state(a0, tx)
            cf.init_state(a0, rx)
            codes, scales = cf.compress(2, a1, tx, None)
            cf.decompress(2, codes, scales, rx)
            pair.append(rx.view(t, h, d))
        cf.kv4_append(cache, *pair, torch.arange(p * t, (p + 1) * t, device=dev))
        keep.append(pair)
    q = torch.randn(t, h, d, device=dev, dtype=torch.bfloat16)
    lens = torch.tensor([peers * t], dtype=torch.int32, device=dev)
    lse = torch.empty(t, h, device=dev)
    out = cf.kv4_attention(q, cache, lens, table_width=peers * t // 16, lse=lse)
    torch.cuda.synchronize()
    kk, vv = (np.concatenate([ref.quantize(host(x[i])) for x in keep]) for i in range(2))
    o, l, bo, bl = ref.attention(host(q.double()), kk, vv, t, d ** -0.5, False, 0)
    assert (np.abs(host(out.double()) - o) <= ref.out_bound(o, bo, peers * t, vv, "bf16", h)).all()
    assert (np.abs(host(lse.double()) - l) <= bl).all()
