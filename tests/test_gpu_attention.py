"""cf_attention against softmax(scale Q K^T) V in 64 bits: packed sequences of lengths from none, shared heads, causal and
windowed rows, more queries than keys and fewer, rows that see nothing, infinities and NaN in hidden and seen places,
strides, rows of no sequence, splits, streams, graphs, and prompts whose K and V go into the 8-bit cache."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import serving_ref as ref
from gpu_util import host, say
from test_gpu_kv8_attention import compare

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
    def __init__(self, cf, dev, nk, nq, hq, hk, dim, dtype, seed=0, spread=1.0):
        rng = np.random.default_rng(seed)
        self.cf, self.nk, self.nq, self.dtype = cf, nk, nq, dtype
        new = lambda n, h, s: torch.from_numpy((rng.standard_normal((n, h, dim)) * s).astype(np.float32)).to(DT[dtype]).to(dev)
        self.q, self.k, self.v = new(sum(nq), hq, 1.0), new(sum(nk), hk, spread), new(sum(nk), hk, 1.0) + 0.25
        self.qs, self.ks = (np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (nq, nk))
        self.q_starts, self.k_starts = (torch.from_numpy(x).to(dev) for x in (self.qs, self.ks))

    def run(self, **kw):
        lse = torch.full(self.q.shape[:2], CANARY, dtype=torch.float32, device=self.q.device)
        kw = {"q_starts": self.q_starts, "k_starts": self.k_starts, **kw}
        out = self.cf.attention(self.q, self.k, self.v, lse=lse, **kw)
        torch.cuda.synchronize()
        return out, lse

    def check(self, out, lse, causal=False, window=0, scale=None):
        q, k, v, out, lse = (host(x.double()) for x in (self.q, self.k, self.v, out, lse))
        step, products = (ref.P_BF16, 1) if self.dtype == "bf16" else (ref.P_PARTS, 6)
        for i in range(len(self.nq)):
            a, b, c, d = self.qs[i], self.qs[i + 1], self.ks[i], self.ks[i + 1]
            want = ref.attention(q[a:b], k[c:d], v[c:d], scale or q.shape[2] ** -0.5, causal, window, step, products, self.dtype)
            compare(out[a:b], lse[a:b], *want, f"sequence {i}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 1), (True, 40)])
@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 2), (6, 2), (8, 1)])
def test_prompts(cf, dev, dtype, dim, causal, window, hq, hk):
    nq = [1, 0, 31, 32, 33, 64, 65, 100, 257]
    say(f"attention {dtype} dim={dim} causal={causal} window={window} heads={hq}/{hk} {nq}")
    c = Case(cf, dev, nq, nq, hq, hk, dim, dtype, seed=hq)
    c.check(*c.run(max_q=max(nq), causal=causal, window=window), causal, window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 7)])
def test_more_and_fewer_keys_than_queries(cf, dev, dtype, dim, causal, window):
    say(f"attention of unequal lengths {dtype} dim={dim} causal={causal} window={window}")
    c = Case(cf, dev, [0, 5, 1, 300, 90, 17, 0], [4, 70, 0, 1, 40, 150, 1], 3, 3, dim, dtype, seed=1)
    c.check(*c.run(causal=causal, window=window), causal, window)
    c = Case(cf, dev, [200, 64, 3], [1, 1, 1], 4, 2, dim, dtype, seed=2)
    c.check(*c.run(max_q=1, causal=causal, window=window), causal, window)
    c.check(*c.run(q_starts=None, causal=causal, window=window), causal, window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq,nk", [(1, 20000), (40, 5000), (300, 2500), (700, 700)])
def test_split_over_workgroups(cf, dev, dtype, nq, nk):
    say(f"attention split {dtype} {nq} queries, {nk} keys")
    c = Case(cf, dev, [nk, 70], [nq, 1], 2, 1, 128, dtype, seed=nq, spread=2.0)
    a = c.run(max_q=nq, causal=True)
    c.check(*a, causal=True)
    b = c.run(max_q=nq, causal=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), "two calls differ"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("nq,nk", [(30, 900), (129, 1300), (200, 2700), (256, 16411)])
def test_an_item_in_many_parts(cf, dev, dtype, dim, nq, nk):
    """Whatever workgroup comes last, and whatever lies in the workspace, the bits are the same."""
    say(f"attention of one item in parts {dtype} dim={dim} {nq} queries, {nk} keys")
    c = Case(cf, dev, [nk], [nq], 1, 1, dim, dtype, seed=nk)
    ws = torch.empty(cf.attention_workspace_bytes(DT[dtype], nq, 1, 1, dim), dtype=torch.uint8, device=dev)
    want = c.run(max_q=nq, workspace=ws)
    c.check(*want)
    for i in range(20):
        if i % 3 == 0:
            ws.random_(0, 256)
        got = c.run(max_q=nq, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), f"call {i} differs"


def test_peaked_rows(cf, dev):
    say("attention peaked rows")
    for dtype in ("bf16", "f32"):
        for dim in (64, 128):
            c = Case(cf, dev, [700, 513], [300, 40], 2, 2, dim, dtype, spread=30.0, seed=9)
            c.check(*c.run(scale=0.5), scale=0.5)
            c.check(*c.run(scale=1e-4, causal=True), scale=1e-4, causal=True)


def test_rising_scores(cf, dev):
    """Each 8 keys beat the last by a little or a lot."""
    say("attention rising scores")
    for dtype in ("bf16", "f32"):
        for step in (0.0625, 0.5, 4.0):
            c = Case(cf, dev, [640], [140], 1, 1, 128, dtype, seed=1)
            c.k.zero_(), c.q.zero_()
            c.k[:, 0, 0] = (step * (torch.arange(640, device=dev) // 8)).to(c.k.dtype)
            c.q[:, :, 0] = torch.linspace(-8, 8, 140, device=dev)[:, None].to(c.q.dtype)
            c.check(*c.run(scale=1.0), scale=1.0)


def test_equal_sizes_need_no_starts(cf, dev):
    say("attention without starts")
    c = Case(cf, dev, [50] * 3, [20] * 3, 4, 2, 64, "bf16")
    a = c.run(causal=True)
    b = c.run(causal=True, q_starts=None, k_starts=None, batch=3)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c.check(*a, causal=True)


def test_wrong_bound_of_queries_is_only_slow(cf, dev):
    say("attention max_q below the longest")
    for dtype in ("bf16", "f32"):
        c = Case(cf, dev, [300, 40], [300, 3], 4, 2, 64, dtype)
        for m in (1, 9, 0, 303):
            c.check(*c.run(max_q=m, causal=True), causal=True)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [40, 300])
def test_nan_and_infinities_reach_only_rows_that_see_them(cf, dev, dim, dtype, nq):
    say(f"attention NaN and infinite keys and values dim={dim} {dtype} nq={nq}")
    for what in ("k", "v", "both"):
        c = Case(cf, dev, [nq, 70, nq], [nq, 70, nq], 2, 1, dim, dtype, seed=4)
        # in the first sequence, seen by its later half; the last row of the second; the third is whole
        at, end = nq // 2, nq + 69
        for bad in (float("nan"), float("inf"), -float("inf")):
            if what != "v":
                c.k[at, 0, 3], c.k[end, 0, 5] = bad, bad
            if what != "k":
                c.v[at, 0, dim - 40], c.v[end, 0, 1] = bad, bad
            for kw in (dict(causal=True), dict(causal=True, window=5)):
                out, lse = c.run(**kw)
                w = kw.get("window", nq)
                hit = torch.zeros(2 * nq + 70, dtype=torch.bool, device=dev)
                hit[at:min(at + w, nq)] = hit[end] = True
                if what != "v":  # a score of -infinity is a key that weighs nothing
                    assert not (np.isnan(bad) and torch.isfinite(out[hit]).all(-1).any())
                else:
                    assert torch.isfinite(lse).all()
                    assert not torch.isfinite(out[at:min(at + w, nq), :, dim - 40]).any() and not torch.isfinite(out[end, :, 1]).any()
                    good = torch.ones(dim, dtype=torch.bool, device=dev)
                    good[dim - 40] = good[1] = False
                    assert torch.isfinite(out[hit][:, :, good]).all()
                assert torch.isfinite(out[~hit]).all() and torch.isfinite(lse[~hit]).all()
                # and the rest is as without them
                k, v = c.k.clone(), c.v.clone()
                c.k, c.v = c.k.nan_to_num(0, 0, 0), c.v.nan_to_num(0, 0, 0)
                want, wl = c.run(**kw)
                want[~hit], wl[~hit] = out[~hit], lse[~hit]
                c.check(want, wl, **kw)
                c.k, c.v = k, v


def test_nan_query_stays_in_its_row(cf, dev):
    say("attention NaN query")
    for dtype in ("bf16", "f32"):
        c = Case(cf, dev, [290], [290], 2, 2, 64, dtype)
        want, wl = c.run()
        c.q[1, 1, 5] = float("nan")
        out, lse = c.run()
        assert out[1, 1].isnan().all() and lse[1, 1].isnan()
        out[1, 1], lse[1, 1] = want[1, 1], wl[1, 1]
        assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
def test_strides_and_rows_of_no_sequence(cf, dev, dtype, dim):
    say(f"attention strides and rows of no sequence {dtype} dim={dim}")
    c = Case(cf, dev, [90, 60], [30, 160], 4, 2, dim, dtype)
    want, wl = c.run(causal=True)
    tq, tk = 190, 150
    for gap in (0, 1):
        # q, k and v out of one product, other rows around them all NaN; a packed output
        n = max(tq, tk) + 3
        x = torch.full((n, 8, dim), float("nan"), dtype=DT[dtype], device=dev)
        x[gap:tq + gap, :4], x[gap:tk + gap, 4:6], x[gap:tk + gap, 6:] = c.q, c.k, c.v
        packed = torch.full((n, 12, dim), CANARY, dtype=DT[dtype], device=dev)
        lse = torch.full((n, 4), CANARY, device=dev)
        cf.attention(x[:, :4], x[:, 4:6], x[:, 6:], q_starts=c.q_starts + gap, k_starts=c.k_starts + gap, causal=True, out=packed[:, 4:8], lse=lse)
        torch.cuda.synchronize()
        assert torch.equal(packed[gap:tq + gap, 4:8], want) and torch.equal(lse[gap:tq + gap], wl)
        assert (packed[:, :4] == CANARY).all() and (packed[:, 8:] == CANARY).all() and (packed[:gap] == CANARY).all()
        assert (packed[tq + gap:] == CANARY).all() and (lse[tq + gap:] == CANARY).all() and (lse[:gap] == CANARY).all()
    # head-major
    q, k, v = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (c.q, c.k, c.v))
    out = torch.empty(4, tq, dim, dtype=DT[dtype], device=dev).transpose(0, 1)
    cf.attention(q, k, v, q_starts=c.q_starts, k_starts=c.k_starts, causal=True, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    # one key row for all tokens, one head for all heads
    k1 = c.k[:1, :1].expand(150, 2, dim)
    a = cf.attention(c.q, k1, c.v, q_starts=c.q_starts, k_starts=c.k_starts)
    b = cf.attention(c.q, k1.contiguous(), c.v, q_starts=c.q_starts, k_starts=c.k_starts)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_keys_past_32_bits(cf, dev):
    """Keys so far apart that their offsets pass 2^32 bytes, in both layouts."""
    say("attention past 4 GiB")
    big = torch.empty((1 << 31) + (1 << 25), dtype=torch.bfloat16, device=dev)
    c = Case(cf, dev, [130], [130], 2, 2, 64, "bf16")
    want, _ = c.run(causal=True)
    for shape in ((1 << 24, 64), (64, 1 << 30)):  # 2^25 bytes from token to token; 2^31 from head to head
        k, v = (torch.as_strided(big, (130, 2, 64), (*shape, 1), at) for at in (0, 256 * 64))
        k.copy_(c.k), v.copy_(c.v)
        out = cf.attention(c.q, k, v, causal=True)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_nothing_to_do(cf, dev):
    say("attention of nothing")
    c = Case(cf, dev, [20], [10], 2, 2, 64, "bf16")
    assert cf.attention(c.q[:0], c.k, c.v).shape == (0, 2, 64)
    out, lse = torch.full_like(c.q, CANARY), torch.full((10, 2), CANARY, device=dev)
    cf.attention(c.q, c.k[:0], c.v[:0], out=out, lse=lse)
    torch.cuda.synchronize()
    assert not out.any() and lse.isneginf().all()
    out.fill_(CANARY)
    z = torch.zeros(4, dtype=torch.int32, device=dev)
    cf.attention(c.q, c.k, c.v, q_starts=z, k_starts=z, out=out)
    torch.cuda.synchronize()
    assert (out == CANARY).all()


def test_many_sequences(cf, dev):
    say("attention of 600 prompts")
    rng = np.random.default_rng(2)
    n = [int(x) for x in rng.integers(0, 50, 600)]
    n[333] = 900
    c = Case(cf, dev, n, n, 2, 1, 64, "bf16", seed=3)
    c.check(*c.run(max_q=900, causal=True), causal=True)


def test_largest_window(cf, dev):
    say("attention with a window past every length")
    c = Case(cf, dev, [170, 5], [170, 90], 2, 2, 64, "bf16")
    want, got = c.run(causal=True), c.run(causal=True, window=2 ** 31 - 1)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_workspace_needs_nothing_and_is_not_overrun(cf, dev):
    say("attention workspace")
    for nq, dtype in ((1, "bf16"), (130, "bf16"), (130, "f32")):
        c = Case(cf, dev, [900, 31], [nq, nq], 2, 2, 128, dtype)
        need = cf.attention_workspace_bytes(DT[dtype], nq, 2, 2, 128)
        want = c.run(max_q=nq)
        for fill in (0xFF, 0x00, 0x7F):
            buf = torch.full((need + 8192,), fill, dtype=torch.uint8, device=dev)
            got = c.run(max_q=nq, workspace=buf[4096:4096 + need])
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            assert (buf[:4096] == fill).all() and (buf[4096 + need:] == fill).all()


def test_side_stream_and_graphs_that_share_a_workspace(cf, dev):
    say("attention on a side stream, and two graphs with one workspace")
    a, b = Case(cf, dev, [300, 33], [300, 33], 8, 2, 128, "bf16", seed=1), Case(cf, dev, [260], [50], 8, 2, 128, "bf16", seed=2)
    side = torch.cuda.Stream()
    want, _ = a.run(causal=True)
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        out = cf.attention(a.q, a.k, a.v, q_starts=a.q_starts, k_starts=a.k_starts, causal=True, stream=side)
        torch.empty(1 << 20, device=dev).fill_(7)
        side.synchronize()
        assert torch.equal(out, want)
    ws = torch.empty(max(cf.attention_workspace_bytes(torch.bfloat16, n, 8, 2, 128) for n in (300, 50)), dtype=torch.uint8, device=dev)
    graphs, outs = [], []
    for c in (a, b):
        o = torch.zeros_like(c.q)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=side):
            cf.attention(c.q, c.k, c.v, q_starts=c.q_starts, k_starts=c.k_starts, causal=True, out=o, workspace=ws)
        graphs.append(g), outs.append(o)
    for i in range(4):
        for c, g in zip((a, b), graphs):
            c.q.copy_(torch.randn_like(c.q)), c.v.copy_(torch.randn_like(c.v))
            if i == 2:  # starts are read at every replay
                c.k_starts[-1:].sub_(7)
            g.replay()
        torch.cuda.synchronize()
        for c, o in zip((a, b), outs):
            want = cf.attention(c.q, c.k, c.v, q_starts=c.q_starts, k_starts=c.k_starts, causal=True)
            torch.cuda.synchronize()
            assert torch.equal(o, want), f"replay {i}"


def test_two_calls_at_once(cf, dev):
    """Items in many parts on two streams, each with a workspace, while the other runs."""
    say("attention on two streams at once")
    cases = [Case(cf, dev, [9000, 700], [200, 31], 4, 2, 128, "bf16", seed=1), Case(cf, dev, [5000], [256], 2, 1, 64, "bf16", seed=2)]
    wants = [c.run(causal=True) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        outs = [[] for _ in cases]
        for _ in range(4):
            for c, s, o in zip(cases, streams, outs):
                o.append(cf.attention(c.q, c.k, c.v, q_starts=c.q_starts, k_starts=c.k_starts, causal=True, stream=s))
        torch.cuda.synchronize()
        for o, (want, _) in zip(outs, wants):
            assert all(torch.equal(x, want) for x in o)


def test_decoded_shards(cf, dev):
    """A receiver's bf16 copies of its peers' reconstructions, attended to where they lie."""
    say("attention over decoded shards")
    t, h, d, peers = 96, 2, 64, 3
    g = torch.Generator().manual_seed(6)
    kv = torch.empty(2, peers * t, h, d, dtype=torch.bfloat16, device=dev)
    for x in kv:
        a0, a1 = (torch.randn(peers * t * h * d, generator=g).to(torch.bfloat16).to(dev) for _ in range(2))
        tx, rx = (torch.empty(peers * t * h * d, device=dev) for _ in range(2))
        cf.init_state(a0, tx)
        cf.init_state(a0, rx)
        codes, scales = cf.compress(2, a1, tx, None)
        cf.decompress(2, codes, scales, rx, out_bf16=x.view(-1))
    q = torch.randn(t, h, d, device=dev, dtype=torch.bfloat16)
    lse = torch.empty(t, h, device=dev)
    out = cf.attention(q, kv[0], kv[1], lse=lse)
    torch.cuda.synchronize()
    want = ref.attention(host(q.double()), host(kv[0].double()), host(kv[1].double()), d ** -0.5, False, 0, ref.P_BF16)
    compare(host(out.double()), host(lse.double()), *want, "shard")


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("alone", [True, False])
def test_no_product_of_fp32_parts_is_left_out(cf, dev, dim, alone):
    """Rows that see one key, in sequences of one token or through a window: nothing hides what a product adds."""
    say(f"attention fp32, one key a row, dim={dim} alone={alone}")
    n = 300
    x = ref.one_key_rows(np.random.default_rng(dim), n, dim)
    want = ref.one_key(*x, 0.25)
    q, k, v = (torch.from_numpy(y).to(dev)[:, None] for y in x)
    lse = torch.full((n, 1), CANARY, device=dev)
    if alone:
        starts = torch.arange(n + 1, dtype=torch.int32, device=dev)
        out = cf.attention(q, k, v, q_starts=starts, k_starts=starts, max_q=1, scale=0.25, lse=lse)
    else:
        out = cf.attention(q, k, v, causal=True, window=1, scale=0.25, lse=lse)
    torch.cuda.synchronize()
    for got, y, b in ((host(out[:, 0].double()), want[0], want[2]), (host(lse[:, 0].double()), want[1], want[3])):
        assert (np.abs(got - y) <= b).all(), f"{(np.abs(got - y) / b).max():.3g} of the bound"
