"""cf_kv4_append and cf_kv4_read: every rounding of the 4-bit format exactly, the stored bytes against
the documented layout, slots, padding, non-finite groups, strides, guard bytes, streams and graphs."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import attn_ref as ref
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


def _rows(rng, *shape):
    x = rng.standard_normal(shape) * np.exp(2 * rng.standard_normal(shape[:-1] + (1,)))
    return x.astype(np.float32)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,heads", [(1, 1), (7, 3), (129, 8), (600, 2)])
def test_round_trip(cf, dev, dim, page, dtype, tokens, heads):
    say(f"kv4 round trip dim={dim} page={page} {dtype} tokens={tokens} heads={heads}")
    rng = np.random.default_rng(tokens + page)
    pages = tokens // page + 3
    cache = cf.KV4Cache.create(pages, page, heads, dim)
    k, v = (torch.from_numpy(_rows(rng, tokens, heads, dim)).to(DT[dtype]) for _ in range(2))
    slots = rng.permutation(pages * page)[:tokens].astype(np.int64)
    cf.kv4_append(cache, k.to(dev), v.to(dev), torch.from_numpy(slots).to(dev))
    for out in ("f32", "bf16"):
        kk, vv = cf.kv4_read(cache, torch.from_numpy(slots).to(dev), DT[out])
        torch.cuda.synchronize()
        assert np.array_equal(host(kk.float()), ref.quantize(k.double().numpy()))
        assert np.array_equal(host(vv.float()), ref.quantize(v.double().numpy()))
    # slots that took nothing still hold the zeros they were made with
    rest = np.setdiff1d(np.arange(pages * page), slots)
    kk, vv = cf.kv4_read(cache, torch.from_numpy(rest).to(dev), torch.float32)
    assert not kk.any() and not vv.any()


def test_every_rounding(cf, dev):
    """All levels, all ties and their neighbours in fp32, at exponents over and past the whole range."""
    say("kv4 every rounding")
    mags = []
    for t in (0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 5.5, 6):
        t = np.float32(t)
        mags += [t, np.nextafter(t, np.float32(9)), max(np.float32(0), np.nextafter(t, np.float32(-9)))]
    mags = np.array(mags, np.float32)
    rows = []
    for e in list(range(-26, 18)) + [-126, -100, 100, 125]:
        for top in (6.0, 3.0, np.nextafter(np.float32(6), np.float32(9)), 4.0, 5.0):
            g = np.concatenate([mags, -mags])
            for part in np.array_split(g, 4):
                x = np.zeros(32, np.float32)
                x[:len(part)] = np.clip(part, -top, top)
                x[31] = top
                rows.append(x * np.float32(2.0) ** np.float32(e))
    rows = np.concatenate(rows)
    rows = np.pad(rows, (0, -len(rows) % 128)).reshape(-1, 1, 128).astype(np.float32)
    n = len(rows)
    cache = cf.KV4Cache.create(n // 16 + 1, 16, 1, 128)
    slots = torch.arange(n, device=dev)
    d = torch.from_numpy(rows).to(dev)
    cf.kv4_append(cache, d, -d, slots)
    k, v = cf.kv4_read(cache, slots, torch.float32)
    torch.cuda.synchronize()
    want = ref.quantize(rows)
    assert np.array_equal(host(k), want) and np.array_equal(host(v), -want)


@pytest.mark.parametrize("dim", [64, 128])
def test_stored_bytes(cf, dev, dim):
    """The bytes of a block are where the header says: a cache is a file format."""
    say(f"kv4 stored bytes dim={dim}")
    page, heads = 32, 3
    rng = np.random.default_rng(5)
    cache = cf.KV4Cache.create(2, page, heads, dim)
    k, v = _rows(rng, 2 * page, heads, dim), _rows(rng, 2 * page, heads, dim)
    cf.kv4_append(cache, torch.from_numpy(k).to(dev), torch.from_numpy(v).to(dev), torch.arange(2 * page, device=dev))
    blocks = host(cache.data)
    a, b = page * dim // 2, page * dim // 32
    value = np.concatenate([ref.LEVELS, -ref.LEVELS])
    kq, vq = ref.quantize(k), ref.quantize(v)
    for p in range(2):
        for h in range(heads):
            blk = blocks[p, h]
            kc = blk[:a].reshape(page, dim // 2)
            vc = blk[a:2 * a].reshape(page // 8, 16, 8, dim // 32)
            ks = blk[2 * a:2 * a + b].reshape(page, dim // 32)
            vs = blk[2 * a + b:].reshape(page // 8, dim // 32, 8)
            for t in range(page):
                for c in range(dim):
                    code = kc[t, c // 2] >> (4 * (c % 2)) & 15
                    x = value[code] * 2.0 ** (int(ks[t, c // 32]) - 127)
                    assert x == kq[p * page + t, h, c]
                    per = dim // 16
                    code = vc[t // 8, c // per, t % 8, c % per // 2] >> (4 * (c % 2)) & 15
                    y = value[code] * 2.0 ** (int(vs[t // 8, c // 32, t % 8]) - 127)
                    assert y == vq[p * page + t, h, c]


def test_padding_slots_and_neighbours(cf, dev):
    say("kv4 padding slots")
    heads, dim, page, pages = 2, 128, 16, 3
    guard = torch.full((pages + 2, heads, page * dim * 17 // 16), 0xA5, dtype=torch.uint8, device=dev)
    cache = cf.KV4Cache(guard[1:-1], page, dim)
    slots = torch.tensor([-1, 5, pages * page, -2 ** 62, 2 ** 62, 47], device=dev)
    x = torch.randn(6, heads, dim, device=dev)
    before = guard.clone()
    cf.kv4_append(cache, x, 2 * x, slots)
    k, v = cf.kv4_read(cache, slots, torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(guard[0], before[0]) and torch.equal(guard[-1], before[-1])
    # two rows of K and V, codes and scale bytes, for each head: nothing else changed hands
    assert int((guard != before).sum()) <= 2 * heads * 2 * (dim // 2 + dim // 32)
    for i in (0, 2, 3, 4):
        assert not k[i].any() and not v[i].any()
    want = ref.quantize(host(x))
    for i in (1, 5):
        assert np.array_equal(host(k[i]), want[i]) and np.array_equal(host(v[i]), 2 * want[i])
    cf.kv4_append(cache, x[:0], x[:0], slots[:0])
    assert cf.kv4_read(cache, slots[:0])[0].shape == (0, heads, dim)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_non_finite_groups_read_nan(cf, dev, dtype):
    say(f"kv4 NaN groups {dtype}")
    x = torch.randn(4, 1, 128, device=dev).to(DT[dtype])
    clean = x.clone()
    x[1, 0, 40], x[2, 0, 127], x[3, 0, 0] = float("nan"), float("inf"), float("-inf")
    cache = cf.KV4Cache.create(1, 16, 1, 128)
    slots = torch.arange(4, device=dev)
    cf.kv4_append(cache, x, x, slots)
    for got in cf.kv4_read(cache, slots, DT[dtype]):
        got = host(got.float())
        want = ref.quantize(clean.double().cpu().numpy())
        want[1, 0, 32:64], want[2, 0, 96:], want[3, 0, :32] = np.nan, np.nan, np.nan
        assert np.array_equal(got, want, equal_nan=True)


def test_strides_stream_and_graph(cf, dev):
    say("kv4 strides, side stream, graph")
    t, h, d = 50, 4, 64
    packed = torch.randn(t, 3 * h, d, device=dev, dtype=torch.bfloat16)
    k, v = packed[:, h:2 * h], packed[:, 2 * h:]
    slots = torch.arange(t, device=dev) + 7
    side = torch.cuda.Stream()
    cache = cf.KV4Cache.create(4, 16, h, d)
    out = torch.zeros(h, t, d, device=dev, dtype=torch.bfloat16), torch.zeros(h, t, d, device=dev, dtype=torch.bfloat16)
    ko, vo = (o.transpose(0, 1) for o in out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        cf.kv4_append(cache, k, v, slots)
        cf.kv4_read(cache, slots, k=ko, v=vo)
    for i in range(4):
        packed.copy_(torch.randn(t, 3 * h, d, device=dev))
        g.replay()
        other = cf.KV4Cache.create(4, 16, h, d)
        cf.kv4_append(other, k.transpose(0, 1).contiguous().transpose(0, 1), v, slots)
        torch.cuda.synchronize()
        assert torch.equal(other.data, cache.data), f"replay {i}"
        assert np.array_equal(host(ko.float()), ref.quantize(host(k.float())))
        assert np.array_equal(host(vo.float()), ref.quantize(host(v.float())))
    cf.kv4_append(cache, k, k, slots, stream=side)
    ks, vs = cf.kv4_read(cache, slots, stream=side)
    side.synchronize()
    assert torch.equal(ks, vs)


def test_offsets_past_32_bits(cf, dev):
    """A cache of more than 2^32 bytes: its last page is as good as its first."""
    say("kv4 cache of 4.5 GB")
    page, heads, dim = 256, 8, 128
    block = page * dim * 17 // 16 * heads
    pages = (9 << 29) // block
    cache = cf.KV4Cache(torch.empty((pages, heads, block // heads), dtype=torch.uint8, device=dev), page, dim)
    assert cache.data.numel() > 1 << 32
    x = torch.randn(40, heads, dim, device=dev, dtype=torch.bfloat16)
    slots = torch.arange(40, device=dev) * 7 + (pages - 2) * page
    cf.kv4_append(cache, x, -x, slots)
    k, v = cf.kv4_read(cache, slots)
    assert torch.equal(k, -v) and np.array_equal(host(k.float()), ref.quantize(host(x.float())))
    # attention over the last page only
    q = torch.randn(1, heads, dim, device=dev, dtype=torch.bfloat16)
    s = torch.arange(40, device=dev) + (pages - 1) * page
    cf.kv4_append(cache, x, -x, s)
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device=dev)
    out = cf.kv4_attention(q, cache, torch.tensor([40], dtype=torch.int32, device=dev), table=table)
    kk = ref.quantize(host(x.float()))
    o, _, bo, _ = ref.attention(host(q.double()), kk, -kk, 1, dim ** -0.5, False, 0)
    assert (np.abs(host(out.double()) - o) <= ref.out_bound(o, bo, 40, -kk, "bf16", heads)).all()
