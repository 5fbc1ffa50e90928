"""cf_kv4_attention where its number formats are at their ends, against 64 bits."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import attn_ref as ref
from gpu_util import host, say
from test_gpu_kv4_attention import Case

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
F32_MAX = float(np.finfo(np.float32).max)


@pytest.fixture(scope="module")
def cf():
    from activation_residual_compression_cf_amd import cf as _cf

    return _cf


@pytest.fixture(scope="module")
def dev(cf):
    return cf.require_device()


def put(cf, dev, c, i, k=None, v=None):
    """Other K or V rows for sequence i of a case."""
    if k is not None:
        c.k[i] = ref.quantize(k)
    if v is not None:
        c.v[i] = ref.quantize(v)
    d = lambda x: torch.from_numpy(x.astype(np.float32)).to(dev)
    cf.kv4_append(c.cache, d(c.k[i]), d(c.v[i]), d(c.slots[i]).long())


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("nq", [1, 20, 50])
def test_largest_fp32_queries(cf, dev, nq, dim):
    """Queries up to the largest fp32, which bf16 does not reach, over the smallest keys: scores of a few units."""
    say(f"kv4 attention of the largest fp32 queries nq={nq} dim={dim}")
    c = Case(cf, dev, [90], [nq], 2, 1, dim, "f32", seed=nq)
    put(cf, dev, c, 0, k=c.k[0] * 2.0 ** -23)
    c.q *= F32_MAX / 2 / c.q.abs().max()
    c.q[:, :, 0], c.q[:, :, dim - 1] = F32_MAX, -F32_MAX
    c.q[0, 0, 1] = 3.3961775e38  # the first that rounds to infinity in bf16
    assert c.q.isfinite().all()
    c.check(*c.run(cf, scale=2.0 ** -108), scale=2.0 ** -108)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kv,nq", [(300, 1), (9000, 1), (250, 20), (400, 60), (9000, 40)])
def test_values_at_the_ends_of_their_exponents(cf, dev, kv, nq, dim, dtype):
    """V from 2^-23, which fp16 holds as a subnormal number, to 6 * 2^13, in whole items and in split ones."""
    say(f"kv4 attention of the smallest and largest V {dtype} dim={dim} kv={kv} nq={nq}")
    rng = np.random.default_rng(5)
    for ends in ([-22, -21, 13, 0], [13, -22, -22, -21]):
        c = Case(cf, dev, [kv, 17], [nq, 1], 2, 1, dim, dtype, seed=3)
        for i in range(2):
            e = np.array(ends)[(np.arange(dim) // 32 + i) % 4]
            level = rng.choice(ref.LEVELS, (c.kv[i], 1, dim)) * rng.choice([-1, 1], (c.kv[i], 1, dim))
            put(cf, dev, c, i, v=level * 2.0 ** e)
            assert np.array_equal(c.v[i], level * 2.0 ** e)  # the least scale differs, the values do not
        out, lse = c.run(cf, max_q=nq)
        c.check(out, lse)
        assert out.any(-1).all()


class Sink:
    """`batch` sequences that share one cache, in which all of the 8 heads hold the same: key `at` takes nearly all
    of the weight and has V = 0, the others have V of about one.  Enough sequences that no workgroup's run of keys is
    much shorter than a sequence.  Row r's first key lies 8 to 32 nats above the others."""

    def __init__(self, cf, dev, length, nq, batch, dim, dtype, at=0, seed=0):
        rng = np.random.default_rng(seed)
        self.length, self.nq, self.batch, self.dim, self.dtype = length, nq, batch, dim, dtype
        page, heads = 64, 8
        pages = -(-length // page)
        self.cache = cf.KV4Cache.create(pages, page, heads, dim, device=dev)
        k, v = np.zeros((length, 1, dim), np.float32), np.ones((length, 1, dim), np.float32)
        k[at, 0, 0] = 6
        k[:, 0, 32] = rng.choice(ref.LEVELS, length)
        k[at, 0, 32] = 0
        v += rng.choice([0, 0.5, 1], (length, 1, dim)).astype(np.float32)
        v[at] = 0
        self.k, self.v = ref.quantize(k), ref.quantize(v)
        wide = lambda x: torch.from_numpy(x).to(dev).expand(length, heads, dim)
        cf.kv4_append(self.cache, wide(k), wide(v), torch.arange(length, device=dev))
        q = np.zeros((nq, heads, dim), np.float32)
        self.scale = dim ** -0.5
        q[:, :, 0] = (np.linspace(8, 32, nq * heads) / (6 * self.scale)).reshape(nq, heads)
        q[:, :, 32] = 0.05 + 0.02 * rng.random((nq, heads))
        self.q = torch.from_numpy(q).to(DT[dtype]).to(dev)
        self.many = self.q.repeat(batch, 1, 1)
        self.table = torch.arange(pages, dtype=torch.int32, device=dev).expand(batch, pages).contiguous()
        self.lens = torch.full((batch,), length, dtype=torch.int32, device=dev)

    def run(self, cf):
        lse = torch.empty(self.many.shape[:2], device=self.many.device)
        out = cf.kv4_attention(self.many, self.cache, self.lens, table=self.table, max_q=self.nq, lse=lse)
        torch.cuda.synchronize()
        shape = (self.batch, self.nq, 8)
        return host(out.double()).reshape(*shape, self.dim), host(lse.double()).reshape(shape)

    def want(self):
        """(out, lse, and their bounds without the rounding of probabilities and the last one): relative to what is
        added up to each result, which is the result, since V is not negative."""
        return ref.attention(host(self.q.double()), self.k, self.v, self.nq, self.scale, False, 0)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("length,nq,batch,at", [(16385, 1, 64, 0), (16385, 1, 64, 9001), (6001, 20, 32, 64), (4099, 40, 32, 0), (4099, 40, 32, 2050)])
def test_long_tail_below_one_key_fp32(cf, dev, dim, length, nq, batch, at):
    """Probabilities of fp32 queries are exact at any size: no term for their rounding."""
    say(f"kv4 attention fp32 tail below key {at} of {length} nq={nq} dim={dim}")
    c = Sink(cf, dev, length, nq, batch, dim, "f32", at)
    out, lse = c.run(cf)
    o, l, bo, bl = c.want()
    far = np.abs(out - o)
    bound = bo + ref.HALF_STEP["f32"] * o
    assert (far <= bound).all(), f"{(far / bound).max():.3g} of the bound, {(far / o).max():.3g} of the value"
    assert (np.abs(lse - l) <= bl).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("length,nq,batch", [(40001, 1, 128), (16385, 40, 64), (16385, 300, 16)])
def test_sums_of_many_keys(cf, dev, dtype, length, nq, batch):
    """One key of nearly all the weight and thousands of a few 2^-25 of it: added to the sum one by one, each would
    be rounded away.  A lane adds up its up to 32 probabilities of 64 keys first, so a sum has the roundings of those,
    of one addition for each 64 keys, and of joining lanes, waves and parts: under length / 64 + 100, of at most
    the sum each, and the parts' own factors are among them."""
    say(f"kv4 attention sum over {length} keys nq={nq} {dtype}")
    c = Sink(cf, dev, length, nq, batch, 64, dtype)
    _, lse = c.run(cf)
    q, k = host(c.q.double())[:, :, [0, 32]], c.k[:, 0, [0, 32]]
    s = q @ k.T * c.scale
    m = s.max(-1)
    want = m + np.log(np.exp(s - m[..., None]).sum(-1))
    # a score's two products, scaled, shifted and raised, as in attention's bound
    err = (64 + 8) * ref.F24 * 2 * np.abs(m)
    far = np.abs(lse - want)
    bound = 2 * err + (length / 64 + 100) * ref.F24
    assert (far <= bound).all(), f"{(far / bound).max():.3g} of the bound"


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("length,nq,batch,at", [(16385, 1, 64, 0), (16385, 1, 64, 9001), (6001, 20, 32, 64), (4099, 40, 32, 0), (4099, 40, 32, 2050)])
def test_long_tail_below_one_key_bf16(cf, dev, dim, length, nq, batch, at):
    """Probabilities are rounded to fp16: off by 2^-11 of the largest of their 64 keys, which for keys of the tail alone is
    at most 1.1 times their own size (their scores differ by at most 0.07 * 6 * 64 ** -0.5 nats); beside the first key by
    up to 2^-32 of that (half a subnormal's step of 2^-24, where the largest is 2^7)."""
    say(f"kv4 attention bf16 tail below key {at} of {length} nq={nq} dim={dim}")
    c = Sink(cf, dev, length, nq, batch, dim, "bf16", at)
    out, lse = c.run(cf)
    o, l, bo, bl = c.want()
    far = np.abs(out - o)
    bound = bo + 1.1 * ref.P_STEP["bf16"] * o + 64 * 2.0 ** -32 * c.v.max() + ref.HALF_STEP["bf16"] * o
    assert (far <= bound).all(), f"{(far / bound).max():.3g} of the bound, {(far / o).max():.3g} of the value"
    assert (np.abs(lse - l) <= bl).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("nq", [1, 20, 50])
def test_scores_that_rise_and_fall_by_a_lot(cf, dev, dtype, dim, nq):
    """Runs of keys whose scores lie up to 300 nats apart, rising, falling and in turn, beside the largest values:
    nothing overflows, and a result is off by no more than its own probabilities' rounding."""
    say(f"kv4 attention, scores that rise and fall {dtype} dim={dim} nq={nq}")
    rng = np.random.default_rng(nq)
    n = 1500
    for shape in ("falling", "rising", "in turn", "steps down"):
        c = Case(cf, dev, [n], [nq], 1, 1, dim, dtype, page=32, seed=nq)
        level = {"falling": 6 - np.arange(n) * 12 / n, "rising": np.arange(n) * 12 / n - 6,
                 "in turn": np.where(np.arange(n) // 100 % 2, 6, -6), "steps down": 6 - np.arange(n) // 200 * 1.5}[shape]
        k = np.zeros((n, 1, dim), np.float32)
        k[:, 0, 0] = level
        k[:, 0, 40] = rng.choice(ref.LEVELS, n)
        v = rng.standard_normal((n, 1, dim)) * 2.0 ** 13
        v[:, 0, 32:] = rng.standard_normal((n, dim - 32))
        put(cf, dev, c, 0, k=k, v=v)
        c.q[:] = 0
        c.q[:, 0, 0] = torch.linspace(0.1, 25, nq, device=dev) if nq > 1 else 25
        c.q[:, 0, 40] = 0.3
        c.check(*c.run(cf, scale=1.0, max_q=nq), scale=1.0)
        c.check(*c.run(cf, scale=1.0, max_q=nq, causal=True, window=700), scale=1.0, causal=True, window=700)
