"""cf_qk_norm_rope against its formulas in 64 bits: every norm and rotation, head layouts and strides,
one token to many, partial rotations, in place, padding and positions behind the table, streams and
graphs."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import attn_ref as ref
from gpu_util import host, say

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CANARY = 77.0


@pytest.fixture(scope="module")
def cf():
    from activation_residual_compression_cf_amd import cf as _cf

    return _cf


@pytest.fixture(scope="module")
def dev(cf):
    return cf.require_device()


def _consts(cf, norm, rope):
    return ({"none": cf.CF_NORM_NONE, "rms": cf.CF_NORM_RMS, "layer": cf.CF_NORM_LAYER}[norm],
            {"none": cf.CF_ROPE_NONE, "interleaved": cf.CF_ROPE_INTERLEAVED, "half": cf.CF_ROPE_HALF}[rope])


def _tables(n_pos, rot):
    a = np.arange(n_pos)[:, None] * 100.0 ** (-np.arange(rot // 2) / max(rot // 2, 1))
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def _params(rng, dim):
    return [(1 + 0.3 * rng.standard_normal(dim)).astype(np.float32) for _ in range(2)], \
        [(0.5 * rng.standard_normal(dim)).astype(np.float32) for _ in range(2)]


def _close(got, x, dtype, args):
    y, size = ref.norm_rope(x, *args)
    far = np.abs(host(got.float()).astype(np.float64) - y)
    assert (far <= ref.norm_rope_bound(y, size, dtype)).all(), float((far / (size + 1e-30)).max())


@pytest.mark.parametrize("norm", ["none", "rms", "layer"])
@pytest.mark.parametrize("rope", ["none", "interleaved", "half"])
@pytest.mark.parametrize("tokens,hq,hk,dim,rot,dtype", [
    (1, 32, 8, 128, 128, "bf16"), (1, 1, 1, 64, 64, "f32"), (37, 5, 1, 64, 32, "bf16"), (300, 24, 24, 128, 64, "f32"),
    (3, 2, 3, 8, None, "f32"), (65, 7, 2, 80, 48, "bf16"), (9, 3, 1, 256, 256, "bf16"), (2049, 30, 30, 64, 64, "bf16"),
    (11, 1, 4, 200, 192, "f32")])
def test_matches_formula(cf, dev, norm, rope, tokens, hq, hk, dim, rot, dtype):
    if rot is None:
        if rope != "none":
            pytest.skip("no rotation fits 8 channels")
        rot = 0
    say(f"norm_rope {norm} {rope} tokens={tokens} heads={hq}+{hk} dim={dim} rot={rot} {dtype}")
    rng = np.random.default_rng(tokens + dim)
    n, r = _consts(cf, norm, rope)
    g = torch.Generator().manual_seed(dim + tokens)
    q = (torch.randn(tokens, hq, dim, generator=g) * 3 + 0.5).to(DT[dtype])
    k = (torch.randn(tokens, hk, dim, generator=g) * 0.01).to(DT[dtype])
    (qw, kw), (qb, kb) = _params(rng, dim)
    cos, sin = _tables(500, rot)
    pos = rng.integers(0, 500, tokens).astype(np.int32)
    d = lambda x: torch.from_numpy(x).to(dev)
    use_b = norm == "layer" or tokens == 37
    qo, ko = cf.qk_norm_rope(q.to(dev), k.to(dev), norm=n, q_weight=d(qw), k_weight=None if tokens == 9 else d(kw),
                             q_bias=d(qb) if use_b else None, k_bias=d(kb) if use_b else None, eps=1e-6, rope=r,
                             cos=d(cos), sin=d(sin), positions=d(pos))
    torch.cuda.synchronize()
    for got, x, w, b in ((qo, q, qw, qb), (ko, k, None if tokens == 9 else kw, kb)):
        _close(got, x.double().numpy(), dtype, (norm, w, b if use_b else None, 1e-6, rope, cos[pos], sin[pos], rot))


@pytest.mark.parametrize("layout", ["packed", "packed_in_place", "head_major", "broadcast"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layouts(cf, dev, layout, dtype):
    tokens, hq, hk, dim = 33, 6, 2, 64
    say(f"norm_rope layout={layout} {dtype}")
    cos, sin = _tables(tokens, dim)
    x = (torch.randn(tokens, hq + 2 * hk, dim, generator=torch.Generator().manual_seed(3))).to(DT[dtype]).to(dev)
    before = x.clone()
    q, k = x[:, :hq], x[:, hq:hq + hk]
    kw = dict(norm=cf.CF_NORM_RMS, rope=cf.CF_ROPE_HALF, cos=torch.from_numpy(cos).to(dev), sin=torch.from_numpy(sin).to(dev))
    qx, kx = q.double().cpu().numpy(), k.double().cpu().numpy()
    if layout == "packed":
        qo, ko = cf.qk_norm_rope(q, k, **kw)
        assert torch.equal(x, before)
    elif layout == "packed_in_place":
        qo, ko = cf.qk_norm_rope(q, k, q_out=q, k_out=k, **kw)
        assert torch.equal(x[:, hq + hk:], before[:, hq + hk:])
    elif layout == "head_major":
        qo = torch.full((hq, tokens + 1, dim), CANARY, dtype=DT[dtype], device=dev)
        ko = torch.full((hk, tokens + 1, dim), CANARY, dtype=DT[dtype], device=dev)
        a, b = qo[:, :tokens].transpose(0, 1), ko[:, :tokens].transpose(0, 1)
        cf.qk_norm_rope(q.transpose(0, 1).contiguous().transpose(0, 1), k, q_out=a, k_out=b, **kw)
        assert (qo[:, tokens] == CANARY).all() and (ko[:, tokens] == CANARY).all()
        qo, ko = a, b
    else:  # one head's row for all of them
        q = q[:, :1].expand(tokens, hq, dim)
        qx = q.double().cpu().numpy()
        qo, ko = cf.qk_norm_rope(q, k, **kw)
    torch.cuda.synchronize()
    for got, v in ((qo, qx), (ko, kx)):
        _close(got, v, dtype, ("rms", None, None, 1e-6, "half", cos, sin, dim))


def test_one_side_only_and_no_tokens(cf, dev):
    say("norm_rope q only, k only, no tokens")
    x = torch.randn(5, 3, 64, device=dev)
    both = cf.qk_norm_rope(x, x)
    q, none = cf.qk_norm_rope(x, None)
    assert none is None and torch.equal(q, both[0])
    none, k = cf.qk_norm_rope(None, x)
    assert none is None and torch.equal(k, both[1])
    q, k = cf.qk_norm_rope(x[:0], x[:0])
    assert q.shape == (0, 3, 64) and k.shape == (0, 3, 64)


def test_padding_and_positions_behind_the_table(cf, dev):
    say("norm_rope padding")
    x = torch.randn(6, 4, 128, device=dev, dtype=torch.bfloat16)
    cos, sin = (torch.from_numpy(t).to(dev) for t in _tables(10, 128))
    pos = torch.tensor([0, -1, 9, 10, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=dev)
    out = torch.full_like(x, CANARY)
    cf.qk_norm_rope(x, None, rope=cf.CF_ROPE_HALF, cos=cos, sin=sin, positions=pos, q_out=out)
    torch.cuda.synchronize()
    assert (out[[1, 5]] == CANARY).all() and out[[3, 4]].isnan().all()
    p = pos.cpu().numpy()[[0, 2]]
    c, s = _tables(10, 128)
    _close(out[[0, 2]], x[[0, 2]].double().cpu().numpy(), "bf16", ("rms", None, None, 1e-6, "half", c[p], s[p], 128))


def test_nan_and_infinity_stay_in_their_row(cf, dev):
    say("norm_rope NaN rows")
    x = torch.randn(4, 5, 64, device=dev)
    y0, _ = cf.qk_norm_rope(x, None)
    x[1, 2, 7], x[2, 0, 0] = float("nan"), float("inf")
    y, _ = cf.qk_norm_rope(x, None)
    assert y[1, 2].isnan().all() and y[2, 0, 0].isnan()
    y[1, 2] = y0[1, 2]
    y[2, 0] = y0[2, 0]
    assert torch.equal(y, y0)
    z = torch.zeros(2, 1, 64, device=dev, dtype=torch.bfloat16)
    assert (cf.qk_norm_rope(z, None, norm=cf.CF_NORM_LAYER)[0] == 0).all()


def test_bf16_nan_payloads_stay_nan(cf, dev):
    say("norm_rope bf16 NaN payloads")
    x = torch.full((1, 1, 64), 0x7FFF, dtype=torch.int16, device=dev).view(torch.bfloat16)
    assert cf.qk_norm_rope(x, None, norm=cf.CF_NORM_NONE)[0].isnan().all()


def test_other_stream_and_graph(cf, dev):
    say("norm_rope on a side stream, and captured")
    x = torch.randn(70, 12, 128, device=dev, dtype=torch.bfloat16)
    q, k = x[:, :8], x[:, 8:]
    cos, sin = (torch.from_numpy(t).to(dev) for t in _tables(70, 128))
    kw = dict(rope=cf.CF_ROPE_INTERLEAVED, cos=cos, sin=sin)
    want = cf.qk_norm_rope(q, k, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = cf.qk_norm_rope(q, k, stream=side, **kw)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    qo, ko = torch.empty(70, 8, 128, dtype=x.dtype, device=dev), torch.empty(70, 4, 128, dtype=x.dtype, device=dev)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        cf.qk_norm_rope(q, k, q_out=qo, k_out=ko, **kw)
    for i in range(4):
        x.copy_(torch.randn(70, 12, 128, device=dev))
        g.replay()
        want = cf.qk_norm_rope(q, k, **kw)
        torch.cuda.synchronize()
        assert torch.equal(qo, want[0]) and torch.equal(ko, want[1]), f"replay {i}"
