"""Refusals of the attention operators' entry points (norms with rotation, 4-bit cache, attention over
it), as in test_abi.py: placeholder addresses that are never read, and valid calls that stop at the
device check where there is no GPU."""
import ctypes
import os

import pytest

from test_abi import (CF_E_ALIAS, CF_E_ALIGN, CF_E_ARG, CF_E_DEVICE, CF_E_NULL, CF_E_SHAPE, CF_E_WORKSPACE, CF_OK)

G = 1 << 36  # placeholder buffers this far apart


@pytest.fixture(scope="module")
def cf():
    from activation_residual_compression_cf_amd import cf as _cf

    return _cf


@pytest.fixture(scope="module")
def L(cf):
    if os.path.exists("/dev/kfd"):
        pytest.skip("valid calls with placeholder pointers would launch on a present GPU")
    return cf.lib


def P(x):
    return ctypes.c_void_p(x) if x else None


def norm(cf, dt=0, tokens=10, hq=4, hk=2, dim=64, q=(G, 256, 64), k=(2 * G, 128, 64), qo=(3 * G, 256, 64),
         ko=(4 * G, 128, 64), n=1, qw=0, qb=0, kw=0, kb=0, eps=1e-6, rope=2, cos=6 * G, sin=7 * G, n_pos=10, rot=64,
         pos=8 * G):
    r = [cf.Rows(*x) if x else None for x in (q, k, qo, ko)]
    return cf.lib.cf_qk_norm_rope(dt, tokens, hq, hk, dim, *r, n, P(qw), P(qb), P(kw), P(kb), eps, rope, P(cos), P(sin),
                                  n_pos, rot, P(pos), None)


def test_norm_rope_refusals(cf, L):
    assert norm(cf) == CF_E_DEVICE
    assert norm(cf, dt=2) == CF_E_ARG
    assert norm(cf, n=3) == CF_E_ARG and norm(cf, n=-1) == CF_E_ARG
    assert norm(cf, rope=3) == CF_E_ARG
    for eps in (-1e-6, float("nan"), float("inf")):
        assert norm(cf, eps=eps) == CF_E_ARG
    assert norm(cf, eps=0.0) == CF_E_DEVICE
    for bad in (dict(tokens=-1), dict(hq=-1), dict(hq=0, hk=0), dict(dim=0), dict(dim=12), dict(dim=264), dict(hq=65536),
                dict(tokens=1 << 40), dict(tokens=(1 << 28) + 1, hq=1, hk=0, dim=8, rope=0), dict(rot=0), dict(rot=8), dict(rot=24), dict(rot=80), dict(n_pos=0),
                dict(pos=0, n_pos=9)):
        assert norm(cf, **bad) == CF_E_SHAPE, bad
    assert norm(cf, rope=0, rot=0, n_pos=0, cos=0, sin=0, pos=0) == CF_E_DEVICE
    assert norm(cf, pos=0) == CF_E_DEVICE
    assert norm(cf, tokens=0, q=None, k=None, qo=None, ko=None) == CF_OK
    for bad in (dict(q=None), dict(q=(0, 256, 64)), dict(ko=None), dict(cos=0), dict(sin=0)):
        assert norm(cf, **bad) == CF_E_NULL, bad
    # a side without heads has no pointers
    assert norm(cf, hk=0, k=None, ko=None, kw=3) == CF_E_DEVICE
    assert norm(cf, hq=0, q=None, qo=None) == CF_E_DEVICE
    for bad in (dict(q=(G + 8, 256, 64)), dict(q=(G, 260, 64)), dict(q=(G, 256, 68)), dict(qw=5 * G + 4), dict(kb=5 * G + 8),
                dict(cos=6 * G + 4), dict(pos=8 * G + 2), dict(ko=(4 * G + 2, 128, 64))):
        assert norm(cf, **bad) == CF_E_ALIGN, bad
    # strides: inputs may repeat rows, outputs may not, none is negative
    assert norm(cf, q=(G, 0, 0)) == CF_E_DEVICE
    for bad in (dict(q=(G, -256, 64)), dict(qo=(3 * G, 192, 64)), dict(qo=(3 * G, 256, 32)), dict(qo=(3 * G, 0, 64)),
                dict(qo=(3 * G, 64, 576)), dict(q=(G, 1 << 50, 64))):
        assert norm(cf, **bad) == CF_E_SHAPE, bad
    assert norm(cf, qo=(3 * G, 64, 640)) == CF_E_DEVICE  # head-major
    assert norm(cf, tokens=1, qo=(3 * G, 0, 64), ko=(4 * G, -5, 64)) == CF_E_DEVICE  # a stride that nothing uses


def test_norm_rope_overlaps(cf, L):
    assert norm(cf, qo=(G, 256, 64), ko=(2 * G, 128, 64)) == CF_E_DEVICE  # in place
    assert norm(cf, qo=(G + 16, 256, 64)) == CF_E_ALIAS
    assert norm(cf, qo=(G, 512, 64)) == CF_E_ALIAS  # the same rows in part only
    assert norm(cf, ko=(G, 128, 64)) == CF_E_ALIAS
    assert norm(cf, ko=(3 * G, 128, 64)) == CF_E_ALIAS
    # q, k and v side by side in one buffer, 8 heads a token, in place
    packed = dict(q=(G, 512, 64), k=(G + 4 * 128, 512, 64))
    assert norm(cf, **packed, qo=packed["q"], ko=packed["k"]) == CF_E_DEVICE
    assert norm(cf, **packed) == CF_E_DEVICE
    assert norm(cf, **packed, qo=(G + 2 * 128, 512, 64)) == CF_E_ALIAS
    assert norm(cf, **packed, qo=packed["q"], ko=(G + 6 * 128, 512, 64)) == CF_E_DEVICE  # into v's place
    assert norm(cf, **packed, qo=packed["q"], ko=(G + 7 * 128, 512, 64)) == CF_E_ALIAS   # one head into the next token's q
    for name in ("qw", "kb", "cos", "sin", "pos"):
        assert norm(cf, **{name: 3 * G + 64}) == CF_E_ALIAS, name
    assert norm(cf, hk=0, k=None, ko=None, kw=3 * G) == CF_E_DEVICE  # not read
    assert norm(cf, qw=5 * G, qb=5 * G) == CF_E_DEVICE               # inputs may share


def test_cache_bytes(cf):
    f = cf.lib.cf_kv4_cache_bytes
    assert f(1, 16, 1, 64) == 16 * 64 * 17 // 16
    assert f(100, 256, 8, 128) == 100 * 8 * 256 * 136
    for bad in ((0, 16, 1, 64), (-1, 16, 1, 64), (1, 8, 1, 64), (1, 24, 1, 64), (1, 512, 1, 64), (1, 16, 0, 64),
                (1, 16, 65536, 64), (1, 16, 1, 96), (1, 16, 1, 256), (1 << 50, 16, 8, 128), (1 << 31, 16, 1, 64)):
        assert f(*bad) == CF_E_SHAPE, bad


def rows_call(cf, read, dt=0, k=(G, 512, 64), v=(2 * G, 512, 64), slots=3 * G, tokens=10, cache=4 * G, pages=8, page=16,
              heads=8, dim=64):
    k, v = (cf.Rows(*x) if x else None for x in (k, v))
    if read:
        return cf.lib.cf_kv4_read(dt, P(cache), pages, page, heads, dim, P(slots), tokens, k, v, None)
    return cf.lib.cf_kv4_append(dt, k, v, P(slots), tokens, P(cache), pages, page, heads, dim, None)


@pytest.mark.parametrize("read", [False, True])
def test_append_and_read_refusals(cf, L, read):
    call = lambda **kw: rows_call(cf, read, **kw)
    assert call() == CF_E_DEVICE
    assert call(dt=7) == CF_E_ARG
    for bad in (dict(pages=0), dict(page=20), dict(heads=0), dict(dim=32), dict(tokens=-1), dict(tokens=1 << 40),
                dict(k=(G, -512, 64)), dict(v=(2 * G, 512, -64))):
        assert call(**bad) == CF_E_SHAPE, bad
    assert call(tokens=0, k=None, v=None, cache=0, slots=0) == CF_OK
    for bad in (dict(k=None), dict(v=(0, 512, 64)), dict(slots=0), dict(cache=0)):
        assert call(**bad) == CF_E_NULL, bad
    for bad in (dict(k=(G + 8, 512, 64)), dict(v=(2 * G, 516, 64)), dict(slots=3 * G + 4), dict(cache=4 * G + 8)):
        assert call(**bad) == CF_E_ALIGN, bad
    size = 8 * 8 * 16 * 64 * 17 // 16
    for bad in (dict(k=(4 * G + size - 16, 512, 64)), dict(v=(4 * G, 512, 64))):
        assert call(**bad) == CF_E_ALIAS, bad
    assert call(k=(4 * G + size, 512, 64)) == CF_E_DEVICE
    # repeated rows and one buffer for both: fine to read from, not to write to
    assert call(k=(G, 0, 0)) == (CF_E_SHAPE if read else CF_E_DEVICE)
    assert call(v=(G, 512, 64)) == (CF_E_ALIAS if read else CF_E_DEVICE)
    assert call(slots=4 * G + 64) == (CF_E_DEVICE if read else CF_E_ALIAS)
    assert call(slots=G + 64) == (CF_E_ALIAS if read else CF_E_DEVICE)


def attn(cf, dt=0, q=(G, 512, 64), total=12, hq=8, cache=2 * G, pages=50, page=16, hk=2, dim=64, batch=3, table=3 * G, width=5,
         lens=4 * G, starts=5 * G, max_q=4, flags=0, window=0, scale=0.125, out=(6 * G, 512, 64), lse=7 * G, ws=8 * G,
         ws_bytes=None):
    if ws_bytes is None:
        ws_bytes = 1 << 33
    q, out = (cf.Rows(*x) if x else None for x in (q, out))
    return cf.lib.cf_kv4_attention(dt, q, total, hq, P(cache), pages, page, hk, dim, batch, P(table), width, P(lens),
                                   P(starts), max_q, flags, window, scale, out, P(lse), P(ws), ws_bytes, None)


def test_attention_refusals(cf, L):
    assert attn(cf) == CF_E_DEVICE
    assert attn(cf, flags=1, window=7) == CF_E_DEVICE
    for bad in (dict(dt=2), dict(flags=2), dict(window=-1, flags=1), dict(window=5), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=2e38)):
        assert attn(cf, **bad) == CF_E_ARG, bad
    for bad in (dict(pages=0), dict(page=17), dict(hk=3), dict(hq=0), dict(hq=9), dict(dim=80), dict(total=-1),
                dict(total=1 << 30), dict(max_q=13), dict(max_q=-1), dict(batch=0), dict(width=0), dict(width=1 << 27),
                dict(table=0, width=17), dict(starts=0, batch=5), dict(out=(6 * G, 448, 64)), dict(out=(6 * G, 0, 64)),
                dict(q=(G, -512, 64))):
        assert attn(cf, **bad) == CF_E_SHAPE, bad
    assert attn(cf, table=0, width=16) == CF_E_DEVICE
    assert attn(cf, starts=0, batch=4) == CF_E_DEVICE
    assert attn(cf, lse=0) == CF_E_DEVICE
    assert attn(cf, max_q=0) == CF_E_DEVICE
    assert attn(cf, total=0, q=None, out=None, max_q=0, batch=0, ws=0, ws_bytes=0) == CF_OK
    for bad in (dict(q=None), dict(out=None), dict(cache=0), dict(lens=0), dict(ws=0), dict(out=(0, 512, 64))):
        assert attn(cf, **bad) == CF_E_NULL, bad
    for bad in (dict(q=(G + 2, 512, 64)), dict(out=(6 * G, 1024, 66)), dict(cache=2 * G + 4), dict(table=3 * G + 2),
                dict(lens=4 * G + 1), dict(starts=5 * G + 2), dict(lse=7 * G + 2), dict(ws=8 * G + 128)):
        assert attn(cf, **bad) == CF_E_ALIGN, bad
    need = cf.lib.cf_kv4_attention_workspace_bytes(0, 4, 8, 2, 64)
    assert need > 0
    assert attn(cf, ws_bytes=need) == CF_E_DEVICE
    assert attn(cf, ws_bytes=need - 1) == CF_E_WORKSPACE
    for bad in (dict(out=(G, 512, 64)), dict(out=(2 * G, 512, 64)), dict(out=(3 * G + 16, 512, 64)), dict(lse=G),
                dict(lse=4 * G), dict(lse=6 * G + 512), dict(ws=G), dict(ws=2 * G), dict(ws=5 * G), dict(ws=7 * G)):
        assert attn(cf, **bad) == CF_E_ALIAS, bad
    # queries and results side by side in one buffer
    assert attn(cf, q=(G, 1024, 64), out=(G + 1024, 1024, 64)) == CF_E_DEVICE
    assert attn(cf, q=(G, 1024, 64), out=(G + 896, 1024, 64)) == CF_E_ALIAS


def test_workspace_bytes(cf):
    f = cf.lib.cf_kv4_attention_workspace_bytes
    for bad in ((3, 1, 8, 2, 64), (0, 0, 8, 2, 64), (0, 1, 8, 3, 64), (0, 1, 0, 1, 64), (0, 1, 8, 0, 64), (0, 1, 8, 2, 32),
                (0, 1 << 31, 8, 2, 64)):
        assert f(*bad) == 0, bad
    for dt in (0, 1):
        for dim in (64, 128):
            sizes = [f(dt, n, 8, 2, dim) for n in (1, 4, 5, 8, 9, 100, 5000)]
            assert all(sizes) and max(sizes) < 1 << 29


def test_binding_refuses(cf):
    """What the C ABI cannot see: element types, shapes, host tensors."""
    import torch

    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensors"):
        cf.qk_norm_rope(x, x, q_out=x.clone(), k_out=x.clone())
    with pytest.raises(ValueError):
        cf.qk_norm_rope(None, None)
    with pytest.raises(ValueError):
        cf.qk_norm_rope(x[0], None)
    with pytest.raises(TypeError, match="activation dtype"):
        cf.qk_norm_rope(x.half(), x.half())
    with pytest.raises(TypeError, match="k is"):
        cf.qk_norm_rope(x, x.float())
    with pytest.raises(ValueError, match="k is"):
        cf.qk_norm_rope(x, x[:3])
    with pytest.raises(ValueError, match="q_out is"):
        cf.qk_norm_rope(x, None, q_out=x[:, :1])
    cache = cf.KV4Cache(torch.zeros(2, 2, 16 * 68, dtype=torch.uint8), 16, 64)
    slots = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="device tensors"):
        cf.kv4_append(cache, x, x, slots)
    with pytest.raises(TypeError, match="slots"):
        cf.kv4_append(cache, x, x, slots.int())
    with pytest.raises(ValueError, match="slots"):
        cf.kv4_append(cache, x, x, slots[:3])
    with pytest.raises(ValueError, match="v is"):
        cf.kv4_append(cache, x, x[:, :1], slots)
    with pytest.raises(ValueError, match="cache data"):
        cf.KV4Cache(cache.data, 32, 64)._args(-2)
    with pytest.raises(TypeError, match="cache"):
        cf.KV4Cache(cache.data.to(torch.int8), 16, 64)._args(-2)
    lens = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError, match="kv_lens"):
        cf.kv4_attention(x, cache, lens.long())
    with pytest.raises(ValueError, match="table"):
        cf.kv4_attention(x, cache, lens, table=torch.zeros(2, 3, dtype=torch.int32))
    with pytest.raises(ValueError, match="q_starts"):
        cf.kv4_attention(x, cache, lens, q_starts=lens)
    with pytest.raises(ValueError, match="rows of"):
        cf.kv4_attention(torch.zeros(4, 2, 128, dtype=torch.bfloat16), cache, lens)
    with pytest.raises(TypeError, match="lse"):
        cf.kv4_attention(x, cache, lens, lse=torch.zeros(4, 2, dtype=torch.float64), out=x.clone(), workspace=slots)
    with pytest.raises(cf.CFError):
        cf.kv4_attention_workspace_bytes(torch.float16, 1, 8, 2, 64)
    with pytest.raises(cf.CFError):
        cf.KV4Cache.create(1, 17, 1, 64, device="cpu")
