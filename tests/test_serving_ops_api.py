"""Refusals of the serving operators' entry points (8-bit cache and attention over it, attention over prompts,
operations on pages): placeholder addresses that are never read, and valid calls that stop at the device check where there
is no GPU."""
import ctypes
import os

import pytest

from test_abi import CF_E_ALIAS, CF_E_ALIGN, CF_E_ARG, CF_E_DEVICE, CF_E_NULL, CF_E_SHAPE, CF_E_WORKSPACE, CF_OK

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


def test_cache_bytes(cf):
    f = cf.lib.cf_kv8_cache_bytes
    assert f(1, 16, 1, 64) == 2 * 16 * 64 + 16
    assert f(100, 128, 8, 128) == 100 * 8 * (2 * 128 * 128 + 16)
    assert f(100, 256, 8, 128) == 100 * 8 * (2 * 256 * 128 + 32)
    for bad in ((0, 16, 1, 64), (-1, 16, 1, 64), (1, 8, 1, 64), (1, 24, 1, 64), (1, 512, 1, 64), (1, 16, 0, 64),
                (1, 16, 65536, 64), (1, 16, 1, 96), (1, 16, 1, 256), (1 << 50, 16, 8, 128), (1 << 31, 16, 1, 64)):
        assert f(*bad) == CF_E_SHAPE, bad


def append(cf, dt=0, k=(G, 512, 64), v=(2 * G, 512, 64), tokens=10, cache=3 * G, pages=50, page=16, heads=8, dim=64, batch=3,
           table=4 * G, width=5, lens=5 * G, starts=6 * G):
    k, v = (cf.Rows(*x) if x else None for x in (k, v))
    return cf.lib.cf_kv8_append(dt, k, v, tokens, P(cache), pages, page, heads, dim, batch, P(table), width, P(lens), P(starts), None)


def test_append_refusals(cf, L):
    assert append(cf) == CF_E_DEVICE
    assert append(cf, dt=7) == CF_E_ARG
    for bad in (dict(pages=0), dict(page=20), dict(heads=0), dict(dim=32), dict(tokens=-1), dict(tokens=(1 << 27) + 1, heads=1), dict(k=(G, -512, 64)),
                dict(v=(2 * G, 512, -64)), dict(batch=0), dict(batch=(1 << 24) + 1), dict(width=0), dict(width=1 << 27),
                dict(table=0, width=17), dict(starts=0)):
        assert append(cf, **bad) == CF_E_SHAPE, bad
    assert append(cf, table=0, width=16) == CF_E_DEVICE
    assert append(cf, starts=0, tokens=9) == CF_E_DEVICE
    assert append(cf, tokens=0, k=None, v=None, cache=0, lens=0, batch=0) == CF_OK
    for bad in (dict(k=None), dict(v=(0, 512, 64)), dict(lens=0), dict(cache=0)):
        assert append(cf, **bad) == CF_E_NULL, bad
    for bad in (dict(k=(G + 8, 512, 64)), dict(v=(2 * G, 516, 64)), dict(cache=3 * G + 8), dict(table=4 * G + 2), dict(lens=5 * G + 1), dict(starts=6 * G + 2)):
        assert append(cf, **bad) == CF_E_ALIGN, bad
    size = 50 * 8 * (2 * 16 * 64 + 16)
    for bad in (dict(k=(3 * G + size - 16, 512, 64)), dict(v=(3 * G, 512, 64)), dict(table=3 * G), dict(lens=3 * G + 64), dict(starts=3 * G + size - 4)):
        assert append(cf, **bad) == CF_E_ALIAS, bad
    assert append(cf, k=(3 * G + size, 512, 64)) == CF_E_DEVICE
    assert append(cf, k=(G, 0, 0), v=(G, 512, 64)) == CF_E_DEVICE  # repeated rows and one buffer for both


def read(cf, dt=0, k=(G, 512, 64), v=(2 * G, 512, 64), slots=3 * G, tokens=10, cache=4 * G, pages=8, page=16, heads=8, dim=64):
    k, v = (cf.Rows(*x) if x else None for x in (k, v))
    return cf.lib.cf_kv8_read(dt, P(cache), pages, page, heads, dim, P(slots), tokens, k, v, None)


def test_read_refusals(cf, L):
    assert read(cf) == CF_E_DEVICE and read(cf, dt=7) == CF_E_ARG
    for bad in (dict(pages=0), dict(page=20), dict(tokens=-1), dict(tokens=1 << 40), dict(k=(G, 0, 0)), dict(v=(2 * G, 512, -64))):
        assert read(cf, **bad) == CF_E_SHAPE, bad
    assert read(cf, tokens=0, k=None, v=None, cache=0, slots=0) == CF_OK
    for bad in (dict(k=None), dict(slots=0), dict(cache=0)):
        assert read(cf, **bad) == CF_E_NULL, bad
    for bad in (dict(k=(G + 8, 512, 64)), dict(slots=3 * G + 4), dict(cache=4 * G + 8)):
        assert read(cf, **bad) == CF_E_ALIGN, bad
    size = 8 * 8 * (2 * 16 * 64 + 16)
    for bad in (dict(k=(4 * G + size - 16, 512, 64)), dict(v=(G, 512, 64)), dict(slots=G + 64)):
        assert read(cf, **bad) == CF_E_ALIAS, bad


def attn8(cf, dt=0, q=(G, 512, 64), total=12, hq=8, cache=2 * G, pages=50, page=16, hk=2, dim=64, batch=3, table=3 * G, width=5,
          lens=4 * G, starts=5 * G, max_q=4, flags=0, window=0, scale=0.125, out=(6 * G, 512, 64), lse=7 * G, ws=8 * G, ws_bytes=1 << 33):
    q, out = (cf.Rows(*x) if x else None for x in (q, out))
    return cf.lib.cf_kv8_attention(dt, q, total, hq, P(cache), pages, page, hk, dim, batch, P(table), width, P(lens),
                                   P(starts), max_q, flags, window, scale, out, P(lse), P(ws), ws_bytes, None)


def test_kv8_attention_refusals(cf, L):
    assert attn8(cf) == CF_E_DEVICE and attn8(cf, flags=1, window=7) == CF_E_DEVICE
    for bad in (dict(dt=2), dict(flags=2), dict(window=-1, flags=1), dict(window=5), dict(scale=0.0), dict(scale=float("nan")), dict(scale=2e38)):
        assert attn8(cf, **bad) == CF_E_ARG, bad
    for bad in (dict(pages=0), dict(page=17), dict(hk=3), dict(hq=0), dict(dim=80), dict(total=-1), dict(total=1 << 30), dict(max_q=13),
                dict(batch=0), dict(width=0), dict(table=0, width=17), dict(starts=0, batch=5), dict(out=(6 * G, 448, 64))):
        assert attn8(cf, **bad) == CF_E_SHAPE, bad
    assert attn8(cf, total=0, q=None, out=None, max_q=9, batch=0, ws=0, ws_bytes=0) == CF_OK
    for bad in (dict(q=None), dict(out=None), dict(cache=0), dict(lens=0), dict(ws=0)):
        assert attn8(cf, **bad) == CF_E_NULL, bad
    for bad in (dict(q=(G + 2, 512, 64)), dict(cache=2 * G + 4), dict(table=3 * G + 2), dict(lse=7 * G + 2), dict(ws=8 * G + 128)):
        assert attn8(cf, **bad) == CF_E_ALIGN, bad
    need = cf.lib.cf_kv8_attention_workspace_bytes(0, 4, 8, 2, 64)
    assert need > 0 and attn8(cf, ws_bytes=need) == CF_E_DEVICE and attn8(cf, ws_bytes=need - 1) == CF_E_WORKSPACE
    # the last byte of a cache is the cache's
    size = 50 * 2 * (2 * 16 * 64 + 16)
    for bad in (dict(out=(G, 512, 64)), dict(out=(2 * G + size - 16, 512, 64)), dict(lse=4 * G), dict(ws=2 * G), dict(ws=7 * G)):
        assert attn8(cf, **bad) == CF_E_ALIAS, bad
    assert attn8(cf, out=(2 * G + size, 512, 64)) == CF_E_DEVICE


def attn(cf, dt=0, q=(G, 512, 64), total=12, hq=8, k=(2 * G, 128, 64), v=(3 * G, 128, 64), keys=30, hk=2, dim=64, batch=3, qs=4 * G,
         ks=5 * G, max_q=4, flags=0, window=0, scale=0.125, out=(6 * G, 512, 64), lse=7 * G, ws=8 * G, ws_bytes=1 << 33):
    q, k, v, out = (cf.Rows(*x) if x else None for x in (q, k, v, out))
    return cf.lib.cf_attention(dt, q, total, hq, k, v, keys, hk, dim, batch, P(qs), P(ks), max_q, flags, window, scale, out, P(lse),
                               P(ws), ws_bytes, None)


def test_attention_refusals(cf, L):
    assert attn(cf) == CF_E_DEVICE and attn(cf, flags=1, window=7) == CF_E_DEVICE
    for bad in (dict(dt=2), dict(flags=2), dict(window=-1, flags=1), dict(window=5), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf"))):
        assert attn(cf, **bad) == CF_E_ARG, bad
    for bad in (dict(hk=3), dict(hq=0), dict(hk=0), dict(dim=80), dict(total=-1), dict(total=1 << 30), dict(keys=-1), dict(keys=(1 << 31) - 255),
                dict(max_q=13), dict(max_q=-1), dict(batch=0), dict(batch=(1 << 24) + 1), dict(qs=0, batch=5), dict(ks=0, batch=4),
                dict(out=(6 * G, 448, 64)), dict(q=(G, -512, 64)), dict(k=(2 * G, (1 << 25) + 8, 64)), dict(v=(3 * G, 1 << 26, 64)),
                dict(dt=1, k=(2 * G, (1 << 24) + 4, 64))):
        assert attn(cf, **bad) == CF_E_SHAPE, bad
    for good in (dict(qs=0), dict(ks=0), dict(lse=0), dict(max_q=0), dict(k=(2 * G, 1 << 25, 64)), dict(keys=1, ks=0, batch=1, k=(2 * G, 1 << 40, 64)),
                 dict(k=(2 * G, 0, 0)), dict(v=(2 * G, 128, 64)), dict(keys=0, k=None, v=None)):
        assert attn(cf, **good) == CF_E_DEVICE, good
    assert attn(cf, total=0, q=None, k=None, v=None, out=None, max_q=0, batch=0, ws=0, ws_bytes=0) == CF_OK
    for bad in (dict(q=None), dict(k=None), dict(v=(0, 128, 64)), dict(out=None), dict(ws=0)):
        assert attn(cf, **bad) == CF_E_NULL, bad
    for bad in (dict(q=(G + 2, 512, 64)), dict(k=(2 * G, 132, 64)), dict(v=(3 * G, 128, 66)), dict(out=(6 * G + 8, 512, 64)), dict(qs=4 * G + 2),
                dict(ks=5 * G + 1), dict(lse=7 * G + 2), dict(ws=8 * G + 128)):
        assert attn(cf, **bad) == CF_E_ALIGN, bad
    need = cf.lib.cf_attention_workspace_bytes(0, 4, 8, 2, 64)
    assert need > 0 and attn(cf, ws_bytes=need) == CF_E_DEVICE and attn(cf, ws_bytes=need - 1) == CF_E_WORKSPACE
    for bad in (dict(out=(G, 512, 64)), dict(out=(2 * G, 512, 64)), dict(out=(3 * G + 128, 512, 64)), dict(out=(4 * G, 512, 64)), dict(lse=G),
                dict(lse=2 * G + 64), dict(lse=6 * G + 512), dict(ws=3 * G), dict(ws=5 * G), dict(ws=7 * G), dict(lse=5 * G)):
        assert attn(cf, **bad) == CF_E_ALIAS, bad
    # q, k, v and results side by side in one buffer
    p = dict(q=(G, 1280, 64), k=(G + 1024, 1280, 64), v=(G + 1280, 1280, 64), keys=12)
    assert attn(cf, **p, out=(G + 1536, 1280, 64)) == CF_E_DEVICE
    assert attn(cf, **p, out=(G + 1408, 1280, 64)) == CF_E_ALIAS


def test_workspace_bytes(cf):
    for f in (cf.lib.cf_kv8_attention_workspace_bytes, cf.lib.cf_attention_workspace_bytes):
        for bad in ((3, 1, 8, 2, 64), (0, 0, 8, 2, 64), (0, 1, 8, 3, 64), (0, 1, 0, 1, 64), (0, 1, 8, 0, 64), (0, 1, 8, 2, 32), (0, 1 << 31, 8, 2, 64)):
            assert f(*bad) == 0, bad
        for dt in (0, 1):
            for dim in (64, 128):
                sizes = [f(dt, n, 8, 2, dim) for n in (1, 4, 5, 8, 9, 32, 33, 64, 65, 100, 5000)]
                assert all(sizes) and max(sizes) < 1 << 29 and sizes == sorted(sizes)
    f = cf.lib.cf_pages_workspace_bytes
    for bad in ((0, 1), (1 << 31, 1), (1, 0), (1, (1 << 20) + 1), (-1, 1)):
        assert f(*bad) == 0, bad
    assert f(100, 10) >= 4 * 121


def pages(cf, op, a=(G, 2 * G, 3 * G), b=(4 * G, 5 * G, 6 * G), n=100, rows=10, width=8, page=16, want=7 * G, src=8 * G, dst=9 * G, count=10 * G,
          ws=11 * G, ws_bytes=1 << 30):
    a, b = (cf.Pages(*x) if x else None for x in (a, b))
    if op == "resize":
        return cf.lib.cf_pages_resize(a, b, n, rows, width, page, P(want), P(count), P(ws), ws_bytes, None)
    if op == "fork":
        return cf.lib.cf_pages_fork(a, b, n, rows, width, page, P(want), P(src), P(dst), P(count), P(ws), ws_bytes, None)
    return cf.lib.cf_pages_compact(a, b, n, rows, width, P(src), P(dst), P(count), P(ws), ws_bytes, None)


@pytest.mark.parametrize("op", ["resize", "fork", "compact"])
def test_pages_refusals(cf, L, op):
    call = lambda **kw: pages(cf, op, **kw)
    assert call() == CF_E_DEVICE
    for bad in (dict(n=0), dict(n=1 << 31), dict(rows=0), dict(rows=(1 << 20) + 1), dict(width=0), dict(rows=1 << 20, width=1025)):
        assert call(**bad) == CF_E_SHAPE, bad
    if op != "compact":
        for bad in (dict(page=0), dict(page=-1), dict(page=1 << 29)):
            assert call(**bad) == CF_E_SHAPE, bad
        assert call(want=0) == CF_E_NULL
    for bad in (dict(a=None), dict(b=None), dict(a=(0, 2 * G, 3 * G)), dict(b=(4 * G, 5 * G, 0)), dict(count=0), dict(ws=0)):
        assert call(**bad) == CF_E_NULL, bad
    for bad in (dict(a=(G + 2, 2 * G, 3 * G)), dict(b=(4 * G, 5 * G + 1, 6 * G)), dict(count=10 * G + 2), dict(ws=11 * G + 2)):
        assert call(**bad) == CF_E_ALIGN, bad
    need = cf.lib.cf_pages_workspace_bytes(100, 10)
    assert call(ws_bytes=need) == CF_E_DEVICE and call(ws_bytes=need - 1) == CF_E_WORKSPACE
    same = CF_E_ALIAS if op == "fork" else CF_E_DEVICE
    assert call(b=(G, 2 * G, 3 * G)) == same and call(b=(4 * G, 2 * G, 6 * G)) == same and call(b=(G, 5 * G, 6 * G)) == CF_E_DEVICE
    for bad in (dict(b=(G + 4, 5 * G, 6 * G)), dict(b=(4 * G, 3 * G, 6 * G)), dict(b=(4 * G, 4 * G, 6 * G)), dict(count=G), dict(count=5 * G),
                dict(ws=2 * G), dict(ws=6 * G + 36), dict(ws=10 * G)):
        assert call(**bad) == CF_E_ALIAS, bad
    if op != "compact":
        assert call(b=(4 * G, 5 * G, 7 * G)) == CF_E_ALIAS
    if op != "resize":
        assert call(src=0) == CF_E_NULL and call(dst=8 * G) == CF_E_ALIAS and call(src=2 * G) == CF_E_ALIAS
    if op == "compact":
        assert call(n=1, src=0, dst=0) == CF_E_DEVICE


def copy(cf, data=G, n_pages=100, size=4096, layers=2, stride=100 * 4096, src=2 * G, dst=3 * G, n=10, count=4 * G):
    return cf.lib.cf_pages_copy(P(data), n_pages, size, layers, stride, P(src), P(dst), n, P(count), None)


def test_copy_refusals(cf, L):
    assert copy(cf) == CF_E_DEVICE and copy(cf, count=0) == CF_E_DEVICE
    for bad in (dict(n_pages=0), dict(n_pages=1 << 31), dict(size=0), dict(size=4104), dict(size=1 << 41), dict(layers=0), dict(layers=65536),
                dict(stride=100 * 4096 - 16), dict(stride=100 * 4096 + 8), dict(n=-1), dict(n=(1 << 30) + 1), dict(stride=1 << 46)):
        assert copy(cf, **bad) == CF_E_SHAPE, bad
    assert copy(cf, layers=1, stride=0) == CF_E_DEVICE and copy(cf, stride=1 << 30) == CF_E_DEVICE
    assert copy(cf, n=0, data=0, src=0, dst=0) == CF_OK
    for bad in (dict(data=0), dict(src=0), dict(dst=0)):
        assert copy(cf, **bad) == CF_E_NULL, bad
    for bad in (dict(data=G + 8), dict(src=2 * G + 2), dict(dst=3 * G + 1), dict(count=4 * G + 2)):
        assert copy(cf, **bad) == CF_E_ALIGN, bad
    for bad in (dict(src=G), dict(dst=G + 2 * 100 * 4096 - 4), dict(count=G + 64)):
        assert copy(cf, **bad) == CF_E_ALIAS, bad
    assert copy(cf, dst=2 * G) == CF_E_DEVICE  # every pair the same: nothing to do


def test_binding_refuses(cf):
    """What the C ABI cannot see: element types, shapes, host tensors."""
    import torch

    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cache = cf.KV8Cache(torch.zeros(2, 2, 2 * 16 * 64 + 16, dtype=torch.uint8), 16, 64)
    lens, slots = torch.zeros(1, dtype=torch.int32), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="device tensors"):
        cf.kv8_append(cache, x, x, lens, table_width=2)
    with pytest.raises(TypeError, match="kv_lens"):
        cf.kv8_append(cache, x, x, lens.long())
    with pytest.raises(ValueError, match="starts"):
        cf.kv8_append(cache, x, x, lens, starts=lens)
    with pytest.raises(ValueError, match="table"):
        cf.kv8_append(cache, x, x, lens, table=torch.zeros(2, 3, dtype=torch.int32))
    with pytest.raises(ValueError, match="v is"):
        cf.kv8_append(cache, x, x[:, :1], lens)
    with pytest.raises(TypeError, match="activation dtype"):
        cf.kv8_append(cache, x.half(), x.half(), lens)
    with pytest.raises(TypeError, match="slots"):
        cf.kv8_read(cache, slots.int())
    with pytest.raises(ValueError, match="cache data"):
        cf.KV8Cache(cache.data, 32, 64)._args(-2)
    with pytest.raises(ValueError, match="cache data"):
        cf.KV8Cache(torch.zeros(2, 2, 16 * 68, dtype=torch.uint8), 16, 64)._args(-2)
    with pytest.raises(ValueError, match="rows of"):
        cf.kv8_attention(torch.zeros(4, 2, 128, dtype=torch.bfloat16), cache, lens)
    with pytest.raises(cf.CFError):
        cf.KV8Cache.create(1, 17, 1, 64, device="cpu")
    with pytest.raises(cf.CFError):
        cf.kv8_attention_workspace_bytes(torch.float16, 1, 8, 2, 64)
    with pytest.raises(ValueError, match="k is"):
        cf.attention(x, x[:, :, :32], x)
    with pytest.raises(ValueError, match="v is"):
        cf.attention(x, x, x[:3])
    with pytest.raises(TypeError, match="k is"):
        cf.attention(x, x.float(), x.float())
    with pytest.raises(TypeError, match="k_starts"):
        cf.attention(x, x, x, k_starts=slots)
    with pytest.raises(ValueError, match="must be"):
        cf.attention(x[0], x, x)
    with pytest.raises(ValueError, match="device tensors"):
        cf.attention(x, x, x)
    with pytest.raises(cf.CFError):
        cf.attention_workspace_bytes(torch.bfloat16, 1, 8, 3, 64)
    t = cf.PageTable.create(8, 2, 3, 16, device="cpu")
    want = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensors"):
        cf.pages_resize(t, want)
    with pytest.raises(ValueError, match="tokens in"):
        cf.pages_resize(t, want, out=cf.PageTable.create(8, 2, 3, 32, device="cpu"))
    with pytest.raises(ValueError, match="table must be"):
        cf.pages_compact(cf.PageTable(t.refs, t.lens, t.lens, 16))
    with pytest.raises(cf.CFError):
        cf.pages_resize(cf.PageTable(t.refs, t.table, t.lens, 1 << 40), want)
    with pytest.raises(TypeError, match="data must be"):
        cf.pages_copy(torch.zeros(8, 64, dtype=torch.uint8), want, want)
    with pytest.raises(ValueError, match="device tensors"):
        cf.pages_copy(torch.zeros(1, 8, 64, dtype=torch.uint8), want, want)


def test_lengths_of_an_append_behind_a_short_resize(cf):
    import torch

    t = cf.PageTable.create(8, 4, 3, 16, device="cpu")
    t.lens.copy_(torch.tensor([17, 16, 0, 5]))
    got = t.append_lens(torch.tensor([17, 17, 0, -1], dtype=torch.int32))
    assert got.tolist() == [17, 0, 0, 0] and got.dtype == torch.int32


def test_fork_own_refusals(cf, L, monkeypatch):
    """All that a fork refuses."""
    monkeypatch.setattr(cf.lib, "cf_pages_fork", cf.lib.cf_pages_fork_own)
    test_pages_refusals(cf, L, "fork")
    import torch

    t = cf.PageTable.create(8, 2, 3, 16, device="cpu")
    with pytest.raises(ValueError, match="device tensors"):
        cf.pages_fork(t, torch.zeros(2, dtype=torch.int32), own=True)
