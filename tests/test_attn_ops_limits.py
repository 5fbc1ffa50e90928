"""Sizes and limits of the attention operators' entry points: workspaces, bounds of the queries, empty calls.
Placeholder addresses that are never read, as in test_attn_ops_api.py."""
import pytest

from test_abi import CF_E_ARG, CF_E_DEVICE, CF_E_SHAPE, CF_E_WORKSPACE, CF_OK
from test_attn_ops_api import G, L, attn, cf  # noqa: F401  (fixtures)


def test_a_workspace_for_more_queries_serves_fewer(cf):
    f = cf.lib.cf_kv4_attention_workspace_bytes
    for dt in (0, 1):
        for dim in (64, 128):
            for share in (1, 2, 3, 8, 16, 40):
                sizes = [f(dt, n, 2 * share, 2, dim) for n in list(range(1, 140)) + [1000, 100000]]
                assert all(a > 0 for a in sizes)
                assert sizes == sorted(sizes), (dt, dim, share)


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("total,batch,starts", [(32, 32, 0), (33, 1, 0), (64, 4, 0), (12, 3, 5 * G), (40, 2, 5 * G), (100, 100, 5 * G)])
def test_the_documented_workspace_is_enough_without_a_bound(cf, L, dt, dim, total, batch, starts):
    """max_q 0: bytes for total_q, with q_starts and without."""
    call = dict(dt=dt, dim=dim, total=total, batch=batch, starts=starts, max_q=0, hq=8, hk=8, q=(G, 8 * dim, dim), out=(6 * G, 8 * dim, dim))
    need = cf.lib.cf_kv4_attention_workspace_bytes(dt, total, 8, 8, dim)
    assert attn(cf, ws_bytes=need, **call) == CF_E_DEVICE
    # and with any bound below it
    for most in range(1, total + 1):
        assert attn(cf, ws_bytes=need, **{**call, "max_q": most}) == CF_E_DEVICE, most
    each = total if starts else total // batch
    assert attn(cf, ws_bytes=cf.lib.cf_kv4_attention_workspace_bytes(dt, each, 8, 8, dim) - 1, **call) == CF_E_WORKSPACE


@pytest.mark.parametrize("max_q", [0, 1, 4, 1 << 40])
def test_no_queries_is_a_valid_call_with_any_bound(cf, L, max_q):
    """A decoding step in which no sequence takes part."""
    assert attn(cf, total=0, max_q=max_q) == CF_OK
    assert attn(cf, total=0, max_q=max_q, q=None, out=None, batch=0, ws=0, ws_bytes=0) == CF_OK
    # what is no bound, and what no call takes, is refused all the same
    assert attn(cf, total=0, max_q=-1) == CF_E_SHAPE
    assert attn(cf, total=0, max_q=max_q, hq=9) == CF_E_SHAPE
    assert attn(cf, total=0, max_q=max_q, flags=2) == CF_E_ARG


def test_binding_cuts_the_bound_to_the_queries(cf, monkeypatch):
    """cf_kv4_attention takes bounds up to total_q; a program's own bound may be above what a step has."""
    import torch

    seen = []
    real = cf.lib.cf_kv4_attention_workspace_bytes

    class Lib:
        def __getattr__(self, name):
            return lambda *a: seen.append((name, a)) or (real(*a) if name.endswith("_bytes") else 0)

    monkeypatch.setattr(cf, "lib", Lib())
    monkeypatch.setattr(cf, "_here", lambda *a: None)  # host tensors: nothing is launched
    monkeypatch.setattr(cf, "_on", lambda *a: None)
    q = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    cache = cf.KV4Cache(torch.zeros(2, 2, 16 * 68, dtype=torch.uint8), 16, 64)
    lens, starts = torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    for most, want in ((4, 3), (3, 3), (2, 2), (0, 0)):
        seen.clear()
        cf.kv4_attention(q, cache, lens, q_starts=starts, table_width=1, max_q=most)
        name, args = seen[-1]
        assert name == "cf_kv4_attention" and args[14] == want
    seen.clear()
    cf.kv4_attention(q[:0], cache, lens, q_starts=starts, table_width=1, max_q=4)
    assert seen[-1][1][14] in (0, 4)


def _on_host(cf, monkeypatch):
    """The binding without a device: calls are noted, and report success."""
    seen = []
    strerror = cf.lib.cf_strerror

    class Lib:
        cf_strerror = staticmethod(strerror)

        def __getattr__(self, name):
            return lambda *a: seen.append((name, a)) or (1 << 20 if name.endswith("_bytes") else 0)

    monkeypatch.setattr(cf, "lib", Lib())
    monkeypatch.setattr(cf, "_here", lambda *a: None)
    monkeypatch.setattr(cf, "_on", lambda *a: None)
    return seen


TOO_BIG = [1 << 31, (1 << 32) + 5, -(1 << 32) + 5, 1 << 70]


@pytest.mark.parametrize("n", TOO_BIG)
def test_binding_refuses_numbers_past_32_bits(cf, monkeypatch, n):
    """An int of the C ABI takes the lowest 32 bits of what it is given: a window of 2^32 + 5 would be one of 5."""
    import torch

    lib = cf.lib
    with pytest.raises(cf.CFError):
        cf.KV4Cache.create(1, 16 + n, 1, 64, device="cpu")
    with pytest.raises(cf.CFError):
        cf.KV4Cache.create(1, 16, 1 + n, 64, device="cpu")
    with pytest.raises(cf.CFError):
        cf.KV4Cache.create(1, 16, 1, 64 + n, device="cpu")
    with pytest.raises(cf.CFError):
        cf.kv4_attention_workspace_bytes(torch.bfloat16, 1, 8 + n, 2, 64)
    with pytest.raises(cf.CFError):
        cf.kv4_attention_workspace_bytes(torch.bfloat16, 1, 8, 2 + n, 64)
    with pytest.raises(cf.CFError):
        cf.kv4_attention_workspace_bytes(torch.bfloat16, 1, 8, 2, 64 + n)
    seen = _on_host(cf, monkeypatch)
    q = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    cache = cf.KV4Cache(torch.zeros(2, 2, 16 * 68, dtype=torch.uint8), 16, 64)
    lens, starts = torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    good = dict(q_starts=starts, table_width=1)
    cf.kv4_attention(q, cache, lens, **good, causal=True, window=(1 << 31) - 1)
    assert seen[-1][1][16] == (1 << 31) - 1
    for bad in (dict(good, causal=True, window=n), dict(good, table_width=n), dict(good, table_width=n, max_q=1)):
        seen.clear()
        with pytest.raises(cf.CFError):
            cf.kv4_attention(q, cache, lens, **bad)
        assert not [x for x in seen if x[0] == "cf_kv4_attention"]
    row = torch.zeros(2, 2, 64)
    for bad in (dict(norm=cf.CF_NORM_RMS + n), dict(rope=cf.CF_ROPE_HALF + n, cos=torch.zeros(4, 32), sin=torch.zeros(4, 32))):
        seen.clear()
        with pytest.raises(cf.CFError):
            cf.qk_norm_rope(row, row, **bad)
        assert not seen
    for bad in (cf.KV4Cache(cache.data, 16, 64 + n), cf.KV4Cache(cache.data, 16 + n, 64)):
        with pytest.raises((ValueError, cf.CFError)):
            cf.kv4_append(bad, q, q, torch.zeros(3, dtype=torch.int64))
    assert lib.cf_kv4_cache_bytes(1, 16, 1, 64) > 0


@pytest.mark.parametrize("n", [1 << 63, -(1 << 63) - 1])
def test_binding_refuses_numbers_past_64_bits(cf, monkeypatch, n):
    """cf_kv4_cache_bytes(2^64 + 1, ...) would be that of one page."""
    import torch

    with pytest.raises(cf.CFError):
        cf.KV4Cache.create(1 + 2 * n, 16, 1, 64, device="cpu")
    with pytest.raises(cf.CFError):
        cf.kv4_attention_workspace_bytes(torch.bfloat16, 1 + 2 * n, 8, 2, 64)
    seen = _on_host(cf, monkeypatch)
    q = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    cache = cf.KV4Cache(torch.zeros(2, 2, 16 * 68, dtype=torch.uint8), 16, 64)
    with pytest.raises(cf.CFError):
        cf.kv4_attention(q, cache, torch.zeros(3, dtype=torch.int32), table_width=1, max_q=-2 * (1 << 63) + 1)
    assert not [x for x in seen if x[0] == "cf_kv4_attention"]


def test_number_of_sequences(cf, L):
    """The plan counts through the sequences in 64s and in 32 bits: 2^31 - 1 of them would never end."""
    most = 1 << 24
    many = dict(total=12, width=1, lens=4 * G, table=9 * G)
    assert attn(cf, batch=most, **many) == CF_E_DEVICE
    for batch in (most + 1, (1 << 31) - 64, (1 << 31) - 1):
        assert attn(cf, batch=batch, **many) == CF_E_SHAPE, batch
        assert attn(cf, batch=batch, **{**many, "total": 0}) == CF_OK


def test_number_of_rows(cf, L):
    """Rows are counted in tiles of up to 128 and in 32 bits: the end of the last tile has to fit."""
    f = cf.lib.cf_kv4_attention_workspace_bytes
    most = (1 << 31) - 256
    big = dict(hq=1, hk=1, pages=50, q=(G, 0, 0), out=(1 << 45, 64, 64), lse=0, max_q=0)
    assert attn(cf, total=most, **big) == CF_E_DEVICE
    assert f(0, most, 1, 1, 64) > 0 and f(0, most // 8, 8, 2, 64) > 0
    for total in (most + 1, (1 << 31) - 1):
        assert attn(cf, total=total, **big) == CF_E_SHAPE, total
        assert f(0, total, 1, 1, 64) == 0
    assert attn(cf, total=most // 8 + 1, q=(G, 0, 0), out=(1 << 45, 512, 64), lse=0, max_q=0) == CF_E_SHAPE
