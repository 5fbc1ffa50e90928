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
