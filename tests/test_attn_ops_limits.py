"""Sizes and limits of the attention operators' entry points: workspaces, bounds of the queries, empty calls.
Placeholder addresses that are never read, as in test_attn_ops_api.py."""
import pytest

from test_abi import CF_E_DEVICE, CF_E_WORKSPACE
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
