"""Which stream's blocks the buffers come from that the binding allocates for a call on another stream than the caller's:
on the CPU with streams, launches and the allocator's entry points recorded."""
from __future__ import annotations

import contextlib

import pytest
import torch

HERE, THERE = 11, 22  # the caller's stream and the launch stream


class Fake:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture(scope="module")
def cf():
    from activation_residual_compression_cf_amd import cf as _cf

    return _cf


@pytest.fixture
def log(cf, monkeypatch):
    """[(current stream, address, bytes)] of allocations, {address: stream} of what is recorded, and what launches were given."""
    now, made, kept, launched = [HERE], [], {}, []

    @contextlib.contextmanager
    def use(stream):
        now.append(stream.cuda_stream)
        yield
        now.pop()

    def watch(owner, name):
        make = getattr(owner, name)

        def f(*a, **k):
            t = make(*a, **k)
            made.append((now[-1], t))
            return t

        monkeypatch.setattr(owner, name, f)

    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Fake(now[-1]))
    monkeypatch.setattr(torch.cuda, "ExternalStream", Fake)
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: kept.__setitem__(id(t), s.cuda_stream))
    watch(torch, "empty")
    watch(torch, "empty_like")
    watch(torch.Tensor, "new_empty")
    monkeypatch.setattr(cf, "_device", lambda t: 0)
    monkeypatch.setattr(cf, "_here", lambda *a: None)
    monkeypatch.setattr(cf, "_ptr", lambda t: None if t is None else t.data_ptr())
    for name in cf._SIG:
        if not name.endswith("bytes"):
            monkeypatch.setattr(cf.lib, name, lambda *a: launched.append(a) or 0)
    return made, kept, launched


def flat(x):
    return [t for y in x for t in flat(y)] if isinstance(x, (tuple, list)) else [x] if isinstance(x, torch.Tensor) else []


def calls(cf):
    rows = lambda n, h=2, d=64, t=torch.bfloat16: torch.zeros(n, h, d, dtype=t)
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)
    c4, c8 = cf.KV4Cache.create(4, 16, 2, 64, device="cpu"), cf.KV8Cache.create(4, 16, 2, 64, device="cpu")
    pt = cf.PageTable.create(8, 2, 3, 16, device="cpu")
    of = lambda t: [t.refs, t.table, t.lens] if isinstance(t, cf.PageTable) else [t]
    several = lambda r: [t for x in r for t in of(x)]
    a = torch.zeros(1, 128, 128)
    state = lambda: torch.zeros(1, 128, 128)
    return {
        "compress": lambda s: cf.compress(1, a, state(), None, stream=s),
        "compress_ablation": lambda s: cf.compress_ablation(0, 1, a, state(), stream=s),
        "topk_compress": lambda s: cf.topk_compress(4, a, state(), None, stream=s),
        "lowrank_compress": lambda s: cf.lowrank_compress(a, state(), None, torch.zeros(1, 128, 8), 8, 1, stream=s),
        "lowrank_compress_16": lambda s: cf.lowrank_compress(a, state(), None, torch.zeros(1, 128, 8), 8, 1, 16, stream=s),
        "qk_norm_rope": lambda s: cf.qk_norm_rope(rows(3), rows(3), stream=s),
        "kv4_read": lambda s: cf.kv4_read(c4, torch.zeros(3, dtype=torch.int64), stream=s),
        "kv8_read": lambda s: cf.kv8_read(c8, torch.zeros(3, dtype=torch.int64), stream=s),
        "kv4_attention": lambda s: cf.kv4_attention(rows(2), c4, i32(1), table_width=4, stream=s),
        "kv8_attention": lambda s: cf.kv8_attention(rows(2), c8, i32(1), table_width=4, stream=s),
        "attention": lambda s: cf.attention(rows(2), rows(3), rows(3), stream=s),
        "pages_resize": lambda s: several(cf.pages_resize(pt, i32(2), stream=s)),
        "pages_fork": lambda s: several(cf.pages_fork(pt, i32(2), stream=s)),
        "pages_fork_own": lambda s: several(cf.pages_fork(pt, i32(2), own=True, stream=s)),
        "pages_compact": lambda s: several(cf.pages_compact(pt, stream=s)),
    }


NAMES = ["compress", "compress_ablation", "topk_compress", "lowrank_compress", "lowrank_compress_16", "qk_norm_rope", "kv4_read", "kv8_read",
         "kv4_attention", "kv8_attention", "attention", "pages_resize", "pages_fork", "pages_fork_own", "pages_compact"]
OWN_WORKSPACE = {"lowrank_compress", "lowrank_compress_16", "kv4_attention", "kv8_attention", "attention", "pages_resize", "pages_fork",
                 "pages_fork_own", "pages_compact"}


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("stream", [None, HERE, THERE])
def test_buffers_are_the_launch_streams(cf, log, monkeypatch, name, stream):
    made, kept, launched = log
    call = calls(cf)[name]
    del made[:], launched[:]
    if stream is None:  # the raw handle of the current stream is asked for, which needs a device
        monkeypatch.setattr(cf, "_on", lambda *a: HERE)
        monkeypatch.setattr(cf, "_stream", lambda s: HERE)
    got = flat(call(stream))
    assert len(launched) == 1
    want = THERE if stream == THERE else HERE
    assert made and {s for s, _ in made} == {want}
    mine = {id(t) for _, t in made}
    assert {id(t) for t in got} <= mine
    assert len(mine) - len(got) == (name in OWN_WORKSPACE)
    # what the caller gets is kept for the caller's stream; the workspace needs nothing
    assert kept == ({id(t): HERE for t in got} if stream == THERE else {})
