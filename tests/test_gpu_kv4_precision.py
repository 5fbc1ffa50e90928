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
