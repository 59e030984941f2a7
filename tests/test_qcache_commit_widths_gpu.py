"""tv_qcache_commit takes another number of threads per request once there are more requests than
the device has SMs: batches of exactly as many, of one more and of one less."""
import numpy as np
import pytest

import workloads
from tests.test_qcache_gpu import Cache, commit, strided

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,Hkv", [(64, 2), (128, 1)])
@pytest.mark.parametrize("more", [-1, 0, 1])
def test_about_as_many_requests_as_sms(d, Hkv, more):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import tree_speculative_verify_tv_gb300 as tv
    tv.build()
    tv.load()
    B = torch.cuda.get_device_properties(0).multi_processor_count + more
    rng = np.random.default_rng(d + more)
    b = workloads.random_batch(rng, [7] * B, 1, 16, 16, depth_cap=7, max_depth=7)
    b.parent[:] = np.tile(np.arange(-1, 6, dtype=np.int32), B)  # chains
    lens = rng.integers(0, 8, B).astype(np.int32)
    path = np.where(np.arange(7) < lens[:, None], np.arange(7), -1).astype(np.int32)
    ctx = rng.integers(0, 120, B)
    c = Cache(rng, B, 2, Hkv, d)
    ((kt, kv), (vt, vv)), stride = strided(rng, b.T, [Hkv * d, Hkv * d], 0)
    new = commit(c, b, ctx, lens, path, kt, vt, stride)
    assert np.array_equal(new, ctx + lens)
    for r in range(B):
        for m in range(lens[r]):
            at = b.node_offsets[r] + m
            c.put(r, int(ctx[r]) + m, kv[at].reshape(Hkv, d), vv[at].reshape(Hkv, d))
    assert np.array_equal(c.fetch(), c.host)
