"""The 4-bit cache at sizes where its calls change shape: page tables so wide that every request
gets an attention launch of its own, commits of more requests than the GPU has SMs."""
import numpy as np
import pytest

import workloads
from tests.test_qcache_gpu import Cache, attend, check_rows, commit, make, strided

pytestmark = pytest.mark.gpu


def test_wide_page_tables():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import tree_speculative_verify_tv_gb300 as tv
    tv.build()
    tv.load()
    # 128 heads to a KV head and 256 nodes are 512 units of 64 rows: with 2^22 pages two
    # requests could have more than 2^31 tiles together
    ctx = [70, 0, 200]
    b, c = make(5, [256, 3, 1], 1, 64, ctx)
    wide = np.full((3, 1 << 22), -1, np.int32)
    wide[:, :c.mp] = c.table
    c.mp = wide.shape[1]
    s, got, args = attend(c, b, ctx, 128, table=wide)
    assert s == 0
    check_rows(got, *args)


@pytest.mark.parametrize("d,Hkv", [(64, 3), (128, 8)])
def test_commits_of_many_requests(d, Hkv):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import tree_speculative_verify_tv_gb300 as tv
    tv.build()
    tv.load()
    rng = np.random.default_rng(d)
    B = 200
    b = workloads.random_batch(rng, rng.integers(0, 12, B), 1, 16, 16, depth_cap=6, max_depth=6)
    lens, path = np.zeros(B, np.int32), np.full((B, 6), -1, np.int32)
    for r in range(B):  # to a random node, or nowhere
        s, n = b.node_offsets[r], b.node_offsets[r + 1] - b.node_offsets[r]
        j, p = int(rng.integers(-1, n)) if n else -1, []
        while j >= 0:
            p.append(j)
            j = int(b.parent[s + j])
        lens[r] = len(p)
        path[r, :len(p)] = p[::-1]
    ctx = rng.integers(0, 120, B)
    c = Cache(rng, B, 2, Hkv, d)
    ((kt, kv), (vt, vv)), stride = strided(rng, b.T, [Hkv * d, Hkv * d], 8)
    new = commit(c, b, ctx, lens, path, kt, vt, stride, in_place=True)
    assert np.array_equal(new, ctx + lens)
    for r in range(B):
        for m in range(lens[r]):
            at = b.node_offsets[r] + path[r, m]
            c.put(r, int(ctx[r]) + m, kv[at].reshape(Hkv, d), vv[at].reshape(Hkv, d))
    assert np.array_equal(c.fetch(), c.host)
