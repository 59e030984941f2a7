"""Attention over the 4-bit cache with page tables so wide that every request gets a launch of
its own."""
import numpy as np
import pytest

from tests.test_qcache_gpu import attend, check_rows, make

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
