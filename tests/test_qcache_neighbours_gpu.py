"""Rows with values that are not numbers, infinite or beyond the range, next to ordinary ones:
a word of V's codes holds eight positions, of which only the odd one may lose anything."""
import numpy as np
import pytest

import oracle
import workloads

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("odd", [np.nan, np.inf, -np.inf, 3e38, -6272.0])
def test_neighbours_of_an_odd_row_keep_their_codes(d, odd):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import tree_speculative_verify_tv_gb300 as tv
    tv.build()
    rng = np.random.default_rng(17)
    n, Hkv = 150, 2
    x = rng.normal(size=(n, Hkv, d)).astype(np.float32)
    rows = [0, 7, 9, 42, 63, 64, 100, 149]
    for r in rows:  # in one group of 32 channels of one head
        x[r, 1, 32 + r % 32] = odd
    bits = workloads.f32_to_bf16_bits(x)
    x = workloads.bf16_bits_to_f32(bits).reshape(n, Hkv, d)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    rec = tv.tv_qcache_bytes(1, 1, d)
    cache = torch.full((4, Hkv, rec), 255, dtype=torch.uint8, device="cuda")
    row = dev(bits).view(torch.bfloat16).reshape(n, Hkv * d)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    start = 5
    tv.tv_qcache_write(1, n, Hkv, d, 4, 4, dev(np.array([0, n], np.int32)),
                       dev(np.array([start], np.int32)), dev(np.array([2, 0, 3, 1], np.int32)),
                       row, row, Hkv * d, cache, st)
    torch.cuda.synchronize()
    assert int(st[0]) == 0
    K, V = oracle.qcache_get(cache.cpu().numpy()[[2, 0, 3, 1]], d)  # [pages, Hkv, 64, d]
    want = oracle.qcache_values(*oracle.qcache_quantise(x.astype(np.float64)))
    for got in (K, V):
        got = got.transpose(0, 2, 1, 3).reshape(-1, Hkv, d)[start:start + n]
        assert np.array_equal(np.isnan(got), np.isnan(want))
        ok = ~np.isnan(want)
        assert np.array_equal(got[ok], want[ok])
