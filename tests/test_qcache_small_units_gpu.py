"""The 4-bit cache at the sizes that the other tests pass by: attention whose requests have at
most 32 rows per KV head (single tokens and small trees, both widths, both output types, with
and without a window, contexts cut between many CTAs), batches of more requests than a launch
or a thread of it takes, and writes of many requests, byte for byte."""
import numpy as np
import pytest

from tests.test_qcache_gpu import Cache, attend, check_rows, make, read, write

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import tree_speculative_verify_tv_gb300 as tv
    tv.build()
    tv.load()


CTX = [0, 1, 63, 64, 65, 127, 128, 129, 700, 3000]


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (100, 4), (130, 70), (1000, 3)])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("nodes,H,Hkv", [(1, 2, 2), (1, 16, 2), (4, 8, 1), (3, 6, 2), (4, 3, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_single_tokens_and_small_trees(d, nodes, H, Hkv, half, window, sinks):
    rng = np.random.default_rng(nodes * H + window)
    sizes = rng.integers(0, nodes + 1, len(CTX))
    sizes[0] = sizes[-1] = nodes
    b, c = make(d + H, sizes.tolist(), Hkv, d, CTX, depth_cap=4)
    assert b.max_nodes * H // Hkv <= 32
    s, got, args = attend(c, b, CTX, H, window=window, sinks=sinks, half=half, pad=8, seed=H)
    assert s == 0
    check_rows(got, *args)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("d,nodes,H,window", [(64, 1, 8, 0), (64, 4, 8, 9000), (128, 1, 32, 9000),
                                              (128, 4, 8, 0)])
def test_one_context_over_the_whole_gpu(d, nodes, H, window, half):
    ctx = [20001]
    b, c = make(d + nodes, [nodes], 1, d, ctx, depth_cap=4)
    s, got, args = attend(c, b, ctx, H, window=window, sinks=5 if window else 0, half=half, seed=nodes)
    assert s == 0
    check_rows(got, *args)


@pytest.mark.parametrize("B", [769, 900, 1024, 1025, 1100, 2100])
@pytest.mark.parametrize("d,H", [(64, 4), (128, 2)])
def test_more_requests_than_threads_and_than_a_launch_takes(B, d, H):
    rng = np.random.default_rng(B + d)
    sizes = rng.integers(0, 3, B)  # a third of them empty
    sizes[-1] = 2
    ctx = rng.integers(0, 140, B).tolist()
    b, c = make(B, sizes.tolist(), 1, d, ctx, depth_cap=2)
    s, got, args = attend(c, b, ctx, H, half=d == 128, seed=B)
    assert s == 0
    check_rows(got, *args)


@pytest.mark.parametrize("B", [896, 897, 1030])
def test_many_requests_of_large_units(B):
    # more than 32 rows per KV head: the kernel of 64-row units
    rng = np.random.default_rng(B)
    sizes = rng.integers(0, 4, B)
    sizes[0] = 3
    ctx = rng.integers(0, 140, B).tolist()
    b, c = make(B, sizes.tolist(), 1, 64, ctx, depth_cap=2)
    s, got, args = attend(c, b, ctx, 16, window=100, sinks=2, seed=B)
    assert s == 0
    check_rows(got, *args)


@pytest.mark.parametrize("B,d,Hkv,most", [(31, 128, 2, 70), (33, 64, 1, 70), (300, 64, 2, 9),
                                          (1025, 128, 1, 4), (1100, 64, 1, 3)])
def test_rows_of_many_requests_byte_for_byte(B, d, Hkv, most):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, most + 1, B)
    lens[B // 2] = 130
    start = rng.integers(0, 60, B)
    c = Cache(rng, B, 3, Hkv, d)
    write(c, rng, lens, start, pad=8)
    assert np.array_equal(c.fetch(), c.host)
    ctx = start + lens // 2 + 1
    gk, gv = read(c, lens, start, ctx, pad=8)
    K, V = c.values()
    at = 0
    for b in range(B):
        live = np.arange(start[b], start[b] + lens[b]) < ctx[b]
        for got, held in ((gk, K), (gv, V)):
            want = held[b][:, start[b]:start[b] + lens[b]].transpose(1, 0, 2) * live[:, None, None]
            np.testing.assert_array_equal(got[at:at + lens[b]], want)
        at += lens[b]


@pytest.mark.parametrize("nodes,H", [(1, 4), (12, 8)])
def test_repeats_are_equal_bit_for_bit(nodes, H):
    # contexts cut between CTAs, a workspace of other contents each time
    ctx = [5000, 1, 900]
    b, c = make(7, [nodes, 1, nodes], 2, 128, ctx)
    _, first, _ = attend(c, b, ctx, H, half=True, seed=2)
    for seed in range(3):
        _, other, _ = attend(c, b, [33, 2, 4], H, half=True, seed=3 + seed)
        s, got, _ = attend(c, b, ctx, H, half=True, seed=2)
        assert s == 0 and np.array_equal(got, first)
