"""Attention over the 4-bit cache with scores as large as fp32 holds."""
import numpy as np
import pytest

import oracle
from tests.test_qcache_gpu import Cache, attend, write
from tests.test_qcache_weights_gpu import U, chain, keys, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import tree_speculative_verify_tv_gb300 as tv
    tv.build()
    tv.load()


@pytest.mark.parametrize("d,H", [(64, 2), (128, 16)])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("e", [12, 24, 31, 33, 62, 100, 120])
def test_finite_scores_of_any_size(d, H, sign, e):
    """Scores of 2^(e - 7) and more, all of one sign (all far below zero, or far above): the
    largest takes all the weight, keys with equal scores share it."""
    L, n = 300, 4
    b = chain(n)
    rng = np.random.default_rng(e)
    c = Cache(rng, 1, 5, 1, d, fill=0)
    first = rng.integers(1, 8, L)
    first[200:] = np.minimum(first[200:] + 2, 7)  # a later tile has smaller ones
    kt = keys(n, d, rng.integers(1, 8, n))
    v, vt = rng.normal(size=(L, d)), rng.normal(size=(n, 1, d))
    write(c, rng, [L], [0], k=keys(L, d, first).reshape(L, -1), v=v)
    q = np.zeros((n, H, d))
    q[:, :, 0] = sign * 2.0 ** e
    q[:, 1::2, 0] = sign * 8.0  # every other head has ordinary scores
    s, got, a = attend(c, b, [L], H, rows=rows_of(q, kt, vt))
    assert s == 0
    want = oracle.qcache_attention(*a[:11])
    assert np.isfinite(got).all()
    # weights of one or zero, shared by at most 304 keys; and ordinary ones (6 u and the scale's
    # roundings; sums of 304 in blocks of 16: 19 + 16 steps of 2 u, numerator and denominator)
    vmax = max(np.abs(a[4]).max(), np.abs(vt).max())
    assert np.abs(got - want).max() <= vmax * 2 * (16 + 70) * U


@pytest.mark.parametrize("e", [31, 62, 110])
def test_scores_that_grow_and_fall_by_far_between_tiles(e):
    """The largest score of a row stands in any tile, with ordinary ones, zeros and far negative
    ones in the others; a window hides whole tiles from some rows."""
    d, H, L, n = 64, 4, 700, 4
    b = chain(n)
    c = Cache(np.random.default_rng(0), 1, 11, 1, d, fill=0)
    for at in (3, 130, 390, 600, 699):
        for low in (False, True):
            rng = np.random.default_rng(at)
            first = np.zeros(L)
            first[rng.integers(0, L, 60)] = 5
            first[at] = -7  # channel 0 is +7 / 8
            if low:
                first = first + 8  # (beyond 7: the step doubles, 1 / 4)
                first = np.maximum(first - first % 2, 2)
            k = keys(L, d, first)
            k[:, 0, 1] = 1.75 if low else 0.875
            v = rng.normal(size=(L, d))
            write(c, rng, [L], [0], k=k.reshape(L, -1), v=v)
            q = np.zeros((n, H, d))
            q[:, :, 0] = 2.0 ** e
            q[:, 1, 0] = -2.0 ** e
            q[:, 2, 0] = 1.0
            vt = rng.normal(size=(n, 1, d))
            for window in (0, 150):
                s, got, a = attend(c, b, [L], H, window=window, sinks=8 if window else 0,
                                   rows=rows_of(q, keys(n, d, [7, 7, 7, 7]) * (2 if low else 1), vt))
                assert s == 0 and np.isfinite(got).all()
                want = oracle.qcache_attention(*a[:11])
                vmax = max(np.abs(a[4]).max(), np.abs(vt).max())
                assert np.abs(got - want).max() <= vmax * 2 * (16 + 2 * (704 // 16 + 16)) * U
