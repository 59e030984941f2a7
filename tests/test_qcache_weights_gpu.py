"""Attention over the 4-bit cache where the weights are known to a few last places.

Scores come from one channel of the queries and keys, so that they are exact in fp32, and
values are exact, too.  Then an output is off by its weights alone.  With u = 2^-24, a weight
2^(s - m), s - m in [-1.3, 0], is off by the exponential's 2 last places (4 u relative) and by
its argument's roundings (the factor log2 e, the product or difference: 2 * 1.3 u, times ln 2:
1.8 u): 6 u.  Numerator and denominator each have one such error in the tile and one in
the join of the pieces (24 u); the parts that a weight enters the value product in leave u
(fp32 outputs); the sums of at most 12 terms, the joins, the quotient and the output round some
20 times by u: 48 u in all.  Without its third part a weight would be off by up to 2^-16 = 256 u.
"""
import numpy as np
import pytest

import oracle
import workloads
from tests.test_qcache_gpu import Cache, attend, bf, write

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import tree_speculative_verify_tv_gb300 as tv
    tv.build()
    tv.load()


def chain(n):
    b = workloads.random_batch(np.random.default_rng(1), [n], 1, 16, 16, depth_cap=4, max_depth=32)
    b.parent[:] = np.arange(-1, n - 1, dtype=np.int32)
    return b


def rows_of(q, kt, vt):
    """The arguments `rows` of attend from arrays [T][heads][d]."""
    wide = np.concatenate([x.reshape(len(x), -1) for x in (q, kt, vt)], axis=1)
    base, val = bf(wide)
    out, at = [], 0
    for x in (q, kt, vt):
        w = x[0].size
        out.append((base[:, at:at + w], val[:, at:at + w]))
        at += w
    return out, at


def keys(n, d, first):
    """Rows of which channel 0 is -first[i] / 8 and channel 1 the 0.875 that makes the step of
    their first 32 channels 1 / 8."""
    k = np.zeros((n, 1, d))
    k[:, 0, 0] = -np.asarray(first) / 8.0
    k[:, 0, 1] = 0.875
    return k


def one_hot(n, d, at):
    v = np.zeros((n, 1, d))
    v[np.arange(n), 0, at] = 0.875
    return v


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H", [1, 8, 32])  # units of 32 rows, 32 rows and 64 rows
@pytest.mark.parametrize("L", [0, 5, 70])
def test_weights_keep_single_precision(d, H, L):
    n = 4
    b = chain(n)
    rng = np.random.default_rng(L + H)
    c = Cache(rng, 1, 2, 1, d, fill=0)
    seen = min(L, 6)  # the others' weights are zero: a window hides them
    window, first = (seen + n if L > seen else 0), rng.integers(0, 8, L)
    vc = one_hot(L, d, (np.arange(L) * 5) % d) if L else np.zeros((0, 1, d))
    if L:
        write(c, rng, [L], [0], k=keys(L, d, first).reshape(L, -1), v=vc.reshape(L, -1))
    # a key's weight against the others': heads with scores of a half and a quarter, too
    q = np.zeros((n, H, d))
    q[:, :, 0] = 0.5 ** (np.arange(H) % 3)[None]
    kt, vt = keys(n, d, [3, 7, 0, 5]), one_hot(n, d, 1 + np.arange(n) * 7)
    # (attend scales by d^-1/2; what its rounding to fp32 moves is within what the smaller
    # scores of d = 128 leave)
    s, got, a = attend(c, b, [L], H, window=window, rows=rows_of(q * 8, kt, vt))
    assert s == 0
    want = oracle.qcache_attention(*a[:11])
    assert np.all(np.abs(got - want) <= 48 * U * np.abs(want))
    assert (want > 0).any(axis=(1, 2)).all()
