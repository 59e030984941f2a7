"""tv_qk_norm_rope at positions up to 2^31, against angles in whole numbers.

Bound per element as in test_qk_norm_rope_gpu (d / 8 + 16 roundings of |a| + |b|), and the angle's
error: turns per position are the product of two doubles, 1 / 2 pi off by 2^-53.8 of itself and the
product by 2^-53, so that an angle of t rad is off by 2^-52 |t| at most."""
from fractions import Fraction

import numpy as np
import pytest

import oracle
from test_qk_norm_rope_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import tree_speculative_verify_tv_gb300 as tv
    tv.build()
    tv.load()


def two_pi(bits=200):
    """2 pi times 2^bits, by Machin's formula pi = 16 atan(1/5) - 4 atan(1/239)."""
    def atan(n):
        total = term = (1 << bits + 20) // n
        k = 1
        while term:
            term //= n * n
            k += 2
            total += -term // k if k % 4 == 3 else term // k
        return total
    return 2 * (16 * atan(5) - 4 * atan(239)) >> 20


def turns(position, inv_freq, bits=200):
    """The fraction of a turn of position * inv_freq rad (a double, taken as it is)."""
    f = Fraction(inv_freq) * (1 << bits) / two_pi(bits)
    return float(f * int(position) % 1)


def test_two_pi():
    assert two_pi() / 2.0 ** 200 == 2 * np.pi


@pytest.mark.parametrize("at", [1 << 24, 1 << 28, 2 ** 31 - 100])
@pytest.mark.parametrize("pairs", [False, True])
def test_far_positions(at, pairs):
    c = Case(51, [20, 30], 2, 1, 128, 128, f32=True, pairs=pairs, base=500000.0)
    c.start[:] = at, at - 1000
    pos = c.positions()
    angle = 2 * np.pi * np.array([[turns(p, f) for f in c.freq] for p in pos])
    lo, hi = (slice(0, None, 2), slice(1, None, 2)) if pairs else (slice(0, 64), slice(64, None))
    outs = c.run()
    assert int(c.status[0]) == 0
    for x, w, out in zip(c.host, c.hw, outs):
        y = oracle.qk_norm_rope(x, 0 * pos, w, c.eps, c.freq, pairs)
        a, b = y[..., lo], y[..., hi]
        want, size = np.empty_like(y), np.empty_like(y)
        want[..., lo] = a * np.cos(angle)[:, None] - b * np.sin(angle)[:, None]
        want[..., hi] = b * np.cos(angle)[:, None] + a * np.sin(angle)[:, None]
        size[..., lo] = size[..., hi] = np.abs(a) + np.abs(b)
        got = out.cpu().numpy().astype(np.float64).reshape(y.shape)
        bound = ((c.d / 8 + 16) * 2.0 ** -24 + 2.0 ** -52 * at) * size
        assert (np.abs(got - want) <= bound).all(), float((np.abs(got - want) / bound).max())


@pytest.mark.parametrize("f", [1.0, 0.75, 3.5, 6.28, 100.3, 1.0e-9, -0.3, -1.0e-12, 0.0])
def test_frequencies_of_any_size_and_sign(f):
    """One frequency for all pairs, at positions to 2^31: radians per position above one and below
    zero are turned as they are."""
    c = Case(52, [40], 1, 1, 64, 64, f32=True)
    c.start[:] = 2 ** 31 - 41
    c.freq = np.full(32, f)
    c.freq[1::2] = f * 0.7
    pos = c.positions()
    angle = 2 * np.pi * np.array([[turns(p, x) for x in c.freq] for p in pos])
    outs = c.run()
    for x, w, out in zip(c.host, c.hw, outs):
        y = oracle.qk_norm_rope(x, 0 * pos, w, c.eps, c.freq, False)
        a, b = y[..., :32], y[..., 32:]
        want = np.concatenate([a * np.cos(angle)[:, None] - b * np.sin(angle)[:, None],
                               b * np.cos(angle)[:, None] + a * np.sin(angle)[:, None]], -1)
        size = np.tile(np.abs(a) + np.abs(b), 2)
        got = out.cpu().numpy().astype(np.float64).reshape(y.shape)
        off = 2.0 ** -52 * np.abs(pos[:, None] * c.freq[None])[:, None, :]
        bound = ((c.d / 8 + 16) * 2.0 ** -24 + np.tile(off, 2)) * size
        assert (np.abs(got - want) <= bound).all()
