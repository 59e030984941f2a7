"""tv_qk_norm_rope against norms and rotations in 64 bits.

Bound per element: the sum of d squares, its root and quotient, two products with weights and
the rotation's two products and sum round at most d / 8 + 12 times at 2^-24, relative to
|a| + |b| of the rotated pair; the turns are exact to 2^-27 of half a turn (angle 2^-25); the
result rounds once to its type."""
import numpy as np
import pytest

import oracle
import workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import tree_speculative_verify_tv_gb300 as tv
    tv.build()
    tv.load()


class Case:
    def __init__(self, seed, lens, H, Hkv, d, rot, *, pairs=False, f32=False, fused=False,
                 trees=False, weights=True, eps=1e-6, at=5000, extra=0, base=10000.0):
        import torch
        rng = np.random.default_rng(seed)
        self.B, self.R = len(lens), int(sum(lens)) + extra
        self.H, self.Hkv, self.d, self.rot, self.pairs, self.f32 = H, Hkv, d, rot, pairs, f32
        self.eps, self.n = eps, int(sum(lens))
        self.offsets = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        self.start = rng.integers(0, at + 1, self.B).astype(np.int32)
        self.depth = rng.integers(1, 33, self.R).astype(np.int32) if trees else None
        self.freq = base ** (-np.arange(0, rot, 2) / max(rot, 1))
        dt = torch.float32 if f32 else torch.bfloat16

        def put(x):
            x = x.astype(np.float32)
            if not f32:
                x = workloads.bf16_bits_to_f32(workloads.f32_to_bf16_bits(x))
            return x.astype(np.float64), torch.from_numpy(x).to("cuda", dt)

        hq, q = put(rng.normal(size=(self.R, H * d)))
        hk, k = put(3 * rng.normal(size=(self.R, Hkv * d)))
        self.host = hq.reshape(self.R, H, d), hk.reshape(self.R, Hkv, d)
        self.stride = (H * d, Hkv * d)
        if fused:
            both = torch.cat([q, k, k], 1)
            q, k, _ = both.split([H * d, Hkv * d, Hkv * d], 1)
            self.stride = (both.shape[1],) * 2
        self.dev = q, k
        w = [put(1 + 0.3 * rng.normal(size=d)) if weights else (None, None) for _ in range(2)]
        self.hw, self.dw = [x[0] for x in w], [x[1] for x in w]

    def run(self, in_place=False, out_pad=0, stream=None):
        import torch
        import tree_speculative_verify_tv_gb300 as tv
        dev = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        outs, strides = self.dev, self.stride
        if not in_place:
            strides = (self.H * self.d + out_pad, self.Hkv * self.d + out_pad)
            outs = [torch.full((self.R, s), float("nan"), dtype=x.dtype, device="cuda")
                    for s, x in zip(strides, self.dev)]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        tv.tv_qk_norm_rope(self.B, self.R, self.H, self.Hkv, self.d, self.rot,
                           tv.TV_ROPE_PAIRS if self.pairs else tv.TV_ROPE_HALVES,
                           tv.TV_F32 if self.f32 else tv.TV_BF16, dev(self.offsets),
                           dev(self.start), dev(self.depth), self.dev[0], self.stride[0],
                           self.dev[1], self.stride[1], self.dw[0], self.dw[1], self.eps,
                           dev(self.freq), outs[0], strides[0], outs[1], strides[1], self.status,
                           stream=stream)
        torch.cuda.synchronize()
        return outs

    def positions(self):
        b = np.repeat(np.arange(self.B), np.diff(self.offsets))
        rows = np.arange(self.n)
        if self.depth is not None:
            return self.start[b].astype(np.int64) + self.depth[:self.n] - 1
        return self.start[b].astype(np.int64) + rows - self.offsets[b]

    def check(self, outs):
        assert int(self.status[0]) == 0
        pos, eps = self.positions(), None if self.eps < 0 else self.eps
        for x, heads, w, out in zip(self.host, (self.H, self.Hkv), self.hw, outs):
            want = oracle.qk_norm_rope(x[:self.n], pos, w, eps, self.freq, self.pairs)
            flat = oracle.qk_norm_rope(x[:self.n], 0 * pos, w, eps, self.freq, self.pairs)
            size = np.abs(flat)  # |a| + |b| of the pair that an element came from
            half = len(self.freq)
            lo, hi = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if self.pairs else
                      (slice(0, half), slice(half, 2 * half)))
            size[..., lo] = size[..., hi] = size[..., lo] + size[..., hi]
            got = out[:, :heads * self.d].float().cpu().numpy().astype(np.float64)
            got = got.reshape(self.R, heads, self.d)[:self.n]
            bound = ((self.d / 8 + 16) * 2.0 ** -24 * size +
                     (2.0 ** -24 if self.f32 else 2.0 ** -8) * np.abs(want) + 1e-37)
            assert (np.abs(got - want) <= bound).all(), float((np.abs(got - want) / bound).max())


@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (256, 256), (128, 64), (64, 8), (256, 96),
                                   (128, 0), (128, 120)])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("f32", [False, True])
def test_widths_layouts_and_types(d, rot, pairs, f32):
    c = Case(1, [1, 0, 40, 7], 5, 2, d, rot, pairs=pairs, f32=f32, fused=True)
    c.check(c.run())
    c.check(c.run(out_pad=24))


@pytest.mark.parametrize("H,Hkv", [(1, 1), (32, 8), (7, 7), (3, 1), (17, 0), (40, 20)])
@pytest.mark.parametrize("lens", [[1], [16] * 9, [300, 1, 55]])
def test_heads_and_rows(H, Hkv, lens):
    c = Case(2, lens, H, Hkv, 128, 128)
    c.check(c.run())


def test_trees():
    c = Case(3, [16, 1, 0, 64], 8, 2, 128, 128, trees=True, at=200000)
    c.check(c.run())


@pytest.mark.parametrize("at", [0, 1 << 20, 2**31 - 200])
@pytest.mark.parametrize("f32", [False, True])
def test_far_positions(at, f32):
    """Angles of 2^31 radians: the position times the frequency in 64 bits is off by 2^-21 there
    (and so is the oracle's), which the bound's angle does not hold."""
    c = Case(4, [50, 70], 2, 1, 64, 64, f32=f32, at=at, base=500000.0)
    if at > 1 << 24:
        c.freq = 2 * np.pi * 2.0 ** -np.arange(3, 35.0)  # whole fractions of a turn: exact
        turns = [(int(p) * 2 ** (40 - i) % 2 ** 40) / 2 ** 40 for p in c.positions()
                 for i in range(3, 35)]
        angle = 2 * np.pi * np.array(turns).reshape(-1, 32)
        outs = c.run()
        for x, w, out in zip(c.host, c.hw, outs):
            y = oracle.qk_norm_rope(x, 0 * c.positions(), w, 1e-6, c.freq, False)
            a, b = y[..., :32], y[..., 32:]
            want = np.concatenate([a * np.cos(angle)[:, None] - b * np.sin(angle)[:, None],
                                   b * np.cos(angle)[:, None] + a * np.sin(angle)[:, None]], -1)
            got = out.float().cpu().numpy().astype(np.float64).reshape(want.shape)
            size = np.tile(np.abs(a) + np.abs(b), 2)
            # 1 / 2 pi rounds to 2^-54 of itself: 2^31 positions of 1/8 turn are off by 2^-26
            bound = 2.0 ** -19 * size + (2.0 ** -24 if f32 else 2.0 ** -8) * np.abs(want)
            assert (np.abs(got - want) <= bound).all()
        return
    c.check(c.run())


@pytest.mark.parametrize("weights,eps", [(False, 1e-5), (True, 0.0), (True, -1.0), (False, -1.0)])
def test_without_weights_or_norm(weights, eps):
    c = Case(5, [20, 3], 4, 2, 128, 128, weights=weights, eps=eps)
    if eps < 0:
        c.hw = [None, None]
    c.check(c.run())


@pytest.mark.parametrize("fused", [False, True])
def test_in_place(fused):
    import torch
    c = Case(6, [33, 70], 6, 3, 128, 64, fused=fused, extra=4)
    before = [x.clone() for x in c.dev]
    want = c.run()
    c.check(want)
    got = c.run(in_place=True)
    for x, y, old in zip(want, got, before):
        assert torch.equal(x[:c.n], y[:c.n])
        assert torch.equal(y[c.n:], old[c.n:])       # rows of no request stay
        assert torch.isnan(x[c.n:].float()).all()


def test_zero_rows_and_huge_values():
    """A row of zeros stays zero (eps keeps the quotient finite; with eps 0 it is NaN)."""
    import torch
    c = Case(7, [4], 2, 1, 64, 64)
    c.dev[0][1].zero_()
    q, _ = c.run()
    assert not q[1].any()
    c.eps = 0.0
    q, _ = c.run()
    assert torch.isnan(q[1].float()).all() and torch.isfinite(q[0].float()).all()


@pytest.mark.parametrize("offsets", [[0, 30, 20, 60], [-1, 20, 40, 60], [0, 20, 40, 99]])
def test_unusable_offsets(offsets):
    import tree_speculative_verify_tv_gb300 as tv
    c = Case(8, [20, 20, 20], 2, 1, 64, 64)
    c.offsets = np.array(offsets, np.int32)
    c.run()
    assert int(c.status[0]) == tv.TV_ERR_TREE
