"""tv_qk_norm_rope: values whose squares leave single precision, and rows of unusable requests.
Bounds are those of test_qk_norm_rope_gpu.Case.check."""
import numpy as np
import pytest

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


def scaled(case, sizes):
    """Row r of both projections times a power of two of `sizes` (in turn)."""
    import torch
    for x, host in zip(case.dev, case.host):
        heads, d = host.shape[1], case.d
        for r in range(case.R):
            row = x[r].view(heads, d)
            for h in range(heads):
                f = 2.0 ** sizes[(r + h) % len(sizes)]
                y = (row[h].double() * f).to(x.dtype)
                y = torch.where(torch.isinf(y), row[h], y)  # (no larger than the type)
                row[h] = y
                host[r, h] = y.double().cpu().numpy()


HUGE = [0, 62, 70, 100, 124, 61, 126, 63]
TINY = [0, -62, -70, -48, -100, -120, -51, -132, -140]


@pytest.mark.parametrize("d,rot", [(64, 64), (128, 64), (256, 256), (128, 0)])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e30])
def test_huge_rows(d, rot, pairs, f32, eps):
    c = Case(21, [9, 1, 8], 7, 3, d, rot, pairs=pairs, f32=f32, eps=eps)
    scaled(c, HUGE)
    c.check(c.run())


@pytest.mark.parametrize("d,rot", [(64, 64), (128, 64), (256, 256)])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("eps", [0.0, 1e-38, 1e-31, 1e-20, 1e-6])
def test_tiny_rows(d, rot, f32, eps):
    """Without eps the norm brings rows of any size to the size of the weights.  (bf16 has nothing
    between 0 and 2^-133: rows times 2^-140 are rows of zeros, 0 / 0 without eps and compared apart.)"""
    import torch
    c = Case(22, [9, 1, 8], 7, 3, d, rot, f32=f32, eps=eps)
    scaled(c, TINY)
    first = [x.clone() for x in c.run()]
    none = [torch.from_numpy(~x.any(-1)).cuda() for x in c.host]
    if eps == 0.0:
        for i, (x, heads) in enumerate(((c.dev[0], 7), (c.dev[1], 3))):
            assert torch.isnan(first[i].view(c.R, heads, d)[none[i]].float()).all()
            x.view(c.R, heads, d)[none[i]] = 1.0
            c.host[i][none[i].cpu().numpy()] = 1.0
    second = c.run()
    c.check(second)
    for i, heads in enumerate((7, 3)):
        keep = ~none[i] if eps == 0.0 else torch.ones_like(none[i])
        x, y = (z[i].view(c.R, heads, d)[keep] for z in (first, second))
        assert torch.equal(x, y)


@pytest.mark.parametrize("f32", [False, True])
def test_bad_rows_beside_huge_ones(f32):
    """A NaN makes its row of that head NaN; an infinity is one over itself and the others are 0.  The
    neighbours are what they are without them."""
    import torch
    c = Case(23, [12], 4, 2, 64, 64, f32=f32)
    scaled(c, HUGE)
    want = [x.clone() for x in c.run()]
    c.check(want)
    c.dev[0].view(12, 4, 64)[3, 1, 5] = float("nan")
    c.dev[0].view(12, 4, 64)[4, 2, 9] = float("inf")
    c.dev[1].view(12, 2, 64)[4, 0, 63] = -float("inf")
    got = c.run()
    q, k = got[0].view(12, 4, 64), got[1].view(12, 2, 64)
    assert torch.isnan(q[3, 1]).all()
    for row, at in ((q[4, 2], (9, 41)), (k[4, 0], (63, 31))):  # the infinity's pair turns with it
        bad = torch.zeros(64, dtype=torch.bool)
        bad[list(at)] = True
        assert torch.isnan(row[bad]).all() and not row[~bad].any()
    for x, y, rows in ((q, want[0].view(12, 4, 64), ((3, 1), (4, 2))),
                       (k, want[1].view(12, 2, 64), ((4, 0),))):
        keep = torch.ones(x.shape[:2], dtype=torch.bool)
        for r in rows:
            keep[r] = False
        assert torch.equal(x[keep], y[keep])


def usable_rows(offsets, R):
    """Rows of usable requests, and the request of each."""
    of = np.full(R, -1)
    for b in range(len(offsets) - 1):
        o, e = offsets[b], offsets[b + 1]
        if 0 <= o <= e <= R:
            of[o:e] = b
    return of


@pytest.mark.parametrize("offsets", [[-1, 20, 40, 60], [0, 20, 40, 99],
                                     [0, 2] + [4] * 30 + [8, 30, 31, 50, 61],
                                     [-7, 2] + [4] * 30 + [8, 30, 31, 50, 60]])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_unusable_requests_stay(offsets, d):
    """Rows of an unusable request keep what the outputs held; the others are right (an offset out
    of range at either end leaves the others' rows their own)."""
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    B = len(offsets) - 1
    c = Case(24, [60] + [0] * (B - 1), 2, 1, d, 64)
    c.offsets = np.array(offsets, np.int32)
    of = usable_rows(offsets, 60)
    outs = [x.cpu() for x in c.run()]
    assert int(c.status[0]) == tv.TV_ERR_TREE
    assert (of >= 0).any() and (of < 0).any()
    for x in outs:
        assert torch.isnan(x[of < 0].float()).all()
    # the usable rows again, as requests of their own
    rows = np.nonzero(of >= 0)[0]
    alone = Case(24, [60] + [0] * (B - 1), 2, 1, d, 64)
    alone.R = alone.n = len(rows)
    lens = [int((of == b).sum()) for b in range(B)]
    alone.offsets = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    alone.dev = [x[torch.from_numpy(rows).cuda()].contiguous() for x in c.dev]
    alone.host = [x[rows] for x in c.host]
    want = alone.run()
    alone.check(want)
    for x, y in zip(outs, want):
        assert torch.equal(x[rows], y.cpu())


def test_overlapping_requests_write_right_rows_or_none():
    """Offsets that fall: the request between is unusable; rows of the others may be left, but none
    is wrong."""
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    c = Case(25, [30, 0, 30], 2, 1, 64, 64)
    want = [x.clone() for x in c.run()]           # requests 0: 0-29, 2: 30-59
    c.start[2] -= 10                              # row 30 stands at its old position when 20 begins
    c.offsets = np.array([0, 30, 20, 60], np.int32)
    got = c.run()
    assert int(c.status[0]) == tv.TV_ERR_TREE
    for x, y in zip(got, want):
        left = torch.isnan(x.float()).all(1)
        right = (x == y).all(1)
        assert (left | right)[:20].all() and (left | right)[30:].all()


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("f32", [False, True])
def test_huge_and_tiny_rows_in_place(pairs, f32):
    """What is scaled is read again after the other heads have been written; a weight of zeros makes
    rows of zeros of these, which are not taken for tiny ones."""
    import torch
    for weights in (True, False):
        c = Case(26, [30, 9], 21, 6, 64, 64, pairs=pairs, f32=f32, eps=0.0)
        scaled(c, [0, 70, -62, 1, 100, -100, 0, 0])
        if weights:
            c.dw[0].zero_()
            c.hw[0][:] = 0.0
        want = c.run()
        c.check(want)
        for x, y in zip(want, c.run(in_place=True)):
            assert torch.equal(x, y)
