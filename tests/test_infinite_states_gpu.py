"""Infinite elements of a state, and decays past single precision's range.

A finite decay above 0 leaves infinity as it is, whatever the decay's rounding; one that is past
2^128 makes infinity of every element that is not 0."""
import numpy as np
import pytest

from recurrence_util import Rows
from test_prefill_gpu import OneRow, decode

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import tree_speculative_verify_tv_gb300 as tv
    tv.build()
    tv.load()


def rows(seed, lens, kind, dk=64, dv=64, H=3, cls=Rows, **kw):
    rng = np.random.default_rng(seed)
    r = cls(rng, lens, H, dk, dv, f32=kind == "f32", diag=kind == "diag", **kw)
    H0, _ = r.state(rng)
    return r, H0


def spoil(H0):
    """Infinities of both signs in every request, head 1."""
    bad = H0.clone()
    bad[:, 1, 5, 7], bad[:, 1, 6, 8] = INF, -INF
    return bad


def check(clean, got, dv_bad=(7, 8)):
    """Infinite where the state was, the same bits elsewhere; outputs of other columns as without."""
    import torch
    state = clean[1].clone()
    state[:, 1, 5, 7], state[:, 1, 6, 8] = INF, -INF
    assert torch.equal(got[1], state)
    keep = torch.ones_like(clean[0], dtype=torch.bool)
    keep[:, 1, list(dv_bad)] = False
    assert torch.equal(got[0][keep], clean[0][keep])
    assert not torch.isfinite(got[0][~keep]).any()


# (0: the decay is 1 exactly; the others' rounding errors have either sign)
GATES = [0.0, -0.1, -0.2, -0.3, -0.5, -0.7, -1.0, -2.0, -5.0, -1e-3, -1e-7, 0.1, 0.3]


@pytest.mark.parametrize("kind", ["tensor", "f32", "diag"])
@pytest.mark.parametrize("g", GATES)
def test_infinite_elements_stay_infinite(kind, g):
    r, H0 = rows(1, [1, 5, 40], kind)
    r.g.fill_(g)
    check(r.prefill(H0), r.prefill(spoil(H0)))


@pytest.mark.parametrize("kind", ["tensor", "f32", "diag"])
@pytest.mark.parametrize("g", GATES)
def test_infinite_elements_stay_infinite_token_by_token(kind, g):
    r, H0 = rows(2, [1, 1], kind, cls=OneRow)
    r.g.fill_(g)
    check(decode(r, H0, True), decode(r, spoil(H0), True))


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (64, 128), (128, 128), (24, 40)])
def test_requests_without_rows_keep_any_state(dk, dv):
    import torch
    r, H0 = rows(3, [0, 70, 0], "tensor", dk, dv)
    H0[0, 0, 3, 4], H0[0, 2, 1, 9], H0[2, 1, 0, 0], H0[2, 1, 0, 1] = INF, -INF, float("nan"), 1e38
    H0[2, 0, 1, 1] = 2.0 ** -149
    _, H_new, status = r.prefill(H0)
    torch.cuda.synchronize()
    assert int(status[0]) == 0
    for b in (0, 2):
        assert torch.equal(torch.isnan(H_new[b]), torch.isnan(H0[b]))
        assert torch.equal(H_new[b].nan_to_num(7.0, INF, -INF), H0[b].nan_to_num(7.0, INF, -INF))


def test_infinite_elements_through_cuts():
    r, H0 = rows(4, [3000], "tensor", H=2, gates="head", decay=1e-4)
    check(r.prefill(H0), r.prefill(spoil(H0)))


@pytest.mark.parametrize("kind", ["tensor", "f32", "diag"])
@pytest.mark.parametrize("g", [89.0, 95.5, 100.0, 101.3, 177.3, 180.0, 700.0])
@pytest.mark.parametrize("step", [False, True])
def test_growth_past_the_range(kind, g, step):
    """A row that grows the state by e^g > 2^128 (k = 0, so that nothing else is added)."""
    import torch
    r, H0 = rows(5, [1, 1], kind, cls=OneRow if step else Rows)
    H0[H0 == 0] = 1.0
    r.dev["k"].zero_()
    r.g.fill_(g)
    H_new = (decode(r, H0, True) if step else r.prefill(H0))[1]
    torch.cuda.synchronize()
    assert torch.equal(H_new, torch.where(H0 > 0, INF, -INF))


def test_growth_past_the_range_in_a_segment():
    """A prompt in segments: the decay of one of them passes 2^128, though no chunk's does."""
    import torch
    import tree_speculative_verify_tv_gb300 as tv
    r, H0 = rows(6, [4096], "tensor", H=1)
    H0[H0 == 0] = 1.0
    assert tv.tv_prefill_workspace_bytes(1, 4096, 4096, 1, 64, 64, tv.TV_DECAY_SCALAR, tv.TV_BF16) > 0
    r.dev["k"].zero_()
    for g in (0.3, 0.31, 0.37, 0.4):  # 19 to 26 a chunk
        r.g.fill_(g)
        H_new = r.prefill(H0)[1]
        torch.cuda.synchronize()
        assert torch.equal(H_new, torch.where(H0 > 0, INF, -INF)), g
